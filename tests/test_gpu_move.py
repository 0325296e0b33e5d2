"""GPU: pages moved inside the pool, bit for bit, with the block tables renumbered."""
import random

import pytest
import torch

import paged_kv_cache_290_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_290_gb300 import build
    build.build()
    pa.load_library()
    assert torch.cuda.is_available()
    pa.get_device_error()


def bits(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    if dtype == torch.uint8:
        return torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)
    return torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, dtype=torch.int16).view(dtype)


def raw(x):
    return x.cpu() if x.dtype == torch.uint8 else x.cpu().view(torch.int16)


def moved(pool, pairs):
    """The same moves one by one from a copy."""
    old, new = raw(pool), raw(pool).clone()
    for s, d in pairs:
        new.select(-4, d).copy_(old.select(-4, s))
    return new


def lists(nb, rng):
    ids = list(range(nb))
    rng.shuffle(ids)
    yield "none", []
    yield "stay", [(i, i) for i in range(nb)]
    yield "one", [(ids[0], ids[1])]
    yield "swap", [(ids[0], ids[1]), (ids[1], ids[0])]
    yield "chain", list(zip(ids, ids[1:]))
    yield "cycle", list(zip(ids, ids[1:] + ids[:1]))
    yield "holes", [(nb - 1 - i, i) for i in range(nb // 2)]
    to = list(range(nb))
    rng.shuffle(to)
    yield "permutation", list(enumerate(to))
    part = rng.sample(list(enumerate(to)), nb // 3)  # chains and pieces of cycles, any order
    yield "part", part


@pytest.mark.parametrize("shape, dtype", [
    ((40, 2, 16, 64), torch.float16), ((3, 41, 1, 16, 64), torch.bfloat16),
    ((2, 70, 3, 32, 128), torch.uint8), ((1, 17, 1, 16, 64), torch.uint8)],
    ids=["f16", "bf16x3", "e4m3x2", "e4m3x1"])
def test_every_kind_of_list(shape, dtype):
    nb = shape[-4]
    rng = random.Random(nb)
    for i, (name, pairs) in enumerate(lists(nb, rng)):
        k, v = bits(shape, dtype, 2 * i), bits(shape, dtype, 2 * i + 1)
        dk, dv = k.cuda(), v.cuda()
        tables = torch.randint(-2, nb + 2, (5, 9), generator=torch.Generator().manual_seed(i),
                               dtype=torch.int32)
        tables[0, 0], tables[1, 1] = 2 ** 31 - 1, -2 ** 31
        wide = torch.full((5, 12), 77, dtype=torch.int32, device="cuda")
        wide[:, 1:10] = tables.cuda()
        pa.move_blocks(dk, dv, pairs, block_tables=wide[:, 1:10])
        assert torch.equal(raw(dk), moved(k, pairs)), name
        assert torch.equal(raw(dv), moved(v, pairs)), name
        new = {s: d for s, d in pairs}
        want = tables.clone().apply_(lambda e: new.get(e, e))
        assert torch.equal(wide[:, 1:10].cpu(), want), name
        assert (wide[:, 0] == 77).all() and (wide[:, 10:] == 77).all(), name


@pytest.mark.parametrize("kind", ["permutation", "cycle", "chain"])
def test_lists_of_several_launches(kind):
    """More moves than one launch takes, through a workspace of one layer and of all."""
    nb, shape = 2500, (3, 2500, 1, 16, 64)
    pairs = dict(lists(nb, random.Random(9)))[kind]
    k, v = bits(shape, torch.uint8, 1), bits(shape, torch.uint8, 2)
    plan = pa.MovePlan(pairs, nb)
    assert plan.staged <= nb // 4  # one or two of a group of eight
    for layers in (1, 3):
        dk, dv = k.cuda(), v.cuda()
        ws = torch.empty(plan.workspace_size(dk, layers, False), dtype=torch.uint8, device="cuda")
        pa.move_blocks(dk, dv, plan, workspace=ws)
        assert torch.equal(raw(dk), moved(k, pairs)) and torch.equal(raw(dv), moved(v, pairs))


@pytest.mark.parametrize("n, shape", [
    (256, (3, 700)), (257, (3, 700)), (9, (300, 900)), (256, (1, 1)), (1100, (40, 50))])
def test_tables_of_many_sizes(n, shape):
    """Renaming beside the moves, by a launch of its own and after long lists."""
    nb = 1500
    rng = random.Random(n)
    to = list(range(nb))
    rng.shuffle(to)
    pairs = rng.sample([(s, d) for s, d in enumerate(to) if s != d], n)
    k, v = bits((nb, 1, 16, 64), torch.uint8, 6), bits((nb, 1, 16, 64), torch.uint8, 7)
    dk, dv = k.cuda(), v.cuda()
    t = torch.randint(-1, nb, shape, generator=torch.Generator().manual_seed(n), dtype=torch.int32)
    dt = t.cuda()
    pa.move_blocks(dk, dv, pairs, block_tables=dt)
    assert torch.equal(raw(dk), moved(k, pairs)) and torch.equal(raw(dv), moved(v, pairs))
    new = torch.arange(nb, dtype=torch.int32)
    new[[s for s, _ in pairs]] = torch.tensor([d for _, d in pairs], dtype=torch.int32)
    assert torch.equal(dt.cpu(), torch.where(t < 0, t, new[t.clamp(min=0).long()]))


def test_layers_of_k_and_v_in_one_buffer():
    both = bits((4, 2, 30, 2, 16, 64), torch.float16, 3)
    d = both.cuda()
    pairs = [(29, 0), (0, 1), (1, 29), (5, 6)]
    pa.move_blocks(d[:, 0], d[:, 1], pairs)
    assert torch.equal(raw(d[:, 0].contiguous()), moved(both[:, 0].contiguous(), pairs))
    assert torch.equal(raw(d[:, 1].contiguous()), moved(both[:, 1].contiguous(), pairs))


def test_replays_in_a_graph_and_ends_with_its_plan():
    nb = 30
    k, v = bits((nb, 2, 16, 64), torch.float16, 4), bits((nb, 2, 16, 64), torch.float16, 5)
    pairs = dict(lists(nb, random.Random(3)))["cycle"]
    dk, dv, t = k.cuda(), v.cuda(), torch.arange(nb, dtype=torch.int32, device="cuda")[None]
    plan = pa.MovePlan(pairs, nb)
    ws = torch.empty(plan.workspace_size(dk), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.move_blocks(dk, dv, plan, block_tables=t, workspace=ws)
    plan.close()
    new = dict(pairs)
    want_t = list(range(nb))
    for _ in range(2):
        graph.replay()
        k, v = moved(k, pairs).view(torch.float16), moved(v, pairs).view(torch.float16)
        want_t = [new[e] for e in want_t]
    torch.cuda.synchronize()
    assert torch.equal(raw(dk), raw(k)) and torch.equal(raw(dv), raw(v))
    assert t[0].tolist() == want_t
