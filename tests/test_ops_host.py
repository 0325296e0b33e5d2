"""Host-side behaviour of the rotary cache write, differential attention and page moves: refused
arguments (nothing is launched), plans, and the block manager's compaction."""
import ctypes
import random

import pytest
import torch

import paged_kv_cache_290_gb300 as pa
from paged_kv_cache_290_gb300 import binding as B
from paged_kv_cache_290_gb300.block_manager import BlockManager
from test_abi import FAKE, T, msg
from test_block_manager import Engine


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_290_gb300 import build
    build.build()
    return B.load_library()


def R(n=16, freq=0.5, axes=None, factor=1.0, adjacent=0):
    f = (ctypes.c_double * max(1, n))(*([freq] * max(0, n)))
    ax = (ctypes.c_int32 * max(1, n))(*axes) if axes else None
    r = B.PARope(n, adjacent, factor, ctypes.cast(f, ctypes.c_void_p),
                 ctypes.cast(ax, ctypes.c_void_p) if axes else None)
    r.keep = (f, ax)
    return r


def call_rope(lib, rope=None, scales=None, **kw):
    t, hq, hkv, d, bs, nb = 5, 4, 2, 64, 16, 10
    a = dict(q=T(B.PA_F16, [t, hq, d], data=0x20000), k=T(B.PA_F16, [t, hkv, d], data=0x30000),
             v=T(B.PA_F16, [t, hkv, d], data=0x40000), pos=T(B.PA_I64, [2, t]),
             kc=T(B.PA_F16, [nb, hkv, bs, d]), vc=T(B.PA_F16, [nb, hkv, bs, d]),
             sm=T(B.PA_I64, [t]), qo=T(B.PA_F16, [t, hq, d], data=0x50000))
    a.update(kw)
    p = {k: ctypes.byref(v) if v is not None else None for k, v in a.items()}
    rope = R() if rope is None else rope
    return lib.pa_rope_and_cache(p["q"], p["k"], p["v"], p["pos"],
                                 ctypes.byref(rope) if rope else None, p["kc"], p["vc"], p["sm"],
                                 p["qo"], ctypes.byref(scales) if scales else None, None)


F8 = dict(kc=T(B.PA_F8E4M3, [10, 2, 16, 64]), vc=T(B.PA_F8E4M3, [10, 2, 16, 64]))


@pytest.mark.parametrize("kw, status, text", [
    (dict(q=None), B.PA_ERR_INVALID_ARG, "q is NULL"),
    (dict(kc=None), B.PA_ERR_INVALID_ARG, "k_cache is NULL"),
    (dict(q=T(B.PA_BF16, [5, 4, 64])), B.PA_ERR_INVALID_ARG, "q must be float16"),
    (dict(q=T(B.PA_F16, [5, 4, 128])), B.PA_ERR_INVALID_ARG, "matching the pool"),
    (dict(v=T(B.PA_F16, [5, 3, 64])), B.PA_ERR_INVALID_ARG, "matching the pool"),
    (dict(k=T(B.PA_F16, [4, 2, 64])), B.PA_ERR_INVALID_ARG, "matching the pool"),
    (dict(qo=T(B.PA_F16, [5, 2, 64])), B.PA_ERR_INVALID_ARG, "q_out must have q's shape"),
    (dict(qo=T(B.PA_F16, [5, 4, 64], data=0x20010)), B.PA_ERR_INVALID_ARG, "overlap"),
    (dict(qo=T(B.PA_F16, [5, 4, 64], data=0x40000 - 64)), B.PA_ERR_INVALID_ARG, "overlap"),
    (dict(q=T(B.PA_F16, [5, 4, 64], stride=[260, 64, 1])), B.PA_ERR_INVALID_ARG, "multiple of 8"),
    (dict(k=T(B.PA_F16, [5, 2, 64], data=FAKE + 8)), B.PA_ERR_INVALID_ARG, "alignment"),
    (dict(q=T(B.PA_F16, [5, 4, 64], stride=[512, 128, 1])), B.PA_ERR_INVALID_ARG, "head stride"),
    (dict(pos=T(B.PA_I32, [2, 5])), B.PA_ERR_INVALID_ARG, "positions must be int64"),
    (dict(pos=T(B.PA_I64, [2, 4])), B.PA_ERR_INVALID_ARG, "positions"),
    (dict(pos=T(B.PA_I64, [0, 5])), B.PA_ERR_INVALID_ARG, "axes"),
    (dict(sm=T(B.PA_I64, [6])), B.PA_ERR_INVALID_ARG, "slot_mapping"),
    (dict(rope=R(12)), B.PA_ERR_INVALID_ARG, "multiple of 8"),
    (dict(rope=R(0)), B.PA_ERR_INVALID_ARG, "multiple of 8"),
    (dict(rope=R(40)), B.PA_ERR_INVALID_ARG, "head_dim"),
    (dict(rope=R(freq=float("nan"))), B.PA_ERR_INVALID_ARG, "inv_freq must be finite"),
    (dict(rope=R(factor=float("inf"))), B.PA_ERR_INVALID_ARG, "factor"),
    (dict(rope=R(axes=[0] * 15 + [2])), B.PA_ERR_INVALID_ARG, "axis"),
    (dict(rope=R(axes=[-1] + [0] * 15)), B.PA_ERR_INVALID_ARG, "axis"),
    (dict(rope=B.PARope(16, 0, 1.0, None, None)), B.PA_ERR_INVALID_ARG, "inv_freq is NULL"),
    (F8, B.PA_ERR_INVALID_ARG, "scales is NULL"),
    (dict(F8, scales=B.PAKVScales(1.0, 0.0)), B.PA_ERR_INVALID_ARG, "finite and > 0"),
    (dict(F8, scales=B.PAKVScales(1.0, 1.0), q=T(B.PA_BF16, [5, 4, 64])), B.PA_ERR_INVALID_ARG,
     "q must be float16"),
])
def test_rope_refuses(lib, kw, status, text):
    assert call_rope(lib, **kw) == status
    assert text in msg(lib), msg(lib)


def test_rope_without_tokens_is_a_no_op(lib):
    e = lambda h: T(B.PA_F16, [0, h, 64])
    assert call_rope(lib, q=e(4), k=e(2), v=e(2), qo=e(4), pos=T(B.PA_I64, [2, 0]),
                     sm=T(B.PA_I64, [0])) == B.PA_OK


def call_diff(lib, hint=(1, 100), ws=None, wsb=0, scale=0.125, lam=T(B.PA_F32, [4]), w=None,
              eps=1e-5, gain=1.0, diff=True, **kw):
    n, hq, hkv, d, bs, nb, mb = 3, 8, 2, 64, 16, 40, 8
    a = dict(q=T(B.PA_F16, [n, hq, d]), kc=T(B.PA_F16, [nb, hkv, bs, d]),
             vc=T(B.PA_F16, [nb, hkv, bs, d]), bt=T(B.PA_I32, [n, mb]), sl=T(B.PA_I32, [n]),
             qsl=T(B.PA_I32, [n + 1]), out=T(B.PA_F16, [n, hq // 2, 2 * d]))
    a.update(kw)
    p = {k: ctypes.byref(v) if v is not None else None for k, v in a.items()}
    df = B.PADiff(ctypes.pointer(lam) if lam is not None else None,
                  ctypes.pointer(w) if w is not None else None, eps, gain)
    return lib.pa_diff_attention(p["q"], p["kc"], p["vc"], p["bt"], p["sl"], p["qsl"],
                                 ctypes.c_float(scale), ctypes.byref(df) if diff else None,
                                 p["out"], ctypes.byref(B.PABatchHint(*hint)) if hint else None,
                                 ws, wsb, None)


@pytest.mark.parametrize("kw, status, text", [
    (dict(kc=None), B.PA_ERR_INVALID_ARG, "k_cache is NULL"),
    (dict(kc=T(B.PA_F8E4M3, [40, 2, 16, 64])), B.PA_ERR_UNSUPPORTED, "FP8"),
    (dict(kc=T(B.PA_F16, [40, 1, 16, 64]), vc=T(B.PA_F16, [40, 1, 16, 64])), B.PA_ERR_INVALID_ARG,
     "even"),
    (dict(q=T(B.PA_F16, [3, 7, 64])), B.PA_ERR_INVALID_ARG, "multiple of num_kv_heads"),
    (dict(q=T(B.PA_F16, [3, 34, 64]), out=T(B.PA_F16, [3, 17, 128])), B.PA_ERR_UNSUPPORTED, "group"),
    (dict(out=T(B.PA_F16, [3, 8, 64])), B.PA_ERR_INVALID_ARG, "out must be [T"),
    (dict(out=T(B.PA_BF16, [3, 4, 128])), B.PA_ERR_INVALID_ARG, "out must be float16"),
    (dict(out=T(B.PA_F16, [3, 4, 128], stride=[1024, 128, 1])), B.PA_ERR_INVALID_ARG, "contiguous"),
    (dict(q=T(B.PA_F16, [3, 8, 64], data=FAKE + 2)), B.PA_ERR_INVALID_ARG, "alignment"),
    (dict(qsl=T(B.PA_I32, [3])), B.PA_ERR_INVALID_ARG, "query_start_loc"),
    (dict(bt=T(B.PA_I32, [2, 8])), B.PA_ERR_INVALID_ARG, "block_tables"),
    (dict(lam=None), B.PA_ERR_INVALID_ARG, "lambda is NULL"),
    (dict(lam=T(B.PA_F32, [8])), B.PA_ERR_INVALID_ARG, "lambda must be"),
    (dict(lam=T(B.PA_F32, [2, 4])), B.PA_ERR_INVALID_ARG, "lambda must be"),
    (dict(lam=T(B.PA_F16, [4])), B.PA_ERR_INVALID_ARG, "lambda must be float32"),
    (dict(w=T(B.PA_F32, [64])), B.PA_ERR_INVALID_ARG, "2 * head_dim"),
    (dict(w=T(B.PA_BF16, [128])), B.PA_ERR_INVALID_ARG, "norm_weight must be float32"),
    (dict(w=T(B.PA_F32, [128]), eps=-1.0), B.PA_ERR_INVALID_ARG, "eps"),
    (dict(w=T(B.PA_F32, [128]), eps=float("nan")), B.PA_ERR_INVALID_ARG, "eps"),
    (dict(gain=float("inf")), B.PA_ERR_INVALID_ARG, "out_scale"),
    (dict(scale=float("nan")), B.PA_ERR_INVALID_ARG, "scale"),
    (dict(diff=False), B.PA_ERR_INVALID_ARG, "diff is NULL"),
    (dict(hint=None), B.PA_ERR_INVALID_ARG, "hint is NULL"),
    (dict(hint=(1, 1000, 0, 512)), B.PA_ERR_UNSUPPORTED, "shared-prefix"),
    (dict(hint=(20, 10)), B.PA_ERR_INVALID_ARG, "max_query_len"),
    (dict(hint=(1, 4000)), B.PA_ERR_WORKSPACE, "workspace needs"),
    (dict(hint=(1, 4000), ws=FAKE + 16, wsb=1 << 40), B.PA_ERR_WORKSPACE, "aligned"),
])
def test_diff_refuses(lib, kw, status, text):
    assert call_diff(lib, **kw) == status
    assert text in msg(lib), msg(lib)


@pytest.mark.parametrize("hq, hkv", [(1024, 2), (6, 3), (8, 1), (7, 2), (0, 2), (2, 4)])
def test_diff_workspace_of_refused_heads_is_empty(lib, hq, hkv):
    h = B.PABatchHint(512, 4096, 4, 0)
    assert lib.pa_diff_attention_workspace_size(4096, 8, hq, hkv, 128, ctypes.byref(h)) == 0
    assert lib.pa_diff_attention_workspace_size(4096, 8, 8, 2, 128, ctypes.byref(h)) > 0


def test_diff_without_rows_is_a_no_op(lib):
    assert call_diff(lib, q=T(B.PA_F16, [0, 8, 64]), out=T(B.PA_F16, [0, 4, 128]),
                     hint=(0, 0)) == B.PA_OK


def test_host_tensors_are_refused():
    x = torch.zeros(2, 4, 64, dtype=torch.float16)
    pool = torch.zeros(3, 2, 16, 64, dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA device"):
        pa.rope_and_cache(x, x, x, i, pa.rope_inv_freq(64), pool, pool, i)
    with pytest.raises(ValueError, match="CUDA device"):
        pa.diff_attention(x, pool, pool, i, i, i, 1.0, i, x, 1, 1)
    with pytest.raises(ValueError, match="CUDA device"):
        pa.move_blocks(pool, pool, [(0, 1)])
    with pytest.raises(ValueError, match="inv_freq"):
        pa.rope_and_cache(x, x, x, i, pa.rope_inv_freq(64).float(), pool, pool, i)
    with pytest.raises(ValueError, match="axes"):
        pa.rope_and_cache(x, x, x, i, pa.rope_inv_freq(64), pool, pool, i, axes=pa.rope_axes([31]))


def test_rope_helpers():
    assert pa.rope_axes([2, 0, 3]).tolist() == [0, 0, 2, 2, 2]
    f = pa.rope_inv_freq(8, 100.0)
    assert torch.allclose(f, torch.tensor([1.0, 100 ** -0.25, 0.1, 100 ** -0.75],
                                          dtype=torch.float64), rtol=1e-15)


@pytest.mark.parametrize("pairs, nb, text", [
    ([(0, 4)], 4, "outside the pool"), ([(-1, 0)], 4, "outside the pool"),
    ([(0, 1), (2, 1)], 4, "into one block"), ([(0, 1), (0, 2)], 4, "out of one block"),
    ([(0, 0), (1, 0)], 4, "into one block"), ([(0, 1)], -1, "bad size"),
])
def test_move_plan_refuses(pairs, nb, text):
    with pytest.raises(B.PAError, match=text):
        pa.MovePlan(pairs, nb)


def call_move(lib, plan, kc, vc, bt=None, ws=None, wsb=0):
    return lib.pa_move_blocks(plan._h if plan else None, ctypes.byref(kc), ctypes.byref(vc),
                              ctypes.byref(bt) if bt is not None else None, ws, wsb, None)


def test_move_refuses(lib):
    plan = pa.MovePlan([(i, (i + 1) % 40) for i in range(40)], 40)  # one cycle
    assert 0 < plan.staged <= 10
    kc = T(B.PA_F16, [40, 2, 16, 64])
    vc = T(B.PA_F16, [40, 2, 16, 64], data=FAKE + (1 << 24))
    size = 40 * 2 * 16 * 64
    for args, status, text in (
            ((None, kc, vc), B.PA_ERR_INVALID_ARG, "plan is NULL"),
            ((plan, T(B.PA_F16, [41, 2, 16, 64]), T(B.PA_F16, [41, 2, 16, 64])),
             B.PA_ERR_INVALID_ARG, "a pool of 40 blocks"),
            ((plan, T(B.PA_F16, [2, 16, 64]), vc), B.PA_ERR_INVALID_ARG, "rank 4 or 5"),
            ((plan, kc, T(B.PA_BF16, [40, 2, 16, 64])), B.PA_ERR_INVALID_ARG, "float16"),
            ((plan, kc, kc), B.PA_ERR_INVALID_ARG, "overlap"),
            ((plan, T(B.PA_F16, [2, 40, 2, 16, 64]), T(B.PA_F16, [2, 40, 2, 16, 64],
                                                      data=FAKE + 2 * size)),
             B.PA_ERR_INVALID_ARG, "overlap"),
            ((plan, T(B.PA_F16, [2, 40, 2, 16, 64], stride=[size // 2, 2048, 1024, 64, 1]),
              T(B.PA_F16, [2, 40, 2, 16, 64], stride=[size // 2, 2048, 1024, 64, 1],
                data=FAKE + (1 << 24))), B.PA_ERR_INVALID_ARG, "must not overlap"),
            ((plan, kc, vc, T(B.PA_I64, [2, 3])), B.PA_ERR_INVALID_ARG, "int32"),
            ((plan, kc, vc), B.PA_ERR_WORKSPACE, "workspace needs"),
            ((plan, kc, vc, None, FAKE + 128, 1 << 30), B.PA_ERR_WORKSPACE, "aligned"),
            ((plan, T(B.PA_F16, [0, 40, 2, 16, 64]), T(B.PA_F16, [0, 40, 2, 16, 64])),
             B.PA_ERR_INVALID_ARG, "layers")):
        assert call_move(lib, *args) == status, text
        assert text in msg(lib), (text, msg(lib))
    assert call_move(lib, pa.MovePlan([(3, 3)], 40), kc, vc) == B.PA_OK  # nothing moves



def test_filling_holes_needs_no_workspace():
    pairs = [(5000 + i, 4999 - i) for i in range(3000)]
    random.Random(1).shuffle(pairs)
    plan = pa.MovePlan(pairs, 8000)
    assert plan.staged == 0
    chain = [(i, i + 1) for i in range(4999)]  # a long chain: one in eight, at group borders
    random.Random(2).shuffle(chain)
    assert pa.MovePlan(chain, 5000).staged <= 5000 // 8


@pytest.mark.parametrize("in_order", [False, True])
@pytest.mark.parametrize("seed", range(6))
def test_compaction_keeps_every_sequence(seed, in_order):
    """Random traffic; after each compaction, with the moves applied to the slots, every live
    sequence finds its own prefix at every position and later traffic goes on as before."""
    rng = random.Random(seed)
    e = Engine(160, 4, caching=bool(seed % 2))
    live, nxt, prompts = [], 0, [[rng.randrange(50) for _ in range(16)] for _ in range(3)]
    compacted = 0
    for _ in range(200):
        op = rng.random()
        try:
            if op < 0.35 or not live:
                e.add(nxt, rng.choice(prompts)[:rng.randint(1, 16)] +
                      [rng.randrange(50) for _ in range(rng.randint(0, 9))] or [1])
                live.append(nxt)
                nxt += 1
            elif op < 0.65:
                e.append(rng.choice(live), [rng.randrange(50) for _ in range(rng.randint(1, 5))])
            elif op < 0.75:
                p = rng.choice(live)
                e.bm.fork(p, nxt)
                e.toks[nxt] = list(e.toks[p])
                live.append(nxt)
                nxt += 1
            elif op < 0.9:
                s = live.pop(rng.randrange(len(live)))
                e.bm.free(s)
                del e.toks[s]
            else:
                before = e.bm.stats()
                moves = e.bm.compact(in_order)
                compacted += bool(moves)
                assert e.bm.stats() == before
                old = dict(e.slots)
                for s, d in moves:
                    for off in range(e.bs):
                        e.slots.pop(d * e.bs + off, None)
                        if s * e.bs + off in old:
                            e.slots[d * e.bs + off] = old[s * e.bs + off]
                used = e.nb - before.free_blocks
                assert all(d < used for _, d in moves)
                if not in_order:
                    assert all(s >= used for s, _ in moves)
                seen = []
                for sid in sorted(live):
                    table = e.bm.sequence(sid)[1]
                    assert all(b < used for b in table)
                    seen += [b for b in table if b not in seen]
                if in_order:
                    assert seen == list(range(len(seen)))
                assert e.bm.compact(in_order) == []  # nothing left to move
        except B.PAError as err:
            assert err.status == B.PA_ERR_NO_BLOCKS
        for sid in live:
            length, table = e.bm.sequence(sid)
            for p in range(length):
                assert e.slots[table[p // e.bs] * e.bs + p % e.bs] == tuple(e.toks[sid][:p + 1])
    assert compacted


def test_compact_refuses_without_changing_anything(lib):
    bm = BlockManager(8, 4, False)
    bm.add(1, [1] * 4)
    bm.add(2, [2] * 12)
    bm.free(1)
    tables = bm.sequence(2)
    n, out = ctypes.c_int32(-1), (ctypes.c_int32 * 2)()
    assert lib.pa_bm_compact(bm._h, 1, out, 0, ctypes.byref(n)) == B.PA_ERR_INVALID_ARG
    assert "needed" in msg(lib) and bm.sequence(2) == tables and n.value == -1
    assert lib.pa_bm_compact(None, 1, out, 1, ctypes.byref(n)) == B.PA_ERR_INVALID_ARG
    assert lib.pa_bm_compact(bm._h, 1, None, 1, ctypes.byref(n)) == B.PA_ERR_INVALID_ARG
    assert lib.pa_bm_compact(bm._h, 1, out, 1, None) == B.PA_ERR_INVALID_ARG
    assert bm.compact() == [(3, 0)] and bm.sequence(2)[1] == [1, 2, 0]
    assert bm.compact(in_order=True) == [(0, 2), (1, 0), (2, 1)]
    assert bm.sequence(2)[1] == [0, 1, 2]
