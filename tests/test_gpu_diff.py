"""GPU: differential attention against the float64 formula on contiguous K/V.

The bound on each value is derived in _diff_ref.py.  Pools hold NaN in every slot no sequence
maps, so a stray read shows.
"""
import pytest
import torch

import paged_kv_cache_290_gb300 as pa
from paged_kv_cache_290_gb300 import binding as B
from paged_kv_cache_290_gb300 import workloads as W
from _cases import small_decode, small_long_chunks, small_mixed, small_spec
from _diff_ref import diff_attention_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_290_gb300 import build
    build.build()
    pa.load_library()
    assert torch.cuda.is_available()
    pa.get_device_error()


def learned(b, per_token=False, seed=5):
    g = torch.Generator().manual_seed(seed)
    shape = (b.num_tokens, b.num_q_heads // 2) if per_token else (b.num_q_heads // 2,)
    lam = 0.7 + 0.2 * torch.randn(shape, generator=g)
    return lam, 1 + 0.2 * torch.randn(2 * b.head_dim, generator=g)


def run(b, lam, weight=None, eps=1e-5, gain=1.0, q=None, stream=None, workspace=None):
    q = b.q.cuda() if q is None else q
    out = torch.full((b.num_tokens, b.num_q_heads // 2, 2 * b.head_dim), float("nan"),
                     dtype=b.q.dtype, device="cuda")
    pa.diff_attention(q, b.k_cache.cuda(), b.v_cache.cuda(), b.block_tables.cuda(),
                      b.seq_lens.cuda(), b.query_start_loc.cuda(), b.scale, lam.cuda(), out,
                      b.max_query_len, b.max_seq_len,
                      norm_weight=None if weight is None else weight.cuda(), eps=eps,
                      out_scale=gain, num_prefill_seqs=b.num_prefill_seqs, workspace=workspace)
    assert pa.get_device_error() == (0, 0)
    return out


def check(out, ref, bound):
    assert torch.isfinite(out).all()
    over = ((out.cpu().double() - ref).abs() / bound).max().item()
    assert over <= 1.0, f"error is {over:.2f} of its bound"


CASES = {
    "decode_d128_g4": lambda: small_decode(),
    "decode_d128_bs32_g8": lambda: small_decode(bs=32, hq=64, hkv=8, seed=9104),
    "decode_d64_g1": lambda: small_decode(d=64, hq=4, hkv=4, seed=9105),
    "decode_d64_bs32_g16": lambda: small_decode(d=64, bs=32, hq=32, hkv=2, seed=9106),
    "decode_d128_g7": lambda: small_decode(hq=28, hkv=4, seed=9107),
    "decode_d128_g12": lambda: small_decode(hq=24, hkv=2, seed=9108),
    "decode_tiny": W.tiny_decode,
    "mixed_d128_g4": lambda: small_mixed(),
    "mixed_d128_bs32_g8": lambda: small_mixed(bs=32, hq=16, hkv=2, seed=9207),
    "mixed_d64_g7": lambda: small_mixed(d=64, hq=28, hkv=4, seed=9208),
    "mixed_d64_bs32_g1": lambda: small_mixed(d=64, bs=32, hq=4, hkv=4, seed=9209),
    "mixed_d128_g16": lambda: small_mixed(hq=32, hkv=2, seed=9210),
    "mixed_d64_g3": lambda: small_mixed(d=64, hq=6, hkv=2, seed=9211),
    "spec_d128_g8": lambda: small_spec(),
    "spec_d64_bs32_g4": lambda: small_spec(d=64, bs=32, hq=16, hkv=4, seed=9401),
    "chunks_alone_d128_g1": lambda: W.build_batch(
        "chunks_alone", [W.SeqSpec(300, 300), W.SeqSpec(129, 128), W.SeqSpec(2, 2)],
        num_q_heads=2, num_kv_heads=2, head_dim=128, block_size=16, seed_base=9220),
}


@pytest.mark.parametrize("bf16", [False, True], ids=["f16", "bf16"])
@pytest.mark.parametrize("name", list(CASES))
def test_matches_the_formula(name, bf16):
    b = CASES[name]()
    b = W.to_bf16(b) if bf16 else b
    lam, weight = learned(b)
    check(run(b, lam, weight, gain=0.4), *diff_attention_ref(b, lam, weight, gain=0.4))


SPLIT = {
    # too few chunk tiles to fill the GPU: their keys are shared out and joined
    "d128_g4": dict(specs=[(5000, 200)], hq=8, hkv=2, d=128),
    "d64_g2": dict(specs=[(5000, 300), (2600, 20)], hq=4, hkv=2, d=64),
    "d128_g3_beside_rows": dict(specs=[(6100, 260), (3000, 1), (40, 1)], hq=6, hkv=2, d=128),
    "d64_g16_bs32": dict(specs=[(4100, 90)], hq=32, hkv=2, d=64, bs=32),
}


def split_batch(name):
    c = SPLIT[name]
    return W.build_batch("split_" + name, [W.SeqSpec(*x) for x in c["specs"]], num_q_heads=c["hq"],
                         num_kv_heads=c["hkv"], head_dim=c["d"], block_size=c.get("bs", 16),
                         seed_base=9230 + len(name))


@pytest.mark.parametrize("bf16", [False, True], ids=["f16", "bf16"])
@pytest.mark.parametrize("name", list(SPLIT))
def test_chunks_whose_keys_are_shared_out(name, bf16):
    b = split_batch(name)
    b = W.to_bf16(b) if bf16 else b
    lam, weight = learned(b)
    check(run(b, lam, weight), *diff_attention_ref(b, lam, weight))
    check(run(b, lam, gain=0.5), *diff_attention_ref(b, lam, gain=0.5))


@pytest.mark.parametrize("d, bs", [(128, 16), (64, 32)])
def test_whole_prompts_alone(d, bs):
    b = W.build_batch("prompts", [W.SeqSpec(900, 900), W.SeqSpec(400, 399), W.SeqSpec(129, 129)],
                      num_q_heads=8, num_kv_heads=2, head_dim=d, block_size=bs, seed_base=9240)
    lam, weight = learned(b)
    check(run(b, lam, weight), *diff_attention_ref(b, lam, weight))


def test_many_sequences():
    """More sequences than the chunk kernel sorts, and than it has threads; some without rows."""
    specs = [W.SeqSpec(1 + i % 5, i % 2) for i in range(700)]
    specs[3], specs[650], specs[699] = W.SeqSpec(600, 512), W.SeqSpec(300, 257), W.SeqSpec(70, 9)
    b = W.build_batch("many", specs, num_q_heads=2, num_kv_heads=2, head_dim=64, block_size=16,
                      seed_base=9241)
    lam, weight = learned(b)
    check(run(b, lam, weight), *diff_attention_ref(b, lam, weight))


def test_hidden_keys_of_the_chunk_do_not_reach_earlier_rows():
    """A key that only later rows see may score anything; earlier rows are the same to the bit."""
    b = W.build_batch("hidden", [W.SeqSpec(700, 600)], num_q_heads=8, num_kv_heads=2, head_dim=64,
                      block_size=16, seed_base=9242)
    lam, weight = learned(b)
    first = run(b, lam, weight)
    blk, off = int(b.block_tables[0, 650 // 16]), 650 % 16
    b.k_cache[blk, :, off] = 3000.0
    b.v_cache[blk, :, off] = -50000.0
    again = run(b, lam, weight)
    seen = 650 - (700 - 600)
    assert torch.equal(first[:seen], again[:seen])
    assert not torch.equal(first[seen:], again[seen:])


def test_scores_that_rise_late():
    """Each block of keys scores far above all before it, so the softmax base has to follow."""
    b = W.build_batch("rising", [W.SeqSpec(900, 300), W.SeqSpec(1400, 1)], num_q_heads=4,
                      num_kv_heads=2, head_dim=64, block_size=16, seed_base=9243)
    step = torch.arange(1400) // 64
    for s in range(2):
        n, base = int(b.seq_lens[s]), int(b.kv_start[s])
        for h in range(2):
            b.k_contig[base:base + n, h] = (step[:n, None] * 3.0).half()
        for i in range(n):
            b.k_cache[int(b.block_tables[s, i // 16]), :, i % 16] = b.k_contig[base + i]
    b.q[:] = b.q.abs()
    lam, weight = learned(b)
    check(run(b, lam, weight), *diff_attention_ref(b, lam, weight))


def test_long_contexts():
    b = small_long_chunks(hq=4, hkv=2)
    lam, weight = learned(b)
    check(run(b, lam, weight), *diff_attention_ref(b, lam, weight))


def test_without_norm_lambda_per_token_strided_q():
    b = small_mixed(d=64, hq=8, hkv=4, seed=9221)
    lam, _ = learned(b, per_token=True)
    wide = torch.full((b.num_tokens, 3 * 8 * 64), float("nan"), dtype=b.q.dtype, device="cuda")
    q = wide[:, 512:1024].view(-1, 8, 64)
    q.copy_(b.q)
    lam_wide = torch.zeros(b.num_tokens, 9)
    lam_wide[:, :4] = lam
    out = run(b, lam_wide.cuda()[:, :4], gain=-1.5, q=q)
    check(out, *diff_attention_ref(b, lam, gain=-1.5))


def test_lambda_zero_is_plain_attention_of_the_first_map():
    """With lambda 0 the result is pa_attention's of q heads 2p over K head 2j, on V's halves."""
    b = small_decode(hq=8, hkv=4, d=64)
    out = run(b, torch.zeros(4))
    check(out, *diff_attention_ref(b, torch.zeros(4)))


def test_equal_maps_cancel():
    """q1 = q2, K1 = K2 and lambda 1: y is exactly 0, and so is the normed result (eps > 0)."""
    b = small_mixed(d=64, hq=4, hkv=2, seed=9222)
    b.q[:, 1::2] = b.q[:, 0::2]
    b.k_cache[:, 1] = b.k_cache[:, 0]
    for weight in (None, torch.ones(128)):
        assert run(b, torch.ones(2), weight).abs().max().item() == 0


def test_large_scores_do_not_overflow():
    b = small_mixed(d=64, hq=8, hkv=4, seed=9223)
    b.q *= 30
    lam, weight = learned(b)
    check(run(b, lam, weight), *diff_attention_ref(b, lam, weight))


@pytest.mark.parametrize("scale", [0.0, -0.2])
def test_zero_and_negative_scale(scale):
    b = small_mixed(d=64, hq=8, hkv=4, seed=9224)
    b.scale = scale
    lam, weight = learned(b)
    check(run(b, lam, weight), *diff_attention_ref(b, lam, weight))


def test_results_do_not_depend_on_the_pages_or_the_run():
    b = small_mixed(hq=16, hkv=4, seed=9225)
    lam, weight = learned(b)
    first = run(b, lam, weight)
    assert torch.equal(first, run(b, lam, weight))
    assert torch.equal(first, run(W.repermute(b, 77), lam, weight))


@pytest.mark.parametrize("make", [small_decode, small_mixed], ids=["decode", "mixed"])
def test_replays_in_a_graph_on_another_stream(make):
    b = make(hq=8, hkv=4, d=64)
    lam, weight = learned(b)
    dev = [x.cuda() for x in (b.q, b.k_cache, b.v_cache, b.block_tables, b.seq_lens,
                              b.query_start_loc)]
    lam, weight = lam.cuda(), weight.cuda()
    out = torch.empty((b.num_tokens, 4, 128), dtype=b.q.dtype, device="cuda")
    ws = torch.empty(max(1, pa.diff_attention_workspace_size(
        b.num_tokens, b.num_seqs, 8, 4, 64, b.max_query_len, b.max_seq_len, b.num_prefill_seqs)),
        dtype=torch.uint8, device="cuda")

    def call():
        pa.diff_attention(*dev, b.scale, lam, out, b.max_query_len, b.max_seq_len,
                          norm_weight=weight, num_prefill_seqs=b.num_prefill_seqs, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (1, 2):  # new queries, the same graph
        b.q = torch.randn(b.q.shape, generator=torch.Generator().manual_seed(seed)).half()
        dev[0].copy_(b.q)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check(out, *diff_attention_ref(b, lam.cpu(), weight.cpu()))
    assert pa.get_device_error() == (0, 0)


def test_bad_descriptors_leave_rows_alone():
    """A block id outside the pool, a table that is too short and a hint that is too small are
    reported; the other sequences' rows are right and nothing else is written."""
    b = small_decode(hq=8, hkv=4, d=64)
    lam, weight = learned(b)
    ref, bound = diff_attention_ref(b, lam, weight)

    def call(tables, lens, max_len, rows=1):
        out = torch.full((b.num_tokens, 4, 128), float("nan"), dtype=b.q.dtype, device="cuda")
        pa.diff_attention(b.q.cuda(), b.k_cache.cuda(), b.v_cache.cuda(), tables.cuda(), lens.cuda(),
                          b.query_start_loc.cuda(), b.scale, lam.cuda(), out, rows, max_len,
                          norm_weight=weight.cuda())
        return out.cpu(), pa.get_device_error()

    def others(out, lost):
        keep = [s for s in range(b.num_seqs) if s not in lost]
        check(out[keep], ref[keep], bound[keep])
        assert out[list(lost)].isnan().all()

    bad = b.block_tables.clone()
    bad[3, 1] = b.num_blocks
    bad[4, 0] = -1
    bad[8, 40] = b.num_blocks + 5  # the second of three partitions
    out, (st, bits) = call(bad, b.seq_lens, b.max_seq_len)
    assert st == B.PA_ERR_OUT_OF_RANGE and bits & 4
    others(out, {3, 4, 8})
    long = b.seq_lens.clone()
    long[0] = b.block_tables.shape[1] * b.block_size + 1
    long[1] = 0
    out, (st, bits) = call(b.block_tables, long, 4096)
    assert st == B.PA_ERR_DESCRIPTOR and bits & 8
    others(out, {0, 1})
    out, (st, bits) = call(b.block_tables, b.seq_lens, 600)
    assert st == B.PA_ERR_DESCRIPTOR and bits & 16
    others(out, {8, 9})  # more than two partitions' keys


def test_too_small_hints_are_reported():
    """More chunks, or longer ones, than the hint says: reported, and the other rows are right."""
    b = small_mixed(d=64, hq=16, hkv=4, seed=9226)
    lam, weight = learned(b)
    ref, bound = diff_attention_ref(b, lam, weight)
    for rows, seqs in ((b.max_query_len, 3), (100, b.num_prefill_seqs)):
        out = torch.full((b.num_tokens, 8, 128), float("nan"), dtype=b.q.dtype, device="cuda")
        pa.diff_attention(b.q.cuda(), b.k_cache.cuda(), b.v_cache.cuda(), b.block_tables.cuda(),
                          b.seq_lens.cuda(), b.query_start_loc.cuda(), b.scale, lam.cuda(), out,
                          rows, b.max_seq_len, norm_weight=weight.cuda(), num_prefill_seqs=seqs)
        st, bits = pa.get_device_error()
        assert st == B.PA_ERR_DESCRIPTOR and bits & 16
        out = out.cpu()
        lost = out.isnan().all(-1).all(-1)
        assert lost.any() and not lost.all()
        check(out[~lost], ref[~lost], bound[~lost])


@pytest.mark.parametrize("hint", [1, 2])
def test_rows_beyond_the_hint_are_reported(hint):
    """Calls that the rows kernel serves alone: a sequence with more rows than the hint allows."""
    b = W.build_batch("beyond", [W.SeqSpec(40, 1), W.SeqSpec(50, 3), W.SeqSpec(300, 1)],
                      num_q_heads=4, num_kv_heads=4, head_dim=64, block_size=16, seed_base=9244)
    lam, weight = learned(b)
    out = torch.full((5, 2, 128), float("nan"), dtype=b.q.dtype, device="cuda")
    pa.diff_attention(b.q.cuda(), b.k_cache.cuda(), b.v_cache.cuda(), b.block_tables.cuda(),
                      b.seq_lens.cuda(), b.query_start_loc.cuda(), b.scale, lam.cuda(), out, hint,
                      b.max_seq_len, norm_weight=weight.cuda())
    st, bits = pa.get_device_error()
    assert st == B.PA_ERR_DESCRIPTOR and bits & 16
    out = out.cpu()
    assert out[1:4].isnan().all()
    ref, bound = diff_attention_ref(b, lam, weight)
    for row in (0, 4):
        check(out[row], ref[row], bound[row])


def test_bad_ids_in_shared_out_keys():
    b = split_batch("d64_g2")
    lam, weight = learned(b)
    bad = b.block_tables.clone()
    bad[0, 200] = b.num_blocks  # in one of the first sequence's ranges
    out = torch.full((b.num_tokens, 2, 128), float("nan"), dtype=b.q.dtype, device="cuda")
    pa.diff_attention(b.q.cuda(), b.k_cache.cuda(), b.v_cache.cuda(), bad.cuda(), b.seq_lens.cuda(),
                      b.query_start_loc.cuda(), b.scale, lam.cuda(), out, b.max_query_len,
                      b.max_seq_len, norm_weight=weight.cuda(), num_prefill_seqs=2)
    st, bits = pa.get_device_error()
    assert st == B.PA_ERR_OUT_OF_RANGE and bits & 4
    assert out[:300].isnan().all()
    ref, bound = diff_attention_ref(b, lam, weight, rows_of={1})
    check(out[300:], ref[300:], bound[300:])


@pytest.mark.parametrize("name", ["decode", "chunks"])
def test_two_streams_at_once(name):
    """Two calls in flight on streams of their own, each with its own workspace."""
    b = small_decode(hq=8, hkv=4, d=64) if name == "decode" else split_batch("d64_g2")
    lam, weight = learned(b)
    ref, bound = diff_attention_ref(b, lam, weight)
    dev = [x.cuda() for x in (b.q, b.k_cache, b.v_cache, b.block_tables, b.seq_lens,
                              b.query_start_loc)]
    lam, weight = lam.cuda(), weight.cuda()
    torch.cuda.synchronize()
    outs = []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                out = torch.empty((b.num_tokens, b.num_q_heads // 2, 2 * b.head_dim),
                                  dtype=b.q.dtype, device="cuda")
            out.record_stream(s)
            pa.diff_attention(*dev, b.scale, lam, out, b.max_query_len, b.max_seq_len,
                              norm_weight=weight, num_prefill_seqs=b.num_prefill_seqs, stream=s)
            outs.append(out)
    torch.cuda.synchronize()
    assert pa.get_device_error() == (0, 0)
    for out in outs:
        check(out, ref, bound)


def test_bad_chunks_leave_their_rows_alone():
    b = small_mixed(d=64, hq=16, hkv=4, seed=9226)
    lam, weight = learned(b)
    ref, bound = diff_attention_ref(b, lam, weight)
    bad = b.block_tables.clone()
    bad[6, 5] = -3  # in every tile of the last chunk
    out = torch.full((b.num_tokens, 8, 128), float("nan"), dtype=b.q.dtype, device="cuda")
    pa.diff_attention(b.q.cuda(), b.k_cache.cuda(), b.v_cache.cuda(), bad.cuda(), b.seq_lens.cuda(),
                      b.query_start_loc.cuda(), b.scale, lam.cuda(), out, b.max_query_len,
                      b.max_seq_len, norm_weight=weight.cuda(),
                      num_prefill_seqs=b.num_prefill_seqs)
    st, bits = pa.get_device_error()
    assert st == B.PA_ERR_OUT_OF_RANGE and bits & 4
    r0, r1 = b.query_start_loc[6:8].tolist()
    assert out[r0:r1].isnan().all()
    keep = [i for i in range(b.num_tokens) if not r0 <= i < r1]
    check(out[keep], ref[keep], bound[keep])
