"""GPU: rotary positions with the cache write against the float64 formula.

Per value, with u the output type's half step: u |y| for the one rounding (2^-25 near fp16's
zero; for E4M3 2^-4 |y|, scale 2^-10 near its zero), and for the float32 arithmetic cos and sin
each within 4e-7 (angle to half a float32 step of pi: 1.9e-7, sincospif 2 ulp: 1.2e-7, times
factor: 0.6e-7), two products and a sum of 2^-24 each: (|a| + |b|) factor 7e-7 in all.
"""
import pytest
import torch

import paged_kv_cache_290_gb300 as pa
from paged_kv_cache_290_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_290_gb300 import build
    build.build()
    pa.load_library()
    assert torch.cuda.is_available()
    pa.get_device_error()


def rotated(x, pos, inv_freq, axes, adjacent, factor):
    """(y, |a| + |b|) in float64."""
    x = x.double()
    theta = pos.double()[axes.long()].T * inv_freq  # [T, pairs]
    c, s = theta.cos()[:, None] * factor, theta.sin()[:, None] * factor
    n = inv_freq.numel()
    i = torch.arange(n)
    ia, ib = (2 * i, 2 * i + 1) if adjacent else (i, i + n)
    y, size = x.clone(), torch.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return y, size


def make(t, hq, hkv, d, rot, axes, dtype, pool, bs, seed, far=1 << 17, fused=True):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(t, (hq + 2 * hkv) * d, generator=g).to(dtype).cuda()
    cut = (qkv[:, :hq * d], qkv[:, hq * d:(hq + hkv) * d], qkv[:, (hq + hkv) * d:])
    q, k, v = (x.view(t, -1, d) if fused else x.contiguous().view(t, -1, d) for x in cut)
    nb = t // bs + 3
    slots = torch.randperm(nb * bs, generator=g)[:t]
    if t > 2:
        slots[1] = -1
    if pool == "e4m3":
        pools = [torch.full((nb, hkv, bs, d), 0x7F, dtype=torch.uint8, device="cuda")
                 for _ in range(2)]
    else:
        pools = [torch.full((nb, hkv, bs, d), float("nan"), dtype=dtype, device="cuda")
                 for _ in range(2)]
    pos = torch.randint(0, far, (axes, t), generator=g)
    axis = torch.randint(0, axes, (rot // 2,), generator=g, dtype=torch.int32)
    return q, k, v, pos, axis, pools, slots


def expect(out, y, size, dtype, factor, scale=1.0):
    if out.dtype == torch.uint8:
        out = out.view(torch.float8_e4m3fn).double() * scale
        y = y.clamp(-448 * scale, 448 * scale)
        bound = y.abs() * 2.0 ** -4 + scale * 2.0 ** -10
    else:
        bound = y.abs() * (torch.finfo(dtype).eps / 2) + 2.0 ** -25
    bound = bound * (1 + 2.0 ** -20) + size * abs(factor) * 7e-7
    over = ((out.double() - y).abs() / bound).max().item()
    assert over <= 1, f"error is {over:.2f} of its bound"


def check(q, k, v, pos, axis, pools, slots, rot, adjacent, factor, q_out, scales=(1.0, 1.0),
          x0=None):
    dtype = q.dtype
    q0, k0, v0 = x0
    inv = pa.rope_inv_freq(rot)
    yq, sq = rotated(q0, pos, inv, axis, adjacent, factor)
    yk, sk = rotated(k0, pos, inv, axis, adjacent, factor)
    expect(q_out.cpu(), yq, sq, dtype, factor)
    nb, hkv, bs, d = pools[0].shape
    keep = (slots >= 0) & (slots < nb * bs)
    for pool, y, size, scale in ((pools[0], yk, sk, scales[0]),
                                 (pools[1], v0.double(), torch.zeros_like(sk), scales[1])):
        rows = pool.cpu().transpose(1, 2).reshape(nb * bs, hkv, d)
        expect(rows[slots[keep]], y[keep], size[keep], dtype, factor, scale)
        other = torch.ones(nb * bs, dtype=torch.bool)
        other[slots[keep]] = False
        left = rows[other]  # untouched: NaN, or the code of NaN
        assert (left == 0x7F).all() if left.dtype == torch.uint8 else left.isnan().all()


CASES = [
    # t, hq, hkv, d, rot, axes, dtype, pool, bs, adjacent, factor
    (1, 4, 2, 64, 64, 1, "f16", "f16", 16, False, 1.0),
    (5, 28, 4, 128, 128, 3, "bf16", "bf16", 16, False, 1.0),
    (33, 32, 8, 128, 64, 2, "f16", "f16", 32, True, 1.0),
    (33, 7, 1, 64, 16, 1, "bf16", "bf16", 32, False, 1.25),
    (1301, 8, 2, 128, 128, 3, "bf16", "bf16", 16, True, 1.0),
    (1303, 64, 8, 64, 32, 3, "f16", "f16", 16, False, 1.0),
    (1, 3, 1, 128, 128, 2, "f16", "e4m3", 16, False, 1.0),
    (70, 28, 4, 64, 64, 2, "f16", "e4m3", 32, True, 1.0),
    (1301, 9, 3, 128, 96, 3, "f16", "e4m3", 16, False, 0.5),
]
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.mark.parametrize("fused", [True, False], ids=["fused", "separate"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_matches_the_formula(case, fused):
    t, hq, hkv, d, rot, axes, dt, pool, bs, adjacent, factor = case
    q, k, v, pos, axis, pools, slots = make(t, hq, hkv, d, rot, axes, TYPES[dt], pool, bs,
                                            t + hq + d, fused=fused)
    x0 = [x.cpu() for x in (q, k, v)]
    scales = (0.0625, 0.03125) if pool == "e4m3" else (None, None)
    out = pa.rope_and_cache(q, k, v, pos.cuda(), pa.rope_inv_freq(rot), *pools, slots.cuda(),
                            axes=axis, adjacent=adjacent, factor=factor, k_scale=scales[0],
                            v_scale=scales[1])
    assert pa.get_device_error() == (0, 0)
    for x, y in zip((q, k, v), x0):
        assert torch.equal(x.cpu(), y)  # the inputs stay
    check(q, k, v, pos, axis, pools, slots, rot, adjacent, factor, out,
          scales if pool == "e4m3" else (1.0, 1.0), x0)


@pytest.mark.parametrize("adjacent", [False, True])
def test_in_place_inside_a_fused_projection(adjacent):
    q, k, v, pos, axis, pools, slots = make(19, 8, 2, 128, 128, 2, torch.bfloat16, "bf16", 16, 3)
    x0 = [x.cpu() for x in (q, k, v)]
    out = pa.rope_and_cache(q, k, v, pos.cuda(), pa.rope_inv_freq(128), *pools, slots.cuda(),
                            q_out=q, axes=axis, adjacent=adjacent)
    assert out is q
    check(q, k, v, pos, axis, pools, slots, 128, adjacent, 1.0, q, x0=x0)
    assert torch.equal(k.cpu(), x0[1]) and torch.equal(v.cpu(), x0[2])


def test_far_and_negative_positions():
    """Exact turns: position 2^31 - 1 and its negative are as good as position 1."""
    q, k, v, _, axis, pools, slots = make(6, 4, 2, 64, 64, 1, torch.float16, "f16", 16, 4)
    pos = torch.tensor([[0, 1, 2 ** 31 - 1, -(2 ** 31 - 1), 1_000_003, -7]])
    x0 = [x.cpu() for x in (q, k, v)]
    # float64 angles are off by 2^-22 rad at 2^31: take the reference's turn from exact integers
    inv = pa.rope_inv_freq(64)
    out = pa.rope_and_cache(q, k, v, pos[0].cuda(), inv, *pools, slots.cuda())
    from fractions import Fraction
    import math
    pi = Fraction(314159265358979323846264338327950288, 10 ** 35)
    theta = torch.tensor([[float((Fraction(int(p)) * Fraction(float(f))) % (2 * pi)) for f in inv]
                          for p in pos[0]], dtype=torch.float64)
    assert math.pi == float(pi)
    c, s = theta.cos()[:, None], theta.sin()[:, None]
    a, b = x0[0].double()[..., :32], x0[0].double()[..., 32:]
    y = torch.cat((a * c - b * s, b * c + a * s), -1)
    size = (a.abs() + b.abs()).repeat(1, 1, 2)
    # f / 2 pi is a float64: 2^-52 of a turn's fraction per position, 2^31 of them: 2 pi 2^-21
    far = (pos[0].abs().double() * 2.0 ** -52 * 2 * math.pi)[:, None, None]
    bound = y.abs() * 2.0 ** -11 + 2.0 ** -25 + size * (7e-7 + far)
    assert ((out.cpu().double() - y).abs() <= bound).all()


def test_slots_past_the_pool_are_reported_and_q_is_rotated():
    q, k, v, pos, axis, pools, slots = make(9, 4, 2, 64, 64, 1, torch.float16, "f16", 16, 6)
    slots[4] = pools[0].shape[0] * 16
    x0 = [x.cpu() for x in (q, k, v)]
    out = pa.rope_and_cache(q, k, v, pos.cuda(), pa.rope_inv_freq(64), *pools, slots.cuda(),
                            axes=axis)
    st, bits = pa.get_device_error()
    assert st == B.PA_ERR_OUT_OF_RANGE and bits & 2
    check(q, k, v, pos, axis, pools, slots, 64, False, 1.0, out, x0=x0)


def test_nan_and_infinity_stay_in_their_pairs():
    q, k, v, pos, axis, pools, slots = make(2, 2, 2, 64, 32, 1, torch.bfloat16, "bf16", 16, 7)
    q[0, 0, 3] = float("nan")
    q[1, 1, 40] = float("inf")
    out = pa.rope_and_cache(q, k, v, pos.cuda(), pa.rope_inv_freq(32), *pools, slots.cuda(),
                            axes=axis).cpu()
    lost = ~torch.isfinite(out)
    assert lost.nonzero().tolist() == [[0, 0, 3], [0, 0, 19], [1, 1, 40]]
    assert out[1, 1, 40] == float("inf")


def test_replays_in_a_graph():
    q, k, v, pos, axis, pools, slots = make(12, 4, 2, 128, 128, 3, torch.float16, "f16", 16, 8)
    inv, dpos, dslots = pa.rope_inv_freq(128), pos.cuda(), slots.cuda()
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    call = lambda: pa.rope_and_cache(q, k, v, dpos, inv, *pools, dslots, q_out=out, axes=axis)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    del inv  # the captured launch holds the frequencies itself
    pos = pos + 100
    dpos.copy_(pos)
    out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    check(q, k, v, pos, axis, pools, slots, 128, False, 1.0, out,
          x0=[x.cpu() for x in (q, k, v)])
