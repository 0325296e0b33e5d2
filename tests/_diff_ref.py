"""Differential attention in float64 from contiguous K/V, with a rigorous bound of what the
kernels' float32 arithmetic and their roundings may change (both per output value).

Sources of error, with u = torch.finfo(dtype).eps / 2 the element type's half step:
* each softmax weight is rounded to the element type for the P V product: u of each weight;
* a score is a float32 sum of d products: at most d 2^-23 of the sum of their magnitudes
  (truncating adders included), S; it changes a weight by S scale and the sum l by the same;
  2^x and the running sums add 2^-20 at most;
* so a map's result is off by at most (u + 2 S scale + 2^-20) A, A = softmax(...) |V|, and
  y = o1 - lambda o2 by E = e1 + |lambda| e2;
* the norm's 1/rms moves by ||E|| / ||y|| relative (both sides of the quotient, doubled for second
  order terms); the output is rounded once, u of it, or 2^-25 near fp16's zero.
"""
import torch


def diff_attention_ref(b, lam, weight=None, eps=1e-5, gain=1.0, rows_of=None):
    """(out, bound), float64 [T, Hq / 2, 2 d], of a PagedBatch (its contiguous K/V)."""
    q, k, v = b.q.double(), b.k_contig.double(), b.v_contig.double()
    hq, hkv, d = b.num_q_heads, b.num_kv_heads, b.head_dim
    g, t = hq // hkv, q.shape[0]
    u = torch.finfo(b.q.dtype).eps / 2
    out = torch.full((t, hq // 2, 2 * d), float("nan"), dtype=torch.float64)
    err = torch.full_like(out, float("nan"))
    lam = lam.double().expand(t, hq // 2) if lam.dim() == 1 else lam.double()
    for s in range(b.num_seqs):
        n, base = int(b.seq_lens[s]), int(b.kv_start[s])
        r0, r1 = int(b.query_start_loc[s]), int(b.query_start_loc[s + 1])
        if r0 == r1 or (rows_of is not None and s not in rows_of):
            continue
        see = torch.arange(n) <= (n - (r1 - r0) + torch.arange(r1 - r0))[:, None]
        for p in range(hq // 2):
            j = p // g
            val = torch.cat((v[base:base + n, 2 * j], v[base:base + n, 2 * j + 1]), 1)
            o, e = [], []
            for m in range(2):
                qq, kk = q[r0:r1, 2 * p + m], k[base:base + n, 2 * j + m]
                z = (qq @ kk.T) * b.scale
                size = (qq.abs() @ kk.abs().T).masked_fill(~see, 0).amax(1, keepdim=True)
                w = torch.softmax(z.masked_fill(~see, -float("inf")), 1)
                o.append(w @ val)
                e.append((w @ val.abs()) *
                         (u + 2 * d * 2.0 ** -23 * size * abs(b.scale) + 2.0 ** -20))
            la = lam[r0:r1, p:p + 1]
            y, E = o[0] - la * o[1], e[0] + la.abs() * e[1]
            if weight is not None:
                rms = (y.square().mean(1, keepdim=True) + eps).sqrt()
                rel = E.norm(dim=1, keepdim=True) / (rms * (2 * d) ** 0.5)
                z = y / rms * weight.double() * gain
                E = (E / rms * weight.double().abs() * abs(gain)) * (1 + 2 * rel) + 2 * rel * z.abs()
            else:
                z, E = y * gain, E * abs(gain)
            out[r0:r1, p] = z
            err[r0:r1, p] = E + (z.abs() + E) * u + z.abs() * 2.0 ** -20 + 2.0 ** -25
    return out, err
