"""Cases of three operators of the paged-attention library, with their plain forms.

rope   rotary positions with one to three axes, and the step's K/V written into their pages
diff   differential attention over the pages: the difference of two softmax maps of a head pair
move   pages moved inside the pool (compaction), with the block tables renumbered

``own`` false: elementary torch operations in float32 (angles in float64); ``own`` true: the
library's calls.
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.uint8}


def listed():
    return [
        # one decode step of 64 sequences deep in their contexts: latency
        {"name": "rope_decode_64", "op": "rope", "tokens": 64, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "axes": 1, "adjacent": False, "dtype": "bf16", "pool": "bf16", "bs": 16},
        # a video or image prompt: one large chunk, time/height/width axes
        {"name": "rope_video_8192", "op": "rope", "tokens": 8192, "hq": 64, "hkv": 8, "d": 128,
         "rot": 128, "axes": 3, "adjacent": False, "dtype": "bf16", "pool": "bf16", "bs": 16},
        # an odd chunk into an FP8 cache, height/width axes on half of each head
        {"name": "rope_fp8_1037", "op": "rope", "tokens": 1037, "hq": 28, "hkv": 4, "d": 64,
         "rot": 32, "axes": 2, "adjacent": True, "dtype": "f16", "pool": "e4m3", "bs": 32},
        # the smallest serving step: four short conversations
        {"name": "diff_decode_tiny", "op": "diff", "decode": 4, "dlo": 1, "dhi": 64, "chunks": 0,
         "rows": 0, "clo": 0, "chi": 0, "hq": 4, "hkv": 2, "d": 64, "dtype": "f16", "bs": 16,
         "norm": True},
        # 64 conversations of ragged length, one token each
        {"name": "diff_decode_ragged_64", "op": "diff", "decode": 64, "dlo": 512, "dhi": 4096,
         "chunks": 0, "rows": 0, "clo": 0, "chi": 0, "hq": 32, "hkv": 8, "d": 128,
         "dtype": "bf16", "bs": 32, "norm": True},
        # 32 sessions of 8k tokens, one token each: the cache streams once
        {"name": "diff_decode_32x8k", "op": "diff", "decode": 32, "dlo": 8192, "dhi": 8192,
         "chunks": 0, "rows": 0, "clo": 0, "chi": 0, "hq": 64, "hkv": 8, "d": 128,
         "dtype": "f16", "bs": 16, "norm": True},
        # four prompts' 512-token chunks over their earlier context
        {"name": "diff_chunk_4x512", "op": "diff", "decode": 0, "dlo": 0, "dhi": 0, "chunks": 4,
         "rows": 512, "clo": 0, "chi": 7488, "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16",
         "bs": 16, "norm": True},
        # one whole prompt of an odd length, small heads
        {"name": "diff_prompt_4001_d64", "op": "diff", "decode": 0, "dlo": 0, "dhi": 0,
         "chunks": 1, "rows": 4001, "clo": 0, "chi": 0, "hq": 32, "hkv": 8, "d": 64,
         "dtype": "f16", "bs": 16, "norm": False},
        # continuous batching: two chunks beside 64 decode rows
        {"name": "diff_mixed_2x512_64", "op": "diff", "decode": 64, "dlo": 256, "dhi": 8000,
         "chunks": 2, "rows": 512, "clo": 0, "chi": 7488, "hq": 32, "hkv": 8, "d": 128,
         "dtype": "f16", "bs": 16, "norm": True},
        # a few holes filled in one layer's pool after a request ended: latency
        {"name": "move_holes_48", "op": "move", "layers": 1, "blocks": 512, "moves": 48,
         "permute": False, "hkv": 8, "d": 128, "dtype": "bf16", "bs": 16, "seqs": 16},
        # a fragmented pool of eight layers put in sequence order: chains and cycles of moves
        {"name": "move_order_8x4096", "op": "move", "layers": 8, "blocks": 4096, "moves": 4096,
         "permute": True, "hkv": 8, "d": 128, "dtype": "f16", "bs": 16, "seqs": 64},
        # holes of an FP8 pool filled, an odd number of them
        {"name": "move_holes_fp8_1501", "op": "move", "layers": 4, "blocks": 6000, "moves": 1501,
         "permute": False, "hkv": 4, "d": 128, "dtype": "e4m3", "bs": 32, "seqs": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "diff", "diff", "move"))
    hq, hkv = rng.choice(((32, 8), (64, 8), (28, 4), (4, 2), (16, 8), (24, 2)))
    bs = rng.choice((16, 32))
    if op == "rope":
        d = rng.choice((64, 128))
        pool = rng.choice(("f16", "bf16", "e4m3"))
        return {"op": op, "tokens": _log(rng, 1, 8192), "hq": hq, "hkv": hkv, "d": d,
                "rot": rng.choice((d, d, d // 2, 16)), "axes": rng.choice((1, 2, 3)),
                "adjacent": rng.random() < 0.4, "dtype": "bf16" if pool == "bf16" else "f16",
                "pool": pool, "bs": bs}
    if op == "diff":
        d = rng.choice((64, 128))
        hq = min(hq, 32)
        kind = rng.choice(("decode", "decode", "chunk", "mixed"))
        decode = _log(rng, 1, 64) if kind != "chunk" else 0
        top = _log(rng, 2, 4096)
        chunks = 0 if kind == "decode" else rng.randint(1, 2)
        ctx = rng.choice((0, _log(rng, 1, 4000))) if chunks else 0
        return {"op": op, "decode": decode, "dlo": max(1, top // 4) if decode else 0,
                "dhi": top if decode else 0, "chunks": chunks,
                "rows": _log(rng, 2, 700) if chunks else 0, "clo": ctx // 2, "chi": ctx,
                "hq": hq, "hkv": hkv, "d": d, "dtype": rng.choice(("f16", "bf16")), "bs": bs,
                "norm": rng.random() < 0.7}
    blocks = _log(rng, 64, 4000)
    permute = rng.random() < 0.5
    return {"op": op, "layers": rng.choice((1, 2, 5)), "blocks": blocks,
            "moves": blocks if permute else rng.randint(1, blocks // 2), "permute": permute,
            "hkv": hkv, "d": rng.choice((64, 128)), "dtype": rng.choice(("f16", "bf16", "e4m3")),
            "bs": bs, "seqs": rng.randint(1, 32)}


def _lengths(case):
    """Row count and key count of every sequence; the same for every seed, as work() needs."""
    g = torch.Generator().manual_seed(case["decode"] * 1009 + case["chunks"] * 31 + case["rows"])
    dec = torch.randint(case["dlo"], case["dhi"] + 1, (case["decode"],), generator=g)
    ctx = torch.randint(case["clo"], case["chi"] + 1, (case["chunks"],), generator=g)
    rows = torch.full((case["chunks"],), case["rows"], dtype=torch.int64)
    return rows, rows + ctx, torch.ones_like(dec), dec


def _random(shape, dtype, g):
    if dtype == torch.uint8:  # E4M3 codes of ordinary values
        x = torch.randn(shape, generator=g, device="cuda")
        return x.to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _inv_freq(rot):
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def _axis_of_pair(pairs, axes):
    """Sections of the pairs, time first: a quarter for time where there are three axes."""
    cut = {1: [pairs], 2: [pairs // 2, pairs - pairs // 2],
           3: [pairs // 4, (pairs - pairs // 4) // 2,
               pairs - pairs // 4 - (pairs - pairs // 4) // 2]}[axes]
    return torch.repeat_interleave(torch.arange(axes, dtype=torch.int32), torch.tensor(cut))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"rope": _prepare_rope, "diff": _prepare_diff, "move": _prepare_move}[case["op"]](case, g)


def _prepare_rope(c, g):
    t, hq, hkv, d, bs = c["tokens"], c["hq"], c["hkv"], c["d"], c["bs"]
    dt, pool = TYPES[c["dtype"]], TYPES[c["pool"]]
    qkv = _random((t, (hq + 2 * hkv) * d), dt, g)  # one projection's output: strided slices
    nb = -(-t // bs) + 8
    slots = torch.randperm(nb * bs, generator=g, device="cuda")[:t]
    slots[torch.rand(t, generator=g, device="cuda") < 0.01] = -1  # padding rows of the batch
    # text far into a context, or a video's grid of patches after it
    base = torch.randint(0, 100000, (1,), generator=g, device="cuda")
    i = torch.arange(t, device="cuda")
    grid = torch.stack((i // 1024, i // 32 % 32, i % 32)) if c["axes"] > 1 else i[None]
    pool_shape = (nb, hkv, bs, d)
    return {"op": "rope", "q": qkv[:, :hq * d].view(t, hq, d),
            "k": qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d),
            "v": qkv[:, (hq + hkv) * d:].view(t, hkv, d),
            "positions": (base + grid[3 - c["axes"] if c["axes"] > 1 else 0:]).contiguous(),
            "inv_freq": _inv_freq(c["rot"]), "axes": _axis_of_pair(c["rot"] // 2, c["axes"]),
            "adjacent": c["adjacent"], "slots": slots, "k_scale": 0.03125, "v_scale": 0.015625,
            "k_cache": _random(pool_shape, pool, g), "v_cache": _random(pool_shape, pool, g),
            "q_out": torch.empty((t, hq, d), dtype=dt, device="cuda")}


def _prepare_diff(c, g):
    hq, hkv, d, bs, dt = c["hq"], c["hkv"], c["d"], c["bs"], TYPES[c["dtype"]]
    crow, clen, drow, dlen = _lengths(c)
    rows, lens = torch.cat((crow, drow)), torch.cat((clen, dlen))
    start = torch.cat((torch.zeros(1, dtype=torch.int64), rows.cumsum(0)))
    t, n = int(start[-1]), len(rows)
    blocks = -(-lens // bs)
    mb, used = int(blocks.max()), int(blocks.sum())
    nb = used + used // 10 + 1
    perm = torch.randperm(nb, generator=g, device="cuda")
    first = blocks.cumsum(0) - blocks
    col = torch.arange(mb)
    at = torch.where(col < blocks[:, None], first[:, None] + col, used)
    tables = perm[at.cuda()].to(torch.int32)

    def group(lo, hi):  # the rows of sequences lo .. hi - 1 as a padded [sequence, row] block
        if lo == hi:
            return None
        r = torch.arange(int(rows[lo:hi].max()))
        real = r < rows[lo:hi, None]
        idx = torch.where(real, start[lo:hi, None] + r, start[lo:hi, None])
        pos = lens[lo:hi, None] - rows[lo:hi, None] + torch.where(real, r, 0)
        w = int(blocks[lo:hi].max())
        return {"rows": idx.cuda(), "real": real.flatten().nonzero()[:, 0].cuda(),
                "pos": pos.cuda(), "tables": tables[lo:hi, :w].long()}

    nc = c["chunks"]
    pool = (nb, hkv, bs, d)
    lam = 0.8 - 0.6 * math.exp(-0.3 * 12) + 0.1 * torch.randn(hq // 2, generator=g, device="cuda")
    return {"op": "diff", "q": _random((t, hq, d), dt, g), "k_cache": _random(pool, dt, g),
            "v_cache": _random(pool, dt, g), "tables": tables,
            "lens": lens.to(torch.int32).cuda(), "start": start.to(torch.int32).cuda(),
            "scale": d ** -0.5, "lam": lam,
            "weight": 1 + 0.1 * torch.randn(2 * d, generator=g, device="cuda") if c["norm"] else None,
            "eps": 1e-5, "gain": 0.2 if c["norm"] else 1.0,
            "out": torch.empty((t, hq // 2, 2 * d), dtype=dt, device="cuda"),
            "max_rows": int(rows.max()), "max_len": int(lens.max()), "chunks": int((rows > 1).sum()),
            "groups": [x for x in (group(0, nc), group(nc, n)) if x is not None],
            "rows_of": rows, "lens_of": lens}


def _prepare_move(c, g):
    nb, m, dt = c["blocks"], c["moves"], TYPES[c["dtype"]]
    shape = (c["layers"], nb, c["hkv"], c["bs"], c["d"])
    if c["permute"]:  # every page to the place that its sequence's order gives it
        src, dst = torch.randperm(nb, generator=g, device="cuda"), torch.arange(nb, device="cuda")
    else:  # pages behind the pool's kept part into the holes in front
        keep = nb - m
        src = keep + torch.randperm(m, generator=g, device="cuda")
        dst = torch.randperm(keep, generator=g, device="cuda")[:m]
    per = nb // c["seqs"]
    tables = torch.randperm(nb, generator=g, device="cuda")[:per * c["seqs"]]
    return {"op": "move", "k_cache": _random(shape, dt, g), "v_cache": _random(shape, dt, g),
            "pairs": torch.stack((src, dst), 1).to(torch.int32).cpu(),
            "tables": tables.view(c["seqs"], per).to(torch.int32)}


def run(state):
    return {"rope": _run_rope, "diff": _run_diff, "move": _run_move}[state["op"]](state)


def _values(pool):
    return pool.view(torch.float8_e4m3fn) if pool.dtype == torch.uint8 else pool


def _run_rope(s):
    if own:
        import paged_kv_cache_290_gb300 as pa
        fp8 = s["k_cache"].dtype == torch.uint8
        pa.rope_and_cache(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["k_cache"],
                          s["v_cache"], s["slots"], s["q_out"], axes=s["axes"],
                          adjacent=s["adjacent"], k_scale=s["k_scale"] if fp8 else None,
                          v_scale=s["v_scale"] if fp8 else None)
    else:
        angle = s["positions"][s["axes"].cuda().long()].T.double() * s["inv_freq"].cuda()
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
        q, k = (_rotated(s[x].float(), cos, sin, s["adjacent"]) for x in ("q", "k"))
        s["q_out"].copy_(q)
        _stored(s["k_cache"], k, s["slots"], s["k_scale"])
        _stored(s["v_cache"], s["v"].float(), s["slots"], s["v_scale"])
    return {"q": s["q_out"], "k": _values(s["k_cache"]), "v": _values(s["v_cache"])}


def _rotated(x, cos, sin, adjacent):
    half = cos.shape[-1]
    x, rest = x[..., :2 * half], x[..., 2 * half:]
    if adjacent:
        a, b = x[..., 0::2], x[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, rest), -1)


def _stored(pool, x, slots, scale):
    bs = pool.shape[2]
    if pool.dtype == torch.uint8:
        x = (x * (1.0 / scale)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    real = slots >= 0
    slots = slots[real]
    pool[slots // bs, :, slots % bs] = x[real].to(pool.dtype)


def _run_diff(s):
    if own:
        import paged_kv_cache_290_gb300 as pa
        return pa.diff_attention(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"],
                                 s["start"], s["scale"], s["lam"], s["out"], s["max_rows"],
                                 s["max_len"], norm_weight=s["weight"], eps=s["eps"],
                                 out_scale=s["gain"], num_prefill_seqs=s["chunks"])
    t = s["q"].shape[0]
    flat = s["out"].view(t, -1)
    for x in s["groups"]:  # chunk rows, then decode rows
        y = _difference(s, x)
        flat[x["rows"].flatten()[x["real"]]] = y.flatten(0, 1)[x["real"]].flatten(1).to(flat.dtype)
    return s["out"]


def _difference(s, x):
    hkv, bs, d = s["k_cache"].shape[1:]
    n, r = x["rows"].shape
    hq = s["q"].shape[1]
    gq = hq // hkv
    keys = lambda pool: pool[x["tables"]].transpose(1, 2).reshape(n, hkv, -1, d).float()  # noqa: E731
    k, v = keys(s["k_cache"]), keys(s["v_cache"])
    v = v.view(n, hkv // 2, 2, -1, d).transpose(2, 3).flatten(3)  # [n, pair, key, 2d]
    q = s["q"][x["rows"]].float().view(n, r, hkv // 2, gq, 2, d)
    q = q.permute(0, 2, 4, 3, 1, 5).reshape(n, hkv, gq * r, d)  # kv head = 2 pair + map
    p = q @ k.transpose(-1, -2) * s["scale"]
    p = p.view(n, hkv, gq, r, -1)
    later = torch.arange(k.shape[2], device="cuda") > x["pos"][:, None, None, :, None]
    p = p.masked_fill(later, -math.inf)
    p = (p - p.amax(-1, keepdim=True)).exp()
    p = p / p.sum(-1, keepdim=True)
    o = p.view(n, hkv // 2, 2 * gq * r, -1) @ v
    o = o.view(n, hkv // 2, 2, gq, r, 2 * d)
    lam = s["lam"].view(hkv // 2, gq, 1, 1)
    y = (o[:, :, 0] - lam * o[:, :, 1]).permute(0, 3, 1, 2, 4).reshape(n, r, hq // 2, 2 * d)
    if s["weight"] is not None:
        y = y * (y.square().mean(-1, keepdim=True) + s["eps"]).rsqrt() * s["weight"]
    return y * s["gain"]


def _run_move(s):
    if own:
        import paged_kv_cache_290_gb300 as pa
        pa.move_blocks(s["k_cache"], s["v_cache"], s["pairs"], block_tables=s["tables"])
    else:
        src, dst = s["pairs"].cuda().long().unbind(1)
        s["k_cache"][:, dst] = s["k_cache"][:, src]
        s["v_cache"][:, dst] = s["v_cache"][:, src]
        new = torch.arange(s["k_cache"].shape[1], device="cuda", dtype=torch.int32)
        new[src] = dst.to(torch.int32)
        s["tables"].copy_(new[s["tables"].long()])
    return {"k": _values(s["k_cache"]), "v": _values(s["v_cache"]), "tables": s["tables"]}


def work(case):
    c = case
    if c["op"] == "rope":
        t, d, page = c["tokens"], c["d"], 1 if c["pool"] == "e4m3" else 2
        heads = c["hq"] + 2 * c["hkv"]
        return {"bytes": t * (heads * d * 2 + c["hq"] * d * 2 + 2 * c["hkv"] * d * page +
                              8 * c["axes"] + 8),
                "flops": t * (c["hq"] + c["hkv"]) * c["rot"] * 3}
    if c["op"] == "diff":
        crow, clen, drow, dlen = _lengths(c)
        rows, lens = torch.cat((crow, drow)), torch.cat((clen, dlen))
        seen = (rows * lens - rows * (rows - 1) // 2).sum()  # keys seen, over all rows
        kv = int(lens.sum()) * 2 * c["hkv"] * c["d"] * 2
        return {"bytes": kv + int(rows.sum()) * c["hq"] * c["d"] * 4 + 4 * int((-(-lens // c["bs"])).sum()),
                "flops": int(seen) * c["hq"] * 6 * c["d"]}
    page = 2 * c["hkv"] * c["bs"] * c["d"] * (1 if c["dtype"] == "e4m3" else 2)
    return {"bytes": 2 * c["layers"] * c["moves"] * page + 8 * c["blocks"], "flops": 0}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "diff": _exact_diff, "move": _exact_move}[case["op"]](s)


def _exact_rope(s):
    """Each pair as a complex number times factor * e^(i theta)."""
    f = s["inv_freq"].cuda()
    turn = torch.polar(torch.ones_like(f),
                       s["positions"].double().index_select(0, s["axes"].cuda()).t() * f)
    n = 2 * f.numel()

    def rotate(x):
        y = x.double().clone()
        z = torch.complex(y[..., 0:n:2], y[..., 1:n:2]) if s["adjacent"] else torch.complex(
            y[..., :n // 2], y[..., n // 2:n])
        z = z * turn.unsqueeze(1)
        if s["adjacent"]:
            y[..., 0:n:2], y[..., 1:n:2] = z.real, z.imag
        else:
            y[..., :n // 2], y[..., n // 2:n] = z.real, z.imag
        return y

    def pages(pool, x, scale):
        p = _values(pool).double().transpose(1, 2).flatten(0, 1).clone()  # [slot, head, d]
        keep = (s["slots"] >= 0).nonzero()[:, 0]
        fp8 = pool.dtype == torch.uint8
        p[s["slots"][keep]] = (x[keep] / scale).clamp(-448, 448) if fp8 else x[keep]
        nb, h, bs, d = pool.shape
        return p.view(nb, bs, h, d).transpose(1, 2).contiguous()

    return {"q": rotate(s["q"]), "k": pages(s["k_cache"], rotate(s["k"]), s["k_scale"]),
            "v": pages(s["v_cache"], s["v"].double(), s["v_scale"])}


def _exact_diff(s):
    """Sequence by sequence and head pair by head pair, from its own keys alone."""
    hq, hkv, bs, d = s["q"].shape[1], *s["k_cache"].shape[1:]
    out = torch.zeros_like(s["out"], dtype=torch.float64)
    row = 0
    for i, (r, n) in enumerate(zip(s["rows_of"].tolist(), s["lens_of"].tolist())):
        b = s["tables"][i, :-(-n // bs)].long()
        hidden = torch.ones(r, n, dtype=torch.bool, device="cuda").triu(n - r + 1)
        for j in range(hkv // 2):
            k1, k2, va, vb = (c[b, 2 * j + h].flatten(0, 1)[:n].double() for c, h in (
                (s["k_cache"], 0), (s["k_cache"], 1), (s["v_cache"], 0), (s["v_cache"], 1)))
            v = torch.cat((va, vb), 1)
            for p in range(j * hq // hkv, (j + 1) * hq // hkv):
                maps = []
                for m, k in ((0, k1), (1, k2)):
                    z = s["q"][row:row + r, 2 * p + m].double() @ k.T * s["scale"]
                    z[hidden] = -math.inf
                    maps.append(torch.softmax(z, 1))
                y = (maps[0] - s["lam"][p].double() * maps[1]) @ v
                if s["weight"] is not None:
                    y = y / (y.pow(2).mean(1, keepdim=True) + s["eps"]).sqrt() * s["weight"].double()
                out[row:row + r, p] = y * s["gain"]
        row += r
    return out


def _exact_move(s):
    """Where each place's page comes from, read off the list of moves."""
    nb = s["k_cache"].shape[1]
    came, went = list(range(nb)), list(range(nb))
    for a, b in s["pairs"].tolist():
        came[b], went[a] = a, b
    came, went = torch.tensor(came, device="cuda"), torch.tensor(went, device="cuda")
    pages = lambda pool: _values(pool.index_select(1, came))  # noqa: E731
    return {"k": pages(s["k_cache"]), "v": pages(s["v_cache"]),
            "tables": went.index_select(0, s["tables"].flatten().long()).view_as(s["tables"]).int()}
