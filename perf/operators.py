"""The operators around the 4-bit KV cache, with the sizes they are measured at.

Four operators of one attention layer: the norms of queries and keys with the
position rotation (``qk_norm_rope``), quantising K and V to 4 bits as they are
written to the paged cache and reading them back (``fp4_kv_write``,
``fp4_kv_read``), and attention over that cache (``fp4_kv_attention``).

Each is here twice: as the framework's call (``own`` true) and in its plain
form, elementary torch operations in fp32 with rounding at the end.  ``exact``
restates the definitions in 64 bits.

The cache.  A value is code * block scale * tensor scale: an E2M1 code (bit 3
the sign, then 0, .5, 1, 1.5, 2, 3, 4, 6), an E4M3 scale per 16 neighbouring
dimensions of one token's head, and an fp32 scale per tensor.  A pool is
uint8 [num_blocks, heads, block_size / 16, 9 * dim]: the last axis is a tile of
16 tokens, 8 * dim bytes of codes (two to a byte, the even dimension low) and
then dim bytes of scales.  K tiles are token-major, V tiles block-major:
    K codes [16 tokens][dim / 2]           K scales [16 tokens][dim / 16]
    V codes [dim / 16][16 tokens][8]       V scales [dim / 16][16 tokens]
"""
import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases


def listed():
    """4 x 128 KV heads and 16-slot blocks are this repository's workloads; 32
    query heads and 4 + 4 KV heads of 128 make a fused projection of 5120."""
    return [
        # one small write of the size of a decode batch, read back: latency
        dict(name="cache_16", kind="cache", tokens=16, heads=4, dim=128, block=16, blocks=64,
             q_heads=32, skipped=2, scales="host", shape_seed=1),
        # a prompt of 4593 tokens into one layer's pool, and back
        dict(name="cache_4593", kind="cache", tokens=4593, heads=4, dim=128, block=16, blocks=8192,
             q_heads=32, skipped=0, scales="device", shape_seed=2),
        # a long cached prefix fetched as bf16, 64-wide heads, 64-slot blocks
        dict(name="read_60001", kind="read", tokens=60001, heads=8, dim=64, block=64, blocks=1200,
             skipped=7, scales="host", shape_seed=3),
        # one user, a short answer: latency
        dict(name="attend_1x517", kind="attend", batch=1, len_lo=517, len_hi=517, q_lo=1, q_hi=1,
             q_heads=32, heads=4, dim=128, block=16, window=0, scales="host", shape_seed=4),
        # a decode batch of uneven histories
        dict(name="attend_64xragged", kind="attend", batch=64, len_lo=1, len_hi=8192, q_lo=1,
             q_hi=1, q_heads=32, heads=4, dim=128, block=16, window=0, scales="device",
             shape_seed=5),
        # one user with a very long document: the long axis has to be split
        dict(name="attend_1x200003", kind="attend", batch=1, len_lo=200003, len_hi=200003, q_lo=1,
             q_hi=1, q_heads=32, heads=4, dim=128, block=16, window=0, scales="host",
             shape_seed=6),
        # a full decode batch: the largest read of the cache
        dict(name="attend_256x4500", kind="attend", batch=256, len_lo=3001, len_hi=6000, q_lo=1,
             q_hi=1, q_heads=32, heads=4, dim=128, block=16, window=0, scales="device",
             shape_seed=7),
        # drafted tokens checked several at a time, five query heads to a KV head
        dict(name="attend_32xdraft", kind="attend", batch=32, len_lo=100, len_hi=4000, q_lo=1,
             q_hi=8, q_heads=40, heads=8, dim=128, block=32, window=0, scales="host",
             shape_seed=8),
        # pieces of prompts against what is cached, sliding window, 64-wide heads,
        # six query heads to a KV head
        dict(name="attend_4xchunk", kind="attend", batch=4, len_lo=2000, len_hi=4001, q_lo=200,
             q_hi=500, q_heads=48, heads=8, dim=64, block=64, window=1024, scales="host",
             shape_seed=9),
        # one decode step of a small batch: latency
        dict(name="rope_16", kind="rope", tokens=16, q_heads=32, heads=4, dim=128, rotary=128,
             interleaved=False, norm=True, start=4000, spread=1, stretch=1.0, shape_seed=10),
        # the same prompt of 4593 tokens
        dict(name="rope_4593", kind="rope", tokens=4593, q_heads=32, heads=4, dim=128, rotary=128,
             interleaved=False, norm=True, start=0, spread=0, stretch=1.0, shape_seed=11),
        # far positions, a quarter of a wide head rotated, neighbours as pairs, no norm
        dict(name="rope_far_1501", kind="rope", tokens=1501, q_heads=16, heads=2, dim=256,
             rotary=64, interleaved=True, norm=False, start=900000, spread=1, stretch=8.0,
             shape_seed=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    kind = rng.choice(("cache", "read", "attend", "attend", "attend", "rope"))
    seed = rng.randrange(1 << 30)
    if kind in ("cache", "read"):
        heads, dim, block = rng.choice((1, 2, 4, 8)), rng.choice((64, 128, 256)), rng.choice((16, 32, 64, 128))
        tokens = _log(rng, 1, min(8192 if kind == "cache" else 60000, 60000 * 512 // (heads * dim)))
        blocks = -(-tokens // block) + rng.randrange(1, 40)
        case = dict(kind=kind, tokens=tokens, heads=heads, dim=dim, block=block, blocks=blocks,
                    skipped=rng.choice((0, tokens // 9)), scales=rng.choice(("host", "device")),
                    shape_seed=seed)
        if kind == "cache":
            case["q_heads"] = heads * rng.choice((1, 4, 8))
        return case
    if kind == "rope":
        heads, dim = rng.choice((1, 2, 4, 8)), rng.choice((64, 128, 256))
        return dict(kind=kind, tokens=_log(rng, 1, 8192 * 512 // (heads * dim) // 2), heads=heads,
                    q_heads=heads * rng.choice((1, 4, 5, 8)), dim=dim,
                    rotary=rng.choice((dim, dim // 2, dim // 4)), interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.7, start=_log(rng, 1, 1000000), spread=rng.choice((0, 1)),
                    stretch=rng.choice((1.0, 4.0, 32.0)), shape_seed=seed)
    heads, dim = rng.choice((1, 2, 4, 8)), rng.choice((64, 128, 128, 256))
    group = rng.choice((1, 2, 4, 5, 6, 8, 12, 16))
    batch = _log(rng, 1, 200)
    hi = _log(rng, 16, max(16, min(131072, 400000 * 512 // (heads * dim) // batch)))
    lo = rng.choice((1, hi, max(1, hi // 3)))
    q_hi = rng.choice((1, 1, 1, 4, 16, 200))
    while q_hi > 1 and 4 * batch * q_hi * heads * group * dim * hi > 18e9:
        q_hi //= 2
    return dict(kind=kind, batch=batch, len_lo=lo, len_hi=hi, q_lo=rng.choice((1, q_hi)), q_hi=q_hi,
                q_heads=heads * group, heads=heads, dim=dim, block=rng.choice((16, 32, 64, 128)),
                window=rng.choice((0, 0, 0, 100, 1024)), scales=rng.choice(("host", "device")),
                shape_seed=seed)


def _lengths(case):
    """Cached tokens and new queries of each sequence: part of the case, the
    same for every seed of the values."""
    rng = random.Random(case["shape_seed"])
    lens = [_log(rng, case["len_lo"], case["len_hi"]) if case["len_lo"] * 10 < case["len_hi"]
            else rng.randint(case["len_lo"], case["len_hi"]) for _ in range(case["batch"])]
    news = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    return lens, news


def _seen(length, new, window, i):
    """Cached tokens that query i of `new` sees."""
    last = length - new + i
    first = max(0, last - window + 1) if window else 0
    return max(0, last - first + 1), first


def work(case):
    row = case["heads"] * case["dim"]
    packed = row * 9 // 16                     # bytes of one token's K or V in the cache
    if case["kind"] in ("cache", "read"):
        live = case["tokens"] - case["skipped"]
        through = 2 if case["kind"] == "cache" else 1
        return dict(bytes=through * (8 * case["tokens"] + 2 * live * (2 * row + packed)),
                    flops=through * 2 * 2 * live * row)
    if case["kind"] == "rope":
        both = case["tokens"] * (case["q_heads"] + case["heads"]) * case["dim"]
        return dict(bytes=4 * both + 8 * case["tokens"] + 4 * case["rotary"] + 4 * case["dim"] * case["norm"],
                    flops=both * (7 if case["norm"] else 3))
    nbytes = flops = 0
    for length, new in zip(*_lengths(case)):
        seen = [_seen(length, new, case["window"], i) for i in range(new)]
        first = min([f for n, f in seen if n], default=length)
        nbytes += 2 * packed * (length - first) + 4 * -(-length // case["block"])
        nbytes += new * case["q_heads"] * (4 * case["dim"] + 4) + 8
        flops += 4 * case["q_heads"] * case["dim"] * sum(n for n, _ in seen)
    return dict(bytes=nbytes, flops=flops)


# ---------------------------------------------------------------------------
# the plain form: the cache


def _quantise(x, scale):
    """Codes (uint8, one to a byte) [..., dim] and E4M3 block scales [..., dim / 16]
    of x.  ``scale`` is a device value: a division by a host number would be a
    product with its reciprocal."""
    b = x.float().unflatten(-1, (-1, 16))
    six = torch.full((), 6.0, device=x.device)
    s = (b.abs().amax(-1) / six / scale).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = s.float() * scale
    r = torch.where(d > 0, 1.0 / d, torch.zeros_like(d))
    y = (b * r.unsqueeze(-1)).abs()
    code = (y > 0.25).to(torch.uint8)                    # ties go to the even code
    code += y >= 0.75
    code += y > 1.25
    code += y >= 1.75
    code += y > 2.5
    code += y >= 3.5
    code += y > 5.0
    code += torch.signbit(b) * 8
    return code.flatten(-2), s.view(torch.uint8)


def _pack(code):
    return code[..., 0::2] | code[..., 1::2] << 4


def _tiles(pool, kind):
    """(codes, scales) of a pool, as views with the token axis third from last
    for V's codes and second from last otherwise: K [nb, h, nt, 16, dim / 2],
    V [nb, h, nt, 16, dim / 16, 8], scales [nb, h, nt, 16, dim / 16]."""
    nb, h, nt, tile = pool.shape
    dim, at = tile // 9, list(pool.stride()[:3])
    first, off = pool.storage_offset(), pool.storage_offset() + 8 * (tile // 9)
    if kind == "k":
        return (pool.as_strided((nb, h, nt, 16, dim // 2), at + [dim // 2, 1], first),
                pool.as_strided((nb, h, nt, 16, dim // 16), at + [dim // 16, 1], off))
    return (pool.as_strided((nb, h, nt, 16, dim // 16, 8), at + [8, 128, 1], first),
            pool.as_strided((nb, h, nt, 16, dim // 16), at + [1, 16], off))


def _values(codes, scales, scale, table):
    """fp32 values [..., dim] of packed codes [..., dim / 2] and block scales."""
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).flatten(-2)
    s = scales.contiguous().view(torch.float8_e4m3fn).float()
    return (v.unflatten(-1, (-1, 16)) * s.unsqueeze(-1) * scale).flatten(-2)


def _place(slots, spare, block):
    """(block, tile, token) of each slot; skipped ones go to a spare block."""
    slots = torch.where(slots < 0, spare * block, slots)
    return slots // block, slots % block // 16, slots % 16


def _plain_write(x, at, pool, kind, scale):
    codes, scales = _tiles(pool, kind)
    code, s = _quantise(x, scale)
    code = _pack(code)
    b, t, k = at
    codes[b, :, t, k] = code.unflatten(-1, (-1, 8)) if kind == "v" else code
    scales[b, :, t, k] = s


def _plain_read(at, pool, kind, scale, table):
    codes, scales = _tiles(pool, kind)
    b, t, k = at
    c = codes[b, :, t, k]
    return _values(c.flatten(2), scales[b, :, t, k], scale, table).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# the plain form: attention and rotation


def _plain_attend(s):
    case = s["case"]
    heads, dim, longest, new = case["heads"], case["dim"], s["longest"], s["most_new"]
    group, lens, start = case["q_heads"] // case["heads"], s["seq_lens"].long(), s["q_start"]
    batch, tokens = lens.shape[0], s["q"].shape[0]
    sc = s["scale_dev"]
    table = s["block_table"].long()
    kc, ks = _tiles(s["k_pool"], "k")
    vc, vs = _tiles(s["v_pool"], "v")

    def rows(codes, scales, scale):            # [batch, heads, longest, dim]
        # [batch, pages, heads, tiles, 16, ...]
        x = _values(codes[table].flatten(5), scales[table], scale, s["e2m1"])
        return x.transpose(1, 2).reshape(batch, heads, -1, dim)[:, :, :longest]

    k, v = rows(kc, ks, sc[0]), rows(vc, vs, sc[1])
    if start is None:
        start = torch.arange(batch + 1, device=lens.device)
    count = (start[1:] - start[:-1]).long()
    i = torch.arange(new, device=lens.device)
    q = s["q"][(start[:-1, None] + i).clamp(max=tokens - 1)].float()       # [batch, new, q_heads, dim]
    q = q.unflatten(2, (heads, group)).permute(0, 2, 3, 1, 4).reshape(batch, heads, group * new, dim)
    a = (q @ k.transpose(-1, -2)) * s["softmax_scale"]
    a = a.view(batch, heads, group, new, longest)
    j = torch.arange(longest, device=lens.device)
    last = (lens - count)[:, None] + i                                     # [batch, new]
    see = (j <= last[..., None]) & (j < lens[:, None, None])
    if case["window"]:
        see &= j > last[..., None] - case["window"]
    a = a.masked_fill(~see[:, None, None], -math.inf)
    top = a.amax(-1, keepdim=True)
    p = (a - torch.where(top == -math.inf, torch.zeros_like(top), top)).exp()
    total = p.sum(-1, keepdim=True)
    o = (p.view(batch, heads, group * new, longest) @ v).view(batch, heads, group, new, dim)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + total.log()).squeeze(-1)
    of = torch.searchsorted(start[1:].long(), torch.arange(tokens, device=lens.device), right=True)
    at = torch.arange(tokens, device=lens.device) - start[of]
    return (o[of, :, :, at].flatten(1, 2).to(torch.bfloat16), lse[of, :, :, at].flatten(1, 2))


def _plain_rope(s):
    case = s["case"]
    half = case["rotary"] // 2
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos = (angle.cos() * s["rope_scale"]).float()[:, None]
    sin = (angle.sin() * s["rope_scale"]).float()[:, None]

    def one(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight.float()
        turn, rest = x[..., :2 * half], x[..., 2 * half:]
        if case["interleaved"]:
            a, b = turn[..., 0::2], turn[..., 1::2]
            turn = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = turn[..., :half], turn[..., half:]
            turn = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((turn, rest), -1).to(torch.bfloat16)

    return one(s["q"], s["q_weight"]), one(s["k"], s["k_weight"])


# ---------------------------------------------------------------------------
# inputs and passes


def _normal(g, *shape, scale=1.0):
    return torch.randn(*shape, device="cuda", generator=g) * scale


def _kv_values(g, *shape):
    """Keys or values: some channels carry more than others, and a few
    elements stand far out."""
    x = _normal(g, *shape)
    x *= 1.0 + 2.0 * (torch.rand(shape[-1], device="cuda", generator=g) < 0.05)
    x[torch.rand(shape, device="cuda", generator=g) < 0.001] *= 20.0
    return x.to(torch.bfloat16)


def _full_pool(g, kind, blocks, heads, tiles, dim, scale):
    """A pool whose every slot holds a token, packed from bf16 values."""
    pool = torch.empty((blocks, heads, tiles, 9 * dim), dtype=torch.uint8, device="cuda")
    codes, scales = _tiles(pool, kind)
    x = _kv_values(g, blocks, heads, tiles, 16, dim)
    code, s = _quantise(x, scale)
    del x
    codes.copy_(_pack(code).view(codes.shape))
    scales.copy_(s)
    return pool


def _fused(g, tokens, *widths):
    """Column ranges of one fused projection's output, as [tokens, heads, dim] views."""
    x = _kv_values(g, tokens, sum(h for h, _ in widths) * widths[0][1])
    out, at = [], 0
    for h, d in widths:
        out.append(x[:, at:at + h * d].unflatten(1, (h, d)))
        at += h * d
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind, heads, dim = case["kind"], case["heads"], case["dim"]
    s = dict(case=case)
    if kind == "rope":
        rng = random.Random(case["shape_seed"])
        t = case["tokens"]
        pos = [case["start"] + (rng.randrange(1000) if case["spread"] else i) for i in range(t)]
        s["q"], s["k"], _ = _fused(g, t, (case["q_heads"], dim), (heads, dim), (heads, dim))
        s["positions"] = torch.tensor(pos, dtype=torch.int64, device="cuda")
        s["inv_freq"] = (torch.arange(0, case["rotary"], 2, dtype=torch.float64, device="cuda")
                         / case["rotary"]).mul(-math.log(1e6)).exp() / case["stretch"]
        s["rope_scale"] = 0.1 * math.log(case["stretch"]) + 1.0
        s["eps"] = 1e-6
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"] = (1.0 + _normal(g, dim, scale=0.2)).to(torch.bfloat16)
            s["k_weight"] = (1.0 + _normal(g, dim, scale=0.2)).to(torch.bfloat16)
        s["q_out"] = torch.empty((t, case["q_heads"], dim), dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty((t, heads, dim), dtype=torch.bfloat16, device="cuda")
        return s
    s["k_scale"], s["v_scale"] = 0.1375, 0.0625 + 0.01 * (seed % 7)
    s["scale_dev"] = torch.tensor([s["k_scale"], s["v_scale"]], device="cuda")
    s["e2m1"] = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    tiles = case["block"] // 16
    if kind in ("cache", "read"):
        t, block, blocks = case["tokens"], case["block"], case["blocks"]
        rng = random.Random(case["shape_seed"] + 7919 * (seed % 1009))
        pages = rng.sample(range(blocks), -(-t // block))
        slots = [pages[i // block] * block + i % block for i in range(t)]
        for i in rng.sample(range(t), case["skipped"]):
            slots[i] = -1
        s["slots"] = torch.tensor(slots, dtype=torch.int64, device="cuda")
        if kind == "cache":
            _, s["k"], s["v"] = _fused(g, t, (case["q_heads"], dim), (heads, dim), (heads, dim))
            both = [torch.zeros((blocks + 1, heads, tiles, 9 * dim), dtype=torch.uint8, device="cuda")
                    for _ in range(2)]
        else:
            both = [_full_pool(g, kv, blocks + 1, heads, tiles, dim, s["scale_dev"][i])
                    for i, kv in enumerate("kv")]
        s["k_all"], s["v_all"] = both          # one spare block behind the pool's own
        s["k_pool"], s["v_pool"] = both[0][:blocks], both[1][:blocks]
        s["k_out"] = torch.zeros((t, heads, dim), dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.zeros((t, heads, dim), dtype=torch.bfloat16, device="cuda")
        return s
    lens, news = _lengths(case)
    pages = [-(-n // case["block"]) for n in lens]
    blocks = sum(pages)
    order = torch.randperm(blocks, device="cuda", generator=g).to(torch.int32)
    table = torch.zeros((len(lens), max(pages)), dtype=torch.int32)
    held = torch.arange(max(pages))[None] < torch.tensor(pages)[:, None]
    table = table.to("cuda")
    table[held.to("cuda")] = order
    s["block_table"] = table
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    tokens = sum(news)
    s["q_start"] = None
    if case["q_hi"] > 1:
        s["q_start"] = torch.tensor([sum(news[:i]) for i in range(len(news) + 1)], dtype=torch.int32,
                                    device="cuda")
    s["longest"], s["most_new"] = max(lens), max(news)
    s["k_pool"] = _full_pool(g, "k", blocks, heads, tiles, dim, s["scale_dev"][0])
    s["v_pool"] = _full_pool(g, "v", blocks, heads, tiles, dim, s["scale_dev"][1])
    s["q"] = _fused(g, tokens, (case["q_heads"], dim), (heads, dim), (heads, dim))[0]
    s["softmax_scale"] = dim ** -0.5
    s["out"] = torch.empty((tokens, case["q_heads"], dim), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty((tokens, case["q_heads"]), dtype=torch.float32, device="cuda")
    return s


def _own_scales(s):
    if s["case"]["scales"] == "device":
        return dict(scale_dev=s["scale_dev"])
    return dict(k_scale=s["k_scale"], v_scale=s["v_scale"])


def run(state):
    s, kind = state, state["case"]["kind"]
    if own:
        import paged_kv_cache_group_b200 as fp8q
        if kind == "rope":
            return fp8q.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_weight"],
                                     s["k_weight"], eps=s["eps"],
                                     interleaved=s["case"]["interleaved"],
                                     rope_scale=s["rope_scale"], q_out=s["q_out"],
                                     k_out=s["k_out"])
        scales = _own_scales(s)
        if kind == "attend":
            return fp8q.fp4_kv_attention(s["q"], s["k_pool"], s["v_pool"], s["block_table"],
                                         s["seq_lens"], softmax_scale=s["softmax_scale"],
                                         q_start=s["q_start"], window=s["case"]["window"],
                                         out=s["out"], lse=s["lse"], **scales)
        if kind == "cache":
            fp8q.fp4_kv_write(s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"], **scales)
        return fp8q.fp4_kv_read(s["slots"], s["k_pool"], s["v_pool"], k_out=s["k_out"],
                                v_out=s["v_out"], **scales)
    if kind == "rope":
        return _plain_rope(s)
    if kind == "attend":
        return _plain_attend(s)
    at = _place(s["slots"], s["case"]["blocks"], s["case"]["block"])
    live = (s["slots"] >= 0)[:, None, None]
    if kind == "cache":
        _plain_write(s["k"], at, s["k_all"], "k", s["scale_dev"][0])
        _plain_write(s["v"], at, s["v_all"], "v", s["scale_dev"][1])
    k = _plain_read(at, s["k_all"], "k", s["scale_dev"][0], s["e2m1"])
    v = _plain_read(at, s["v_all"], "v", s["scale_dev"][1], s["e2m1"])
    return torch.where(live, k, s["k_out"]), torch.where(live, v, s["v_out"])


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def _f32(x):
    return x.to(torch.float32).to(torch.float64)


def _exact_e4m3(bits):
    b = bits.to(torch.int64)
    e, m = b >> 3 & 15, (b & 7).double()
    return torch.where(e > 0, (8 + m) * torch.exp2((e - 10).double()), m * 2.0 ** -9)


def _exact_nearest(y, step):
    """y / step to the nearest whole number, ties to even, times step."""
    return torch.round(y / step) * step


def _exact_quantised(x, scale):
    """What x stands for once it is in the cache: its definition in 64 bits,
    rounded to fp32 where the definition says so."""
    x = x.double().unflatten(-1, (-1, 16))
    scale = _f32(torch.tensor(scale, dtype=torch.float64)).item()
    t = _f32(_f32(x.abs().amax(-1) / 6.0) / scale).clamp(max=448.0)
    e = torch.floor(torch.log2(t.clamp(min=2.0 ** -6)))
    b = _exact_nearest(t, torch.exp2(e - 3)).clamp(max=448.0)
    d = _f32(b * scale)
    y = torch.where((d > 0)[..., None], _f32(x * _f32(1.0 / d.clamp(min=1e-300))[..., None]), 0.0 * x)
    a = y.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.sign(y) * _exact_nearest(a, step) * b[..., None] * scale).flatten(-2)


def _exact_rows(pool, kind, blocks, scale):
    """[heads, len(blocks) * block_size, dim] values of some blocks of a pool."""
    p = pool[blocks]                           # [n, heads, tiles, 9 dim]
    n, heads, tiles, dim = *p.shape[:3], p.shape[3] // 9
    codes, scales = p[..., :8 * dim], p[..., 8 * dim:]
    if kind == "k":
        codes = codes.reshape(n, heads, tiles, 16, dim // 16, 8)
        scales = scales.reshape(n, heads, tiles, 16, dim // 16)
    else:
        codes = codes.reshape(n, heads, tiles, dim // 16, 16, 8).transpose(3, 4)
        scales = scales.reshape(n, heads, tiles, dim // 16, 16).transpose(3, 4)
    nib = torch.stack((codes % 16, codes // 16), -1).flatten(-2).to(torch.int64)
    mag = nib % 8
    e, m = mag // 2, (mag % 2).double()
    v = torch.where(e > 0, (1 + m / 2) * torch.exp2((e - 1).double()), m / 2)
    v = torch.where(nib >= 8, -v, v) * _exact_e4m3(scales)[..., None] * _f32(torch.tensor(scale, dtype=torch.float64)).item()
    return v.flatten(-2).transpose(0, 1).reshape(heads, -1, dim)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "rope":
        turn = torch.polar(torch.full((1,), s["rope_scale"], dtype=torch.float64, device="cuda"),
                           s["positions"].double()[:, None] * s["inv_freq"])[:, None]
        outs = []
        for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
            x = x.double()
            if w is not None:
                x = x / (x.pow(2).mean(-1, keepdim=True) + s["eps"]).sqrt() * w.double()
            r, half = case["rotary"], case["rotary"] // 2
            first = slice(0, r, 2) if case["interleaved"] else slice(0, half)
            second = slice(1, r, 2) if case["interleaved"] else slice(half, r)
            z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
            x = x.clone()
            x[..., first], x[..., second] = z.real, z.imag
            outs.append(x)
        return tuple(outs)
    if kind == "cache":
        live = (s["slots"] >= 0)[:, None, None]
        return tuple(torch.where(live, _exact_quantised(s[n], s[n + "_scale"]), 0.0) for n in ("k", "v"))
    if kind == "read":
        outs = []
        for n in ("k", "v"):
            out = torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda")
            rows = _exact_rows(s[n + "_pool"], n, torch.arange(case["blocks"], device="cuda"), s[n + "_scale"])
            out[s["slots"] >= 0] = rows[:, s["slots"][s["slots"] >= 0]].transpose(0, 1)
            outs.append(out)
        return tuple(outs)
    lens, news = _lengths(case)
    group = case["q_heads"] // case["heads"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    t = 0
    for b, (length, new) in enumerate(zip(lens, news)):
        blocks = s["block_table"][b, :-(-length // case["block"])].long()
        k = _exact_rows(s["k_pool"], "k", blocks, s["k_scale"])
        v = _exact_rows(s["v_pool"], "v", blocks, s["v_scale"])
        for i in range(new):
            n, first = _seen(length, new, case["window"], i)
            if n:
                q = s["q"][t + i].double().view(case["heads"], group, -1)
                a = torch.einsum("hgd,hjd->hgj", q, k[:, first:first + n]) * s["softmax_scale"]
                lse[t + i] = torch.logsumexp(a, -1).flatten()
                out[t + i] = torch.einsum("hgj,hjd->hgd", torch.softmax(a, -1), v[:, first:first + n]).flatten(0, 1)
        t += new
    return out, lse
