"""Plain restatement of the 4-bit KV cache, attention over it, and the norm and
rotation of queries and keys, in 64-bit numpy on the host.

Values that the definitions round to fp32 are rounded by a cast from fp64; a
quotient or product of fp32 numbers rounded to fp64 first and to fp32 then is
the correctly rounded one (53 >= 2 * 24 + 2).
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
# every E4M3 magnitude by its code; 0x7F is NaN
E4M3 = np.array([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
                 for e in range(16) for m in range(8)])
E4M3[127] = np.nan


def _f32(x):
    return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def _nearest(values, grid):
    """Index of the nearest of an ascending grid, ties to the even index."""
    mid = (grid[1:] + grid[:-1]) / 2
    below = np.searchsorted(mid, values, side="left")        # a tie stays below
    tie = np.isin(values, mid)
    return np.where(tie & (below % 2 == 1), below + 1, below)


def quantise(x, scale):
    """Codes (one a byte) and E4M3 block scale codes of x [..., dim]; ``scale``
    is an fp32 number."""
    b = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, 16)
    mag = np.abs(b)
    amax = np.where(np.isnan(mag), 0.0, mag).max(-1)
    with np.errstate(over="ignore"):
        t = _f32(_f32(amax / 6.0) / float(np.float32(scale)))
    s = _nearest(np.minimum(t, 448.0), E4M3[:127])
    d = _f32(E4M3[s] * float(np.float32(scale)))
    r = np.where(d > 0, _f32(1.0 / np.where(d > 0, d, 1.0)), 0.0)[..., None]
    with np.errstate(over="ignore", invalid="ignore"):
        y = _f32(mag * r)
        y = np.where(np.isnan(y), np.where(np.isinf(mag) & (r == 0), np.nan, y), y)
    code = np.where(np.isnan(y), 7, _nearest(np.minimum(y, 6.0), E2M1[:8]))
    code = code + 8 * (np.signbit(b) & ~np.isnan(y))
    return code.astype(np.uint8).reshape(x.shape), s.astype(np.uint8)


def values(code, scale_code):
    """code * block scale, exact in fp64."""
    b = E2M1[code].reshape(*code.shape[:-1], -1, 16) * E4M3[scale_code & 127][..., None]
    return b.reshape(code.shape)


def _offsets(tok, dim, kind):
    """Byte offsets in a tile of token ``tok``: [dim / 2] of the code bytes and
    [dim / 16] of the scale bytes."""
    byte, blk = np.arange(dim // 2), np.arange(dim // 16)
    if kind == "k":
        return tok * (dim // 2) + byte, 8 * dim + tok * (dim // 16) + blk
    return byte // 8 * 128 + tok * 8 + byte % 8, 8 * dim + blk * 16 + tok


def write(x, slots, pool, kind, scale):
    """Quantise x [T, heads, dim] into pool [blocks, heads, tiles, 9 * dim]."""
    size = pool.shape[2] * 16
    code, s = quantise(x, scale)
    packed = code[..., 0::2] | code[..., 1::2] << 4
    for t, slot in enumerate(slots):
        if 0 <= slot < pool.shape[0] * size:
            blk, off = divmod(int(slot), size)
            c, z = _offsets(off % 16, x.shape[2], kind)
            for h in range(x.shape[1]):
                tile = pool[blk, h, off // 16]
                tile[c] = packed[t, h]
                tile[z] = s[t, h]


def read(slots, pool, kind):
    """code * block scale of the tokens at ``slots``: fp64 [T, heads, dim]."""
    size, dim = pool.shape[2] * 16, pool.shape[3] // 9
    out = np.zeros((len(slots), pool.shape[1], dim))
    for t, slot in enumerate(slots):
        blk, off = divmod(int(slot), size)
        c, z = _offsets(off % 16, dim, kind)
        tile = pool[blk, :, off // 16]
        code = np.empty((pool.shape[1], dim), np.uint8)
        code[:, 0::2], code[:, 1::2] = tile[:, c] & 15, tile[:, c] >> 4
        out[t] = values(code, tile[:, z])
    return out


def attention(q, k, v, softmax_scale, news, window=0):
    """One sequence: q [news, q_heads, dim] are the last tokens of the cached
    k, v [length, heads, dim] (tensor scales included).  Returns out, lse, and
    what error bounds need: the weighted mean of |v| and the largest
    softmax_scale * sum |q k|, per row."""
    length, heads, dim = k.shape
    group = q.shape[1] // heads
    out, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    mean_abs, reach = np.zeros(q.shape), np.zeros(q.shape[:2])
    for i in range(news):
        last = length - news + i
        first = max(0, last - window + 1) if window else 0
        if last < first or last < 0:
            continue
        for h in range(q.shape[1]):
            kk, vv = k[first:last + 1, h // group], v[first:last + 1, h // group]
            a = kk @ q[i, h] * softmax_scale
            reach[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * softmax_scale
            top = a.max()
            p = np.exp(a - top)
            lse[i, h] = top + np.log(p.sum())
            out[i, h] = p @ vv / p.sum()
            mean_abs[i, h] = p @ np.abs(vv) / p.sum()
    return out, lse, mean_abs, reach


def norm_rope(x, positions, inv_freq, weight, eps, interleaved, rope_scale):
    """x [T, heads, dim] normed (with a weight) and rotated; also |a| + |b| of
    each rotary pair at its two places, and |y| elsewhere."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    out, size = x.copy(), np.abs(x)
    n = len(inv_freq)
    a_at, b_at = (np.arange(n) * 2, np.arange(n) * 2 + 1) if interleaved else \
        (np.arange(n), np.arange(n) + n)
    turn = np.exp(1j * np.asarray(positions, np.float64)[:, None] * inv_freq) * rope_scale
    z = (x[..., a_at] + 1j * x[..., b_at]) * turn[:, None]
    out[..., a_at], out[..., b_at] = z.real, z.imag
    both = (size[..., a_at] + size[..., b_at]) * abs(rope_scale)
    size[..., a_at] = size[..., b_at] = both
    return out, size
