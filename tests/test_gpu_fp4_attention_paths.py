"""fp4_kv_attention where it divides its work differently: many rows to a KV
head, one, two and four heads a block, items split and not, windows over pages
that are gone, pools past 2^31 bytes.  Bounds as in test_gpu_fp4_attention,
but for the weights of the kernel for many rows: it takes scores against a
reference up to 2^4 below the maximum and holds p * 2^11 in fp16, so a weight
below the normal range is off by up to 2^-36 of the largest, not 2^-40, and the
bound's last term is n 2^-35 max|v|.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_group_b200 as fp8q
from gpu_util import dev
from oracle import fp4
from test_gpu_fp4_attention import Batch

pytestmark = pytest.mark.gpu


class Many(Batch):
    """A batch checked with the bound of the kernel for many rows."""

    def check(self, out, lse, window=0, scale=None):
        scale = self.dim ** -0.5 if scale is None else scale
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b, n in enumerate(self.lens):
            rows = slice(self.start[b], self.start[b + 1])
            k, v = self.kv(b)
            want, want_lse, mean, reach = fp4.attention(self.q64[rows], k, v, float(np.float32(scale)),
                                                        self.news[b], window)
            e = (self.dim + 16) * 2.0 ** -23 * reach + 2.0 ** -21 * reach
            most = np.abs(v).max() if v.size else 0.0
            bound = 2.0 ** -8 * np.abs(want) + n * 2.0 ** -35 * most + \
                (2.0 ** -11 + 2 * (e + 2.0 ** -22) + n * 2.0 ** -26)[..., None] * mean
            off = np.abs(out[rows] - want)
            assert np.all(off <= bound), (b, n, float((off - bound).max()))
            none = np.isneginf(want_lse)
            assert np.array_equal(np.isneginf(lse[rows]), none) and np.all(out[rows][none] == 0)
            lse_bound = e + 2.0 ** -20 + n * 2.0 ** -26 + 2.0 ** -22 * np.abs(np.where(none, 0, want_lse))
            with np.errstate(invalid="ignore"):
                off = np.where(none, 0.0, np.abs(lse[rows] - want_lse))
            assert np.all(off <= lse_bound), (b, n, float((off - lse_bound).max()))
        assert fp8q.fp8q_device_error(clear=True) == 0


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,group,size", [(1, 1, 16), (2, 3, 48), (3, 7, 32), (1, 16, 64)])
@pytest.mark.parametrize("window", [0, 1, 130])
def test_many_rows(dim, heads, group, size, window):
    # every edge of the 128-row and 128-token tiles; rows that see nothing
    b = Many(dim + group + window, dim, heads, group, size, [129, 128, 300, 40, 3, 0, 1],
             [129, 1, 127, 40, 60, 0, 1])
    b.check(*b.call(window=window), window=window)


def uneven(dim, heads, group, lens, news, seed):
    return Many(seed, dim, heads, group, 16, lens, news)


@pytest.mark.parametrize("dim,heads,group", [(64, 8, 8), (128, 8, 8), (256, 4, 8)])
def test_one_long_sequence_among_many_rows(dim, heads, group):
    """Enough row tiles that items stay whole: with room for parts the long
    one's are split all the same, without it they are not."""
    b = uneven(dim, heads, group, [2500, 900, 5], [1, 900, 2], dim)
    b.check(*b.call())
    n = fp8q.fp4_kv_attention_workspace(3, b.tokens, heads * group, heads, dim)
    assert n < fp8q.fp4_kv_attention_workspace(3, b.tokens, heads * group, heads, dim, uneven=True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    b.check(*b.call(workspace=ws, k_scale=b.k_scale, v_scale=b.v_scale))


@pytest.mark.parametrize("dim,heads,group", [(64, 4, 8), (128, 4, 4), (128, 8, 5), (128, 4, 16), (64, 4, 11), (256, 4, 8)])
@pytest.mark.parametrize("size", [16, 32, 48])
@pytest.mark.parametrize("window", [0, 33])
def test_four_heads_a_block(dim, heads, group, size, window):
    """Wide tables let blocks take four heads at once."""
    g = np.random.default_rng(dim + size)
    b = Batch(dim + group, dim, heads, group, size, g.integers(0, 200, 40))
    wide = np.full((40, 40000 // size), -7, np.int32)
    wide[:, :b.table.shape[1]] = b.table
    b.table = wide
    b.check(*b.call(window=window), window=window)


@pytest.mark.parametrize("heads", [1, 2, 3, 4, 6, 8])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_any_number_of_heads(heads, dim):
    b = Batch(heads, dim, heads, 2, 16, [0, 70, 33, 400, 1])
    b.check(*b.call())
    b.check(*b.call(window=40), window=40)


@pytest.mark.parametrize("news,cls", [([1, 1, 1], Batch), ([50, 44, 41], Many)])
@pytest.mark.parametrize("size", [16, 32, 48])
def test_pages_before_the_window_are_not_looked_at(news, cls, size):
    lens, window = [300, 250, 170], 60
    b = cls(31, 64, 2, 4, size, lens, news if cls is Many else None)
    want = [(b.kv(i)[0].copy(), b.kv(i)[1].copy()) for i in range(3)]
    b.kv = lambda i: want[i]
    for i, (n, m) in enumerate(zip(lens, news)):
        first = n - m + 1 - window
        for page in range(first // size):
            b.kp[b.table[i, page]] = 0xFF
            b.vp[b.table[i, page]] = 0xFF
            b.table[i, page] = (1 << 30) - page
        # what lies before the first seen token in its own page
        for tok in range(first // size * size, first):
            for pool, kind in ((b.kp, "k"), (b.vp, "v")):
                c, z = fp4._offsets(tok % 16, 64, kind)
                tile = pool[b.table[i, tok // size], :, tok % size // 16]
                tile[:, c] = 0xFF
                tile[:, z] = 0xFF
    b.check(*b.call(window=window), window=window)


def test_many_rows_with_a_nan_keep_it_to_themselves():
    b = Many(32, 64, 1, 4, 16, [200, 90], [30, 30])
    clean = b.call()
    b.q[3, 1, 5] = float("nan")
    b.q[40, 2, 0] = float("inf")
    out, lse = b.call()
    keep = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    keep[3, 1] = keep[40, 2] = False
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])
    assert bool(torch.isnan(out[3, 1]).all()) and bool(torch.isnan(lse[3, 1]))


def test_one_row_with_a_nan_gives_nan():
    b = Batch(33, 128, 1, 4, 16, [90])
    b.q[0, 1, 7] = float("nan")
    out, lse = b.call()
    assert bool(torch.isnan(out[0, 1]).all()) and bool(torch.isnan(lse[0, 1]))


@pytest.mark.parametrize("sharp", [1e-30, 1e-3, 30.0, 1e4])
def test_flat_and_peaked_weights_of_many_rows(sharp):
    b = Many(34, 128, 1, 8, 16, [400, 70], [20, 9], sharp=sharp)
    b.check(*b.call())


def test_growing_scores_of_many_rows():
    """Every tile's largest score is far above the last one's: the reference
    moves each time."""
    b = Many(35, 64, 1, 8, 16, [900], [10])
    code, z = fp4._offsets(0, 64, "k")
    for page in range(57):
        for tok in range(16):
            c, zz = fp4._offsets(tok, 64, "k")
            tile = b.kp[b.table[0, page], 0, 0]
            tile[c] = 0x22
            tile[zz] = 0x08 + page                           # block scales double every 8 pages
    b.q[:] = 0.25
    b.q64 = b.q.double().cpu().numpy()
    b.k_scale = 1.0
    b.check(*b.call(scale=1.0), scale=1.0)


def test_many_rows_repeat_bit_for_bit_and_follow_a_graph():
    b = Many(36, 128, 2, 4, 16, [900, 40, 300], [60, 1, 100])
    other = Many(37, 128, 2, 4, 16, [333, 880, 60], [4, 142, 15])
    first = b.call()
    again = b.call()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])

    def inputs(x, wide, blocks):
        table = np.full((3, wide), -1, np.int32)
        table[:, :x.table.shape[1]] = x.table
        pools = [np.concatenate([p, np.full((blocks - len(p), *p.shape[1:]), 255, np.uint8)]) for p in (x.kp, x.vp)]
        return [dev(p) for p in pools] + [dev(table), dev(np.array(x.lens, np.int32)), dev(x.start), x.q]

    wide, blocks = max(x.table.shape[1] for x in (b, other)), max(len(x.kp) for x in (b, other))
    held, want = inputs(b, wide, blocks), inputs(other, wide, blocks)
    out = torch.zeros(b.q.shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(b.q.shape[:2], device="cuda")

    def call():
        fp8q.fp4_kv_attention(held[5], *held[:4], q_start=held[4], k_scale=b.k_scale, v_scale=b.v_scale,
                              out=out, lse=lse)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    b.check(out, lse)
    for x, y in zip(held, want):
        x.copy_(y)
    graph.replay()
    other.check(out, lse)


def test_pools_past_two_to_the_31_bytes():
    heads, dim, blocks = 4, 128, 600000                      # 2.8 GB each
    kp, vp = fp8q.fp4_kv_pools(blocks, 16, heads, dim)
    table = torch.arange(blocks - 40, blocks, dtype=torch.int32, device="cuda").flip(0).view(2, 20)
    g = torch.Generator().manual_seed(5)
    lens, q = [300, 111], torch.randn((2, 16, dim), generator=g).to(torch.bfloat16)
    k, v = (torch.randn((sum(lens), heads, dim), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    slots = torch.cat([table[i].long().repeat_interleave(16)[:n] * 16 + torch.arange(n, device="cuda") % 16
                       for i, n in enumerate(lens)])
    fp8q.fp4_kv_write(k, v, slots, kp, vp, 0.01, 0.01)
    kr, vr = fp8q.fp4_kv_read(slots, kp, vp, 0.01, 0.01)
    lens_dev = torch.tensor(lens, dtype=torch.int32, device="cuda")
    small = [p[-40:].clone() for p in (kp, vp)]
    kr2, vr2 = fp8q.fp4_kv_read(slots - (blocks - 40) * 16, *small, 0.01, 0.01)
    assert torch.equal(kr, kr2) and torch.equal(vr, vr2) and bool(kr.any())
    for start, rows in ((None, q), (torch.tensor([0, 20, 24], dtype=torch.int32, device="cuda"),
                                    torch.randn((24, 16, dim), generator=g).to(torch.bfloat16))):
        far = fp8q.fp4_kv_attention(rows.cuda(), kp, vp, table, lens_dev, q_start=start)
        near = fp8q.fp4_kv_attention(rows.cuda(), *small, table - (blocks - 40), lens_dev, q_start=start)
        assert torch.equal(far, near) and bool(torch.isfinite(far).all()) and bool(far.any())
    assert fp8q.fp8q_device_error(clear=True) == 0


@pytest.mark.parametrize("news,cls", [(1, Batch), (70, Many)])
def test_few_live_sequences_among_many_empty_ones(news, cls):
    count, live = 4000, (0, 1777, 3999)
    lens, new = [0] * count, [0] * count
    for i, b in enumerate(live):
        lens[b], new[b] = 90 + 60 * i, news
    b = cls(38, 64, 2, 2, 16, lens, new)
    b.check(*b.call())


def test_only_empty_sequences():
    b = Batch(39, 64, 2, 2, 16, [0, 7, 0], [0, 0, 0], spare=4)
    out, lse = b.call()
    assert bool((out == 3.0).all()) and bool((lse == 3.0).all())
    b = Batch(40, 64, 2, 40, 16, [0, 0], [40, 30])           # new tokens of sequences without any cached
    out, lse = b.call()
    assert not bool(out.any()) and bool(torch.isneginf(lse).all())
    assert fp8q.fp8q_device_error(clear=True) == 0
