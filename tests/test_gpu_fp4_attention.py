"""fp4_kv_attention against the 64-bit oracle on the same pool bytes.

Bounds.  Let A = sum p|v| / sum p, and R the largest softmax_scale * sum |q k|
of a row.  A score accumulates dim products in fp32, a unit in the last place
each (2^-23), and is rounded a few times more: |da| <= e = (dim + 16) 2^-23 R,
plus 2^-22 |a - max| <= 2^-21 R for the running differences and 2^-22 for the
exponential; numerator and denominator both carry it.  Weights are rounded to
fp16: 2^-11 of their value, or 2^-40 of the largest below the normal range.
Sums over n tokens add n / 8 units of 2^-23 (16 products an instruction, both
ways).  The output is rounded to bf16, 2^-8 of its value.  So
    |out error| <= 2^-8 |out| + (2^-11 + 2 (e + 2^-21 R + 2^-22) + n 2^-26) A + n 2^-39 max|v|
    |lse error| <= e + 2^-21 R + 2^-20 + n 2^-26 + 2^-22 |lse|
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_group_b200 as fp8q
from gpu_util import dev, host
from oracle import fp4

pytestmark = pytest.mark.gpu


class Batch:
    """Sequences in a pool of random codes.  Unused slots hold 0xFF: a NaN
    scale byte wherever they are looked at; unused table entries are far out."""

    def __init__(self, seed, dim, heads, group, size, lens, news=None, pad=0, sharp=1.0, spare=0):
        g = np.random.default_rng(seed)
        self.dim, self.heads, self.group, self.size, self.lens = dim, heads, group, size, list(lens)
        self.news = [1] * len(lens) if news is None else list(news)
        self.k_scale, self.v_scale = float(np.float32(0.011)), float(np.float32(0.37))
        pages = [-(-n // size) for n in lens]
        blocks = sum(pages) + 2
        shape = (blocks, heads, size // 16, 9 * dim)
        self.kp, self.vp = np.full(shape, 0xFF, np.uint8), np.full(shape, 0xFF, np.uint8)
        order = g.permutation(blocks)
        self.table = np.full((len(lens), max(pages + [1]) + 1), -7, np.int32)
        self.table[:, -1] = 1 << 30
        at = 0
        for b, n in enumerate(lens):
            mine = order[at:at + pages[b]]
            at += pages[b]
            self.table[b, :pages[b]] = mine
            for page in range(pages[b]):
                live = min(size, n - page * size)
                for tok in range(live):
                    for pool, kind in ((self.kp, "k"), (self.vp, "v")):
                        c, z = fp4._offsets(tok % 16, dim, kind)
                        tile = pool[mine[page], :, tok // 16]
                        tile[:, c] = g.integers(0, 256, (heads, dim // 2))
                        tile[:, z] = g.integers(0x28, 0x48, (heads, dim // 16))
        self.start = np.concatenate([[0], np.cumsum(self.news)]).astype(np.int32)
        self.tokens = int(self.start[-1]) + spare
        x = torch.from_numpy(g.standard_normal((self.tokens, heads * group * dim + pad)) * sharp)
        x = x.to(torch.bfloat16)
        cut = (slice(None), slice(0, heads * group * dim))
        self.q = x.cuda()[cut].unflatten(1, (heads * group, dim))
        self.q64 = x[cut].unflatten(1, (heads * group, dim)).double().numpy()
        self.ragged = news is not None

    def call(self, window=0, scale=None, **kw):
        out = torch.full(self.q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(self.q.shape[:2], 3.0, device="cuda")
        got = fp8q.fp4_kv_attention(
            self.q, dev(self.kp), dev(self.vp), dev(self.table), dev(np.array(self.lens, np.int32)),
            softmax_scale=scale, q_start=dev(self.start) if self.ragged else None, window=window,
            out=out, lse=lse, **(kw or dict(k_scale=self.k_scale, v_scale=self.v_scale)))
        assert got[0] is out and got[1] is lse
        return out, lse

    def kv(self, b):
        j = np.arange(self.lens[b])
        slots = self.table[b, j // self.size].astype(np.int64) * self.size + j % self.size
        return (fp4.read(slots, self.kp, "k") * self.k_scale,
                fp4.read(slots, self.vp, "v") * self.v_scale)

    def check(self, out, lse, window=0, scale=None):
        scale = self.dim ** -0.5 if scale is None else scale
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.all(out[self.start[-1]:] == 3.0) and np.all(lse[self.start[-1]:] == 3.0)
        for b, n in enumerate(self.lens):
            rows = slice(self.start[b], self.start[b + 1])
            k, v = self.kv(b)
            want, want_lse, mean, reach = fp4.attention(self.q64[rows], k, v, float(np.float32(scale)),
                                                        self.news[b], window)
            e = (self.dim + 16) * 2.0 ** -23 * reach + 2.0 ** -21 * reach
            most = np.abs(v).max() if v.size else 0.0
            bound = 2.0 ** -8 * np.abs(want) + n * 2.0 ** -39 * most + \
                (2.0 ** -11 + 2 * (e + 2.0 ** -22) + n * 2.0 ** -26)[..., None] * mean
            off = np.abs(out[rows] - want)
            assert np.all(off <= bound), (b, n, float((off - bound).max()))
            none = np.isneginf(want_lse)
            assert np.array_equal(np.isneginf(lse[rows]), none), (b, n)
            assert np.all(out[rows][none] == 0)
            lse_bound = e + 2.0 ** -20 + n * 2.0 ** -26 + 2.0 ** -22 * np.abs(np.where(none, 0, want_lse))
            with np.errstate(invalid="ignore"):
                off = np.where(none, 0.0, np.abs(lse[rows] - want_lse))
            assert np.all(off <= lse_bound), (b, n, float((off - lse_bound).max()))
        assert fp8q.fp8q_device_error(clear=True) == 0


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 127, 128, 129, 161, 257]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 8])
@pytest.mark.parametrize("size", [16, 48])
def test_single_tokens(dim, group, size):
    b = Batch(dim + group, dim, 2, group, size, EDGES)
    b.check(*b.call())


@pytest.mark.parametrize("dim,heads,group", [(64, 1, 16), (64, 3, 9), (64, 1, 33), (128, 2, 12), (128, 1, 40), (256, 1, 17)])
def test_many_query_heads_to_a_kv_head(dim, heads, group):
    b = Batch(group, dim, heads, group, 32, [1, 40, 300])
    b.check(*b.call())


@pytest.mark.parametrize("dim,group", [(64, 1), (64, 5), (128, 4), (128, 5), (256, 2)])
@pytest.mark.parametrize("window", [0, 1, 20, 1000])
def test_several_new_tokens_causal_and_windowed(dim, group, window):
    # one token, none, more new than cached (rows that see nothing), all new, an odd piece
    b = Batch(dim * 7 + window, dim, 2, group, 16, [5, 40, 3, 19, 150, 0, 260],
              [1, 0, 7, 19, 33, 2, 70], spare=3)
    b.check(*b.call(window=window), window=window)


@pytest.mark.parametrize("dim,heads,lens", [(128, 1, [5000]), (64, 2, [3001, 1, 4000]), (256, 1, [2500]),
                                            (128, 4, [700] * 3)])
def test_long_sequences_split_over_blocks(dim, heads, lens):
    b = Batch(11, dim, heads, 4, 16, lens)
    b.check(*b.call())
    b.check(*b.call(window=777), window=777)


def test_many_short_sequences():
    g = np.random.default_rng(1)
    b = Batch(12, 64, 2, 2, 16, g.integers(0, 60, 700))
    b.check(*b.call())


def test_strided_queries_and_outputs_and_padded_blocks():
    b = Batch(13, 128, 2, 4, 32, [100, 37], [2, 5], pad=72)
    kp, vp = dev(b.kp), dev(b.vp)
    n, block = kp.shape[0], kp[0].numel()
    wide = [torch.full((n, block + 48), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for w, p in zip(wide, (kp, vp)):
        w[:, :block] = p.view(n, block)
    kp, vp = (w.as_strided(p.shape, (block + 48, *p.stride()[1:])) for w, p in zip(wide, (kp, vp)))
    out = torch.full((7, 8 * 128 + 24), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((7, 8), device="cuda")
    table = torch.full((2, 9), -1, dtype=torch.int32, device="cuda")
    table[:, :b.table.shape[1]] = dev(b.table)
    fp8q.fp4_kv_attention(b.q, kp, vp, table[:, :b.table.shape[1]], dev(np.array(b.lens, np.int32)),
                          q_start=dev(b.start), out=out[:, :1024].unflatten(1, (8, 128)), lse=lse,
                          scale_dev=torch.tensor([b.k_scale, b.v_scale], device="cuda"))
    assert bool((out[:, 1024:] == 3.0).all())
    b.check(out[:, :1024].unflatten(1, (8, 128)), lse)


@pytest.mark.parametrize("sharp", [1e-30, 1e-3, 30.0, 1e4])
def test_flat_and_peaked_weights(sharp):
    b = Batch(14, 128, 1, 8, 16, [300, 70], sharp=sharp)
    b.check(*b.call())


def test_queries_of_very_different_size_in_one_row():
    b = Batch(15, 64, 1, 4, 16, [200])
    b.q[..., ::7] *= 2.0 ** 60
    b.q[..., 1::7] *= 2.0 ** -60
    b.q[0, 2] = 0.0
    b.q64 = b.q.double().cpu().numpy()
    b.check(*b.call(scale=2.0 ** -62), scale=2.0 ** -62)


def test_one_token_far_above_many_small_ones():
    # 4000 weights of about e^-14 against one of 1: together they are 0.3% of the sum
    b = Batch(16, 64, 1, 1, 16, [4000])
    code, z = fp4._offsets(0, 64, "k")
    b.kp[:, :, :, :] = 0
    b.vp[..., 8 * 64:] = 0x38
    b.vp[..., :8 * 64] = 0x22                                # every value is 1.0 ...
    first = b.table[0, 0]
    c, _ = fp4._offsets(0, 64, "v")
    b.vp[first, 0, 0, c] = 0xAA                              # ... the first token's -1.0
    b.kp[first, 0, 0, code] = 0x22
    b.kp[first, 0, 0, z] = 0x38                              # q . k = 14 for the first, else 0
    b.q[:] = 14.0 / 64
    b.q64 = b.q.double().cpu().numpy()
    b.k_scale = b.v_scale = 1.0
    out, lse = b.call(scale=1.0)
    b.check(out, lse, scale=1.0)
    assert abs(float(lse[0, 0]) - np.log(np.exp(14.0) + 3999)) < 1e-5


def test_results_repeat_bit_for_bit():
    b = Batch(17, 128, 2, 8, 16, [3000, 17, 900])
    first = b.call()
    for _ in range(3):
        again = b.call()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_a_captured_call_follows_its_inputs():
    b = Batch(18, 128, 2, 4, 16, [900, 40, 300], [2, 1, 4])
    other = Batch(19, 128, 2, 4, 16, [33, 880, 500], [4, 2, 1])
    names = ("q", "kp", "vp", "table", "lens", "start")

    def inputs(x):
        return dict(q=x.q, kp=dev(x.kp), vp=dev(x.vp), table=dev(x.table),
                    lens=dev(np.array(x.lens, np.int32)), start=dev(x.start))

    held = inputs(b)
    want = inputs(other)
    wide = max(held["table"].shape[1], want["table"].shape[1])
    for x in (held, want):
        x["table"] = torch.nn.functional.pad(x["table"], (0, wide - x["table"].shape[1]), value=-1)
    most = max(held["kp"].shape[0], want["kp"].shape[0])
    for x in (held, want):
        for n in ("kp", "vp"):
            x[n] = torch.cat([x[n], x[n].new_full((most - x[n].shape[0], *x[n].shape[1:]), 255)])
    out = torch.zeros(b.q.shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(b.q.shape[:2], device="cuda")

    def call():
        fp8q.fp4_kv_attention(held["q"], held["kp"], held["vp"], held["table"], held["lens"],
                              q_start=held["start"], k_scale=b.k_scale, v_scale=b.v_scale, out=out,
                              lse=lse)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    b.check(out, lse)
    for n in names:
        held[n].copy_(want[n])
    graph.replay()
    other.check(out, lse)


def test_two_streams_with_a_workspace_each():
    batches = [Batch(20, 128, 2, 4, 16, [2500, 10]), Batch(21, 128, 2, 4, 16, [90, 1800])]
    sides = [torch.cuda.Stream() for _ in batches]
    sets = []
    for b in batches:
        n = fp8q.fp4_kv_attention_workspace(2, 2, 8, 2, 128)
        sets.append([dev(b.kp), dev(b.vp), dev(b.table), dev(np.array(b.lens, np.int32)),
                     torch.empty(n, dtype=torch.uint8, device="cuda")])
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, (b, side) in enumerate(zip(batches, sides)):
            kp, vp, table, lens, ws = sets[i]
            lse = torch.empty((2, 8), device="cuda")
            outs[i].append(fp8q.fp4_kv_attention(b.q, kp, vp, table, lens, k_scale=b.k_scale,
                                                 v_scale=b.v_scale, lse=lse, workspace=ws, stream=side))
    torch.cuda.synchronize()
    for b, got in zip(batches, outs):
        for o, l in got:
            b.check(o, l)


def test_bad_lengths_tables_and_ranges_are_cut_and_reported():
    b = Batch(22, 64, 1, 2, 16, [20, 30, 25])
    lens = np.array([-5, 30, 1000], np.int32)
    kp, vp = dev(b.kp), dev(b.vp)
    kp[kp == 255], vp[vp == 255] = 0, 0                     # what is cut to may be any block
    table = np.zeros_like(b.table)
    out = fp8q.fp4_kv_attention(b.q, kp, vp, dev(table), dev(lens))
    assert fp8q.fp8q_device_error(clear=True) == fp8q.DEVERR_BAD_SEQUENCE
    assert not bool(out[0].any()) and bool(torch.isfinite(out).all())
    table[:] = -1
    out = fp8q.fp4_kv_attention(b.q, kp, vp, dev(table), dev(np.array(b.lens, np.int32)))
    assert fp8q.fp8q_device_error(clear=True) == fp8q.DEVERR_SLOT_OUT_OF_RANGE
    assert bool(torch.isfinite(out).all())
    for start in ([0, 1, 9, 3], [-4, 1, 2, 3], [3, 1, 2, 3]):
        fp8q.fp4_kv_attention(b.q, kp, vp, dev(np.zeros_like(table)), dev(np.array(b.lens, np.int32)),
                              q_start=dev(np.array(start, np.int32)))
        assert fp8q.fp8q_device_error(clear=True) == fp8q.DEVERR_BAD_SEQUENCE


def test_a_bad_device_scale_leaves_the_outputs_alone():
    b = Batch(23, 64, 1, 2, 16, [300])
    for pair in ((float("nan"), 1.0), (1.0, -2.0)):
        out, lse = b.call(scale_dev=torch.tensor(pair, device="cuda"))
        assert fp8q.fp8q_device_error(clear=True) == fp8q.DEVERR_BAD_SCALE
        assert bool((out == 3.0).all()) and bool((lse == 3.0).all())


def test_a_row_with_a_nan_keeps_it_to_itself():
    b = Batch(24, 128, 1, 8, 16, [200])
    clean = b.call()
    b.q[0, 3, 5] = float("nan")
    b.q[0, 6, 0] = float("inf")
    out, lse = b.call()
    keep = [i for i in range(8) if i not in (3, 6)]
    assert torch.equal(out[0, keep], clean[0][0, keep]) and torch.equal(lse[0, keep], clean[1][0, keep])


def test_refusals_of_device_tensors():
    b = Batch(25, 64, 2, 2, 16, [20, 30])
    kp, vp, table, lens = dev(b.kp), dev(b.vp), dev(b.table), dev(np.array(b.lens, np.int32))
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")

    def call(q=b.q, kp=kp, vp=vp, table=table, lens=lens, **kw):
        return fp8q.fp4_kv_attention(q, kp, vp, table, lens, **kw)

    call()
    call(q_start=start)
    for bad in (dict(q=b.q[:, :3]), dict(q=b.q[:1]), dict(table=table[:1]), dict(table=table.long()),
                dict(table=table.t().contiguous().t()), dict(lens=lens.long()), dict(q_start=start[:2]),
                dict(q_start=start.long()), dict(lens=lens.cpu()), dict(table=table.cpu()),
                dict(out=torch.empty_like(b.q)[:, :2]), dict(lse=torch.empty((2, 3), device="cuda")),
                dict(lse=torch.empty((2, 4), dtype=torch.float64, device="cuda")),
                dict(scale_dev=torch.ones(2)), dict(vp=vp[:1])):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), dict(window=-1),
                dict(softmax_scale=-1.0), dict(k_scale=0.0)):
        with pytest.raises(fp8q.Fp8qError):
            call(**bad)
    assert fp8q.fp8q_device_error(clear=True) == 0
