"""What fp4_kv_attention promises beside its values, where a KV head has many query
rows: bad lengths, pages, ranges and scales, rows that no sequence owns, strided
outputs and padded blocks, two streams.  Items are split over blocks in the first
batch and whole in the second, which has enough of them."""
import numpy as np
import pytest
import torch

import paged_kv_cache_group_b200 as fp8q
from gpu_util import dev
from test_gpu_fp4_attention_paths import Many

pytestmark = pytest.mark.gpu

SPLIT = dict(dim=64, heads=1, group=4, size=16, lens=[120, 230, 45], news=[50, 44, 41])
WHOLE = dict(dim=128, heads=8, group=8, size=32, lens=[900, 90], news=[850, 80])


class Owned(Many):
    """A batch whose rows behind the last sequence have to stay as they were."""

    def check(self, out, lse, window=0, scale=None):
        last = int(self.start[-1])
        assert bool((out[last:] == 3.0).all()) and bool((lse[last:] == 3.0).all())
        super().check(out, lse, window, scale)


def batch(sizes, seed, **kw):
    b = Owned(seed, **sizes, **kw)
    assert b.tokens * b.group > 32 * len(b.lens)             # by rows
    least, most = (fp8q.fp4_kv_attention_workspace(len(b.lens), b.tokens, b.heads * b.group, b.heads, b.dim, uneven)
                   for uneven in (False, True))
    assert (least < most) == (sizes is WHOLE)                # whole items need no parts
    return b


def pools_without_nan(b):
    kp, vp = dev(b.kp), dev(b.vp)
    kp[kp == 255], vp[vp == 255] = 0, 0                      # what is cut to may be any block
    return kp, vp


def attend(b, kp, vp, table, lens, start=None):
    out, lse = (torch.full(s, 3.0, dtype=t, device="cuda")
                for s, t in ((b.q.shape, torch.bfloat16), (b.q.shape[:2], torch.float32)))
    fp8q.fp4_kv_attention(b.q, kp, vp, dev(table), dev(np.array(lens, np.int32)),
                          q_start=dev(b.start if start is None else np.array(start, np.int32)),
                          k_scale=b.k_scale, v_scale=b.v_scale, out=out, lse=lse)
    return out, lse


@pytest.mark.parametrize("sizes", [SPLIT, WHOLE], ids=["split", "whole"])
@pytest.mark.parametrize("window", [0, 40])
def test_rows_behind_the_last_sequence(sizes, window):
    b = batch(sizes, 60, spare=150)
    b.check(*b.call(window=window), window=window)


@pytest.mark.parametrize("sizes", [SPLIT, WHOLE], ids=["split", "whole"])
def test_bad_lengths(sizes):
    b = batch(sizes, 61)
    kp, vp = pools_without_nan(b)
    lens = list(b.lens)
    lens[0], lens[-1] = -5, 1 << 20
    out, lse = attend(b, kp, vp, np.zeros_like(b.table), lens)
    assert fp8q.fp8q_device_error(clear=True) == fp8q.DEVERR_BAD_SEQUENCE
    first = slice(0, int(b.start[1]))
    assert not bool(out[first].any()) and bool(torch.isneginf(lse[first]).all())
    assert bool(torch.isfinite(out).all()) and bool(out[int(b.start[-2]):].any())


@pytest.mark.parametrize("sizes", [SPLIT, WHOLE], ids=["split", "whole"])
@pytest.mark.parametrize("entry", [-1, 1 << 30, "blocks"])
def test_pages_outside_the_pool(sizes, entry):
    b = batch(sizes, 62)
    kp, vp = pools_without_nan(b)
    table = np.full_like(b.table, kp.shape[0] if entry == "blocks" else entry)
    out, lse = attend(b, kp, vp, table, b.lens)
    assert fp8q.fp8q_device_error(clear=True) == fp8q.DEVERR_SLOT_OUT_OF_RANGE
    want = attend(b, kp, vp, np.zeros_like(table), b.lens)   # block 0 is read
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert fp8q.fp8q_device_error(clear=True) == 0


@pytest.mark.parametrize("sizes", [SPLIT, WHOLE], ids=["split", "whole"])
def test_bad_ranges_of_queries(sizes):
    b = batch(sizes, 63)
    kp, vp = pools_without_nan(b)
    good = b.start.tolist()
    for at, value, untouched in ((0, -4, None), (len(good) - 1, 1 << 20, None),
                                 (0, good[-1] + 60, slice(0, good[1])), (len(good) - 1, -1, slice(good[-2], None))):
        start = list(good)
        start[at] = value
        out, lse = attend(b, kp, vp, np.zeros_like(b.table), b.lens, start)
        assert fp8q.fp8q_device_error(clear=True) == fp8q.DEVERR_BAD_SEQUENCE, start
        assert bool(torch.isfinite(out).all())
        if untouched is not None:
            assert bool((out[untouched] == 3.0).all()) and bool((lse[untouched] == 3.0).all()), start


@pytest.mark.parametrize("sizes", [SPLIT, WHOLE], ids=["split", "whole"])
def test_a_bad_device_scale_leaves_the_outputs_alone(sizes):
    b = batch(sizes, 64)
    for pair in ((float("nan"), 1.0), (1.0, -2.0), (0.0, 1.0), (1.0, float("inf"))):
        out, lse = b.call(scale_dev=torch.tensor(pair, device="cuda"))
        assert fp8q.fp8q_device_error(clear=True) == fp8q.DEVERR_BAD_SCALE
        assert bool((out == 3.0).all()) and bool((lse == 3.0).all())


@pytest.mark.parametrize("sizes", [SPLIT, WHOLE], ids=["split", "whole"])
def test_strided_queries_and_outputs_and_padded_blocks(sizes):
    b = batch(sizes, 65, pad=72)
    heads, dim = b.heads * b.group, b.dim
    kp, vp = dev(b.kp), dev(b.vp)
    n, block = kp.shape[0], kp[0].numel()
    wide = [torch.full((n, block + 48), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for w, p in zip(wide, (kp, vp)):
        w[:, :block] = p.view(n, block)
    kp, vp = (w.as_strided(p.shape, (block + 48, *p.stride()[1:])) for w, p in zip(wide, (kp, vp)))
    out = torch.full((b.tokens, heads * dim + 24), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((b.tokens, heads), device="cuda")
    table = torch.full((len(b.lens), b.table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    table[:, :b.table.shape[1]] = dev(b.table)
    rows = out[:, :heads * dim].unflatten(1, (heads, dim))
    fp8q.fp4_kv_attention(b.q, kp, vp, table[:, :b.table.shape[1]], dev(np.array(b.lens, np.int32)),
                          q_start=dev(b.start), out=rows, lse=lse,
                          scale_dev=torch.tensor([b.k_scale, b.v_scale], device="cuda"))
    assert bool((out[:, heads * dim:] == 3.0).all())
    b.check(rows, lse)


def test_two_streams_with_a_workspace_each():
    other = dict(SPLIT, lens=[45, 300, 130], news=[45, 60, 30])
    batches = [batch(SPLIT, 66), batch(other, 67)]
    sides = [torch.cuda.Stream() for _ in batches]
    sets = []
    for b in batches:
        n = fp8q.fp4_kv_attention_workspace(3, b.tokens, 4, 1, 64)
        sets.append([dev(b.kp), dev(b.vp), dev(b.table), dev(np.array(b.lens, np.int32)), dev(b.start),
                     torch.empty(n, dtype=torch.uint8, device="cuda")])
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, (b, side) in enumerate(zip(batches, sides)):
            kp, vp, table, lens, start, ws = sets[i]
            lse = torch.empty((b.tokens, 4), device="cuda")
            outs[i].append(fp8q.fp4_kv_attention(b.q, kp, vp, table, lens, q_start=start, k_scale=b.k_scale,
                                                 v_scale=b.v_scale, lse=lse, workspace=ws, stream=side))
    torch.cuda.synchronize()
    for b, got in zip(batches, outs):
        b.check(*got[0])
        assert all(torch.equal(o, got[0][0]) and torch.equal(l, got[0][1]) for o, l in got[1:])
