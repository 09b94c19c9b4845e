"""fp4_kv_write and fp4_kv_read against the 64-bit oracle: whole pools byte for
byte, read-back values bit for bit."""
import numpy as np
import pytest
import torch

import paged_kv_cache_group_b200 as fp8q
from gpu_util import dev, dev_bf16, first_mismatch, host
from oracle import fp4

pytestmark = pytest.mark.gpu
SENTINEL = 0x5A


def rows(g, tokens, heads, dim, pad=0, std=1.0):
    """bf16 [tokens, heads, dim] on the device (rows `pad` elements apart) and in fp64."""
    x = torch.from_numpy(g.standard_normal((tokens, heads * dim + pad)) * std)
    hit = torch.from_numpy(g.random(x.shape) < 0.01)
    x[hit] *= 30.0
    x = x.to(torch.bfloat16)
    view = x.cuda()[:, :heads * dim].unflatten(1, (heads, dim))
    return view, x[:, :heads * dim].unflatten(1, (heads, dim)).double().numpy()


def pools(blocks, size, heads, dim):
    shape = fp8q.fp4_kv_pool_shape(blocks, size, heads, dim)
    return np.full(shape, SENTINEL, np.uint8), np.full(shape, SENTINEL, np.uint8)


def bf16_of(values, scale):
    """bf16(fp32(value * scale)) as fp32 numpy."""
    p = torch.from_numpy(values * float(np.float32(scale))).float()
    return p.to(torch.bfloat16).float().numpy()


def same(got, want, what):
    assert np.array_equal(got, want), what + ": " + first_mismatch(got, want)


@pytest.mark.parametrize("tokens,heads,dim,size,pad,skip", [
    (1, 1, 64, 16, 0, 0), (1, 4, 128, 16, 0, 0), (16, 4, 128, 16, 0, 2), (15, 3, 256, 32, 8, 1),
    (17, 5, 64, 48, 40, 3), (257, 8, 128, 128, 0, 29), (600, 2, 64, 16, 128, 0), (33, 1, 256, 16, 0, 0)])
@pytest.mark.parametrize("device_scales", [False, True])
def test_write_and_read_back(tokens, heads, dim, size, pad, skip, device_scales):
    g = np.random.default_rng(tokens * 1000 + heads * 10 + dim)
    blocks = -(-tokens // size) + 3
    k, k64 = rows(g, tokens, heads, dim, pad)
    v, v64 = rows(g, tokens, heads, dim, 2 * pad, 5.0)
    slots = g.permutation(blocks * size)[:tokens].astype(np.int64)
    slots[g.permutation(tokens)[:skip]] = -1
    ks, vs = 0.0123, 0.31
    kw = dict(scale_dev=torch.tensor([ks, vs], device="cuda")) if device_scales else \
        dict(k_scale=ks, v_scale=vs)
    kp, vp = pools(blocks, size, heads, dim)
    dkp, dvp = dev(kp), dev(vp)
    fp8q.fp4_kv_write(k, v, dev(slots), dkp, dvp, **kw)
    fp4.write(k64, slots, kp, "k", ks)
    fp4.write(v64, slots, vp, "v", vs)
    same(host(dkp), kp, "K pool")
    same(host(dvp), vp, "V pool")
    ko = torch.full((tokens, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = torch.full((tokens, heads * dim + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    vo3 = vo[:, :heads * dim].unflatten(1, (heads, dim))
    fp8q.fp4_kv_read(dev(slots), dkp, dvp, k_out=ko, v_out=vo3, **kw)
    live = slots >= 0
    for got, pool, kind, s in ((ko, kp, "k", ks), (vo3, vp, "v", vs)):
        got = got.float().cpu().numpy()
        same(got[live], bf16_of(fp4.read(slots[live], pool, kind), s), kind)
        assert np.all(got[~live] == 7.0)
    assert bool((vo[:, heads * dim:] == 7.0).all())
    same(host(dkp), kp, "K pool after the read")
    assert fp8q.fp8q_device_error(clear=True) == 0


@pytest.mark.parametrize("scale", [1.0, 0.0123, 2.0 ** -96, 2.0 ** 96, 3.0e-12])
def test_every_bf16_value(scale):
    # each value with three block maxima, one of them its own; NaN and infinity included
    bits = np.arange(65536, dtype=np.uint16)
    x = np.repeat(bits[:, None], 64, 1)
    g = np.random.default_rng(2)
    x[:, 17] = g.integers(0, 0x7F80, 65536)                # blocks 1 and 2: a random finite maximum
    x[:, 40] = g.permutation(bits & 0x7FFF)
    k = dev_bf16(x.reshape(65536, 1, 64))
    k64 = k.double().cpu().numpy()
    kp, vp = pools(4096, 16, 1, 64)
    dkp, dvp = dev(kp), dev(vp)
    slots = np.arange(65536, dtype=np.int64)
    fp8q.fp4_kv_write(k, k, dev(slots), dkp, dvp, scale, scale)
    for got, kind in ((dkp, "k"), (dvp, "v")):
        # the oracle's pool, laid out at once
        code, s = fp4.quantise(k64[:, 0], scale)
        got = host(got).reshape(4096, 576)
        c = np.stack([got[:, fp4._offsets(t, 64, kind)[0]] for t in range(16)], 1).reshape(65536, 32)
        z = np.stack([got[:, fp4._offsets(t, 64, kind)[1]] for t in range(16)], 1).reshape(65536, 4)
        same(z, s, "scale codes")
        same(c, code[:, 0::2] | code[:, 1::2] << 4, "codes")
        assert not np.any((z & 0x7F) == 0x7F)              # no NaN in the cache


def test_slots_past_the_pool_are_reported():
    k = torch.ones((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    kp, vp = (dev(p) for p in pools(2, 16, 2, 64))
    slots = dev(np.array([32, 5, 1 << 40], np.int64))
    fp8q.fp4_kv_write(k, k, slots, kp, vp)
    assert fp8q.fp8q_device_error(clear=True) == fp8q.DEVERR_SLOT_OUT_OF_RANGE
    want = pools(2, 16, 2, 64)[0]
    fp4.write(np.ones((1, 2, 64)), [5], want, "k", 1.0)
    same(host(kp), want, "K pool")
    out = torch.full((3, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    out2 = out.clone()
    fp8q.fp4_kv_read(slots, kp, vp, k_out=out, v_out=out2)
    assert fp8q.fp8q_device_error(clear=True) == fp8q.DEVERR_SLOT_OUT_OF_RANGE
    # 1 / 6 is 11/64 in E4M3, 1 / (11/64) = 5.8 is code 6: 6 * 11/64
    assert out[:, 0, 0].tolist() == [9.0, 1.03125, 9.0] and torch.equal(out, out2)


@pytest.mark.parametrize("scales,k_written,v_written", [
    ((float("nan"), 1.0), False, True), ((1.0, 0.0), True, False), ((-1.0, 1e30), False, False)])
def test_bad_device_scales_leave_their_tensor_alone(scales, k_written, v_written):
    k = torch.ones((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    kp, vp = (dev(p) for p in pools(1, 16, 1, 64))
    sd = torch.tensor(scales, device="cuda")
    slots = dev(np.zeros(1, np.int64))
    fp8q.fp4_kv_write(k, k, slots, kp, vp, scale_dev=sd)
    assert fp8q.fp8q_device_error(clear=True) == fp8q.DEVERR_BAD_SCALE
    assert bool((kp != SENTINEL).any()) == k_written and bool((vp != SENTINEL).any()) == v_written
    ko, vo = (torch.full((1, 1, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fp8q.fp4_kv_read(slots, kp, vp, scale_dev=sd, k_out=ko, v_out=vo)
    assert fp8q.fp8q_device_error(clear=True) == fp8q.DEVERR_BAD_SCALE
    assert bool((ko == 9).all()) != k_written and bool((vo == 9).all()) != v_written


def test_a_slot_may_be_read_many_times_and_outputs_default_to_zero():
    g = np.random.default_rng(4)
    k, k64 = rows(g, 2, 2, 128)
    kp, vp = fp8q.fp4_kv_pools(2, 16, 2, 128)
    fp8q.fp4_kv_write(k, k, dev(np.array([3, 20], np.int64)), kp, vp)
    ko, vo = fp8q.fp4_kv_read(dev(np.array([20, 3, -1, 20], np.int64)), kp, vp)
    assert torch.equal(ko, vo) and torch.equal(ko[0], ko[3]) and not bool(ko[2].any())
    code, s = fp4.quantise(k64, 1.0)
    same(ko[:2].float().cpu().numpy(), bf16_of(fp4.values(code, s)[::-1].copy(), 1.0), "rows")


def test_blocks_more_than_four_gigabytes_apart():
    stride = (1 << 30) + 16
    both = [torch.full((5 * stride,), SENTINEL, dtype=torch.uint8, device="cuda") for _ in range(2)]
    kp, vp = (t.as_strided((5, 1, 1, 576), (stride, 576, 576, 1)) for t in both)
    g = np.random.default_rng(6)
    k, k64 = rows(g, 5, 1, 64)
    slots = np.array([79, 64, 50, 2, 16], np.int64)
    fp8q.fp4_kv_write(k, k, dev(slots), kp, vp)
    for p, kind in ((kp, "k"), (vp, "v")):
        want = pools(5, 16, 1, 64)[0]
        fp4.write(k64, slots, want, kind, 1.0)
        same(host(p.contiguous()), want, kind)
    assert bool((both[0][576:stride] == SENTINEL).all())
    ko, _ = fp8q.fp4_kv_read(dev(slots), kp, vp)
    code, s = fp4.quantise(k64, 1.0)
    same(ko.float().cpu().numpy(), bf16_of(fp4.values(code, s), 1.0), "rows")
    # attention over a block behind the fourth gigabyte: one token, so out is its V
    out = fp8q.fp4_kv_attention(k[:1], kp, vp, dev(np.array([[4]], np.int32)),
                                dev(np.array([1], np.int32)))
    want = fp4.read([64], host(vp.contiguous()), "v")
    same(out.float().cpu().numpy(), bf16_of(want, 1.0), "attention")


def test_on_a_stream_of_its_own():
    g = np.random.default_rng(8)
    k, _ = rows(g, 300, 4, 128)
    slots = dev(np.arange(300, dtype=np.int64))
    kp, vp = fp8q.fp4_kv_pools(20, 16, 4, 128)
    kp2, vp2 = fp8q.fp4_kv_pools(20, 16, 4, 128)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    fp8q.fp4_kv_write(k, k, slots, kp, vp, stream=side)
    a = fp8q.fp4_kv_read(slots, kp, vp, stream=side.cuda_stream)
    torch.cuda.synchronize()
    fp8q.fp4_kv_write(k, k, slots, kp2, vp2)
    b = fp8q.fp4_kv_read(slots, kp2, vp2)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(kp, kp2)


def test_refusals_of_device_tensors():
    k = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    kp, vp = fp8q.fp4_kv_pools(2, 16, 2, 64)
    slots = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        fp8q.fp4_kv_write(k[:, :1], k[:, :1], slots, kp, vp)              # other heads than the pool
    with pytest.raises(ValueError):
        fp8q.fp4_kv_write(k.transpose(1, 2), k.transpose(1, 2), slots, kp, vp)
    with pytest.raises(ValueError):
        fp8q.fp4_kv_write(k, k, slots.int(), kp, vp)
    with pytest.raises(ValueError):
        fp8q.fp4_kv_write(k, k, slots[:3], kp, vp)
    with pytest.raises(ValueError):
        fp8q.fp4_kv_write(k, k, slots, kp, vp[:1])
    with pytest.raises(TypeError):
        fp8q.fp4_kv_write(k, k, slots, kp.view(torch.int8), vp)
    with pytest.raises(ValueError):
        fp8q.fp4_kv_write(k, k, slots, kp, vp, scale_dev=torch.ones(2))
    with pytest.raises(fp8q.Fp8qError):
        fp8q.fp4_kv_write(k.expand(4, 2, 64)[:1].expand(4, 2, 64), k, slots, kp, vp)   # stride 0
    with pytest.raises(fp8q.Fp8qError):
        fp8q.fp4_kv_write(k, k, slots, kp, vp, 0.0, 1.0)
