"""qk_norm_rope against the 64-bit oracle.

Bound.  fp32 throughout: the mean square carries at most dim additions of
2^-24, halved by the root, and rsqrt 2^-22; cosine and sine are off by at most
2^-21 (an fp32 half turn in [-1, 1] and two units of the function); products
and sums add 4 * 2^-24.  All of it scales with |a| + |b| of a pair:
    |error| <= 2^-8 |out| + (dim 2^-25 + 2^-20) (|a| + |b|)
and the result is rounded to bf16 (2^-8; 2^-134 below the normal range).
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_group_b200 as fp8q
from gpu_util import dev
from oracle import fp4

pytestmark = pytest.mark.gpu


def make(seed, tokens, heads, dim, pad=0, std=1.0):
    g = np.random.default_rng(seed)
    x = torch.from_numpy(g.standard_normal((tokens, heads * dim + pad)) * std).to(torch.bfloat16)
    x = x.cuda()
    return x[:, :heads * dim].unflatten(1, (heads, dim))


def check(got, x, positions, freq, weight, eps, interleaved, rope_scale):
    w = None if weight is None else weight.double().cpu().numpy()
    want, size = fp4.norm_rope(x.double().cpu().numpy(), positions, freq, w, float(np.float32(eps)),
                               interleaved, float(np.float32(rope_scale)))
    got = got.double().cpu().numpy()
    bound = 2.0 ** -8 * np.abs(want) + (x.shape[2] * 2.0 ** -25 + 2.0 ** -20) * size + 2.0 ** -133
    off = np.abs(got - want)
    assert np.all(off <= bound), float((off - bound).max())


@pytest.mark.parametrize("tokens,q_heads,k_heads,dim", [
    (1, 1, 1, 64), (1, 32, 4, 128), (3, 5, 1, 256), (16, 40, 8, 128), (17, 7, 3, 64), (1300, 2, 1, 64),
    (257, 16, 2, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("part", [1, 2, 4])
def test_norm_and_rotation(tokens, q_heads, k_heads, dim, interleaved, part):
    g = np.random.default_rng(dim + part)
    q, k = make(1, tokens, q_heads, dim), make(2, tokens, k_heads, dim, std=20.0)
    positions = g.integers(0, 5000, tokens)
    freq = fp8q.rope_inv_freq(dim // part, 1e4)
    wq, wk = make(3, 1, 1, dim)[0, 0], make(4, 1, 1, dim)[0, 0]
    qo, ko = fp8q.qk_norm_rope(q, k, dev(positions), freq, wq, wk, interleaved=interleaved,
                               rope_scale=1.25)
    f = freq.cpu().numpy()
    check(qo, q, positions, f, wq, 1e-6, interleaved, 1.25)
    check(ko, k, positions, f, wk, 1e-6, interleaved, 1.25)


@pytest.mark.parametrize("weights", [(False, False), (True, False), (False, True)])
def test_norm_of_either_only(weights):
    q, k = make(5, 9, 4, 128), make(6, 9, 2, 128)
    w = [make(7 + i, 1, 1, 128)[0, 0] if on else None for i, on in enumerate(weights)]
    positions = np.arange(9)
    freq = fp8q.rope_inv_freq(128)
    qo, ko = fp8q.qk_norm_rope(q, k, dev(positions), freq, *w)
    check(qo, q, positions, freq.cpu().numpy(), w[0], 1e-6, False, 1.0)
    check(ko, k, positions, freq.cpu().numpy(), w[1], 1e-6, False, 1.0)


def test_far_and_negative_positions():
    # the angle reaches 1e9 radians; fp64 positions * frequencies are off by 2^-23 of a turn there
    positions = np.array([0, 1, -1, 131071, 1000003, -999999, 10 ** 9, 2 ** 31 + 7], np.int64)
    q, k = make(8, 8, 2, 64), make(9, 8, 1, 64)
    freq = fp8q.rope_inv_freq(64, 1e6)
    qo, ko = fp8q.qk_norm_rope(q, k, dev(positions), freq)
    check(qo, q, positions, freq.cpu().numpy(), None, 0, False, 1.0)
    check(ko, k, positions, freq.cpu().numpy(), None, 0, False, 1.0)


def test_no_rotation():
    q, k = make(10, 5, 3, 64), make(11, 5, 1, 64)
    w = make(12, 1, 1, 64)[0, 0]
    none = torch.zeros(0, dtype=torch.float64, device="cuda")
    positions = np.arange(5)
    qo, ko = fp8q.qk_norm_rope(q, k, dev(positions), none, w)
    check(qo, q, positions, np.zeros(0), w, 1e-6, False, 1.0)
    assert torch.equal(ko, k)                                # neither norm nor rotation: a copy


def test_in_place_on_a_fused_projection():
    x = make(13, 21, 6, 128)                                 # 4 query, 1 key, 1 value head
    before = x.clone()
    q, k, v = x[:, :4], x[:, 4:5], x[:, 5:]
    positions = dev(np.arange(21) + 100)
    freq = fp8q.rope_inv_freq(128)
    w = make(14, 1, 1, 128)[0, 0]
    want = fp8q.qk_norm_rope(q, k, positions, freq, w, w)
    got = fp8q.qk_norm_rope(q, k, positions, freq, w, w, q_out=q, k_out=k)
    assert got[0].data_ptr() == x.data_ptr()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, before[:, 5:])


def test_strided_rows_keep_what_lies_between():
    q, k = make(15, 30, 4, 64, pad=40), make(16, 30, 2, 64, pad=8)
    base = torch.full((30, 4 * 64 + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    positions = np.arange(30) * 3
    freq = fp8q.rope_inv_freq(32)
    qo, ko = fp8q.qk_norm_rope(q, k, dev(positions), freq, q_out=base[:, :256].unflatten(1, (4, 64)))
    check(qo, q, positions, freq.cpu().numpy(), None, 0, False, 1.0)
    check(ko, k, positions, freq.cpu().numpy(), None, 0, False, 1.0)
    assert bool((base[:, 256:] == 5.0).all())


def test_zero_rows_and_eps():
    q, k = make(17, 4, 2, 64), make(18, 4, 1, 64)
    q[1] = 0.0
    w = make(19, 1, 1, 64)[0, 0]
    freq = fp8q.rope_inv_freq(64)
    qo, _ = fp8q.qk_norm_rope(q, k, dev(np.arange(4)), freq, w, eps=0.5)
    check(qo, q, np.arange(4), freq.cpu().numpy(), w, 0.5, False, 1.0)
    assert not bool(qo[1].any())


def test_a_head_with_a_nan_keeps_it_to_itself():
    q, k = make(20, 4, 4, 64), make(21, 4, 2, 64)
    w = make(22, 1, 1, 64)[0, 0]
    freq = fp8q.rope_inv_freq(64)
    clean = fp8q.qk_norm_rope(q, k, dev(np.arange(4)), freq, w, w)
    q[2, 1, 7] = float("nan")
    qo, ko = fp8q.qk_norm_rope(q, k, dev(np.arange(4)), freq, w, w)
    assert bool(qo[2, 1].isnan().all()) and torch.equal(ko, clean[1])
    qo[2, 1] = clean[0][2, 1]
    assert torch.equal(qo, clean[0])


def test_refusals_of_device_tensors():
    q, k = make(23, 4, 4, 64), make(24, 4, 2, 64)
    pos, freq = dev(np.arange(4)), fp8q.rope_inv_freq(64)
    w = make(25, 1, 1, 64)[0, 0]
    for args, kw in (((q, k, pos.int(), freq), {}), ((q, k, pos[:3], freq), {}),
                     ((q, k, pos, freq.float()), {}), ((q, k, pos, freq, w[:32]), {}),
                     ((q, k, pos, freq, w.float()), {}), ((q, k, pos.cpu(), freq), {}),
                     ((q, k, pos, freq.cpu()), {}), ((q, k, pos, freq), dict(q_out=k)),
                     ((q.transpose(1, 2), k.transpose(1, 2), pos, freq), {})):
        with pytest.raises(ValueError):
            fp8q.qk_norm_rope(*args, **kw)
    with pytest.raises(fp8q.Fp8qError):
        fp8q.qk_norm_rope(q, k, pos, fp8q.rope_inv_freq(128))            # wider than the head
    with pytest.raises(fp8q.Fp8qError):
        fp8q.qk_norm_rope(q, k, pos, freq, eps=-1.0)
