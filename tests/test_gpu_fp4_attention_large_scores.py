"""fp4_kv_attention with scores far above what fp32 resolves to a unit.

Codes, block scales and queries are chosen so that every score is an exact
multiple of a step: with q = +-2^m, block scales that are powers of two times
1 + i/8 in [2^-2, 2^3) and K's scale 1, q.k is a whole multiple of 2^(m-6) below
2^(m+15) for 256 dimensions, 21 bits, so its sum in fp32 is exact.  With
softmax_scale = 2^-3 different scores of a row are at least 2^(m-9) apart, 32
or more here: every weight but those of the largest score is below e^-32,
and the output is the mean of the tokens that share it.  One such weight is
off by nothing, an fp16 weight below it by at most 2^-36 of the largest, so
    |out error| <= 2^-8 |out| + (2^-11 + 2^-20) mean|v| + n (e^-32 + 2^-35) max|v|
and lse, some ten roundings of 2^-24 each of a number near the largest score,
    |lse error| <= 2^-20 |lse|
"""
import numpy as np
import pytest
import torch

from oracle import fp4
from test_gpu_fp4_attention import Batch

pytestmark = pytest.mark.gpu


def check(b, window=0):
    out, lse = b.call(window=window, scale=2.0 ** -3, k_scale=1.0, v_scale=b.v_scale)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    for i, n in enumerate(b.lens):
        rows = slice(b.start[i], b.start[i + 1])
        k, v = b.kv(i)
        want, want_lse, mean, _ = fp4.attention(b.q64[rows], k, v, 2.0 ** -3, b.news[i], window)
        bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -20) * mean + \
            n * (np.exp(-32.0) + 2.0 ** -35) * np.abs(v).max()
        off = np.abs(out[rows] - want)
        assert np.all(off <= bound), (i, n, float((off - bound).max()))
        off = np.abs(lse[rows] - want_lse) - 2.0 ** -20 * np.abs(want_lse)
        assert np.all(off <= 0), (i, n, float(off.max()))


def batch(dim, heads, group, lens, news, m):
    b = Batch(50 + dim + m, dim, heads, group, 16, lens, news)
    b.k_scale = 1.0
    b.q.copy_(torch.where(b.q < 0, -1.0, 1.0) * 2.0 ** m)
    b.q64 = b.q.double().cpu().numpy()
    return b


@pytest.mark.parametrize("m", [14, 17, 20, 30, 60, 100])
@pytest.mark.parametrize("dim,heads,group,lens,news", [
    (64, 1, 1, [700, 33], None), (128, 2, 8, [1500, 40, 1], None), (256, 1, 4, [300, 5], None),
    (128, 4, 12, [2500], None), (64, 2, 5, [90, 260], [3, 5]),
    (64, 2, 8, [300, 700], [20, 40]), (128, 1, 12, [400, 90], [30, 7]), (256, 1, 16, [300, 64], [9, 9])])
def test_the_largest_score_takes_all(dim, heads, group, lens, news, m):
    check(batch(dim, heads, group, lens, news, m))


@pytest.mark.parametrize("news,group", [([1, 1], 4), ([40, 50], 8)])
@pytest.mark.parametrize("m", [14, 40])
def test_in_a_window(news, group, m):
    check(batch(64, 2, group, [500, 700], news, m), window=150)


def test_tokens_with_the_same_largest_score_share_it():
    for news, group in ((None, 4), ([30, 30], 4)):
        b = batch(64, 1, group, [600, 250], news, 33)
        b.kp[:] = np.where(b.kp == 255, b.kp, 0)
        for i in range(2):                                   # all keys are alike: any weight is 1 / n
            for page in b.table[i, :-(-b.lens[i] // 16)]:
                b.kp[page, ..., :8 * 64], b.kp[page, ..., 8 * 64:] = 0x27, 0x38
        check(b)
