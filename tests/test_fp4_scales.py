"""The tensor scales that a calibrator freezes for the FP8 cache, as scales of the
4-bit one.

Bound.  With a normal block scale b = amax / 6 / s (1 + e), |e| <= 2^-4, a value is
off by at most half an E2M1 step times b s, 1 * amax / 6 (1 + 2^-4) = 0.1771 amax, or,
where b was rounded down, by what lies beyond the largest code: 2^-4 amax.  fp32
roundings add 2^-20 of it."""
import numpy as np
import pytest

from oracle import core, fp4


@pytest.mark.parametrize("headroom", [1.0, 1.25, 2.0, 6.0])
@pytest.mark.parametrize("size", [1e-6, 1.0, 3e4])
def test_a_frozen_scale_keeps_every_normal_block(headroom, size):
    g = np.random.default_rng(9)
    x = g.standard_normal((4000, 16)) * 10.0 ** g.uniform(-5, 0, (4000, 1)) * size
    x = (x.astype(np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32).astype(np.float64)
    amax = np.abs(x).max()
    scale = float(core.freeze_scale(amax, headroom))
    x = np.concatenate([x, x[:50] * (5.9 * headroom * amax / np.abs(x[:50]).max())])   # more than was calibrated
    code, s = fp4.quantise(x, scale)
    assert s.max() <= 0x7E
    back = fp4.values(code, s) * scale
    most = np.abs(x).max(-1, keepdims=True)
    normal = (most >= 6 * 2.0 ** -6 * scale)[:, 0]
    assert normal[most[:, 0] >= amax * headroom / 4778].all() and (~normal).any()
    assert np.all(np.abs(back - x)[normal] <= (0.1771 + 2.0 ** -20) * most[normal])
    assert np.all(s[~normal] <= 0x08)
