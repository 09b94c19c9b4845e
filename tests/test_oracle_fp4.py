"""Pins of the 4-bit cache oracle: torch's E4M3 cast, brute force over exact
fractions, hand-worked blocks, and scalar loops."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import fp4


def test_e4m3_table_is_torchs():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(fp4.E4M3[:127], codes)


def _nearest_by_fractions(x, grid):
    best = min(range(len(grid)), key=lambda i: (abs(Fraction(float(x)) - Fraction(float(grid[i]))), i % 2))
    return best


@pytest.mark.parametrize("scale", [1.0, 0.1375, 3.0e-5, 2.0 ** 90])
def test_quantise_matches_brute_force(scale):
    g = np.random.default_rng(7)
    x = torch.from_numpy(g.standard_normal((40, 16)) * scale * 10.0 ** g.uniform(-4, 3, (40, 1)))
    x = x.to(torch.bfloat16).double().numpy()
    code, s = fp4.quantise(x, scale)
    s32 = np.float32(scale)
    for row in range(40):
        t = np.float32(np.float32(np.abs(x[row]).max()) / np.float32(6)) / s32
        assert s[row, 0] == _nearest_by_fractions(min(t, np.float32(448)), fp4.E4M3[:127])
        d = np.float32(fp4.E4M3[s[row, 0]]) * s32
        r = np.float32(1) / d if d > 0 else np.float32(0)
        for i in range(16):
            y = np.float32(abs(x[row, i])) * r
            want = _nearest_by_fractions(min(y, np.float32(6)), fp4.E2M1[:8])
            assert code[row, i] == want + 8 * bool(np.signbit(x[row, i]))


def test_hand_worked_block():
    x = np.array([[6.0, -6.0, 3.0, -3.0, 2.5, 3.5, 5.0, 1.75, 0.25, 0.75, 1.25, -0.25, 0.0, -0.0, 0.3, 7.0]])
    x[0, 15] = 5.5
    code, s = fp4.quantise(x, 1.0)
    assert s.tolist() == [[0x38]]                    # 6 / 6 = 1.0
    assert code[0].tolist() == [7, 15, 5, 13, 4, 6, 6, 4, 0, 2, 2, 8, 0, 8, 1, 7]


def test_zero_and_special_blocks():
    x = np.zeros((4, 16))
    x[1, 3] = np.inf
    x[2, 5] = np.nan
    x[2, 6] = 6.0
    x[3, 0] = -1e-30                                 # its scale rounds to zero
    code, s = fp4.quantise(x, 1.0)
    assert s[:, 0].tolist() == [0, 0x7E, 0x38, 0]
    assert code[1, 3] == 7 and code[2, 5] == 7 and code[2, 6] == 7
    assert code[3, 0] == 8 and fp4.values(code, s)[3, 0] == 0


@pytest.mark.parametrize("kind", ["k", "v"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_tile_has_every_byte_once(kind, dim):
    seen = np.concatenate([np.concatenate(fp4._offsets(t, dim, kind)) for t in range(16)])
    assert sorted(seen.tolist()) == list(range(9 * dim))


@pytest.mark.parametrize("kind", ["k", "v"])
def test_write_then_read(kind):
    g = np.random.default_rng(3)
    x = g.standard_normal((5, 2, 64))
    pool = np.zeros((3, 2, 2, 576), np.uint8)
    slots = np.array([95, 0, 17, 40, 33])
    fp4.write(x, slots, pool, kind, 0.5)
    code, s = fp4.quantise(x, 0.5)
    assert np.array_equal(fp4.read(slots, pool, kind), fp4.values(code, s))
    assert np.abs(fp4.read(slots, pool, kind) * 0.5 - x).max() < 0.6


def test_attention_matches_scalar_loops():
    g = np.random.default_rng(5)
    q, k, v = (g.standard_normal(s) for s in ((3, 4, 8), (6, 2, 8), (6, 2, 8)))
    out, lse, _, _ = fp4.attention(q, k, v, 0.4, 3, window=2)
    for i in range(3):
        for h in range(4):
            seen = [j for j in range(6) if 3 + i - 2 < j <= 3 + i]
            w = [np.exp(0.4 * sum(q[i, h, d] * k[j, h // 2, d] for d in range(8))) for j in seen]
            assert np.isclose(lse[i, h], np.log(sum(w)), rtol=1e-13)
            for d in range(8):
                want = sum(x * v[j, h // 2, d] for x, j in zip(w, seen)) / sum(w)
                assert np.isclose(out[i, h, d], want, rtol=1e-12, atol=1e-14)
    out, lse, _, _ = fp4.attention(q, k[:1], v[:1], 0.4, 3)      # two rows see nothing
    assert np.all(out[:2] == 0) and np.all(np.isneginf(lse[:2])) and np.all(out[2, 0] == v[0, 0])


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_by_hand(interleaved):
    x = np.array([[[3.0, 4.0, 0.0, 5.0]]])
    w = np.array([1.0, 2.0, 3.0, 4.0])
    out, _ = fp4.norm_rope(x, [2], np.array([np.pi / 4]), w, 0.0, interleaved, 1.0)
    y = x[0, 0] / np.sqrt(50 / 4) * w                # a quarter turn of the first pair
    assert np.allclose(out[0, 0], [-y[1], y[0], y[2], y[3]], atol=1e-15)
    out, _ = fp4.norm_rope(x, [1], np.array([0.0, np.pi / 2]), None, 0.0, interleaved, 2.0)
    want = [6, 8, -10, 0] if interleaved else [6, -10, 0, 8]
    assert np.allclose(out[0, 0], want, atol=1e-14)
