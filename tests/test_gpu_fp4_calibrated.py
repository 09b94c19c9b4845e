"""A calibrator's frozen device pair as the scales of the 4-bit cache: written, read
back and attended to, against the oracle at the same scales."""
import numpy as np
import pytest
import torch

import paged_kv_cache_group_b200 as fp8q
from gpu_util import dev, host
from oracle import fp4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("headroom", [1.0, 1.5])
def test_write_read_and_attend_at_the_frozen_scales(headroom):
    heads, dim, tokens = 2, 64, 48
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn((tokens, heads, dim), generator=g).to(torch.bfloat16).cuda() * s for s in (3.0, 0.2))
    slots = torch.arange(tokens, device="cuda")
    calibrator = fp8q.KvCalibration(tokens, headroom, heads, dim, "cuda")
    assert calibrator.observe(k, v, slots) == fp8q.STEP_FREEZE
    fp8 = [torch.zeros((3, 16, heads, dim), dtype=torch.uint8, device="cuda") for _ in range(2)]
    calibrator.freeze_replay(*fp8)
    pair = calibrator.scale_dev
    scales = [float(x) for x in pair.cpu()]
    assert scales == [pytest.approx(float(t.abs().max()) * headroom / 448, rel=1e-6) for t in (k, v)]
    kp, vp = fp8q.fp4_kv_pools(3, 16, heads, dim)
    fp8q.fp4_kv_write(k, v, slots, kp, vp, scale_dev=pair)
    ko, vo = fp8q.fp4_kv_read(slots, kp, vp, scale_dev=pair)
    q = torch.randn((1, 4, dim), generator=g).to(torch.bfloat16).cuda()
    lens = torch.tensor([tokens], dtype=torch.int32, device="cuda")
    out = fp8q.fp4_kv_attention(q, kp, vp, dev(np.arange(3, dtype=np.int32)[None]), lens, scale_dev=pair)
    kept = []
    for x, pool, back, kind, scale in ((k, kp, ko, "k", scales[0]), (v, vp, vo, "v", scales[1])):
        x64 = x.double().cpu().numpy()
        want = np.zeros(pool.shape, np.uint8)
        fp4.write(x64, range(tokens), want, kind, scale)
        assert np.array_equal(host(pool), want)
        kept.append(fp4.read(range(tokens), want, kind) * scale)
        # 0.1771 of a block's largest as in the cache, and a rounding to bf16
        most = np.abs(x64).reshape(tokens, heads, -1, 16).max(-1).repeat(16, -1)
        assert np.all(np.abs(back.double().cpu().numpy() - x64) <= (0.1772 + 2.0 ** -8) * most)
    want, _, mean, reach = fp4.attention(q.double().cpu().numpy(), *kept, dim ** -0.5, 1)
    # as in test_gpu_fp4_attention: bf16 of the output, fp16 weights, fp32 scores
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -12 * (1 + reach[..., None])) * mean
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= bound)
    assert fp8q.fp8q_device_error(clear=True) == 0
