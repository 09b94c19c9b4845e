"""qk_norm_rope of queries alone or keys alone: a tensor without heads has no part in
the call, whatever weight comes with it."""
import pytest
import torch

import paged_kv_cache_group_b200 as fp8q
from test_gpu_qk_norm_rope import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,tokens", [(64, 1), (128, 37), (256, 5)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_one_side_without_heads(dim, tokens, interleaved):
    q, k = make(1, tokens, 4, dim), make(2, tokens, 2, dim)
    w = [make(3 + i, 1, 1, dim)[0, 0] for i in range(2)]
    positions = torch.arange(tokens, device="cuda") * 7
    freq = fp8q.rope_inv_freq(dim, 1e5)
    qo, ko = fp8q.qk_norm_rope(q, k, positions, freq, *w, interleaved=interleaved)
    none, only_k = fp8q.qk_norm_rope(q[:, :0], k, positions, freq, *w, interleaved=interleaved)
    assert none.shape == (tokens, 0, dim) and torch.equal(only_k, ko)
    only_q, none = fp8q.qk_norm_rope(q, k[:, :0], positions, freq, *w, interleaved=interleaved)
    assert none.shape == (tokens, 0, dim) and torch.equal(only_q, qo)
    # a weight at an odd place of a larger parameter is refused, with heads or without
    odd = torch.cat([w[0], w[0]])[1:dim + 1]
    for heads in (4, 0):
        with pytest.raises(fp8q.Fp8qError):
            fp8q.qk_norm_rope(q[:, :heads], k, positions, freq, odd, w[1])
