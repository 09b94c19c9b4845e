"""Refusals of the 4-bit cache's calls and of qk_norm_rope, each from a call that
is taken as it stands, at addresses that do not overlap.  Without a GPU a call
that is not refused fails at its launch instead; with one these tests do not
run, since the addresses are not memory."""
import pytest
import torch

import paged_kv_cache_group_b200 as fp8q
from paged_kv_cache_group_b200 import _abi

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not memory")

L = fp8q.lib
M = 1 << 20
ROPE = dict(q=M, k=2 * M, qs=4096, ks=512, qo=3 * M, ko=4 * M, qos=4096, kos=512, pos=5 * M, freq=6 * M,
            qw=7 * M, kw=None, t=4, qh=32, kh=4, d=128, r=128, inter=0, eps=1e-6, scale=1.0)


def rope(**changes):
    a = dict(ROPE, **changes)
    return L.qk_norm_rope(*(a[n] for n in ROPE), None)


@pytest.mark.parametrize("heads,weight", [(dict(qh=0, q=None, qo=None), "qw"), (dict(kh=0, k=None, ko=None), "kw")])
def test_a_weight_without_heads_is_checked_all_the_same(heads, weight):
    assert rope(**heads) == _abi.ECUDA
    assert rope(**heads, **{weight: 8 * M}) == _abi.ECUDA
    for off in (2, 8):
        assert rope(**heads, **{weight: 8 * M + off}) == _abi.EINVAL
