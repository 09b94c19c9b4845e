"""Refusals of the 4-bit cache's calls and of qk_norm_rope, each from a call that
is taken as it stands, at addresses that do not overlap.  Without a GPU a call
that is not refused fails at its launch instead; with one these tests do not
run, since the addresses are not memory."""
import random

import pytest
import torch

import paged_kv_cache_group_b200 as fp8q
import test_fp4_checks as checks
from paged_kv_cache_group_b200 import _abi

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not memory")

L = fp8q.lib
M = 1 << 30                                    # apart, and from the addresses of checks
CACHE = dict(checks.CACHE, k=M, v=2 * M, slots=3 * M, kp=4 * M, vp=5 * M)
ATTEND = dict(checks.ATTEND, q=M, kp=2 * M, vp=3 * M, table=4 * M, lens=5 * M, out=6 * M, ws=7 * M)
ROPE = dict(checks.ROPE, q=M, k=2 * M, qo=3 * M, ko=4 * M, pos=5 * M, freq=6 * M, qw=7 * M)


def call(name, base, **changes):
    a = dict(base, **changes)
    return getattr(L, name)(*(a[n] for n in base), None)


def rope(**changes):
    return call("qk_norm_rope", ROPE, **changes)


def refused(test):
    """The changes that a test of checks has refused."""
    return next(m.args[1] for m in test.pytestmark if m.name == "parametrize" and m.args[0] == "bad")


@pytest.mark.parametrize("name,base,test", [
    ("fp4_kv_write", CACHE, checks.test_cache_refusals), ("fp4_kv_read", CACHE, checks.test_cache_refusals),
    ("fp4_kv_attention", ATTEND, checks.test_attention_refusals), ("qk_norm_rope", ROPE, checks.test_rope_refusals)])
def test_each_refusal_alone(name, base, test):
    assert call(name, base) == _abi.ECUDA
    for bad in refused(test):
        apart = bad == dict(qos=4104)          # a stride of its own is refused in place alone, see below
        assert call(name, base, **bad) == (_abi.ECUDA if apart else _abi.EINVAL), bad


@pytest.mark.parametrize("heads,weight", [(dict(qh=0, q=None, qo=None), "qw"), (dict(kh=0, k=None, ko=None), "kw")])
def test_a_weight_without_heads_is_checked_all_the_same(heads, weight):
    assert rope(**heads) == _abi.ECUDA
    assert rope(**heads, **{weight: 9 * M}) == _abi.ECUDA
    for off in (2, 8):
        assert rope(**heads, **{weight: 9 * M + off}) == _abi.EINVAL


# Bytes between rows of 32 heads of 128 and of 4: 8192 and 1024.
def test_rows_that_share_memory_are_refused():
    at = ATTEND["q"]
    for out, stride, status in ((at, 4096, _abi.EINVAL), (at + 2 * 4096, 4096, _abi.EINVAL),
                                (at + 3 * 8192 - 16, 4096, _abi.EINVAL), (at + 3 * 8192, 4096, _abi.ECUDA),
                                (at - 3 * 8192 + 16, 4096, _abi.EINVAL), (at - 3 * 8192, 4096, _abi.ECUDA),
                                (at - 8192, 8192, _abi.EINVAL), (at + 8192, 5120, _abi.EINVAL)):
        assert call("fp4_kv_attention", ATTEND, out=out, os=stride) == status, (out - at, stride)
    # column ranges of one buffer
    assert call("fp4_kv_attention", ATTEND, qs=8192, out=at + 8192, os=8192) == _abi.ECUDA
    assert call("fp4_kv_attention", ATTEND, qs=8192, out=at + 8192 - 16, os=8192) == _abi.EINVAL
    assert call("fp4_kv_attention", ATTEND, qs=8192, out=at + 8192 + 16, os=8192) == _abi.EINVAL
    assert call("fp4_kv_read", CACHE, v=CACHE["k"]) == _abi.EINVAL
    assert call("fp4_kv_write", CACHE, v=CACHE["k"]) == _abi.ECUDA
    assert call("fp4_kv_read", CACHE, ks=1024, vs=1024, v=CACHE["k"] + 1024) == _abi.ECUDA


def test_rotation_in_place_and_across():
    q, k = ROPE["q"], ROPE["k"]
    assert rope(qo=q, ko=k) == _abi.ECUDA
    assert rope(qo=q, qos=4104) == _abi.EINVAL
    for bad in (dict(qo=k), dict(ko=q), dict(qo=q + 256), dict(ko=ROPE["qo"]), dict(qo=k - 3 * 8192)):
        assert rope(**bad) == _abi.EINVAL, bad
    fused = dict(q=M, k=M + 8192, qs=5120, ks=5120)             # 32 + 4 + 4 heads
    assert rope(**fused) == _abi.ECUDA
    assert rope(**fused, qo=M, ko=M + 8192, qos=5120, kos=5120) == _abi.ECUDA
    assert rope(**fused, qo=M + 1024, ko=4 * M, qos=5120) == _abi.EINVAL
    assert rope(**fused, ko=M + 9216, kos=5120) == _abi.ECUDA   # the value columns
    assert rope(**fused, qo=M, ko=M + 7168, qos=5120, kos=5120) == _abi.EINVAL
    assert rope(qo=k, kh=0, k=None, ko=None) == _abi.ECUDA


def test_shared_memory_against_every_byte():
    g = random.Random(3)
    for _ in range(400):
        t, h = g.randrange(1, 6), g.choice((1, 2))
        width = 64 * h
        qs, stride = (width + 8 * g.randrange(0, 40) for _ in range(2))
        if g.random() < 0.5:
            stride = qs
        off = 16 * g.randrange(-60 * t, 60 * t)
        a = {M + 2 * (i * qs) + x for i in range(t) for x in range(0, 2 * width, 16)}
        b = {M + off + 2 * (i * stride) + x for i in range(t) for x in range(0, 2 * width, 16)}
        got = call("fp4_kv_attention", ATTEND, b=t, t=t, h=h, qh=h, d=64, stride=9 * 64 * h, qs=qs, out=M + off, os=stride)
        assert got == (_abi.EINVAL if a & b else _abi.ECUDA), (t, h, qs, stride, off)
