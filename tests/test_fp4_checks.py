"""Refusals of the 4-bit cache and of qk_norm_rope that need no GPU: every call
returns before anything is enqueued, and the pointers are never followed."""
import math

import pytest
import torch

import paged_kv_cache_group_b200 as fp8q
from paged_kv_cache_group_b200 import _abi

L = fp8q.lib
F = 1 << 20
CACHE = dict(k=F, v=F, ks=512, vs=512, slots=F, t=4, h=4, d=128, kp=F, vp=F, bs=16, stride=4608,
             nb=8, ksc=1.0, vsc=1.0, sd=None)


@pytest.mark.parametrize("name", ["fp4_kv_write", "fp4_kv_read"])
@pytest.mark.parametrize("bad", [
    dict(t=-1), dict(h=0), dict(h=65537), dict(d=96), dict(d=0), dict(ks=504), dict(vs=516),
    dict(bs=0), dict(bs=8), dict(bs=24), dict(stride=4592), dict(stride=4616), dict(nb=-1),
    dict(nb=1 << 62), dict(k=None), dict(v=F + 8), dict(slots=None), dict(slots=F + 4),
    dict(kp=None), dict(vp=F + 8), dict(ksc=0.0), dict(vsc=-1.0), dict(ksc=math.nan),
    dict(vsc=math.inf), dict(ksc=1e-30), dict(vsc=1e30), dict(sd=F + 4)],
    ids=lambda b: "-".join(f"{k}={v}" for k, v in b.items()))
def test_cache_refusals(name, bad):
    a = dict(CACHE, **bad)
    assert getattr(L, name)(*(a[n] for n in CACHE), None) == _abi.EINVAL


@pytest.mark.parametrize("name", ["fp4_kv_write", "fp4_kv_read"])
def test_no_tokens_is_a_no_op(name):
    a = dict(CACHE, t=0, k=None, v=None, slots=None, kp=None, vp=None, nb=0)
    assert getattr(L, name)(*(a[n] for n in CACHE), None) == _abi.OK


ATTEND = dict(q=F, qs=4096, kp=F, vp=F, bs=16, stride=4608, nb=8, h=4, d=128, table=F, ts=10,
              tw=10, lens=F, start=None, b=3, t=3, qh=32, scale=0.1, window=0, ksc=1.0, vsc=1.0,
              sd=None, out=F, os=4096, lse=None, ws=F, wsb=1 << 30)


@pytest.mark.parametrize("bad", [
    dict(b=-1), dict(t=4), dict(t=-1, start=F), dict(qh=30), dict(qh=0), dict(h=0), dict(d=80),
    dict(t=1 << 30, start=F), dict(qs=4088), dict(os=4100), dict(ts=9), dict(tw=-1),
    dict(tw=1 << 27, ts=1 << 27), dict(ts=1 << 61, b=1 << 29, t=1 << 29, qh=4, h=1, qs=512, os=512),
    dict(window=-1), dict(scale=0.0), dict(scale=math.nan), dict(scale=math.inf), dict(q=None),
    dict(q=F + 8), dict(out=None), dict(out=F + 2), dict(lens=None), dict(lens=F + 2),
    dict(start=F + 2), dict(lse=F + 1), dict(table=None), dict(table=F + 2), dict(ws=None),
    dict(ws=F + 8), dict(wsb=100), dict(kp=None), dict(ksc=0.0), dict(bs=12), dict(stride=4600)],
    ids=lambda b: "-".join(f"{k}={v}" for k, v in b.items()))
def test_attention_refusals(bad):
    a = dict(ATTEND, **bad)
    assert L.fp4_kv_attention(*(a[n] for n in ATTEND), None) == _abi.EINVAL


@pytest.mark.parametrize("empty", [dict(b=0, t=0), dict(t=0, start=F)])
def test_attention_of_nothing_is_a_no_op(empty):
    a = dict(ATTEND, q=None, out=None, ws=None, wsb=0, **empty)
    assert L.fp4_kv_attention(*(a[n] for n in ATTEND), None) == _abi.OK


def test_workspace_sizes():
    f = fp8q.fp4_kv_attention_workspace
    assert f(0, 0, 32, 4, 128) == 0
    assert 0 < f(1, 1, 32, 4, 128) < 1 << 23
    assert f(4, 4000, 32, 4, 128) <= 1 << 24
    for bad in ((-1, 1, 32, 4, 128), (1, 1, 30, 4, 128), (1, 1, 32, 4, 100), (1, 1 << 31, 32, 4, 128)):
        with pytest.raises(ValueError):
            f(*bad)


ROPE = dict(q=F, k=F, qs=4096, ks=512, qo=F, ko=F, qos=4096, kos=512, pos=F, freq=F, qw=F, kw=None,
            t=4, qh=32, kh=4, d=128, r=128, inter=0, eps=1e-6, scale=1.0)


@pytest.mark.parametrize("bad", [
    dict(t=-1), dict(t=1 << 31), dict(qh=-1), dict(kh=-1), dict(qh=0, kh=0), dict(qh=65536),
    dict(d=96), dict(r=136), dict(r=4), dict(r=-8), dict(eps=-1.0), dict(eps=math.nan),
    dict(scale=math.inf), dict(q=None), dict(ko=None), dict(q=F + 8), dict(qo=F + 2),
    dict(qw=F + 8), dict(qs=4088), dict(kos=516), dict(ks=1 << 62), dict(pos=None),
    dict(pos=F + 4), dict(freq=None), dict(freq=F + 4), dict(qos=4104)],
    ids=lambda b: "-".join(f"{k}={v}" for k, v in b.items()))
def test_rope_refusals(bad):
    a = dict(ROPE, **bad)
    assert L.qk_norm_rope(*(a[n] for n in ROPE), None) == _abi.EINVAL


def test_rope_of_no_tokens_is_a_no_op():
    a = dict(ROPE, t=0, q=None, k=None, qo=None, ko=None, pos=None, freq=None)
    assert L.qk_norm_rope(*(a[n] for n in ROPE), None) == _abi.OK


# ---- the binding, on host tensors ----------------------------------------

K = torch.zeros((16, 4, 128), dtype=torch.bfloat16)
SLOTS = torch.zeros(16, dtype=torch.int64)
POOL = torch.zeros(fp8q.fp4_kv_pool_shape(4, 32, 4, 128), dtype=torch.uint8)


def test_pool_shapes():
    assert fp8q.fp4_kv_pool_shape(4, 32, 4, 128) == (4, 4, 2, 1152)
    k, v = fp8q.fp4_kv_pools(2, 16, 1, 64, device="cpu")
    assert k.shape == v.shape == (2, 1, 1, 576) and not k.any()
    for bad in ((4, 8, 4, 128), (4, 0, 4, 128), (4, 16, 4, 96)):
        with pytest.raises(ValueError):
            fp8q.fp4_kv_pool_shape(*bad)


@pytest.mark.parametrize("v", [K[:15], K[:, :, :64], K[:, :2], K.view(16, 512)],
                         ids=["rows", "width", "heads", "rank"])
def test_mismatched_v_is_refused(v):
    with pytest.raises(ValueError):
        fp8q.fp4_kv_write(K, v, SLOTS, POOL, POOL)


def test_host_tensors_are_refused():
    with pytest.raises(TypeError):
        fp8q.fp4_kv_write(K, K, SLOTS, POOL, POOL)
    with pytest.raises(TypeError):
        fp8q.fp4_kv_read(SLOTS, POOL, POOL)
    with pytest.raises(TypeError):
        fp8q.fp4_kv_attention(K, POOL, POOL, torch.zeros((16, 2), dtype=torch.int32),
                              torch.zeros(16, dtype=torch.int32))
    with pytest.raises(TypeError):
        fp8q.qk_norm_rope(K, K, SLOTS, torch.zeros(64, dtype=torch.float64))


@pytest.mark.parametrize("q,k", [(K[:15], K), (K[:, :, :64], K), (K.view(16, 512), K)],
                         ids=["rows", "width", "rank"])
def test_mismatched_q_and_k_are_refused(q, k):
    with pytest.raises(ValueError):
        fp8q.qk_norm_rope(q, k, SLOTS, torch.zeros(64, dtype=torch.float64))


def test_inv_freq():
    plain = fp8q.rope_inv_freq(64, 1e6, device="cpu")
    assert plain.dtype == torch.float64 and plain.shape == (32,)
    assert plain.tolist() == [1e6 ** (-2.0 * i / 64) for i in range(32)]
    assert torch.allclose(fp8q.rope_inv_freq(64, 1e6, 8.0, device="cpu"), plain / 8, rtol=1e-15)
    parts = fp8q.rope_inv_freq(64, 1e6, 8.0, trained_length=32768, device="cpu")
    turns = 32768 * plain / (2 * math.pi)
    assert torch.equal(parts[turns > 64], plain[turns > 64])
    assert torch.allclose(parts[turns < 0.5], plain[turns < 0.5] / 8, rtol=1e-15)
    ratio = parts / plain
    assert bool((ratio[1:] <= ratio[:-1]).all()) and 0.125 < ratio[15] < 1
    for bad in (dict(rotary_dim=63), dict(rotary_dim=64, base=1.0), dict(rotary_dim=64, stretch=0.5),
                dict(rotary_dim=64, stretch=2.0, trained_length=0)):
        with pytest.raises(ValueError):
            fp8q.rope_inv_freq(device="cpu", **bad)


@pytest.mark.parametrize("name", ["fp4_kv_write", "fp4_kv_read", "fp4_kv_attention", "qk_norm_rope"])
def test_binding_exposes_the_abi_names(name):
    assert callable(getattr(fp8q, name)) and name in _abi.SIGNATURES
