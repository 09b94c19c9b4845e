"""FP8 E4M3 quantization for B200: per-token 1x128-group activation
quantization, the paged KV-cache quantize-and-scatter, and online calibration
of the KV scales; and a paged KV cache held in 4 bits: written, read back and
attended to, with the norm and rotation of queries and keys before it.

The compute is the CUDA library libfp8q.so (C ABI: include/fp8q.h).  This
module only marshals torch tensors (device memory) and streams into those
calls; every step runs in the library's kernels.  Function names match the C
ABI.  Importing fails if the library has not been built.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from . import _abi
from ._abi import (CALIB_STATE_BYTES, DEVERR_BAD_SCALE, DEVERR_BAD_SEQUENCE,  # noqa: F401
                   DEVERR_SLOT_OUT_OF_RANGE, DEVERR_WAIT, MAX_STAGED_TOKENS, PROVISIONAL_SCALE, STEP_FREEZE, STEP_FROZEN, STEP_STAGE,
                   STEP_STAGE_DECLINED, CalibStats, Fp8qError)

lib = _abi.load()

_BYTE_TYPES = (torch.uint8, torch.float8_e4m3fn)


def _check(name: str, status: int) -> None:
    if status != _abi.OK:
        raise Fp8qError(name, status, lib.fp8q_status_string(status).decode())


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _bf16_rows(t: torch.Tensor, name: str):
    """``[T, ...]`` bf16 whose rows (all dimensions after the first) are
    contiguous; returns (rows, row stride in elements, elements per row)."""
    if t.dtype != torch.bfloat16 or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA bfloat16 tensor")
    if t.dim() < 2:
        raise ValueError(f"{name} must have a row dimension and at least one more")
    rows = t.shape[0]
    inner = 1
    for size in t.shape[1:]:
        inner *= size
    if t.numel() == 0:          # no data: any strides (an empty array may carry zeros)
        return rows, inner, inner
    expect = 1
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and stride != expect:
            raise ValueError(f"{name} rows must be contiguous")
        expect *= size
    return rows, (t.stride(0) if rows > 1 else inner), inner


def _kv_rows(k: torch.Tensor, v: torch.Tensor):
    """K and V ``[T, heads, dim]`` of the same shape (rows contiguous, row
    strides may differ); returns (T, key_stride, value_stride, heads, dim).
    The shapes are checked before anything else, so a mismatched V is refused
    whatever device it is on."""
    if k.dim() != 3 or v.dim() != 3:
        raise ValueError("k and v must both be [T, heads, dim]")
    if tuple(k.shape) != tuple(v.shape):
        raise ValueError(f"k and v must have the same shape, got {tuple(k.shape)} and "
                         f"{tuple(v.shape)}")
    t, ks, _ = _bf16_rows(k, "k")
    _, vs, _ = _bf16_rows(v, "v")
    return t, ks, vs, k.shape[1], k.shape[2]


def _check_slots(slot_mapping: torch.Tensor, t: int) -> None:
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() < t:
        raise ValueError("slot_mapping must be int64 with one entry per token")
    if t and (not slot_mapping.is_cuda or not slot_mapping.is_contiguous()):
        raise ValueError("slot_mapping must be a contiguous CUDA tensor")


def _check_scale_pair(t: torch.Tensor | None, name: str) -> None:
    """A device ``{k, v}`` fp32 pair the library reads or writes."""
    if t is None:
        return
    if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous() or t.numel() < 2:
        raise ValueError(f"{name} must be a contiguous CUDA float32 tensor of 2 elements")


# ---------------------------------------------------------------------------
# activation quantization


def fp8_group_quant(x: torch.Tensor, q: torch.Tensor | None = None,
                    scales: torch.Tensor | None = None, stream=None):
    """Quantize a bf16 ``[m, k]`` activation (k % 128 == 0, rows may be
    strided) into E4M3 codes ``q [m, k]`` and fp32 ``scales [m, k/128]``."""
    m, stride, k = _bf16_rows(x, "x")
    if q is None:
        q = torch.empty((m, k), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((m, k // 128), dtype=torch.float32, device=x.device)
    if q.dtype not in _BYTE_TYPES or not q.is_contiguous() or q.numel() < m * k:
        raise ValueError("q must be a contiguous uint8/float8_e4m3fn tensor of m*k elements")
    if scales.dtype != torch.float32 or not scales.is_contiguous() or \
            scales.numel() < m * (k // 128):
        raise ValueError("scales must be a contiguous float32 tensor of m*(k/128) elements")
    _check("fp8_group_quant", lib.fp8_group_quant(
        _ptr(x), stride, _ptr(q), _ptr(scales), m, k, _stream(stream)))
    return q, scales


def ceil16(m: int) -> int:
    """Rows a GEMM padded to 16-row tiles is handed for an m-row activation."""
    return (m + 15) // 16 * 16


def fp8_group_quant_kmajor(x: torch.Tensor, m_pad: int | None = None,
                           q: torch.Tensor | None = None, scales_km: torch.Tensor | None = None,
                           stream=None):
    """Quantize a bf16 ``[m, k]`` activation for a padded FP8 GEMM: codes
    ``q [m_pad, k]`` with rows m..m_pad-1 zero, and fp32 scales K-major
    ``scales_km [k/128, m_pad]`` with the pad columns zero.  ``m_pad``
    defaults to ceil16(m)."""
    m, stride, k = _bf16_rows(x, "x")
    m_pad = ceil16(m) if m_pad is None else int(m_pad)
    if m_pad < m:
        raise ValueError("m_pad must be >= the number of rows")
    if q is None:
        q = torch.empty((m_pad, k), dtype=torch.uint8, device=x.device)
    if scales_km is None:
        scales_km = torch.empty((k // 128, m_pad), dtype=torch.float32, device=x.device)
    if q.dtype not in _BYTE_TYPES or not q.is_contiguous() or q.numel() < m_pad * k:
        raise ValueError("q must be a contiguous uint8/float8_e4m3fn tensor of m_pad*k elements")
    if scales_km.dtype != torch.float32 or not scales_km.is_contiguous() or \
            scales_km.numel() < m_pad * (k // 128):
        raise ValueError("scales_km must be a contiguous float32 tensor of (k/128)*m_pad elements")
    _check("fp8_group_quant_kmajor", lib.fp8_group_quant_kmajor(
        _ptr(x) if m else None, stride, _ptr(q), _ptr(scales_km), m, m_pad, k, _stream(stream)))
    return q, scales_km


# ---------------------------------------------------------------------------
# paged KV write


def _pool_geometry(k_pool: torch.Tensor, v_pool: torch.Tensor, elems: int):
    """Pools ``[num_blocks, block_size, heads, dim]`` (block stride may be padded)."""
    for name, p in (("k_pool", k_pool), ("v_pool", v_pool)):
        if p.dtype not in _BYTE_TYPES or not p.is_cuda:
            raise TypeError(f"{name} must be a CUDA uint8/float8_e4m3fn tensor")
    if k_pool.shape != v_pool.shape or k_pool.stride() != v_pool.stride():
        raise ValueError("k_pool and v_pool must have the same shape and strides")
    num_blocks, block_size = k_pool.shape[0], k_pool.shape[1]
    inner = k_pool[0].numel() if num_blocks else block_size * elems
    if inner != block_size * elems:
        raise ValueError("pool block does not hold block_size * num_kv_heads * head_dim codes")
    if num_blocks and not k_pool[0].is_contiguous():
        raise ValueError("each pool block must be contiguous")
    return num_blocks, block_size, k_pool.stride(0)


def fp8_kv_write(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                 k_pool: torch.Tensor, v_pool: torch.Tensor, k_scale: float = 1.0,
                 v_scale: float = 1.0, scale_dev: torch.Tensor | None = None, stream=None):
    """reshape_and_cache_fp8: K, V ``[T, heads, dim]`` bf16 into the pools at
    ``slot_mapping`` (int64, -1 skips), per-tensor scales by value or from the
    device ``scale_dev [2]``."""
    t, ks, vs, heads, dim = _kv_rows(k, v)
    _check_slots(slot_mapping, t)
    _check_scale_pair(scale_dev, "scale_dev")
    nb, bs, cs = _pool_geometry(k_pool, v_pool, heads * dim)
    _check("fp8_kv_write", lib.fp8_kv_write(
        _ptr(k), _ptr(v), ks, vs, _ptr(slot_mapping), t, heads, dim, _ptr(k_pool),
        _ptr(v_pool), bs, cs, nb, float(k_scale), float(v_scale), _ptr(scale_dev),
        _stream(stream)))


def fp8_kv_write_layers(ks, vs, slot_mappings, k_pools, v_pools, k_scales=None, v_scales=None,
                        scale_devs=None, stream=None):
    """reshape_and_cache_fp8 for several layers in one launch.  Per layer:
    K, V ``[T, heads, dim]`` (same shape and row strides for all layers), an
    int64 slot mapping and the layer's pools; scales by value (``k_scales``,
    ``v_scales``) or from device ``scale_devs[i]``."""
    n = len(ks)
    if not (len(vs) == len(slot_mappings) == len(k_pools) == len(v_pools) == n):
        raise ValueError("one k, v, slot_mapping, k_pool and v_pool per layer")
    if n > _abi.MAX_LAYERS:
        raise ValueError(f"at most {_abi.MAX_LAYERS} layers per launch")
    if n == 0:
        return
    t, kst, vst, heads, dim = _kv_rows(ks[0], vs[0])
    e = heads * dim
    nb, bs, cs = _pool_geometry(k_pools[0], v_pools[0], e)
    arr = (_abi.KvLayer * n)()
    for i in range(n):
        ti, ksi, vsi, hi, di = _kv_rows(ks[i], vs[i])
        if (ti, ksi, vsi, hi, di) != (t, kst, vst, heads, dim):
            raise ValueError("all layers must share the row shape and strides")
        _check_slots(slot_mappings[i], t)
        if _pool_geometry(k_pools[i], v_pools[i], e) != (nb, bs, cs):
            raise ValueError("all layers' pools must share one geometry")
        sd = None if scale_devs is None else scale_devs[i]
        _check_scale_pair(sd, "scale_devs[i]")
        arr[i] = _abi.KvLayer(_ptr(ks[i]), _ptr(vs[i]), _ptr(slot_mappings[i]), _ptr(k_pools[i]),
                              _ptr(v_pools[i]), _ptr(sd),
                              float(k_scales[i]) if k_scales is not None else 1.0,
                              float(v_scales[i]) if v_scales is not None else 1.0)
    _check("fp8_kv_write_layers", lib.fp8_kv_write_layers(
        arr, n, kst, vst, t, heads, dim, bs, cs, nb, _stream(stream)))


def fp8_kv_amax_observe(k: torch.Tensor, v: torch.Tensor, amax_dev: torch.Tensor, stream=None):
    """Max-accumulate max|K| and max|V| into the device fp32 ``amax_dev [2]``."""
    t, ks, vs, heads, dim = _kv_rows(k, v)
    _check_scale_pair(amax_dev, "amax_dev")
    _check("fp8_kv_amax_observe", lib.fp8_kv_amax_observe(
        _ptr(k), _ptr(v), ks, vs, t, heads, dim, _ptr(amax_dev), _stream(stream)))


# ---------------------------------------------------------------------------
# calibration


def fp8_kv_graphs_ready(states) -> bool:
    """``states``: per layer None (no calibrator), False (in window), True (frozen)."""
    arr = (ctypes.c_int8 * len(states))(*[-1 if s is None else int(bool(s)) for s in states])
    r = lib.fp8_kv_graphs_ready(arr, len(states))
    if r < 0:
        raise Fp8qError("fp8_kv_graphs_ready", r, "invalid argument")
    return bool(r)


class KvCalibration:
    """The calibrator of one attention layer (fp8_kv_calib_* of the C ABI).

    Device memory (staging for the window's bf16 K/V and slots, and the
    16-byte state) is allocated here with torch and handed to the library."""

    def __init__(self, window_tokens: int, headroom: float, num_kv_heads: int, head_dim: int,
                 device, stage_capacity: int | None = None, stream=None,
                 state: torch.Tensor | None = None) -> None:
        self.num_kv_heads = num_kv_heads
        self.head_dim = head_dim
        e = num_kv_heads * head_dim
        window = min(int(window_tokens), MAX_STAGED_TOKENS)
        cap = window if stage_capacity is None else int(stage_capacity)
        self.stage_k = torch.empty((max(cap, 1), e), dtype=torch.bfloat16, device=device)
        self.stage_v = torch.empty((max(cap, 1), e), dtype=torch.bfloat16, device=device)
        self.stage_slots = torch.empty(max(cap, 1), dtype=torch.int64, device=device)
        if state is None:
            state = torch.empty(4, dtype=torch.float32, device=device)
        if state.dtype != torch.float32 or state.numel() != 4 or not state.is_contiguous():
            raise ValueError("state must be a contiguous float32 tensor of 4 elements")
        self.state = state
        self._h = ctypes.c_void_p()
        self.handle = None
        _check("fp8_kv_calib_create", lib.fp8_kv_calib_create(
            int(window_tokens), float(headroom), num_kv_heads, head_dim, _ptr(self.stage_k),
            _ptr(self.stage_v), _ptr(self.stage_slots), cap, _ptr(self.state), _stream(stream),
            ctypes.byref(self._h)))
        self.handle = self._h.value

    def close(self) -> None:
        if self.handle:
            lib.fp8_kv_calib_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def scale_dev(self) -> torch.Tensor:
        """Device ``{k_scale, v_scale}``: provisional until the freeze, frozen after."""
        return self.state[2:4]

    def observe(self, k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                stream=None) -> int:
        t, ks, vs, heads, dim = _kv_rows(k, v)
        _check_slots(slot_mapping, t)
        step = ctypes.c_int32()
        _check("fp8_kv_calib_observe", lib.fp8_kv_calib_observe(
            self.handle, _ptr(k), _ptr(v), ks, vs, _ptr(slot_mapping), t, heads, dim,
            _stream(stream), ctypes.byref(step)))
        return step.value

    def freeze_replay(self, k_pool: torch.Tensor, v_pool: torch.Tensor, stream=None) -> int:
        nb, bs, cs = _pool_geometry(k_pool, v_pool, self.num_kv_heads * self.head_dim)
        n = ctypes.c_int64()
        _check("fp8_kv_freeze_replay", lib.fp8_kv_freeze_replay(
            self.handle, _ptr(k_pool), _ptr(v_pool), bs, cs, nb, _stream(stream),
            ctypes.byref(n)))
        return n.value

    def observe_write(self, k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                      k_pool: torch.Tensor, v_pool: torch.Tensor, stream=None) -> int:
        t, ks, vs, heads, dim = _kv_rows(k, v)
        _check_slots(slot_mapping, t)
        nb, bs, cs = _pool_geometry(k_pool, v_pool, heads * dim)
        step = ctypes.c_int32()
        _check("fp8_kv_calib_observe_write", lib.fp8_kv_calib_observe_write(
            self.handle, _ptr(k), _ptr(v), ks, vs, _ptr(slot_mapping), t, heads, dim,
            _ptr(k_pool), _ptr(v_pool), bs, cs, nb, _stream(stream), ctypes.byref(step)))
        return step.value

    def restore(self, k_scale: float, v_scale: float, stream=None) -> None:
        """Start frozen at saved scales (only before the first observe)."""
        _check("fp8_kv_calib_restore", lib.fp8_kv_calib_restore(
            self.handle, float(k_scale), float(v_scale), _stream(stream)))

    def saved_scales(self, stream=None) -> dict:
        """The frozen scales as exact hex floats, for save_scales()/restore()."""
        if self.stats()["state"] != 2:
            raise Fp8qError("saved_scales", _abi.ESTATE, "the calibrator has not frozen")
        _, _, ks, vs = self.read_state(stream)
        return {"k_scale": float(ks).hex(), "v_scale": float(vs).hex()}

    def stats(self) -> dict:
        s = CalibStats()
        _check("fp8_kv_calib_stats_get", lib.fp8_kv_calib_stats_get(self.handle, ctypes.byref(s)))
        return {name: getattr(s, name) for name, _ in CalibStats._fields_}

    def read_state(self, stream=None):
        """(k_amax, v_amax, k_scale, v_scale); synchronizes the stream."""
        out = (ctypes.c_float * 4)()
        _check("fp8_kv_calib_read_state", lib.fp8_kv_calib_read_state(
            self.handle, _stream(stream), out))
        return tuple(out)


def fp8_kv_calib_window_noalloc(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                                batch_tokens, window_tokens: int, headroom: float,
                                k_pool: torch.Tensor, v_pool: torch.Tensor,
                                scales_out: torch.Tensor | None = None, stream=None) -> None:
    """One layer's calibration window in one call, with no device memory from
    the caller or the library's user: the scratch is a fixed array inside the
    library (see include/fp8q.h).  ``k``/``v`` hold every batch's rows back to
    back; ``batch_tokens`` lists each batch's token count."""
    t, ks, vs, heads, dim = _kv_rows(k, v)
    counts = [int(n) for n in batch_tokens]
    if sum(counts) != t:
        raise ValueError("batch_tokens must add up to the rows of k and v")
    _check_slots(slot_mapping, t)
    _check_scale_pair(scales_out, "scales_out")
    nb, bs, cs = _pool_geometry(k_pool, v_pool, heads * dim)
    arr = (ctypes.c_int64 * max(len(counts), 1))(*counts)
    _check("fp8_kv_calib_window_noalloc", lib.fp8_kv_calib_window_noalloc(
        _ptr(k), _ptr(v), ks, vs, _ptr(slot_mapping), arr, len(counts), heads, dim,
        int(window_tokens), float(headroom), _ptr(k_pool), _ptr(v_pool), bs, cs, nb,
        _ptr(scales_out), _stream(stream)))


def allreduce_kv_maxima(calibrator, group=None, stream=None) -> None:
    """KV heads sharded over ranks, one scale for all of them: after
    ``observe()`` returns STEP_FREEZE for the batch that reaches the window and
    before ``freeze_replay()``, make every rank's device |K| and |V| maxima the
    maximum over the group (one all-reduce of two fp32 values).  Every rank
    then freezes the same scales.  Pass the ``stream`` that ``observe()`` and
    ``freeze_replay()`` use (default: the current stream): the all-reduce is
    ordered after that stream's absmax kernels and before its replay."""
    import torch.distributed as dist
    if stream is None or isinstance(stream, int):
        dist.all_reduce(calibrator.state[0:2], op=dist.ReduceOp.MAX, group=group)
        return
    with torch.cuda.stream(stream):
        dist.all_reduce(calibrator.state[0:2], op=dist.ReduceOp.MAX, group=group)


def save_scales(calibrators, path: str) -> None:
    """Write every layer's frozen scales to a JSON file (exact hex floats)."""
    import json
    with open(path, "w") as fh:
        json.dump({"fp8_kv_scales": [c.saved_scales() for c in calibrators]}, fh, indent=1)


def load_scales(path: str) -> list[tuple[float, float]]:
    """Read scales written by save_scales(): [(k_scale, v_scale)] per layer."""
    import json
    with open(path) as fh:
        data = json.load(fh)["fp8_kv_scales"]
    return [(float.fromhex(d["k_scale"]), float.fromhex(d["v_scale"])) for d in data]


# ---------------------------------------------------------------------------
# the 4-bit paged KV cache


try:                       # what the public functions wrap, at a tenth of the time
    from torch._C import _cuda_getCurrentRawStream as _current_raw_stream
    from torch._C import _cuda_getDevice as _current_device
except ImportError:
    def _current_raw_stream(device):
        return torch.cuda.current_stream(device).cuda_stream
    _current_device = torch.cuda.current_device


_BF16, _U8, _I32, _I64, _F32 = torch.bfloat16, torch.uint8, torch.int32, torch.int64, torch.float32


def _rows3(t: torch.Tensor, shape, name: str) -> int:
    """Row stride in elements of a CUDA bf16 ``[T, heads, dim]`` tensor of this
    shape whose rows are contiguous."""
    if t.dtype != _BF16 or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA bfloat16 tensor")
    n, heads, dim = shape
    s0, s1, s2 = t.stride()
    if s1 != dim or s2 != 1:
        if ((s2 != 1 and dim != 1) or (s1 != dim and heads != 1)) and t.numel():
            raise ValueError(f"{name} rows must be contiguous")
    return s0 if n > 1 else heads * dim


def _same_device(device: int, names: str, *tensors) -> None:
    for i, t in enumerate(tensors):
        if t is not None and t.get_device() != device:
            raise ValueError(f"{names.split()[i]} must be on the same CUDA device as the other tensors")


def _call_on(device: int, stream, name: str, fn, *args) -> None:
    """Call the library with ``device`` current; no stream given means the
    current stream of that device."""
    if stream is None:
        raw = _current_raw_stream(device)
    else:
        raw = stream if isinstance(stream, int) else stream.cuda_stream
    if _current_device() == device:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            status = fn(*args, raw)
    if status:
        _check(name, status)


def fp4_kv_pool_shape(num_blocks: int, block_size: int, num_kv_heads: int, head_dim: int):
    """Shape of one 4-bit pool (uint8): a block holds ``block_size / 16`` tiles
    of 16 tokens for each head, ``9 * head_dim`` bytes each (include/fp8q.h)."""
    if block_size <= 0 or block_size % 16:
        raise ValueError("block_size must be a positive multiple of 16")
    if head_dim not in (64, 128, 256):
        raise ValueError("head_dim must be 64, 128 or 256")
    return num_blocks, num_kv_heads, block_size // 16, 9 * head_dim


def fp4_kv_pools(num_blocks: int, block_size: int, num_kv_heads: int, head_dim: int, device="cuda"):
    """A zeroed ``(k_pool, v_pool)`` pair of the 4-bit cache."""
    shape = fp4_kv_pool_shape(num_blocks, block_size, num_kv_heads, head_dim)
    return (torch.zeros(shape, dtype=torch.uint8, device=device),
            torch.zeros(shape, dtype=torch.uint8, device=device))


def _fp4_geometry(k_pool: torch.Tensor, v_pool: torch.Tensor):
    """Pools ``[num_blocks, heads, block_size / 16, 9 * dim]`` (block stride may
    be padded): (num_blocks, heads, block_size, dim, block stride in bytes)."""
    if k_pool.dtype != _U8 or v_pool.dtype != _U8 or not k_pool.is_cuda or not v_pool.is_cuda:
        raise TypeError("k_pool and v_pool must be CUDA uint8 tensors")
    shape, stride = k_pool.shape, k_pool.stride()
    if shape != v_pool.shape or stride != v_pool.stride():
        raise ValueError("k_pool and v_pool must have the same shape and strides")
    if len(shape) != 4 or shape[3] % 9:
        raise ValueError("pools must be [num_blocks, num_kv_heads, block_size / 16, 9 * head_dim]")
    num_blocks, heads, tiles, tile = shape
    if num_blocks and (stride[3] != 1 or (tiles != 1 and stride[2] != tile)
                       or (heads != 1 and stride[1] != tiles * tile)):
        raise ValueError("each pool block must be contiguous")
    return (num_blocks, heads, 16 * tiles, tile // 9,
            stride[0] if num_blocks > 1 else heads * tiles * tile)


def _fp4_rows(k: torch.Tensor, v: torch.Tensor, slot_mapping, k_pool, v_pool, scale_dev):
    """Shared argument checks of fp4_kv_write and fp4_kv_read; their arguments
    up to the scales."""
    shape = k.shape
    if len(shape) != 3 or shape != v.shape:
        raise ValueError(f"k and v must both be [T, heads, dim] of one shape, got {tuple(k.shape)} "
                         f"and {tuple(v.shape)}")
    ks, vs = _rows3(k, shape, "k"), _rows3(v, shape, "v")
    t, heads, dim = shape
    _check_slots(slot_mapping, t)
    _check_scale_pair(scale_dev, "scale_dev")
    nb, pool_heads, bs, pool_dim, stride = _fp4_geometry(k_pool, v_pool)
    if (heads, dim) != (pool_heads, pool_dim):
        raise ValueError(f"pools hold {pool_heads} heads of {pool_dim}, k and v have {heads} of {dim}")
    device = k.get_device()
    _same_device(device, "v k_pool v_pool scale_dev slot_mapping", v, k_pool, v_pool, scale_dev,
                 slot_mapping if t else None)
    return device, (k.data_ptr(), v.data_ptr(), ks, vs, slot_mapping.data_ptr(), t, heads, dim,
                    k_pool.data_ptr(), v_pool.data_ptr(), bs, stride, nb)


def fp4_kv_write(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                 k_pool: torch.Tensor, v_pool: torch.Tensor, k_scale: float = 1.0,
                 v_scale: float = 1.0, scale_dev: torch.Tensor | None = None, stream=None) -> None:
    """Quantise K, V ``[T, heads, dim]`` bf16 (rows may be strided) to 4 bits and
    scatter them into the pools at ``slot_mapping`` (int64, negative skips)."""
    device, args = _fp4_rows(k, v, slot_mapping, k_pool, v_pool, scale_dev)
    _call_on(device, stream, "fp4_kv_write", lib.fp4_kv_write, *args, k_scale, v_scale,
             _ptr(scale_dev))


def fp4_kv_read(slot_mapping: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                k_scale: float = 1.0, v_scale: float = 1.0,
                scale_dev: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                v_out: torch.Tensor | None = None, stream=None):
    """Gather the tokens at ``slot_mapping`` back as bf16 ``[T, heads, dim]``.
    Rows of negative slots keep what ``k_out`` and ``v_out`` held (zeros when
    they are allocated here)."""
    if k_out is None or v_out is None:
        _, heads, _, dim, _ = _fp4_geometry(k_pool, v_pool)
        shape = (slot_mapping.numel(), heads, dim)
        with _allocating_for(stream, k_pool.device):
            if k_out is None:
                k_out = torch.zeros(shape, dtype=torch.bfloat16, device=k_pool.device)
            if v_out is None:
                v_out = torch.zeros(shape, dtype=torch.bfloat16, device=k_pool.device)
    device, args = _fp4_rows(k_out, v_out, slot_mapping, k_pool, v_pool, scale_dev)
    _call_on(device, stream, "fp4_kv_read", lib.fp4_kv_read, *args, k_scale, v_scale,
             _ptr(scale_dev))
    return k_out, v_out


_HERE = contextlib.nullcontext()


def _allocating_for(stream, device: torch.device):
    """Context in which tensors belong to ``stream``, so that their memory is
    not handed out again before the stream's work on them is done."""
    if stream is None:
        return _HERE if device.index == _current_device() else torch.cuda.device(device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    return torch.cuda.stream(stream)


def _check_index(t: torch.Tensor, name: str, *shape) -> None:
    if t.dtype != _I32 or t.shape != shape:
        raise ValueError(f"{name} must be int32 {list(shape)}")


@functools.lru_cache(maxsize=256)
def fp4_kv_attention_workspace(batch: int, num_tokens: int, num_q_heads: int, num_kv_heads: int,
                               head_dim: int, uneven: bool = False) -> int:
    """Bytes of workspace fp4_kv_attention needs for these sizes; with
    ``uneven`` what it can use where sequences differ much in length."""
    f = lib.fp4_kv_attention_workspace_uneven if uneven else lib.fp4_kv_attention_workspace
    n = f(batch, num_tokens, num_q_heads, num_kv_heads, head_dim)
    if n < 0:
        raise ValueError("sizes fp4_kv_attention does not take")
    return n


def fp4_kv_attention(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                     block_table: torch.Tensor, seq_lens: torch.Tensor,
                     softmax_scale: float | None = None, q_start: torch.Tensor | None = None,
                     window: int = 0, k_scale: float = 1.0, v_scale: float = 1.0,
                     scale_dev: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream=None):
    """Causal attention of the new tokens ``q [T, q_heads, dim]`` (bf16, rows may
    be strided) over the 4-bit cache.

    ``seq_lens`` int32 ``[batch]`` counts each sequence's cached tokens, the new
    ones included; ``block_table`` int32 ``[batch, width]`` lists its blocks;
    ``q_start`` int32 ``[batch + 1]`` says where its rows of q begin (None: one
    new token each).  A new token sees the cached tokens up to itself, of them
    only the last ``window`` when that is positive.  ``softmax_scale`` defaults
    to dim ** -0.5.  Returns ``out``, or ``(out, lse)`` when an fp32 ``lse
    [T, q_heads]`` is given to be filled.  ``workspace`` (uint8, at least
    fp4_kv_attention_workspace() bytes) is allocated for the call when not
    given, for sequences of any lengths; calls that may overlap need one each."""
    shape = q.shape
    if len(shape) != 3:
        raise ValueError("q must be [T, heads, dim]")
    q_stride = _rows3(q, shape, "q")
    t, q_heads, dim = shape
    nb, heads, bs, pool_dim, stride = _fp4_geometry(k_pool, v_pool)
    if dim != pool_dim or heads == 0 or q_heads % heads:
        raise ValueError(f"pools hold {heads} heads of {pool_dim}, q has {q_heads} of {dim}")
    batch = seq_lens.shape[0] if seq_lens.dim() == 1 else -1
    _check_index(seq_lens, "seq_lens", batch)
    table_shape = block_table.shape
    if block_table.dtype != _I32 or len(table_shape) != 2 or table_shape[0] != batch:
        raise ValueError("block_table must be int32 [batch, width]")
    width = table_shape[1]
    table_stride, step = block_table.stride()
    if step != 1 and width > 1:
        raise ValueError("block_table rows must be contiguous")
    if batch <= 1:
        table_stride = width
    if batch > 1 and seq_lens.stride(0) != 1:
        raise ValueError("seq_lens must be contiguous")
    if q_start is not None:
        _check_index(q_start, "q_start", batch + 1)
        if batch and q_start.stride(0) != 1:
            raise ValueError("q_start must be contiguous")
    elif t != batch:
        raise ValueError("without q_start, q must have one row for each sequence")
    _check_scale_pair(scale_dev, "scale_dev")
    device = q.get_device()
    if out is None or workspace is None:
        with _allocating_for(stream, q.device):
            if out is None:
                out = torch.empty(shape, dtype=_BF16, device=q.device)
            if workspace is None:
                workspace = torch.empty(fp4_kv_attention_workspace(batch, t, q_heads, heads, dim, True),
                                        dtype=_U8, device=q.device)
    if out.shape != shape:
        raise ValueError("out must have the shape of q")
    out_stride = _rows3(out, shape, "out")
    if lse is not None and (lse.dtype != _F32 or lse.shape != (t, q_heads)
                            or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 tensor [T, q_heads]")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _same_device(device, "k_pool v_pool block_table seq_lens q_start scale_dev out lse workspace",
                 k_pool, v_pool, block_table, seq_lens, q_start, scale_dev, out, lse, workspace)
    _call_on(device, stream, "fp4_kv_attention", lib.fp4_kv_attention,
             q.data_ptr(), q_stride, k_pool.data_ptr(), v_pool.data_ptr(), bs, stride, nb, heads,
             dim, block_table.data_ptr(), table_stride, width, seq_lens.data_ptr(), _ptr(q_start),
             batch, t, q_heads, dim ** -0.5 if softmax_scale is None else softmax_scale, window,
             k_scale, v_scale, _ptr(scale_dev), out.data_ptr(), out_stride, _ptr(lse),
             workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out if lse is None else (out, lse)


# ---------------------------------------------------------------------------
# norms of queries and keys with the position rotation


def rope_inv_freq(rotary_dim: int, base: float = 10000.0, stretch: float = 1.0,
                  trained_length: int | None = None, fast: float = 32.0, slow: float = 1.0,
                  device="cuda") -> torch.Tensor:
    """Rotation frequencies ``base ** (-2i / rotary_dim)``, fp64
    ``[rotary_dim / 2]``, for contexts ``stretch`` times as long as the trained
    ones.  Without ``trained_length`` every frequency is divided by ``stretch``
    (positions interpolated).  With it, frequencies that turn at least ``fast``
    times over the trained length stay, those that turn at most ``slow`` times
    are divided, and the ones between are blended linearly in their index
    (interpolation by parts, as YaRN does)."""
    if rotary_dim < 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even")
    if not (base > 1 and stretch >= 1):
        raise ValueError("base must be > 1 and stretch >= 1")
    import math
    freq = [base ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)]
    if trained_length is None:
        keep = [0.0] * len(freq)
    else:
        if not (trained_length > 0 and fast > slow > 0):
            raise ValueError("trained_length must be > 0 and fast > slow > 0")

        def index(turns):      # where a frequency turns that often over trained_length
            return rotary_dim * math.log(trained_length / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo = max(math.floor(index(fast)), 0)
        hi = max(min(math.ceil(index(slow)), rotary_dim - 1), lo + 0.001)
        keep = [1.0 - min(max((i - lo) / (hi - lo), 0.0), 1.0) for i in range(len(freq))]
    return torch.tensor([f * (w + (1.0 - w) / stretch) for f, w in zip(freq, keep)],
                        dtype=torch.float64, device=device)


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor,
                 inv_freq: torch.Tensor, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                 interleaved: bool = False, rope_scale: float = 1.0,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                 stream=None):
    """Root-mean-square norm of each head of ``q [T, q_heads, dim]`` and ``k
    [T, kv_heads, dim]`` (bf16, rows may be strided; no norm without a weight),
    then the rotation of its first ``2 * len(inv_freq)`` elements by
    ``positions[t] * inv_freq`` (fp64): halves paired, or neighbours when
    ``interleaved``.  ``rope_scale`` multiplies cosine and sine.  ``q_out`` and
    ``k_out`` may be ``q`` and ``k``."""
    q_shape, k_shape = q.shape, k.shape
    if len(q_shape) != 3 or len(k_shape) != 3 or q_shape[0] != k_shape[0] or q_shape[2] != k_shape[2]:
        raise ValueError(f"q and k must be [T, heads, dim] with the same T and dim, got "
                         f"{tuple(q.shape)} and {tuple(k.shape)}")
    q_stride, k_stride = _rows3(q, q_shape, "q"), _rows3(k, k_shape, "k")
    t, q_heads, dim = q_shape
    k_heads = k_shape[1]
    if positions.dtype != _I64 or positions.shape != (t,) or (t > 1 and positions.stride(0) != 1):
        raise ValueError("positions must be a contiguous int64 tensor [T]")
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous float64 tensor [rotary_dim / 2]")
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and (w.dtype != _BF16 or w.shape != (dim,) or not w.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous bfloat16 tensor [dim]")
    device = q.get_device()
    if q_out is None or k_out is None:
        with _allocating_for(stream, q.device):
            if q_out is None:
                q_out = torch.empty(q_shape, dtype=_BF16, device=q.device)
            if k_out is None:
                k_out = torch.empty(k_shape, dtype=_BF16, device=q.device)
    if q_out.shape != q_shape or k_out.shape != k_shape:
        raise ValueError("q_out and k_out must have the shapes of q and k")
    qo_stride, ko_stride = _rows3(q_out, q_shape, "q_out"), _rows3(k_out, k_shape, "k_out")
    _same_device(device, "k positions inv_freq q_weight k_weight q_out k_out", k, positions, inv_freq,
                 q_weight, k_weight, q_out, k_out)
    _call_on(device, stream, "qk_norm_rope", lib.qk_norm_rope,
             q.data_ptr(), k.data_ptr(), q_stride, k_stride, q_out.data_ptr(), k_out.data_ptr(),
             qo_stride, ko_stride, positions.data_ptr(), inv_freq.data_ptr(), _ptr(q_weight),
             _ptr(k_weight), t, q_heads, k_heads, dim, 2 * inv_freq.shape[0], int(interleaved),
             eps, rope_scale)
    return q_out, k_out


def fp8q_device_error(clear: bool = True) -> int:
    """Sticky device error bits of the current device (synchronizes)."""
    bits = ctypes.c_uint32()
    _check("fp8q_device_error", lib.fp8q_device_error(ctypes.byref(bits), int(clear)))
    return bits.value


def version() -> int:
    return lib.fp8q_version()


def launch_count() -> int:
    """Kernels the library has launched (or recorded into a graph) so far."""
    return lib.fp8q_launch_count()


# Module-level spellings of the calibrator entry points, with the C ABI's names.
def fp8_kv_calib_create(window_tokens: int, headroom: float, num_kv_heads: int, head_dim: int,
                        device, stage_capacity: int | None = None, stream=None) -> KvCalibration:
    return KvCalibration(window_tokens, headroom, num_kv_heads, head_dim, device,
                         stage_capacity, stream)


def fp8_kv_calib_observe(calib: KvCalibration, k, v, slot_mapping, stream=None) -> int:
    return calib.observe(k, v, slot_mapping, stream)


def fp8_kv_freeze_replay(calib: KvCalibration, k_pool, v_pool, stream=None) -> int:
    return calib.freeze_replay(k_pool, v_pool, stream)


def fp8_kv_calib_observe_write(calib: KvCalibration, k, v, slot_mapping, k_pool, v_pool,
                               stream=None) -> int:
    return calib.observe_write(k, v, slot_mapping, k_pool, v_pool, stream)
