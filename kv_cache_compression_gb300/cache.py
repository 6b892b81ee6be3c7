"""Python binding of include/snapkv_cache.h: operators on a cache that is being decoded over.

Decode attention with grouped queries that keeps a running score of every cached row, eviction by
that score, and a cache held in 4 bits. As in ``snapkv``, every computation runs in the library's
CUDA kernels and arguments mirror the header; calls run on ``stream`` (default: the current stream
of the tensors' device), allocate what the caller does not pass, and raise on a refused call. Tensors
start on 16 bytes: of stacked scores [layers, B, H, cap] every layer's slice does if B * H * cap is a
multiple of four.

A decode step makes several of these calls, and its kernels take microseconds each: the checks are
written to cost little where they pass, and calls with their buffers (``out``, ``workspace``, ...)
passed in cost less still.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache, wraps

import torch

from . import snapkv as _sk
from .snapkv import ERR_INVALID_ARG, OK, SnapKVError

GROUP = 64   # channels of a 4-bit row that share one (h, z)

_INT32, _FP32, _BF16, _BYTE = torch.int32, torch.float32, torch.bfloat16, torch.uint8
_DTYPES = {_FP32: _sk.F32, _BF16: _sk.BF16}


class _Q4Struct(ctypes.Structure):
    """Mirror of snapkv_q4_cache."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_meta", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_meta", ctypes.c_void_p), ("cap", ctypes.c_int64), ("batch", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


_functions = {}   # name -> library function with its prototype


def lib():
    """The loaded library with the prototypes of include/snapkv_cache.h."""
    L = _sk.lib()
    if "snapkv_q4_evict" not in _functions:
        P, I32, I64, SZ, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        C = ctypes.POINTER(_Q4Struct)
        found = {}
        for name, res, args in [
                ("snapkv_scored_workspace_size", SZ, [I32, I32, I32, I32, I64, I32]),
                ("snapkv_decode_attend_scored", I32,
                 [P, P, P, I64, P, P, F, P, I32, I32, I32, I32, I32, P, SZ, P, P]),
                ("snapkv_q4_append", I32, [C, P, P, I64, P, P, P, I32, P, P]),
                ("snapkv_q4_read", I32, [C, P, I64, P, P, I32, P]),
                ("snapkv_q4_decode_attend", I32, [P, C, P, P, F, P, I32, I32, P, SZ, P, P]),
                ("snapkv_evict_workspace_size", SZ, [I32, I32, I64]),
                ("snapkv_evict", I32, [P, P, I64, P, P, P, I64, I64, P, I32, I32, I32, I32, P, SZ, P, P]),
                ("snapkv_q4_evict", I32, [C, P, P, P, I64, I64, P, P, SZ, P, P])]:
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
            found[name] = f
        _functions.update(found)
    return L


def _check(name, t, shape, dtype, device):
    """One tensor argument: shape, type, device and density (the kernels take dense tensors)."""
    if t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous():
        return
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    raise ValueError(f"{name} must be contiguous")


def _code(dtype):
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype} (bf16 or fp32)")
    return code


def _status(t, device):
    if t is None:
        return None
    if t.dtype != _INT32 or t.device != device or t.numel() < 1:
        raise ValueError(f"dev_status must be an int32 tensor on {device}")
    return t.data_ptr()


def _room(workspace, need, device):
    """The caller's workspace or a new one (None where nothing is needed), its address and its bytes."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=_BYTE, device=device)
        return workspace, workspace.data_ptr(), need
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _on_stream(f):
    """Adds the ``stream`` argument: the whole call runs with that stream current, so that what it allocates
    belongs to the stream that uses it. The stream has to be one of the tensors' device."""
    @wraps(f)
    def call(*args, stream=None, **kwargs):
        if stream is None:
            return f(*args, **kwargs)
        for t in (*args, *kwargs.values()):
            dev = getattr(t, "device", None)   # (of a tensor or a cache; NumPy's numbers have one that is text)
            if isinstance(dev, torch.device) and dev != stream.device:
                raise ValueError(f"stream is of {stream.device}, but a tensor is on {dev}")
        with torch.cuda.stream(stream):
            return f(*args, **kwargs)
    return call


def _call(name, device, *args):
    """Calls a library function with `device` current (kernels launch there) on the device's current stream."""
    if device.type != "cuda":
        raise ValueError(f"{name} needs CUDA tensors, not {device}")
    f = _functions.get(name)
    if f is None:
        for load in _loaders:
            load()
        f = _functions[name]
    index = device.index
    handle = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        st = f(*args, handle)
    else:
        with torch.cuda.device(index):
            st = f(*args, handle)
    if st != OK:
        raise SnapKVError(st, name)


class Q4Cache:
    """A K/V cache held in 4 bits (the layout of snapkv_q4_cache): k_codes, v_codes uint8 [B,H,cap,d/2] and
    k_meta, v_meta bfloat16 [B,H,cap,d/64,2] (step h, centre z). 144 bytes per row of K and V at d = 128,
    against 512 in bf16."""
    __slots__ = ("k_codes", "k_meta", "v_codes", "v_meta", "shape", "device")

    def __init__(self, k_codes, k_meta, v_codes, v_meta):
        shape, dev = k_codes.shape, k_codes.device
        if len(shape) != 4 or shape[3] not in (32, 64):
            raise ValueError("k_codes must be [B, H, cap, d / 2] with d 64 or 128")
        B, H, cap, half = shape
        _check("k_codes", k_codes, shape, _BYTE, dev)
        _check("v_codes", v_codes, shape, _BYTE, dev)
        meta = (B, H, cap, half * 2 // GROUP, 2)
        _check("k_meta", k_meta, meta, _BF16, dev)
        _check("v_meta", v_meta, meta, _BF16, dev)
        self.k_codes, self.k_meta, self.v_codes, self.v_meta = k_codes, k_meta, v_codes, v_meta
        self.shape, self.device = (B, H, cap, 2 * half), dev   # B, H, cap, d

    def _struct(self):
        B, H, cap, d = self.shape
        return _Q4Struct(self.k_codes.data_ptr(), self.k_meta.data_ptr(), self.v_codes.data_ptr(),
                         self.v_meta.data_ptr(), cap, B, H, d)

    @classmethod
    def empty(cls, batch, heads, cap, head_dim, device):
        """An uninitialised cache (rows are written by q4_append)."""
        codes = [torch.empty((batch, heads, cap, head_dim // 2), dtype=_BYTE, device=device) for _ in "kv"]
        meta = [torch.empty((batch, heads, cap, head_dim // GROUP, 2), dtype=_BF16, device=device) for _ in "kv"]
        return cls(codes[0], meta[0], codes[1], meta[1])


_loaders = [lib]   # of the headers whose functions _call calls


@lru_cache(maxsize=256)
def scored_workspace_size(batch, q_heads, heads, head_dim, cap, scored=True, dtype=None) -> int:
    """snapkv_scored_workspace_size: bytes for calls of either type, or of ``dtype`` alone."""
    lib()
    if dtype is _BF16 and 8 * heads < q_heads <= 16 * heads and q_heads % heads == 0 and \
            scored_workspace_size(batch, heads, heads, head_dim, cap, scored) == 0:
        return 0   # one pass without workspace (or sizes that are invalid)
    return int(_functions["snapkv_scored_workspace_size"](batch, q_heads, heads, head_dim, cap, bool(scored)))


@lru_cache(maxsize=256)
def evict_workspace_size(batch, heads, cap) -> int:
    lib()
    return int(_functions["snapkv_evict_workspace_size"](batch, heads, cap))


def _attend_args(where, q, shape, dev, len_, score, out, workspace):
    """Checks and completes what the two attention calls share."""
    B, H, cap, d = shape
    if q.dim() != 3:
        raise ValueError("q must be [B, q_heads, d]")
    q_heads = q.shape[1]
    if H < 1 or q_heads < 1 or q_heads % H:
        raise SnapKVError(ERR_INVALID_ARG, where)
    _check("q", q, (B, q_heads, d), q.dtype, dev)
    _check("len_", len_, (B,), _INT32, dev)
    if score is not None:
        _check("score", score, (B, H, cap), _FP32, dev)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check("out", out, q.shape, q.dtype, dev)
    room = _room(workspace, scored_workspace_size(B, q_heads, H, d, cap, score is not None, q.dtype), dev)
    return q_heads, None if score is None else score.data_ptr(), out, room


@_on_stream
def decode_attend_scored(q, k_cache, v_cache, len_, score=None, *, decay=1.0, out=None, workspace=None,
                         dev_status=None):
    """snapkv_decode_attend_scored: q [B,Hq,d] over rows < len_[b] of k_cache, v_cache [B,H,cap,d] (Hq a
    multiple of H) -> out [B,Hq,d]. ``score`` fp32 [B,H,cap], if given, becomes decay * score + the
    attention each row received, in place (rows < len_[b] only; clear it before the first step)."""
    shape, dev, dtype = k_cache.shape, k_cache.device, q.dtype
    if len(shape) != 4:
        raise ValueError("k_cache must be [B, H, cap, d]")
    _check("k_cache", k_cache, shape, dtype, dev)
    _check("v_cache", v_cache, shape, dtype, dev)
    q_heads, score_at, out, room = _attend_args("snapkv_decode_attend_scored", q, shape, dev, len_, score, out,
                                                workspace)
    B, H, cap, d = shape
    _call("snapkv_decode_attend_scored", dev, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), cap,
          len_.data_ptr(), score_at, decay, out.data_ptr(), B, q_heads, H, d, _code(dtype), room[1], room[2],
          _status(dev_status, dev))
    return out


@_on_stream
def q4_decode_attend(q, cache, len_, score=None, *, decay=1.0, out=None, workspace=None, dev_status=None):
    """snapkv_q4_decode_attend: decode_attend_scored over a Q4Cache; q and out are bf16 or fp32."""
    dev = cache.device
    q_heads, score_at, out, room = _attend_args("snapkv_q4_decode_attend", q, cache.shape, dev, len_, score, out,
                                                workspace)
    _call("snapkv_q4_decode_attend", dev, q.data_ptr(), cache._struct(), len_.data_ptr(), score_at, decay,
          out.data_ptr(), q_heads, _code(q.dtype), room[1], room[2], _status(dev_status, dev))
    return out


def _new_lengths(len_in, len_out, batch, dev):
    _check("len_in", len_in, (batch,), _INT32, dev)
    if len_out is None:
        return torch.empty_like(len_in)
    _check("len_out", len_out, (batch,), _INT32, dev)
    return len_out


@_on_stream
def q4_append(cache, k_new, v_new, len_in, len_out=None, *, n_new=None, dev_status=None):
    """snapkv_q4_append: quantises k_new, v_new [B,H,rows,d] (or [B,H,d], one row) into rows len_in[b] on of a
    Q4Cache, n_new[b] of them if given. Returns len_out [B] (len_in is only read)."""
    B, H, _, d = cache.shape
    dev, dtype = cache.device, k_new.dtype
    if k_new.dim() == 4:
        rows = k_new.shape[2]
        shape = (B, H, rows, d)
    else:
        rows = 1
        shape = (B, H, d)
    _check("k_new", k_new, shape, dtype, dev)
    _check("v_new", v_new, shape, dtype, dev)
    if n_new is not None:
        _check("n_new", n_new, (B,), _INT32, dev)
    len_out = _new_lengths(len_in, len_out, B, dev)
    _call("snapkv_q4_append", dev, cache._struct(), k_new.data_ptr(), v_new.data_ptr(), rows,
          None if n_new is None else n_new.data_ptr(), len_in.data_ptr(), len_out.data_ptr(), _code(dtype),
          _status(dev_status, dev))
    return len_out


@_on_stream
def q4_read(cache, rows, *, start=None, dtype=None, k_out=None, v_out=None):
    """snapkv_q4_read: the values (dtype: bf16 or fp32, default bf16) that rows start[b] .. start[b] + rows - 1
    of a Q4Cache stand for, as k, v [B,H,rows,d]; rows outside the cache are zeros."""
    B, H, _, d = cache.shape
    dev = cache.device
    if dtype is None:
        dtype = _BF16 if k_out is None else k_out.dtype
    code = _code(dtype)
    if start is not None:
        _check("start", start, (B,), _INT32, dev)
    shape = (B, H, int(rows), d)
    if k_out is None:
        k_out = torch.empty(shape, dtype=dtype, device=dev)
    else:
        _check("k_out", k_out, shape, dtype, dev)
    if v_out is None:
        v_out = torch.empty_like(k_out)
    else:
        _check("v_out", v_out, shape, dtype, dev)
    _call("snapkv_q4_read", dev, cache._struct(), None if start is None else start.data_ptr(), shape[2],
          k_out.data_ptr(), v_out.data_ptr(), code)
    return k_out, v_out


def _evict_args(where, shape, dev, score, len_in, len_out, keep, recent, idx_out, want_idx, workspace):
    """Checks and completes what the two evictions share."""
    B, H, cap, _ = shape
    if (keep | recent) >> 62:   # (negative, or more than the call's integers hold)
        raise SnapKVError(ERR_INVALID_ARG, where)
    _check("score", score, (B, H, cap), _FP32, dev)
    len_out = _new_lengths(len_in, len_out, B, dev)
    left = keep + recent
    if idx_out is not None:
        _check("idx_out", idx_out, (B, H, left), _INT32, dev)
    elif want_idx and 0 < left <= cap:   # (else the library refuses the call)
        idx_out = torch.empty((B, H, left), dtype=_INT32, device=dev)
    room = _room(workspace, evict_workspace_size(B, H, cap), dev)
    return len_out, idx_out, None if idx_out is None else idx_out.data_ptr(), room


@_on_stream
def evict(k_cache, v_cache, score, len_in, len_out=None, *, keep, recent, idx_out=None, want_idx=True,
          workspace=None, dev_status=None):
    """snapkv_evict: brings sequences of more than keep + recent rows down to the ``keep`` rows of largest score
    and the newest ``recent``, per head and in place (k_cache, v_cache [B,H,cap,d], score [B,H,cap]). Returns
    (len_out [B], idx [B,H,keep+recent] or None): the new lengths and the slot each row came from."""
    shape, dev, dtype = k_cache.shape, k_cache.device, k_cache.dtype
    if len(shape) != 4:
        raise ValueError("k_cache must be [B, H, cap, d]")
    _check("k_cache", k_cache, shape, dtype, dev)
    _check("v_cache", v_cache, shape, dtype, dev)
    len_out, idx_out, idx_at, room = _evict_args("snapkv_evict", shape, dev, score, len_in, len_out, keep, recent,
                                                 idx_out, want_idx, workspace)
    B, H, cap, d = shape
    _call("snapkv_evict", dev, k_cache.data_ptr(), v_cache.data_ptr(), cap, score.data_ptr(),
          len_in.data_ptr(), len_out.data_ptr(), keep, recent, idx_at, B, H, d, _code(dtype), room[1], room[2],
          _status(dev_status, dev))
    return len_out, idx_out


@_on_stream
def q4_evict(cache, score, len_in, len_out=None, *, keep, recent, idx_out=None, want_idx=True, workspace=None,
             dev_status=None):
    """snapkv_q4_evict: evict for a Q4Cache."""
    dev = cache.device
    len_out, idx_out, idx_at, room = _evict_args("snapkv_q4_evict", cache.shape, dev, score, len_in, len_out, keep,
                                                 recent, idx_out, want_idx, workspace)
    _call("snapkv_q4_evict", dev, cache._struct(), score.data_ptr(), len_in.data_ptr(), len_out.data_ptr(),
          keep, recent, idx_at, room[1], room[2], _status(dev_status, dev))
    return len_out, idx_out
