"""Python binding of include/snapkv_draft.h: operators for several tokens at a time over a cache.

Attention of a tree of drafted tokens (or of tokens that read cached states alone) over a dense cache or
one held in 8 bits, and the accepted tokens' rows appended to either. As in ``cache``, every computation
runs in the library's CUDA kernels and arguments mirror the header; calls run on ``stream`` (default: the
current stream of the tensors' device), allocate what the caller does not pass, and raise on a refused call.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache

import torch

from . import snapkv as _sk
from .cache import _call, _check, _code, _functions, _loaders, _new_lengths, _on_stream, _room, _status
from .snapkv import ERR_INVALID_ARG, SnapKVError

_INT32, _FP32, _BF16, _BYTE = torch.int32, torch.float32, torch.bfloat16, torch.uint8


class _Q8Struct(ctypes.Structure):
    """Mirror of snapkv_q8_cache."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_step", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("v_step", ctypes.c_void_p), ("cap", ctypes.c_int64), ("batch", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


def lib():
    """The loaded library with the prototypes of include/snapkv_draft.h."""
    L = _sk.lib()
    if "snapkv_tree_attend" not in _functions:
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        C = ctypes.POINTER(_Q8Struct)
        found = {}
        for name, res, args in [
                ("snapkv_tree_workspace_size", SZ, [I32, I32, I32, I32, I32, I64]),
                ("snapkv_q8_tree_attend", I32, [P, C, P, P, P, P, P, I64, P, P, I32, I32, I32, P, SZ, P, P]),
                ("snapkv_append_rows", I32, [P, P, I64, P, P, I64, P, I64, P, P, P, I32, I32, I32, I32, P, P]),
                ("snapkv_q8_append", I32, [C, P, P, I64, P, I64, P, P, P, I32, P, P]),
                ("snapkv_q8_read", I32, [C, P, I64, P, P, I32, P]),
                ("snapkv_tree_attend", I32,
                 [P, P, P, I64, P, P, P, P, P, I64, P, P, I32, I32, I32, I32, I32, I32, P, SZ, P, P])]:
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
            found[name] = f
        _functions.update(found)
    return L


_loaders.append(lib)


class Q8Cache:
    """A K/V cache held in 8 bits (the layout of snapkv_q8_cache): k_codes, v_codes uint8 [B,H,cap,d] and k_step,
    v_step float32 [B,H,cap]. 264 bytes per row of K and V at d = 128, against 512 in bf16 and 144 in 4 bits."""
    __slots__ = ("k_codes", "k_step", "v_codes", "v_step", "shape", "device")

    def __init__(self, k_codes, k_step, v_codes, v_step):
        shape, dev = k_codes.shape, k_codes.device
        if len(shape) != 4 or shape[3] not in (64, 128):
            raise ValueError("k_codes must be [B, H, cap, d] with d 64 or 128")
        _check("k_codes", k_codes, shape, _BYTE, dev)
        _check("v_codes", v_codes, shape, _BYTE, dev)
        _check("k_step", k_step, shape[:3], _FP32, dev)
        _check("v_step", v_step, shape[:3], _FP32, dev)
        self.k_codes, self.k_step, self.v_codes, self.v_step = k_codes, k_step, v_codes, v_step
        self.shape, self.device = tuple(shape), dev   # B, H, cap, d

    def _struct(self):
        B, H, cap, d = self.shape
        return _Q8Struct(self.k_codes.data_ptr(), self.k_step.data_ptr(), self.v_codes.data_ptr(),
                         self.v_step.data_ptr(), cap, B, H, d)

    @classmethod
    def empty(cls, batch, heads, cap, head_dim, device):
        """An uninitialised cache (rows are written by q8_append)."""
        codes = [torch.empty((batch, heads, cap, head_dim), dtype=_BYTE, device=device) for _ in "kv"]
        steps = [torch.empty((batch, heads, cap), dtype=_FP32, device=device) for _ in "kv"]
        return cls(codes[0], steps[0], codes[1], steps[1])


@lru_cache(maxsize=256)
def tree_workspace_size(batch, q_heads, heads, head_dim, tokens, cap) -> int:
    lib()
    return int(_functions["snapkv_tree_workspace_size"](batch, q_heads, heads, head_dim, tokens, cap))


def _at(t):
    return None if t is None else t.data_ptr()


def _attend_args(where, q, shape, dev, len_, k_new, v_new, mask, n_new, lse, out, workspace):
    """Checks and completes what the two attention calls share."""
    B, H, cap, d = shape
    if q.dim() != 4:
        raise ValueError("q must be [B, q_heads, tokens, d]")
    q_heads, tokens = q.shape[1], q.shape[2]
    if H < 1 or q_heads < 1 or q_heads % H or tokens < 1:
        raise SnapKVError(ERR_INVALID_ARG, where)
    dtype = q.dtype
    _check("q", q, (B, q_heads, tokens, d), dtype, dev)
    _check("len_", len_, (B,), _INT32, dev)
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new go together")
    if k_new is not None:
        _check("k_new", k_new, (B, H, tokens, d), dtype, dev)
        _check("v_new", v_new, (B, H, tokens, d), dtype, dev)
    stride = 0
    if mask is not None:
        if k_new is None:
            raise ValueError("a mask is over drafted rows: it needs k_new and v_new")
        if mask.dtype not in (torch.bool, _BYTE):
            raise TypeError(f"mask is {mask.dtype}, expected torch.bool or torch.uint8")
        one = mask.dim() == 2
        _check("mask", mask, (tokens, tokens) if one else (B, tokens, tokens), mask.dtype, dev)
        stride = 0 if one else tokens * tokens
    if n_new is not None:
        _check("n_new", n_new, (B,), _INT32, dev)
    if lse is not None:
        _check("lse", lse, (B, q_heads, tokens), _FP32, dev)
    if out is None:
        out = torch.empty_like(q)
    else:
        _check("out", out, q.shape, dtype, dev)
    room = _room(workspace, tree_workspace_size(B, q_heads, H, d, tokens, cap), dev)
    return (_at(k_new), _at(v_new), _at(n_new), _at(mask), stride, out.data_ptr(), _at(lse)), q_heads, tokens, out, room


@_on_stream
def tree_attend(q, k_cache, v_cache, len_, k_new=None, v_new=None, mask=None, *, n_new=None, lse=None, out=None,
                workspace=None, dev_status=None):
    """snapkv_tree_attend: q [B,Hq,T,d] over rows < len_[b] of k_cache, v_cache [B,H,cap,d] and over the tokens' own
    rows k_new, v_new [B,H,T,d] that ``mask`` (bool [B,T,T] or one [T,T] for all; None: causal) lets each token see
    -> out [B,Hq,T,d]. Without k_new and v_new: attention to the cache alone. ``n_new`` [B]: how many tokens each
    sequence has (None: T); ``lse`` fp32 [B,Hq,T], if given, receives the logarithms of the softmax sums."""
    shape, dev, dtype = k_cache.shape, k_cache.device, q.dtype
    if len(shape) != 4:
        raise ValueError("k_cache must be [B, H, cap, d]")
    _check("k_cache", k_cache, shape, dtype, dev)
    _check("v_cache", v_cache, shape, dtype, dev)
    rest, q_heads, tokens, out, room = _attend_args("snapkv_tree_attend", q, shape, dev, len_, k_new, v_new, mask, n_new,
                                                    lse, out, workspace)
    B, H, cap, d = shape
    _call("snapkv_tree_attend", dev, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), cap, len_.data_ptr(), *rest, B,
          q_heads, H, d, tokens, _code(dtype), room[1], room[2], _status(dev_status, dev))
    return out


@_on_stream
def q8_tree_attend(q, cache, len_, k_new=None, v_new=None, mask=None, *, n_new=None, lse=None, out=None, workspace=None,
                   dev_status=None):
    """snapkv_q8_tree_attend: tree_attend over a Q8Cache; q, k_new, v_new and out are bf16 or fp32."""
    dev = cache.device
    rest, q_heads, tokens, out, room = _attend_args("snapkv_q8_tree_attend", q, cache.shape, dev, len_, k_new, v_new, mask,
                                                    n_new, lse, out, workspace)
    _call("snapkv_q8_tree_attend", dev, q.data_ptr(), cache._struct(), len_.data_ptr(), *rest, q_heads, tokens,
          _code(q.dtype), room[1], room[2], _status(dev_status, dev))
    return out


def _append_args(where, shape, dev, dtype, k_new, v_new, len_in, len_out, n_new, pick):
    """Checks and completes what the two appends share."""
    B, H, _, d = shape
    rows = k_new.shape[2] if k_new.dim() == 4 else 1
    new = (B, H, rows, d) if k_new.dim() == 4 else (B, H, d)
    _check("k_new", k_new, new, dtype, dev)
    _check("v_new", v_new, new, dtype, dev)
    picks = 0
    if pick is not None:
        if pick.dim() != 2:
            raise ValueError("pick must be [B, picks]")
        picks = pick.shape[1]
        _check("pick", pick, (B, picks), _INT32, dev)
        if picks < 1:   # (such a tensor's address is 0, which the library takes for no pick: all rows)
            raise SnapKVError(ERR_INVALID_ARG, where)
    if n_new is not None:
        _check("n_new", n_new, (B,), _INT32, dev)
    len_out = _new_lengths(len_in, len_out, B, dev)
    return rows, picks, len_out


@_on_stream
def append_rows(k_cache, v_cache, k_new, v_new, len_in, len_out=None, *, n_new=None, pick=None, dev_status=None):
    """snapkv_append_rows: rows pick[b,i], i < n_new[b], of k_new, v_new [B,H,rows,d] (without ``pick`` [B,picks]: rows i) go
    to rows len_in[b] + i of k_cache, v_cache [B,H,cap,d]. Returns len_out [B] (len_in is only read). A step that accepts nothing
    has n_new[b] = 0; a pick without columns (picks = 0) is refused."""
    shape, dev, dtype = k_cache.shape, k_cache.device, k_cache.dtype
    if len(shape) != 4:
        raise ValueError("k_cache must be [B, H, cap, d]")
    _check("k_cache", k_cache, shape, dtype, dev)
    _check("v_cache", v_cache, shape, dtype, dev)
    rows, picks, len_out = _append_args("snapkv_append_rows", shape, dev, dtype, k_new, v_new, len_in, len_out, n_new, pick)
    B, H, cap, d = shape
    _call("snapkv_append_rows", dev, k_cache.data_ptr(), v_cache.data_ptr(), cap, k_new.data_ptr(), v_new.data_ptr(), rows,
          _at(pick), picks, _at(n_new), len_in.data_ptr(), len_out.data_ptr(), B, H, d, _code(dtype),
          _status(dev_status, dev))
    return len_out


@_on_stream
def q8_append(cache, k_new, v_new, len_in, len_out=None, *, n_new=None, pick=None, dev_status=None):
    """snapkv_q8_append: append_rows for a Q8Cache, whose rows are quantised as they are written."""
    dev, dtype = cache.device, k_new.dtype
    rows, picks, len_out = _append_args("snapkv_q8_append", cache.shape, dev, dtype, k_new, v_new, len_in, len_out, n_new,
                                       pick)
    _call("snapkv_q8_append", dev, cache._struct(), k_new.data_ptr(), v_new.data_ptr(), rows, _at(pick), picks, _at(n_new),
          len_in.data_ptr(), len_out.data_ptr(), _code(dtype), _status(dev_status, dev))
    return len_out


@_on_stream
def q8_read(cache, rows, *, start=None, dtype=None, k_out=None, v_out=None):
    """snapkv_q8_read: the values (dtype: bf16 or fp32, default bf16) that rows start[b] .. start[b] + rows - 1 of a
    Q8Cache stand for, as k, v [B,H,rows,d]; rows outside the cache are zeros."""
    B, H, _, d = cache.shape
    dev = cache.device
    if dtype is None:
        dtype = _BF16 if k_out is None else k_out.dtype
    code = _code(dtype)
    if start is not None:
        _check("start", start, (B,), _INT32, dev)
    rows = int(rows)
    if rows < 1:
        raise SnapKVError(ERR_INVALID_ARG, "snapkv_q8_read")
    shape = (B, H, rows, d)
    if k_out is None:
        k_out = torch.empty(shape, dtype=dtype, device=dev)
    else:
        _check("k_out", k_out, shape, dtype, dev)
    if v_out is None:
        v_out = torch.empty_like(k_out)
    else:
        _check("v_out", v_out, shape, dtype, dev)
    _call("snapkv_q8_read", dev, cache._struct(), _at(start), rows, k_out.data_ptr(), v_out.data_ptr(), code)
    return k_out, v_out
