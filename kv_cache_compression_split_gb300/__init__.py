"""Python binding of libkvc.so -- the GB300 compressed-KV decode library.

This module only marshals arguments: it builds the C descriptor structs from
torch tensors (device memory owned by the caller) and calls the C ABI declared
in include/kvc.h with the same function names.  Every step of the path runs in
the library's CUDA kernels; there is no Python or CPU fallback -- if the
library is missing, importing a function raises.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
import threading
from dataclasses import dataclass
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkvc.so")
_lib = None
_lock = threading.Lock()

KVC_OK, KVC_ERR_INVALID_ARG, KVC_ERR_UNSUPPORTED, KVC_ERR_CAPACITY = 0, 1, 2, 3
KVC_ERR_WORKSPACE, KVC_ERR_CUDA, KVC_ERR_DEVICE = 4, 5, 6
KVC_DEV_CAPACITY, KVC_DEV_TIMEOUT = 0x1, 0x2
KVC_KIND_SLOTS, KVC_KIND_KIVI = 0, 1
KVC_H2O_DECODE, KVC_H2O_PREFILL = 0, 1
KIVI_GROUP = 32
PAGE_SLOTS = 64            # KVC_PAGE_SLOTS: slots per page of the paged layout
KIVI_PAGE_GROUPS = 4       # KVC_KIVI_PAGE_GROUPS: 32-token groups per KIVI page
H2O_ONCHIP_MAX_SLOTS = 1024   # KVC_H2O_ONCHIP_MAX_SLOTS: fused H2O with logits kept on chip
PLAN_MAX_UNITS = 65536     # KVC_PLAN_MAX_UNITS: units of one kvc_append_plan
KVC_NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024


class KvcError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {kvc_status_string(status)}")


class SlotCacheDesc(C.Structure):
    _fields_ = [("B", C.c_int), ("Hkv", C.c_int), ("D", C.c_int), ("C", C.c_int),
                ("K", C.c_void_p), ("V", C.c_void_p), ("pos", C.c_void_p), ("n", C.c_void_p),
                ("seqlen", C.c_void_p), ("block_table", C.c_void_p), ("num_pages", C.c_int)]


class QuantCacheDesc(C.Structure):
    _fields_ = [("B", C.c_int), ("Hkv", C.c_int), ("D", C.c_int), ("bits", C.c_int),
                ("R", C.c_int), ("Cq", C.c_int), ("k_blocks", C.c_void_p),
                ("v_blocks", C.c_void_p), ("k_res", C.c_void_p), ("v_res", C.c_void_p),
                ("len", C.c_void_p), ("block_table", C.c_void_p), ("num_pages", C.c_int),
                ("k_gear", C.c_void_p), ("v_gear", C.c_void_p)]


class AttendArgs(C.Structure):
    _fields_ = [("kind", C.c_int), ("Hq", C.c_int), ("q", C.c_void_p), ("o", C.c_void_p),
                ("slots", C.POINTER(SlotCacheDesc)), ("quant", C.POINTER(QuantCacheDesc)),
                ("logits", C.c_void_p), ("lse", C.c_void_p), ("workspace", C.c_void_p),
                ("workspace_bytes", C.c_size_t), ("num_splits", C.c_int),
                ("softmax_scale", C.c_float), ("h2o_scores", C.c_void_p),
                ("h2o_decay", C.c_float)]


class H2OArgs(C.Structure):
    _fields_ = [("mode", C.c_int), ("B", C.c_int), ("Hq", C.c_int), ("Hkv", C.c_int),
                ("D", C.c_int), ("C", C.c_int), ("scores", C.c_void_p), ("logits", C.c_void_p),
                ("lse", C.c_void_p), ("n", C.c_void_p), ("L", C.c_int), ("qp", C.c_void_p),
                ("kp", C.c_void_p), ("kp_cap", C.c_int), ("workspace", C.c_void_p),
                ("workspace_bytes", C.c_size_t), ("softmax_scale", C.c_float),
                ("decay", C.c_float)]


_I64x2, _I64x3 = C.c_int64 * 2, C.c_int64 * 3


class PromptArgs(C.Structure):
    _fields_ = [("B", C.c_int), ("Hq", C.c_int), ("Hkv", C.c_int), ("D", C.c_int),
                ("L", C.c_int), ("q", C.c_void_p), ("k", C.c_void_p), ("v", C.c_void_p),
                ("o", C.c_void_p), ("lse", C.c_void_p), ("cu_seqlens", C.c_void_p),
                ("lens", C.c_void_p), ("q_stride", _I64x3), ("k_stride", _I64x3),
                ("v_stride", _I64x3), ("o_stride", _I64x3), ("softmax_scale", C.c_float)]


class ChunkArgs(C.Structure):
    _fields_ = [("Hq", C.c_int), ("T", C.c_int), ("cache", C.POINTER(SlotCacheDesc)),
                ("q", C.c_void_p), ("o", C.c_void_p), ("cu_new", C.c_void_p),
                ("lse", C.c_void_p), ("q_stride", _I64x2), ("o_stride", _I64x2),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t),
                ("num_splits", C.c_int), ("softmax_scale", C.c_float)]


class PagePoolDesc(C.Structure):
    _fields_ = [("pages", C.c_void_p), ("free_list", C.c_void_p), ("count", C.c_void_p)]


def lib():
    """Load libkvc.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(f"{LIB_PATH} is missing: build it with "
                                  "`python -m kv_cache_compression_split_gb300.build`")
            L = C.CDLL(LIB_PATH)
            P, i, st = C.c_void_p, C.c_int, C.c_int
            sig = {
                "kvc_kivi_block_bytes": (C.c_size_t, [i, i]),
                "kvc_gear_side_bytes": (C.c_size_t, [i]),
                "kvc_append": (st, [C.POINTER(SlotCacheDesc), P, P, i, P]),
                "kvc_append_quant": (st, [C.POINTER(QuantCacheDesc), P, P, i, P]),
                "kvc_workspace_size": (C.c_size_t, [C.POINTER(AttendArgs)]),
                "kvc_decode_attend": (st, [C.POINTER(AttendArgs), P]),
                "kvc_decode_attend_noalloc": (st, [C.POINTER(AttendArgs), P]),
                "kvc_h2o_workspace_size": (C.c_size_t, [C.POINTER(H2OArgs)]),
                "kvc_h2o_accumulate": (st, [C.POINTER(H2OArgs), P]),
                "kvc_h2o_evict": (st, [C.POINTER(SlotCacheDesc), P, i, i, P]),
                "kvc_h2o_evict_when": (st, [C.POINTER(SlotCacheDesc), P, i, i, i, P]),
                "kvc_stream_evict": (st, [C.POINTER(SlotCacheDesc), i, i, P]),
                "kvc_stream_append": (st, [C.POINTER(SlotCacheDesc), P, P, i, i, P]),
                "kvc_h2o_decode_step": (st, [C.POINTER(SlotCacheDesc), P, i, P, P, P, P, P, i, i,
                                             C.c_float, P]),
                "kvc_stream_decode_step": (st, [C.POINTER(SlotCacheDesc), i, P, P, P, P, P, i, i,
                                                P]),
                "kvc_random_evict": (st, [C.POINTER(SlotCacheDesc), i, C.c_double, C.c_uint64,
                                          C.c_uint32, P]),
                "kvc_prompt_attend": (st, [P, P]),
                "kvc_chunk_workspace_size": (C.c_size_t, [P]),
                "kvc_chunk_attend": (st, [P, P]),
                "kvc_append_plan": (st, [P, P, P, i, i, P, P, P, P]),
                "kvc_append_packed": (st, [P, P, P, P, P, i, P, P]),
                "kvc_status_string": (C.c_char_p, [i]),
                "kvc_read_device_status": (st, [C.POINTER(C.c_int), P]),
            }
            for name, (res, args) in sig.items():
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
            _lib = L
    return _lib


# ----------------------------------------------------------------------------- helpers

def _ptr(t):
    """Device address of tensor t for a descriptor field.  Every tensor handed to the library
    must be contiguous and live on the current CUDA device: a host tensor's address given to
    a kernel would be read as device memory (or, where the GPU can reach host memory, read
    silently)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError(f"kvc: tensor on {t.device}; the library takes CUDA tensors")
    if t.get_device() != torch.cuda.current_device() or not t.is_contiguous():
        if t.device.index != torch.cuda.current_device():
            raise ValueError(f"kvc: tensor on {t.device}, expected the current device "
                             f"cuda:{torch.cuda.current_device()}")
        raise ValueError("kvc: tensor arguments must be contiguous")
    return t.data_ptr()


# torch's raw current-stream query, where this torch version has it (a few hundred ns
# against a few microseconds for torch.cuda.current_stream())
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current_device():
    """Index of the current device; -2, which no tensor's device equals, on a machine without
    one (the checks of the arguments then say what is wrong)."""
    try:
        return torch.cuda.current_device()
    except (RuntimeError, AssertionError):
        return -2


def _desc_key(tensors):
    """What a cache descriptor depends on: the current device, which the fields were checked
    against, and each field tensor's address, device, shape and strides (None for an absent
    field)."""
    return (_current_device(),) + tuple(
        None if t is None else (t.data_ptr(), t.get_device(), t.shape, t.stride())
        for t in tensors)


_DESC_CACHE_KEYS = ("_desc", "_desc_key", "_desc_p")


def _state_without_desc(obj):
    """A cache object's state for pickling and copying: its fields, without the kept ctypes
    descriptor (rebuilt on the next call; ctypes pointers do not pickle)."""
    state = dict(obj.__dict__)
    for k in _DESC_CACHE_KEYS:
        state.pop(k, None)
    return state



_F16, _F32, _I32 = torch.float16, torch.float32, torch.int32


class _Refused(Exception):
    """Rows that a call does not take; _explain says why."""


def _rows(t, shape, dev):
    """Device address and strides of binary16 rows of this shape: the last dimension is
    contiguous, the others may have any strides, which the call passes on."""
    st = t.stride()
    if (t.dtype is not _F16 or t.shape != shape or t.get_device() != dev or
            (st[-1] != 1 and shape[-1] != 1)):
        raise _Refused
    if 1 in shape:   # a dimension of size 1 is never stepped over: any stride stands for it
        st = tuple([8 if n == 1 else x for n, x in zip(shape, st)])
    return t.data_ptr(), st


def _explain(rows, dev, index):
    """Raise what is wrong with one of these (name, tensor, shape): the rows of a call and the
    int32 tensor that goes with them.  Types and shapes come before the device."""
    for what, t, _ in rows:
        if t.dtype is not _F16:
            raise ValueError(f"kvc: {what} must be float16, got {t.dtype}")
    for what, t, shape in rows:
        if t.shape != shape:
            raise ValueError(f"kvc: {what} must be of shape {tuple(shape)}, got "
                             f"{tuple(t.shape)}: the arguments do not belong together")
    what, t, shape = index
    if t is not None and (t.dtype is not _I32 or t.shape != shape):
        _typed(t, what, _I32, shape, dev)
    for what, t, _ in rows:
        if t.get_device() != dev:
            _wrong_device(t, dev)
        if t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError(f"kvc: the last dimension of {what} must be contiguous")


def _typed(t, what, dtype, shape, dev):
    """Device address of a contiguous tensor of this type and shape (0 for None)."""
    if t is None:
        return 0
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"kvc: {what} must be {dtype} of shape {tuple(shape)}, got {t.dtype} of "
                         f"{tuple(t.shape)}")
    if t.get_device() != dev:
        _wrong_device(t, dev)
    raise ValueError("kvc: tensor arguments must be contiguous")


def _wrong_device(t, dev):
    if not t.is_cuda:
        raise ValueError(f"kvc: tensor on {t.device}; the library takes CUDA tensors")
    raise ValueError(f"kvc: tensor on {t.device}, expected the current device cuda:{dev}")


# The argument structs packed field by field in one call (a ctypes assignment per field took
# longer than the launch); the field order is that of PromptArgs and ChunkArgs.
_pack_prompt = struct.Struct("@5i4x7P12qf4x").pack
_pack_chunk = struct.Struct("@2i5P4qPNif").pack
_pack_2q = struct.Struct("@2q").pack
_pack_3p = struct.Struct("@3P").pack


def _device(stream):
    """Index of the current device, and the stream's handle."""
    dev = _current_device()
    if dev < 0:
        return dev, 0
    if stream is None:
        return dev, _raw_stream(dev) if _raw_stream is not None else _stream(None)
    return dev, _stream(stream)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != KVC_OK:
        raise KvcError(status, where)


# ----------------------------------------------------------------------------- C ABI, same names

def kvc_status_string(status: int) -> str:
    return lib().kvc_status_string(int(status)).decode()


def kvc_kivi_block_bytes(D: int, bits: int) -> int:
    return int(lib().kvc_kivi_block_bytes(D, bits))


def kvc_append(cache: "SlotCache", k_new, v_new, stream=None):
    d = cache.desc()
    _check(lib().kvc_append(C.byref(d), _ptr(k_new), _ptr(v_new), int(k_new.shape[2]),
                            _stream(stream)), "kvc_append")


def kvc_append_quant(cache: "QuantCache", k_new, v_new, stream=None):
    d = cache.desc()
    _check(lib().kvc_append_quant(C.byref(d), _ptr(k_new), _ptr(v_new), int(k_new.shape[2]),
                                  _stream(stream)), "kvc_append_quant")


def _attend_args(cache, q, o, logits=None, lse=None, workspace=None, num_splits=0, scale=0.0,
                 h2o_scores=None, h2o_decay=0.0, shape_only=False):
    a = AttendArgs()
    keep = []
    d = cache.desc()
    keep.append(d)
    if isinstance(cache, SlotCache):
        a.kind = KVC_KIND_SLOTS
        a.slots = cache.__dict__["_desc_p"]
    else:
        a.kind = KVC_KIND_KIVI
        a.quant = cache.__dict__["_desc_p"]
    a.Hq = int(q.shape[1])
    # a size query reads only q's shape (the library plans from the dimensions)
    a.q, a.o = (None, None) if shape_only else (_ptr(q), _ptr(o))
    a.logits, a.lse = _ptr(logits), _ptr(lse)
    a.workspace = _ptr(workspace)
    a.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    a.num_splits = int(num_splits)
    a.softmax_scale = float(scale)
    a.h2o_scores = _ptr(h2o_scores)
    a.h2o_decay = float(h2o_decay)
    return a, keep


def kvc_gear_side_bytes(D: int) -> int:
    return int(lib().kvc_gear_side_bytes(D))


def kvc_workspace_size(cache, q, num_splits: int = 0) -> int:
    a, _keep = _attend_args(cache, q, None, num_splits=num_splits, shape_only=True)
    return int(lib().kvc_workspace_size(C.byref(a)))


def kvc_decode_attend(cache, q, o, logits=None, lse=None, workspace=None, num_splits: int = 0,
                      softmax_scale: float = 0.0, h2o_scores=None, h2o_decay: float = 0.0,
                      stream=None):
    a, _keep = _attend_args(cache, q, o, logits, lse, workspace, num_splits, softmax_scale,
                            h2o_scores, h2o_decay)
    _check(lib().kvc_decode_attend(C.byref(a), _stream(stream)), "kvc_decode_attend")


def kvc_decode_attend_noalloc(cache, q, o, logits=None, lse=None, num_splits: int = 0,
                              softmax_scale: float = 0.0, h2o_scores=None, h2o_decay: float = 0.0,
                              stream=None):
    """kvc_decode_attend without a caller workspace: for callers that cannot allocate device
    memory on their decode path, the split scratch comes from a fixed array the library owns
    (KVC_NOALLOC_SCRATCH_BYTES per GPU).  Calls that may overlap on the GPU race on it."""
    a, _keep = _attend_args(cache, q, o, logits, lse, None, num_splits, softmax_scale,
                            h2o_scores, h2o_decay)
    _check(lib().kvc_decode_attend_noalloc(C.byref(a), _stream(stream)),
           "kvc_decode_attend_noalloc")


def _h2o_args(mode, B, Hq, Hkv, D, Cc, scores, logits=None, lse=None, n=None, L=0, qp=None,
              kp=None, kp_cap=0, workspace=None, scale=0.0, decay=0.0):
    a = H2OArgs()
    a.mode, a.B, a.Hq, a.Hkv, a.D, a.C = mode, B, Hq, Hkv, D, Cc
    a.scores, a.logits, a.lse, a.n = _ptr(scores), _ptr(logits), _ptr(lse), _ptr(n)
    a.L, a.qp, a.kp, a.kp_cap = int(L), _ptr(qp), _ptr(kp), int(kp_cap)
    a.workspace = _ptr(workspace)
    a.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    a.softmax_scale = float(scale)
    a.decay = float(decay)
    return a


def kvc_h2o_workspace_size(B: int, Hq: int, L: int) -> int:
    a = _h2o_args(KVC_H2O_PREFILL, B, Hq, 1, 128, 1, None, L=L)
    return int(lib().kvc_h2o_workspace_size(C.byref(a)))


def kvc_h2o_accumulate_decode(cache: "SlotCache", scores, logits, lse, Hq: int,
                              decay: float = 0.0, stream=None):
    a = _h2o_args(KVC_H2O_DECODE, cache.B, Hq, cache.Hkv, cache.D, cache.C, scores, logits, lse,
                  cache.n, decay=decay)
    _check(lib().kvc_h2o_accumulate(C.byref(a), _stream(stream)), "kvc_h2o_accumulate")


def kvc_h2o_accumulate_prefill(qp, kp, scores, workspace, L: int, lse=None, stream=None):
    """lse: optional [B, Hq, L] fp32 natural-log row normalisers (skips the row pass)."""
    B, Hq, _, D = qp.shape
    _, Hkv, kp_cap, _ = kp.shape
    a = _h2o_args(KVC_H2O_PREFILL, B, Hq, Hkv, D, int(scores.shape[-1]), scores, lse=lse, L=L,
                  qp=qp, kp=kp, kp_cap=kp_cap, workspace=workspace)
    _check(lib().kvc_h2o_accumulate(C.byref(a), _stream(stream)), "kvc_h2o_accumulate")


def kvc_h2o_accumulate(args: H2OArgs, stream=None):
    _check(lib().kvc_h2o_accumulate(C.byref(args), _stream(stream)), "kvc_h2o_accumulate")


def kvc_h2o_evict(cache: "SlotCache", scores, n_heavy: int, n_recent: int, stream=None):
    d = cache.desc()
    _check(lib().kvc_h2o_evict(C.byref(d), _ptr(scores), n_heavy, n_recent, _stream(stream)),
           "kvc_h2o_evict")


def kvc_h2o_evict_when(cache: "SlotCache", scores, n_heavy: int, n_recent: int, trigger: int,
                       stream=None):
    d = cache.desc()
    _check(lib().kvc_h2o_evict_when(C.byref(d), _ptr(scores), n_heavy, n_recent, int(trigger),
                                    _stream(stream)), "kvc_h2o_evict_when")


def kvc_stream_evict(cache: "SlotCache", n_sink: int, n_recent: int, stream=None):
    d = cache.desc()
    _check(lib().kvc_stream_evict(C.byref(d), n_sink, n_recent, _stream(stream)),
           "kvc_stream_evict")


def kvc_stream_append(cache: "SlotCache", k_new, v_new, n_sink: int, n_recent: int, stream=None):
    """One StreamingLLM decode token per sequence ([B, Hkv, 1, D]); the token leaving the
    window gives up its slot (see kvc.h)."""
    if int(k_new.shape[2]) != 1 or int(v_new.shape[2]) != 1:
        raise ValueError("kvc_stream_append takes one token per sequence")
    d = cache.desc()
    _check(lib().kvc_stream_append(C.byref(d), _ptr(k_new), _ptr(v_new), n_sink, n_recent,
                                   _stream(stream)), "kvc_stream_append")


def kvc_h2o_decode_step(cache: "SlotCache", scores, q, k_new, v_new, o, lse=None,
                        n_heavy: int = 64, n_recent: int = 448, decay: float = 0.0, stream=None):
    """One H2O decode step (append + attention + score update + eviction) in one launch."""
    d = cache.desc()
    _check(lib().kvc_h2o_decode_step(C.byref(d), _ptr(scores), int(q.shape[1]), _ptr(q),
                                     _ptr(k_new), _ptr(v_new), _ptr(o), _ptr(lse), n_heavy,
                                     n_recent, float(decay), _stream(stream)),
           "kvc_h2o_decode_step")


def kvc_stream_decode_step(cache: "SlotCache", q, k_new, v_new, o, lse=None, n_sink: int = 64,
                           n_recent: int = 448, stream=None):
    """One StreamingLLM decode step (append into the leaving token's slot + attention) in one
    launch."""
    d = cache.desc()
    _check(lib().kvc_stream_decode_step(C.byref(d), int(q.shape[1]), _ptr(q), _ptr(k_new),
                                        _ptr(v_new), _ptr(o), _ptr(lse), n_sink, n_recent,
                                        _stream(stream)), "kvc_stream_decode_step")


def kvc_random_evict(cache: "SlotCache", prompt_len: int, keep_ratio: float, seed: int,
                     epoch: int, stream=None):
    d = cache.desc()
    _check(lib().kvc_random_evict(C.byref(d), prompt_len, float(keep_ratio),
                                  seed & (2**64 - 1), epoch & 0xffffffff, _stream(stream)),
           "kvc_random_evict")


def kvc_prompt_attend(q, k, v, o, cu_seqlens=None, lens=None, lse=None,
                      softmax_scale: float = 0.0, stream=None):
    """Causal attention over whole prompts (see kvc.h).  Packed: q, o [T, Hq, D], k, v
    [T, Hkv, D], cu_seqlens [B + 1] int32, lse [Hq, T].  Padded: q, o [B, Hq, L, D], k, v
    [B, Hkv, >= L, D], optional lens [B] int32, lse [B, Hq, L].  Rows may be strided."""
    dev, stream = _device(stream)
    shape = q.shape
    if cu_seqlens is not None:
        if lens is not None:
            raise ValueError("kvc_prompt_attend takes cu_seqlens (packed) or lens (padded)")
        L, Hq, D = shape
        Hkv = k.shape[1]
        kv = (L, Hkv, D)
        B = cu_seqlens.numel() - 1
        try:
            qp, (q2, q1, _) = _rows(q, shape, dev)
            kp, (k2, k1, _) = _rows(k, kv, dev)
            vp, (v2, v1, _) = _rows(v, kv, dev)
            op, (o2, o1, _) = _rows(o, shape, dev)
        except _Refused:
            _explain((("q", q, shape), ("k", k, kv), ("v", v, kv), ("o", o, shape)), dev,
                     ("cu_seqlens", cu_seqlens, (B + 1,)))
        args = _pack_prompt(B, Hq, Hkv, D, L, qp, kp, vp, op,
                            0 if lse is None else _typed(lse, "lse", _F32, (Hq, L), dev),
                            _typed(cu_seqlens, "cu_seqlens", _I32, (B + 1,), dev), 0, 0, q1, q2, 0,
                            k1, k2, 0, v1, v2, 0, o1, o2, softmax_scale)
    else:
        B, Hq, L, D = shape
        Hkv = k.shape[1]
        if k.dim() == 4 and k.shape[2] > L:
            k = k[:, :, :L]
        if v.dim() == 4 and v.shape[2] > L:
            v = v[:, :, :L]
        kv = (B, Hkv, L, D)
        try:
            (qp, qs), (kp, ks) = _rows(q, shape, dev), _rows(k, kv, dev)
            (vp, vs), (op, os_) = _rows(v, kv, dev), _rows(o, shape, dev)
        except _Refused:
            _explain((("q", q, shape), ("k", k, kv), ("v", v, kv), ("o", o, shape)), dev,
                     ("lens", lens, (B,)))
        args = _pack_prompt(B, Hq, Hkv, D, L, qp, kp, vp, op,
                            0 if lse is None else _typed(lse, "lse", _F32, (B, Hq, L), dev), 0,
                            _typed(lens, "lens", _I32, (B,), dev), *qs[:3], *ks[:3], *vs[:3],
                            *os_[:3], softmax_scale)
    _check((_lib or lib()).kvc_prompt_attend(args, stream), "kvc_prompt_attend")


def kvc_chunk_workspace_size(cache: "SlotCache", q, num_splits: int = 0) -> int:
    """Bytes of workspace for kvc_chunk_attend (only q's shape is read).  Fewer tokens may need
    more than many: a workspace kept for several T has the largest of their sizes."""
    cache.desc()
    args = _pack_chunk(q.shape[1], q.shape[0], C.addressof(cache.__dict__["_desc"]), 0, 0, 0, 0, 0, 0,
                       0, 0, 0, 0, num_splits, 0.0)
    return int((_lib or lib()).kvc_chunk_workspace_size(args))


def kvc_chunk_attend(cache: "SlotCache", q, cu_new, o, lse=None, workspace=None,
                     num_splits: int = 0, softmax_scale: float = 0.0, stream=None):
    """Attention of each sequence's chunk of new tokens over the slot cache, which already
    holds their rows in the last slots (see kvc.h): q, o [T, Hq, D] packed by cu_new [B + 1]
    int32 (rows may be strided), lse [Hq, T].  Where an append was refused
    (kvc_read_device_status: KVC_DEV_CAPACITY) the results of that head are not its chunk's."""
    dev, stream = _device(stream)
    d = cache.desc(dev)
    shape = q.shape
    T, Hq, D = shape
    if D != d.D:
        raise ValueError(f"kvc_chunk_attend: q must be [T, Hq, {d.D}], got {tuple(shape)}")
    try:
        qp, (q2, q1, _) = _rows(q, shape, dev)
        op, (o2, o1, _) = _rows(o, shape, dev)
    except _Refused:
        _explain((("q", q, shape), ("o", o, shape)), dev, ("cu_new", cu_new, (d.B + 1,)))
    ws = size = 0
    if workspace is not None:
        ws, size = _ptr(workspace), workspace.nbytes
    args = _pack_chunk(Hq, T, C.addressof(d), qp, op,
                       _typed(cu_new, "cu_new", _I32, (d.B + 1,), dev),
                       0 if lse is None else _typed(lse, "lse", _F32, (Hq, T), dev), q1, q2, o1, o2,
                       ws, size, num_splits, softmax_scale)
    _check((_lib or lib()).kvc_chunk_attend(args, stream), "kvc_chunk_attend")


def kvc_append_plan(cache: "SlotCache", cu_new, slot_map, pool: "Optional[PagePool]" = None,
                    out: "Optional[SlotCache]" = None, pool_out: "Optional[PagePool]" = None,
                    release: bool = False, stream=None):
    """Page tables, slot map [T, Hkv] int32, positions and lengths of a ragged batch of new
    tokens (cu_new [B + 1] int32).  A paged cache takes its pages from `pool`.  `out` and
    `pool_out` receive the new state (default: the cache and the pool, in place)."""
    dev, stream = _device(stream)
    d = cache.desc(dev)
    n = out.desc(dev) if out is not None else d
    pi = pool.desc(d, dev) if pool is not None else None
    po = pool_out.desc(n, dev) if pool_out is not None else pi
    T = slot_map.shape[0]
    _check((_lib or lib()).kvc_append_plan(
        C.addressof(d), pi, _typed(cu_new, "cu_new", _I32, (d.B + 1,), dev), T,
        1 if release else 0, C.addressof(n), po,
        _typed(slot_map, "slot_map", _I32, (T, d.Hkv), dev), stream), "kvc_append_plan")


def kvc_append_packed(cache: "SlotCache", k_new, v_new, slot_map, stream=None):
    """Packed rows k_new, v_new [T, Hkv, D] (rows may be strided) to the cache rows that
    slot_map [T, Hkv] names (kvc_append_plan writes it); n and pos are not touched."""
    dev, stream = _device(stream)
    d = cache.desc(dev)
    T, H = slot_map.shape[0], d.Hkv
    shape = (T, H, d.D)
    try:
        kp, (k0, k1, _) = _rows(k_new, shape, dev)
        vp, (v0, v1, _) = _rows(v_new, shape, dev)
    except _Refused:
        _explain((("k_new", k_new, shape), ("v_new", v_new, shape)), dev,
                 ("slot_map", slot_map, (T, H)))
    _check((_lib or lib()).kvc_append_packed(
        C.addressof(d), kp, _pack_2q(k0, k1), vp, _pack_2q(v0, v1), T,
        _typed(slot_map, "slot_map", _I32, (T, H), dev), stream), "kvc_append_packed")


def kvc_read_device_status(stream=None) -> int:
    out = C.c_int(0)
    st = lib().kvc_read_device_status(C.byref(out), _stream(stream))
    if st not in (KVC_OK, KVC_ERR_DEVICE):
        raise KvcError(st, "kvc_read_device_status")
    return out.value


# ----------------------------------------------------------------------------- cache holders

@dataclass
class SlotCache:
    """fp16 slot cache in device memory (layout documented in include/kvc.h).  Dense layout:
    K, V [B, Hkv, C, D].  Paged layout: K, V are page pools [num_pages, 64, D] and
    block_table [B, Hkv, C // 64] int32 maps each unit's 64-slot pages into them."""
    K: torch.Tensor
    V: torch.Tensor
    pos: torch.Tensor
    n: torch.Tensor
    seqlen: torch.Tensor
    block_table: Optional[torch.Tensor] = None

    @property
    def B(self): return self.pos.shape[0]

    @property
    def Hkv(self): return self.pos.shape[1]

    @property
    def C(self): return self.pos.shape[2]

    @property
    def D(self): return self.K.shape[-1]

    @property
    def num_pages(self): return self.K.shape[0] if self.block_table is not None else 0

    @classmethod
    def empty(cls, B, Hkv, C_, D, device="cuda"):
        return cls(K=torch.zeros(B, Hkv, C_, D, dtype=torch.float16, device=device),
                   V=torch.zeros(B, Hkv, C_, D, dtype=torch.float16, device=device),
                   pos=torch.full((B, Hkv, C_), -1, dtype=torch.int32, device=device),
                   n=torch.zeros(B, Hkv, dtype=torch.int32, device=device),
                   seqlen=torch.zeros(B, dtype=torch.int32, device=device))

    @classmethod
    def empty_paged(cls, B, Hkv, C_, D, num_pages, block_table=None, device="cuda"):
        """Paged cache: pools of num_pages pages of 64 slots; block_table [B, Hkv, C_ // 64]
        (default: unit u owns pages u * C_ / 64 .. (u + 1) * C_ / 64 - 1)."""
        if C_ % PAGE_SLOTS:
            raise ValueError("C must be a multiple of 64 in the paged layout")
        if block_table is None:
            block_table = torch.arange(B * Hkv * (C_ // PAGE_SLOTS), dtype=torch.int32,
                                       device=device).view(B, Hkv, C_ // PAGE_SLOTS)
        return cls(K=torch.zeros(num_pages, PAGE_SLOTS, D, dtype=torch.float16, device=device),
                   V=torch.zeros(num_pages, PAGE_SLOTS, D, dtype=torch.float16, device=device),
                   pos=torch.full((B, Hkv, C_), -1, dtype=torch.int32, device=device),
                   n=torch.zeros(B, Hkv, dtype=torch.int32, device=device),
                   seqlen=torch.zeros(B, dtype=torch.int32, device=device),
                   block_table=block_table.to(device=device, dtype=torch.int32).contiguous())

    def __getstate__(self):
        return _state_without_desc(self)

    def desc(self, dev: Optional[int] = None) -> SlotCacheDesc:
        # built once and kept while the current device (dev, where the caller has it), the
        # fields' storage and shapes stay the same and they are contiguous (a field replaced or
        # resized in place is noticed, and the fields are checked again)
        own = self.__dict__
        if dev is None:
            dev = _current_device()
        K, V, pos, n, sl, bt = self.K, self.V, self.pos, self.n, self.seqlen, self.block_table
        key = own.get("_desc_key")
        if key is not None:
            on, k_p, v_p, kv, pos_p, pos_s, n_p, n_s, sl_p, sl_s, bt_p, bt_s = key
            if (on == dev and K.data_ptr() == k_p and V.data_ptr() == v_p and
                    pos.data_ptr() == pos_p and n.data_ptr() == n_p and sl.data_ptr() == sl_p and
                    K.shape == kv and V.shape == kv and pos.shape == pos_s and n.shape == n_s and
                    sl.shape == sl_s and K.is_contiguous() and V.is_contiguous() and
                    pos.is_contiguous() and n.is_contiguous() and sl.is_contiguous() and
                    (bt_p is None if bt is None else
                     bt.data_ptr() == bt_p and bt.shape == bt_s and bt.is_contiguous())):
                return own["_desc"]
        d = SlotCacheDesc(self.B, self.Hkv, self.D, self.C, _ptr(self.K), _ptr(self.V),
                          _ptr(self.pos), _ptr(self.n), _ptr(self.seqlen),
                          _ptr(self.block_table), self.num_pages)
        own["_desc"] = d
        own["_desc_p"] = C.pointer(d)
        # last: another thread that finds the key finds its descriptor
        own["_desc_key"] = (dev, K.data_ptr(), V.data_ptr(), K.shape, pos.data_ptr(), pos.shape,
                            n.data_ptr(), n.shape, sl.data_ptr(), sl.shape,
                            None if bt is None else bt.data_ptr(),
                            None if bt is None else bt.shape)
        return d


@dataclass
class PagePool:
    """Pages of a paged slot cache (see kvc_append_plan): pages [B, Hkv] int32 held by each
    unit, free [num_pages] int32 a stack of the pages nobody holds, count [1] int32."""
    pages: torch.Tensor
    free: torch.Tensor
    count: torch.Tensor

    @classmethod
    def empty(cls, cache: "SlotCache"):
        """Every page free, none held; the cache's table becomes -1 throughout."""
        dev = cache.n.device
        cache.block_table.fill_(-1)
        return cls(pages=torch.zeros_like(cache.n),
                   free=torch.arange(cache.num_pages - 1, -1, -1, dtype=torch.int32, device=dev),
                   count=torch.full((1,), cache.num_pages, dtype=torch.int32, device=dev))

    def desc(self, cache: SlotCacheDesc, dev: int) -> bytes:
        """The kvc_page_pool struct (the fields of PagePoolDesc) for a cache's descriptor."""
        return _pack_3p(_typed(self.pages, "pages", _I32, (cache.B, cache.Hkv), dev),
                        _typed(self.free, "free", _I32, (cache.num_pages,), dev),
                        _typed(self.count, "count", _I32, (1,), dev))


@dataclass
class QuantCache:
    """KIVI cache in device memory (layout documented in include/kvc.h).  Dense layout:
    k_blocks, v_blocks [B, Hkv, Cq / 32, block_bytes].  Paged layout: pools
    [num_pages, 4, block_bytes] of 4-group (128-token) pages, block_table [B, Hkv, Cq / 128]."""
    k_blocks: torch.Tensor
    v_blocks: torch.Tensor
    k_res: torch.Tensor
    v_res: torch.Tensor
    len: torch.Tensor
    bits: int
    R: int
    block_table: Optional[torch.Tensor] = None
    Cq_paged: int = 0
    k_gear: Optional[torch.Tensor] = None   # GEAR side blocks [B, Hkv, Cq / 32, side_bytes]
    v_gear: Optional[torch.Tensor] = None

    @property
    def B(self): return self.k_res.shape[0]

    @property
    def Hkv(self): return self.k_res.shape[1]

    @property
    def D(self): return self.k_res.shape[3]

    @property
    def Cq(self):
        return self.Cq_paged if self.block_table is not None else self.k_blocks.shape[2] * KIVI_GROUP

    @property
    def num_pages(self): return self.k_blocks.shape[0] if self.block_table is not None else 0

    @classmethod
    def empty(cls, B, Hkv, Cq, D, bits, R, device="cuda", gear=False):
        """KIVI cache; gear=True adds the GEAR side blocks (sparse + rank-2 corrections)."""
        assert Cq % KIVI_GROUP == 0
        bb = KIVI_GROUP * D * bits // 8 + 4 * D
        ng = Cq // KIVI_GROUP
        sb = kvc_gear_side_bytes(D) if gear else 0
        return cls(k_blocks=torch.zeros(B, Hkv, ng, bb, dtype=torch.uint8, device=device),
                   v_blocks=torch.zeros(B, Hkv, ng, bb, dtype=torch.uint8, device=device),
                   k_res=torch.zeros(B, Hkv, R + KIVI_GROUP, D, dtype=torch.float16, device=device),
                   v_res=torch.zeros(B, Hkv, R + KIVI_GROUP, D, dtype=torch.float16, device=device),
                   len=torch.zeros(B, dtype=torch.int32, device=device), bits=bits, R=R,
                   k_gear=torch.zeros(B, Hkv, ng, sb, dtype=torch.uint8, device=device)
                   if gear else None,
                   v_gear=torch.zeros(B, Hkv, ng, sb, dtype=torch.uint8, device=device)
                   if gear else None)

    @classmethod
    def empty_paged(cls, B, Hkv, Cq, D, bits, R, num_pages, block_table=None, device="cuda",
                    gear=False):
        """Paged KIVI cache: pools of num_pages pages of 4 groups; block_table [B, Hkv, Cq / 128]
        (default: unit u owns pages u * Cq / 128 .. (u + 1) * Cq / 128 - 1).  gear=True adds
        GEAR side-block pools [num_pages, 4, side_bytes] behind the same table."""
        page = KIVI_GROUP * KIVI_PAGE_GROUPS
        if Cq % page:
            raise ValueError("Cq must be a multiple of 128 in the paged layout")
        if block_table is None:
            block_table = torch.arange(B * Hkv * (Cq // page), dtype=torch.int32,
                                       device=device).view(B, Hkv, Cq // page)
        bb = KIVI_GROUP * D * bits // 8 + 4 * D
        pool = (num_pages, KIVI_PAGE_GROUPS, bb)
        side = (num_pages, KIVI_PAGE_GROUPS, kvc_gear_side_bytes(D))
        return cls(k_blocks=torch.zeros(pool, dtype=torch.uint8, device=device),
                   v_blocks=torch.zeros(pool, dtype=torch.uint8, device=device),
                   k_res=torch.zeros(B, Hkv, R + KIVI_GROUP, D, dtype=torch.float16, device=device),
                   v_res=torch.zeros(B, Hkv, R + KIVI_GROUP, D, dtype=torch.float16, device=device),
                   len=torch.zeros(B, dtype=torch.int32, device=device), bits=bits, R=R,
                   block_table=block_table.to(device=device, dtype=torch.int32).contiguous(),
                   Cq_paged=Cq,
                   k_gear=torch.zeros(side, dtype=torch.uint8, device=device) if gear else None,
                   v_gear=torch.zeros(side, dtype=torch.uint8, device=device) if gear else None)

    def __getstate__(self):
        return _state_without_desc(self)

    def desc(self) -> QuantCacheDesc:
        # kept while the fields' storage, shapes and strides stay the same (see SlotCache)
        t = (self.k_blocks, self.v_blocks, self.k_res, self.v_res, self.len, self.block_table,
             self.k_gear, self.v_gear)
        key = _desc_key(t) + (self.bits, self.R, self.Cq_paged)
        if self.__dict__.get("_desc_key") == key:
            return self.__dict__["_desc"]
        d = QuantCacheDesc(self.B, self.Hkv, self.D, self.bits, self.R, self.Cq,
                           _ptr(self.k_blocks), _ptr(self.v_blocks), _ptr(self.k_res),
                           _ptr(self.v_res), _ptr(self.len), _ptr(self.block_table),
                           self.num_pages, _ptr(self.k_gear), _ptr(self.v_gear))
        self.__dict__["_desc"] = d
        self.__dict__["_desc_p"] = C.pointer(d)
        self.__dict__["_desc_key"] = key      # last, as in SlotCache
        return d
