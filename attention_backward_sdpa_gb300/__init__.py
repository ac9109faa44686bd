"""GB300 (sm_103a) scaled-dot-product-attention backward.

A thin ctypes binding over ``libsdpa_bwd.so`` (C ABI in ``include/sdpa_bwd.h``).
Every step of the backward runs in the library's CUDA kernels; this module
only checks tensor properties and passes pointers, sizes and the current CUDA
stream. PyTorch is used for device memory and streams.

There is no fallback: if the library cannot be loaded, or the device is not
an sm_103 GPU, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import math
import operator
import os
import struct
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

from . import _build

__all__ = ["sdpa_bwd", "sdpa_fwd", "mask_plan", "MaskPlan", "rope_fwd", "rope_bwd", "rope_inv_freq", "rope_axes",
           "KVCache", "kv_cache", "kv_append", "kv_gather", "sdpa_fwd_cached", "cached_workspace_size",
           "workspace_size", "nvfp4_fake_quant", "sdpa_fwd_nvfp4_qat",
           "sdpa_bwd_nvfp4_qat", "nvfp4_qat_workspace_size", "check_device_status", "debug_relay",
           "profile_enable", "profile_read", "library_path", "load", "SdpaError", "KERNEL_NAMES"]

KERNEL_NAMES = ("preprocess", "main", "dq")

_STATUS = {0: "SDPA_OK", 1: "SDPA_ERR_INVALID", 2: "SDPA_ERR_UNSUPPORTED", 3: "SDPA_ERR_ALIGN",
           4: "SDPA_ERR_WORKSPACE", 5: "SDPA_ERR_CUDA", 6: "SDPA_ERR_TIMEOUT", 7: "SDPA_ERR_BOUNDS",
           8: "SDPA_ERR_PAGE"}


class SdpaError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {_STATUS.get(code, code)} ({_lib_status_string(code)})")


_lib = None


def library_path() -> str:
    """The library this process loads: libsdpa_bwd.so, or the build named by the
    SDPA_BWD_LIBRARY environment variable (for example the debug-bounds build,
    libsdpa_bwd_debug.so, whose kernels check their global accesses)."""
    return os.environ.get("SDPA_BWD_LIBRARY") or _build.LIB


def load(build_if_missing: bool = False):
    """Loads libsdpa_bwd.so (optionally building it first) and declares its ABI."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if build_if_missing and (not os.path.exists(path) or _build.is_stale()):
        _build.build()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m attention_backward_sdpa_gb300._build`"
                           " (or __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.sdpa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, ctypes.c_float,
                             i, i, i, i, i, vp, vp, vp, sz, vp]
    lib.sdpa_bwd.restype = i
    lib.sdpa_bwd_sink.argtypes = list(lib.sdpa_bwd.argtypes[:-1]) + [vp, vp, vp]
    lib.sdpa_bwd_sink.restype = i
    lib.sdpa_bwd_bias.argtypes = list(lib.sdpa_bwd.argtypes[:-1]) + [vp, vp, vp, i, i, vp, vp]
    lib.sdpa_bwd_bias.restype = i
    lib.sdpa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, ctypes.c_float, i, i, i, i,
                             vp, vp, vp, vp]
    lib.sdpa_fwd.restype = i
    lib.sdpa_fwd_bias.argtypes = list(lib.sdpa_fwd.argtypes[:-1]) + [vp, i, i, vp]
    lib.sdpa_fwd_bias.restype = i
    lib.sdpa_bwd_typed.argtypes = [i] + list(lib.sdpa_bwd.argtypes[:-1]) + [vp, vp, vp, i, i, vp, i, vp]
    lib.sdpa_bwd_typed.restype = i
    lib.sdpa_fwd_typed.argtypes = [i] + list(lib.sdpa_fwd.argtypes[:-1]) + [vp, i, i, vp]
    lib.sdpa_fwd_typed.restype = i
    lib.sdpa_fwd_scored.argtypes = [i] + list(lib.sdpa_fwd.argtypes[:-1]) + [ctypes.c_float, vp, vp, vp]
    lib.sdpa_fwd_scored.restype = i
    lib.sdpa_bwd_scored.argtypes = [i] + list(lib.sdpa_bwd.argtypes[:-1]) + [vp, vp, ctypes.c_float, vp, vp, vp]
    lib.sdpa_bwd_scored.restype = i
    lib.sdpa_bwd_scored_workspace_size.argtypes = [i] * 13
    lib.sdpa_bwd_scored_workspace_size.restype = sz
    lib.sdpa_mask_plan_size.argtypes = [i, i, i]
    lib.sdpa_mask_plan_size.restype = sz
    lib.sdpa_mask_plan_rows.argtypes = [vp, vp, i, i, i, vp, sz, vp]
    lib.sdpa_mask_plan_rows.restype = i
    lib.sdpa_mask_plan_docs.argtypes = [vp, vp, i, i, i, i, vp, sz, vp]
    lib.sdpa_mask_plan_docs.restype = i
    lib.sdpa_rope.argtypes = [i, vp, vp, vp, vp, i, i, i, i, i, vp, vp, i,
                              ctypes.c_float, vp, i, i, i, i, vp]
    lib.sdpa_rope.restype = i
    lib.sdpa_rope_axes.argtypes = [i, vp, vp, vp, vp, i, i, i, i, i, vp, vp, i,
                                   ctypes.c_float, vp, i, i, vp, i, i, vp]
    lib.sdpa_rope_axes.restype = i
    lib.sdpa_kv_append.argtypes = [i, i] + [vp] * 11 + [i] * 8 + [vp, vp, i, ctypes.c_float, vp, i, i, vp, i, vp]
    lib.sdpa_kv_append.restype = i
    lib.sdpa_kv_gather.argtypes = [i, i] + [vp] * 8 + [i] * 7 + [vp]
    lib.sdpa_kv_gather.restype = i
    lib.sdpa_fwd_cached_workspace_size.argtypes = [i] * 8
    lib.sdpa_fwd_cached_workspace_size.restype = sz
    lib.sdpa_fwd_cached.argtypes = [i, i] + [vp] * 10 + [i] * 8 + [ctypes.c_float, i, i, i, vp, ctypes.c_float, vp, vp,
                                                                  sz, vp]
    lib.sdpa_fwd_cached.restype = i
    lib.sdpa_nvfp4_fake_quant.argtypes = [vp, vp, ctypes.c_longlong, vp]
    lib.sdpa_nvfp4_fake_quant.restype = i
    lib.sdpa_bwd_nvfp4_qat_workspace_size.argtypes = [i, i, i, i, i, i, i]
    lib.sdpa_bwd_nvfp4_qat_workspace_size.restype = sz
    lib.sdpa_bwd_nvfp4_qat.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i,
                                       ctypes.c_float, i, i, i, i, vp, vp, vp, sz, vp]
    lib.sdpa_bwd_nvfp4_qat.restype = i
    lib.sdpa_bwd_workspace_size.argtypes = [i] * 13
    lib.sdpa_bwd_workspace_size.restype = sz
    lib.sdpa_status_string.argtypes = [i]
    lib.sdpa_status_string.restype = ctypes.c_char_p
    lib.sdpa_bwd_debug_relay.argtypes = [ctypes.c_ulonglong, i]
    lib.sdpa_bwd_debug_relay.restype = i
    lib.sdpa_bwd_check_device_status.argtypes = [vp]
    lib.sdpa_bwd_check_device_status.restype = i
    lib.sdpa_bwd_profile_enable.argtypes = [i]
    lib.sdpa_bwd_profile_enable.restype = i
    lib.sdpa_bwd_profile_read.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int), i]
    lib.sdpa_bwd_profile_read.restype = i
    lib.sdpa_bwd_version.restype = i
    _lib = lib
    return lib


def _lib_status_string(code: int) -> str:
    try:
        return load().sdpa_status_string(code).decode()
    except Exception:  # pragma: no cover - only used while formatting an error
        return "?"


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _addr(t: Optional[torch.Tensor]):
    """The address as a plain integer (ctypes takes it for a pointer; no object is made)."""
    return None if t is None else t.data_ptr()


def _stream_handle(stream: Optional[torch.cuda.Stream]):
    if stream is not None:
        return stream.cuda_stream
    # (torch.cuda.current_stream() builds a Stream object: 2.9 us a call on the Arm
    # host against 0.1 us for the handle itself)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _empty(shape, dtype: torch.dtype, device: torch.device, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """A tensor that a call on a stream given to it makes (a call without one takes torch.empty
    itself, which is 0.6 us less). The memory is that stream's, so that its work comes after
    whatever held the block before, and the current stream, where the caller has the tensor
    in hand, is recorded as a user of it: dropped on either side, the block serves nothing
    else before both have passed that point."""
    if stream is None or device.type != "cuda":  # (the checks refuse the latter)
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _empty_like(t: torch.Tensor, stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    return torch.empty_like(t) if stream is None else _empty(t.shape, t.dtype, t.device, stream)


def _is(t, dtype, dev: int, shape) -> bool:
    """Whether t is a contiguous tensor of this type, device index and shape: the checks
    of a call in one test. A call whose tensors fail it goes through the checks
    that name what is wrong; small calls spend most of their time on the host."""
    return type(t) is torch.Tensor and t.dtype is dtype and t.get_device() == dev and t.shape == shape \
        and t.is_contiguous()


def _optional(t, dtype, dev: int, numel: int) -> bool:
    """The same for an optional tensor of numel elements in any shape."""
    return t is None or (type(t) is torch.Tensor and t.dtype is dtype and t.get_device() == dev
                         and t.numel() == numel and t.is_contiguous())


def workspace_size(B, Hq, Hkv, Sq, Skv, Dqk, Dv, deterministic=False, *, causal=False,
                   bottom_right=False, window_left=-1, window_right=-1, padded=False,
                   scored=False) -> int:
    """Workspace bytes of sdpa_bwd for this shape and mask (``padded``: length
    arrays will be passed; ``scored``: softcap, alibi_slopes or a mask_plan will be).
    The defaults (no mask) give the largest size for the shape, which serves every mask."""
    lib = load()
    size = lib.sdpa_bwd_scored_workspace_size if scored else lib.sdpa_bwd_workspace_size
    return int(size(B, Hq, Hkv, Sq, Skv, Dqk, Dv, int(causal), int(bottom_right), int(window_left),
                    int(window_right), int(deterministic), int(padded)))


@functools.lru_cache(maxsize=4096)
def _scored_workspace(lib, *sizes) -> int:
    return int(lib.sdpa_bwd_scored_workspace_size(*sizes))


def _check_bf16(name, t, shape, dtype=torch.bfloat16):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _check_lens(B, seq_q_lens, seq_kv_lens):
    for name, lens in (("seq_q_lens", seq_q_lens), ("seq_kv_lens", seq_kv_lens)):
        if lens is not None and (lens.dtype != torch.int32 or not lens.is_cuda or lens.numel() != B
                                 or not lens.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous int32 CUDA tensor of B elements")


def _check_lse(lse, B, Hq, Sq):
    if lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous() \
            or lse.numel() != B * Hq * Sq:
        raise ValueError("lse must be a contiguous fp32 CUDA tensor with B*Hq*Sq elements")


def _check_workspace(workspace) -> int:
    if workspace is None:
        return 0
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return workspace.numel() * workspace.element_size()


def _check_sink(sink, dsink, Hq, stream=None):
    """Validates the fp32 (Hq,) sink logits; returns dsink (allocated when None)."""
    if sink.dtype != torch.float32 or not sink.is_cuda or not sink.is_contiguous() \
            or sink.numel() != Hq:
        raise ValueError("sink must be a contiguous fp32 CUDA tensor of Hq elements")
    dsink = _empty_like(sink, stream) if dsink is None else dsink
    if dsink.dtype != torch.float32 or not dsink.is_cuda or not dsink.is_contiguous() \
            or dsink.numel() != Hq:
        raise ValueError("dsink must be a contiguous fp32 CUDA tensor of Hq elements")
    return dsink


def _check_same_device(ref: torch.Tensor, _ref: str = "q", **tensors) -> None:
    """Every tensor argument lives on ref's device (the library takes raw pointers
    and launches on one device)."""
    for name, t in tensors.items():
        if t is not None and t.device != ref.device:
            raise ValueError(f"{name} is on {t.device} but {_ref} is on {ref.device}: "
                             "all tensors must be on one device")


def _check_launch_device(ref: torch.Tensor) -> None:
    """The library launches on the current CUDA device: it must be the tensors' one."""
    if ref.get_device() != torch._C._cuda_getDevice():
        raise ValueError(f"the tensors are on {ref.device} but the current device is "
                         f"cuda:{torch.cuda.current_device()}: call under torch.cuda.device({ref.device})")


_INT32 = 1 << 31  # (ctypes would take a larger int modulo 2^32)

# io element types of the C ABI (sdpa_dtype) for the typed entry points.
_IO_CODES = {torch.bfloat16: 0, torch.float16: 2}

_MAX_AXES = 16  # axes of rotary positions


def _io_dtype(q):
    if not isinstance(q, torch.Tensor) or q.dtype not in _IO_CODES:
        raise ValueError("q must be a bf16 or fp16 tensor")
    return q.dtype


def sdpa_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, do: torch.Tensor,
             lse: torch.Tensor, *, scale: Optional[float] = None, causal: bool = False,
             bottom_right: bool = False, window_left: int = -1, window_right: int = -1,
             deterministic: bool = False, seq_q_lens: Optional[torch.Tensor] = None,
             seq_kv_lens: Optional[torch.Tensor] = None, dq: Optional[torch.Tensor] = None,
             dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None, sink: Optional[torch.Tensor] = None,
             dsink: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
             dbias: Optional[torch.Tensor] = None, bias_grad: bool = True,
             dbias_dtype: torch.dtype = torch.float32, softcap: float = 0.0,
             alibi_slopes: Optional[torch.Tensor] = None, mask_plan: Optional["MaskPlan"] = None,
             stream: Optional[torch.cuda.Stream] = None):
    """dQ, dK, dV of scaled-dot-product attention (see include/sdpa_bwd.h).

    q (B,Hq,Sq,Dqk), k (B,Hkv,Skv,Dqk), v (B,Hkv,Skv,Dv), o/do (B,Hq,Sq,Dv): bf16 or fp16
    (one type for all) CUDA tensors on the current device, contiguous. lse (B,Hq,Sq) fp32 natural-log forward statistic. Lengths: int32 (B,) CUDA.
    Outputs are allocated when not given. Runs on ``stream`` (default: current stream; the
    caller orders the inputs before it and the outputs' uses after it).
    With ``sink`` (fp32 (Hq,) CUDA sink logits, already folded into ``lse`` by the
    forward) the call goes through sdpa_bwd_sink and returns (dq, dk, dv, dsink).
    With ``bias`` ((1|B, Hq, Sq, Skv) bf16, fp16 or fp32 CUDA, contiguous: the additive
    bias that ``lse`` was computed with) the call goes through sdpa_bwd_bias and,
    unless ``bias_grad`` is False, appends the fp32 dBias (shaped like ``bias``) to
    the returned tuple (``dbias_dtype`` float32, or bfloat16 / float16 for the
    io-type dBias of the general entry point).
    With ``softcap`` (> 0), ``alibi_slopes`` (fp32 (Hq,) CUDA) or ``mask_plan`` the call
    goes through sdpa_bwd_scored: the gradient of sdpa_fwd with the same three (not
    together with ``bias``; a plan with ``deterministic`` only at D_qk 128, 192 and 256).
    """
    lib = load()
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be (B, H, S, D)")
    io = _io_dtype(q)
    B, Hq, Sq, Dqk = q.shape
    Hkv, Skv = k.shape[1], k.shape[2]
    Dv = v.shape[3]
    fresh = dq is None and dk is None and dv is None  # (outputs made here need no checks)
    dq = _empty_like(q, stream) if dq is None else dq
    dk = _empty_like(k, stream) if dk is None else dk
    dv = _empty_like(v, stream) if dv is None else dv
    ws_bytes = _check_workspace(workspace)
    if sink is not None:
        dsink = _check_sink(sink, dsink, Hq, stream)
    dev, q_shape, k_shape, o_shape = q.get_device(), (B, Hq, Sq, Dqk), (B, Hkv, Skv, Dqk), (B, Hq, Sq, Dv)
    if not (q.is_cuda and _is(q, io, dev, q_shape) and _is(k, io, dev, k_shape) and _is(v, io, dev, (B, Hkv, Skv, Dv))
            and _is(o, io, dev, o_shape) and _is(do, io, dev, o_shape)
            and (fresh or _is(dq, io, dev, q_shape) and _is(dk, io, dev, k_shape)
                 and _is(dv, io, dev, (B, Hkv, Skv, Dv)))
            and lse is not None and _optional(lse, torch.float32, dev, B * Hq * Sq)
            and (seq_q_lens is None or _optional(seq_q_lens, torch.int32, dev, B))
            and (seq_kv_lens is None or _optional(seq_kv_lens, torch.int32, dev, B))
            and workspace is None and sink is None and bias is None):
        _check_bf16("q", q, q_shape, io)
        _check_bf16("k", k, k_shape, io)
        _check_bf16("v", v, (B, Hkv, Skv, Dv), io)
        _check_bf16("o", o, o_shape, io)
        _check_bf16("do", do, o_shape, io)
        _check_lse(lse, B, Hq, Sq)
        _check_lens(B, seq_q_lens, seq_kv_lens)
        _check_bf16("dq", dq, q.shape, io)
        _check_bf16("dk", dk, k.shape, io)
        _check_bf16("dv", dv, v.shape, io)
        _check_same_device(q, k=k, v=v, o=o, do=do, lse=lse, seq_q_lens=seq_q_lens,
                           seq_kv_lens=seq_kv_lens, dq=dq, dk=dk, dv=dv, workspace=workspace,
                           sink=sink, dsink=dsink if sink is not None else None, bias=bias,
                           dbias=dbias if bias is not None and bias_grad else None)
    scored = _check_score_mods(q, B, Hq, Sq, Skv, softcap, alibi_slopes, mask_plan, bias, window_left, window_right)
    _check_launch_device(q)
    sc = 0.0 if scale is None else float(scale)
    if scored:
        if workspace is None and stream is None:
            # From torch's allocator, which keeps it for the next call. (The library's own
            # comes from the stream-ordered pool, which returns its memory at every
            # synchronization and maps it again at the next call: 2,018 us for the first
            # call after one instead of 447 at B 1, Hq 32, S 4096, D 128, deterministic.)
            # A call on a stream given to it leaves this to the library, whose allocation is
            # ordered on that stream.
            ws_bytes = _scored_workspace(lib, B, Hq, Hkv, Sq, Skv, Dqk, Dv, int(causal), int(bottom_right),
                                         int(window_left), int(window_right), int(deterministic),
                                         int(seq_q_lens is not None or seq_kv_lens is not None))
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device) if ws_bytes else None
        rc = lib.sdpa_bwd_scored(_IO_CODES[io], q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
                                 lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv, Sq, Skv, Dqk,
                                 Dv, sc, int(causal), int(bottom_right), int(window_left), int(window_right),
                                 int(deterministic), _addr(seq_q_lens), _addr(seq_kv_lens), _addr(workspace), ws_bytes,
                                 _addr(sink), None if sink is None else dsink.data_ptr(), float(softcap),
                                 _addr(alibi_slopes),
                                 None if mask_plan is None else mask_plan._on(stream), _stream_handle(stream))
        if rc != 0:
            raise SdpaError(rc, "sdpa_bwd_scored")
        return (dq, dk, dv) + ((dsink,) if sink is not None else ())
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk),
            _ptr(dv), B, Hq, Hkv, Sq, Skv, Dqk, Dv, sc, int(causal), int(bottom_right),
            int(window_left), int(window_right), int(deterministic), _ptr(seq_q_lens),
            _ptr(seq_kv_lens), _ptr(workspace), ws_bytes)
    if io == torch.float16 or (bias is not None and bias_grad and dbias_dtype != torch.float32):
        # the general typed entry: fp16 io, or an io-type dBias (sink and bias optional)
        bias_dtype, bias_batch = 0, 0
        if bias is not None:
            bias_dtype = _check_bias(bias, B, Hq, Sq, Skv)
            bias_batch = int(bias.shape[0])
            if bias_grad:
                if dbias_dtype not in (torch.float32, torch.bfloat16, torch.float16):
                    raise ValueError("dbias_dtype must be float32, bfloat16 or float16")
                dbias = _empty(bias.shape, dbias_dtype, bias.device, stream) if dbias is None else dbias
                if dbias.dtype != dbias_dtype or not dbias.is_cuda or not dbias.is_contiguous() \
                        or tuple(dbias.shape) != tuple(bias.shape):
                    raise ValueError("dbias must be a contiguous CUDA tensor shaped like bias, of dbias_dtype")
            else:
                dbias = None
        else:
            dbias = None
        dbias_code = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16,
                      torch.float16: DTYPE_F16}[dbias.dtype] if dbias is not None else DTYPE_F32
        rc = lib.sdpa_bwd_typed(_IO_CODES[io], *args, _ptr(sink), _ptr(dsink if sink is not None else None),
                                _ptr(bias), bias_dtype, bias_batch, _ptr(dbias), dbias_code,
                                _stream_handle(stream))
        if rc != 0:
            raise SdpaError(rc, "sdpa_bwd_typed")
        out = (dq, dk, dv) + ((dsink,) if sink is not None else ())
        return out + ((dbias,) if bias is not None and bias_grad else ())
    if sink is None and bias is None:
        rc = lib.sdpa_bwd(*args, _stream_handle(stream))
        if rc != 0:
            raise SdpaError(rc, "sdpa_bwd")
        return dq, dk, dv
    if bias is None:
        rc = lib.sdpa_bwd_sink(*args, _ptr(sink), _ptr(dsink), _stream_handle(stream))
        if rc != 0:
            raise SdpaError(rc, "sdpa_bwd_sink")
        return dq, dk, dv, dsink
    bias_dtype = _check_bias(bias, B, Hq, Sq, Skv)
    if bias_grad:
        dbias = _empty(bias.shape, torch.float32, bias.device, stream) if dbias is None else dbias
        if dbias.dtype != torch.float32 or not dbias.is_cuda or not dbias.is_contiguous() \
                or tuple(dbias.shape) != tuple(bias.shape):
            raise ValueError("dbias must be a contiguous fp32 CUDA tensor shaped like bias")
    else:
        dbias = None
    rc = lib.sdpa_bwd_bias(*args, _ptr(sink), _ptr(dsink if sink is not None else None), _ptr(bias),
                           bias_dtype, int(bias.shape[0]), _ptr(dbias), _stream_handle(stream))
    if rc != 0:
        raise SdpaError(rc, "sdpa_bwd_bias")
    out = (dq, dk, dv) + ((dsink,) if sink is not None else ())
    return out + ((dbias,) if bias_grad else ())


# Element-type codes of the C ABI (sdpa_dtype).
DTYPE_BF16, DTYPE_F32, DTYPE_F16 = 0, 1, 2


def _check_bias(bias, B, Hq, Sq, Skv) -> int:
    if not isinstance(bias, torch.Tensor) or not bias.is_cuda or not bias.is_contiguous():
        raise ValueError("bias must be a contiguous CUDA tensor")
    if bias.dtype not in (torch.bfloat16, torch.float16, torch.float32):
        raise ValueError("bias must be bf16, fp16 or fp32")
    if bias.dim() != 4 or bias.shape[0] not in (1, B) or tuple(bias.shape[1:]) != (Hq, Sq, Skv):
        raise ValueError(f"bias must be (1|B, Hq, Sq, Skv), got {tuple(bias.shape)}")
    return {torch.float32: DTYPE_F32, torch.float16: DTYPE_F16}.get(bias.dtype, DTYPE_BF16)


class MaskPlan:
    """The key range of every query row of a batch, with the tile summaries that the
    kernels take their loop bounds from; made by mask_plan()."""

    def __init__(self, B: int, Sq: int, Skv: int, buffer: torch.Tensor, home: Optional[int] = None):
        self.B, self.Sq, self.Skv, self.buffer = B, Sq, Skv, buffer
        self._home = home  # the stream whose memory the buffer is, as a handle

    def _on(self, stream: Optional[torch.cuda.Stream]) -> int:
        """The buffer's address, for work on ``stream`` (None: the current one): recorded as a
        user of the buffer, so that a plan may be dropped while work that reads it is queued."""
        if _stream_handle(stream) != self._home:
            self.buffer.record_stream(torch.cuda.current_stream(self.buffer.device) if stream is None else stream)
        return self.buffer.data_ptr()

    def __repr__(self) -> str:
        return f"MaskPlan(B={self.B}, Sq={self.Sq}, Skv={self.Skv}, device={self.buffer.device})"


def _check_int32(name, t, shapes):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous() \
            or tuple(t.shape) not in shapes:
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor of shape "
                         + " or ".join(str(s) for s in shapes))


def mask_plan(B: int, Sq: int, Skv: int, *, doc_ids: Optional[torch.Tensor] = None,
              prefix_lens: Optional[torch.Tensor] = None, causal: bool = False,
              row_lo: Optional[torch.Tensor] = None, row_hi: Optional[torch.Tensor] = None,
              device: Optional[torch.device] = None, plan: Optional[MaskPlan] = None,
              stream: Optional[torch.cuda.Stream] = None) -> MaskPlan:
    """The mask plan that sdpa_fwd and sdpa_bwd take as ``mask_plan``, made once per
    batch for every layer and both directions.

    Packed documents and prefixes (Sq = Skv): ``doc_ids`` int32 (B, Sq), a document being
    a maximal run of equal consecutive ids; a row sees its own document, with ``causal``
    the part up to itself. ``prefix_lens`` int32 (B,), or (B, Sq) for a length at each
    position, lets every row of a document see its first keys too (needs ``causal``).
    The attention call then takes causal=False: the plan holds the causal side.
    Or any ranges: row i of batch row b sees keys [row_lo[b, i], row_hi[b, i]), int32
    (B, Sq) both. ``plan``: one of the same sizes to write into again.
    """
    lib = load()
    B, Sq, Skv = int(B), int(Sq), int(Skv)
    if not all(0 < n < _INT32 for n in (B, Sq, Skv)):
        raise ValueError("B, Sq and Skv must be positive 32-bit sizes")
    rows = row_lo is not None or row_hi is not None
    if rows and (row_lo is None or row_hi is None or doc_ids is not None or prefix_lens is not None or causal):
        raise ValueError("row_lo and row_hi come together, without doc_ids, prefix_lens or causal")
    if not rows and Sq != Skv:
        raise ValueError("documents and prefixes need Sq = Skv: pass row_lo and row_hi")
    if prefix_lens is not None and not causal:
        raise ValueError("prefix_lens widen a causal mask: pass causal=True")
    tensors = {"row_lo": row_lo, "row_hi": row_hi, "doc_ids": doc_ids, "prefix_lens": prefix_lens}
    for name, t in tensors.items():
        if t is not None:
            _check_int32(name, t, ((B,), (B, Sq)) if name == "prefix_lens" else ((B, Sq),))
    size = int(lib.sdpa_mask_plan_size(B, Sq, Skv))
    if size == 0:
        raise SdpaError(1, "sdpa_mask_plan_size")
    if plan is None:
        given = next((t for t in tensors.values() if t is not None), None)
        dev = given.device if given is not None else torch.device("cuda" if device is None else device)
        plan = MaskPlan(B, Sq, Skv, _empty(size, torch.uint8, dev, stream), _stream_handle(stream))
    elif (plan.B, plan.Sq, plan.Skv) != (B, Sq, Skv):
        raise ValueError(f"plan was made for {plan!r}, not for B={B}, Sq={Sq}, Skv={Skv}")
    _check_same_device(plan.buffer, _ref="the plan", **tensors)
    _check_launch_device(plan.buffer)
    if rows:
        rc = lib.sdpa_mask_plan_rows(_ptr(row_lo), _ptr(row_hi), B, Sq, Skv, plan._on(stream), size,
                                     _stream_handle(stream))
    else:
        rc = lib.sdpa_mask_plan_docs(_ptr(doc_ids), _ptr(prefix_lens),
                                     int(prefix_lens is not None and prefix_lens.dim() == 2), int(causal), B, Sq,
                                     plan._on(stream), size, _stream_handle(stream))
    if rc != 0:
        raise SdpaError(rc, "sdpa_mask_plan_rows" if rows else "sdpa_mask_plan_docs")
    return plan


def _check_score_mods(q, B, Hq, Sq, Skv, softcap, alibi_slopes, mask_plan, bias, window_left, window_right) -> bool:
    """Whether the call modifies its scores (and then that it may)."""
    if not (softcap == 0.0 or 2.0 ** -126 <= softcap < math.inf):  # (a smaller one may be 0 in fp32: no cap)
        raise ValueError("softcap must be 0 (none) or a positive finite number, normal in fp32")
    if softcap == 0.0 and alibi_slopes is None and mask_plan is None:
        return False
    if bias is not None:
        raise ValueError("softcap, alibi_slopes and mask_plan do not combine with bias")
    if not (-_INT32 <= window_left < _INT32 and -_INT32 <= window_right < _INT32):
        raise ValueError("window_left and window_right are 32-bit numbers of keys")
    if alibi_slopes is not None and (
            not isinstance(alibi_slopes, torch.Tensor) or alibi_slopes.dtype != torch.float32
            or not alibi_slopes.is_cuda or not alibi_slopes.is_contiguous() or tuple(alibi_slopes.shape) != (Hq,)):
        raise ValueError("alibi_slopes must be a contiguous fp32 CUDA tensor of shape (Hq,)")
    if mask_plan is not None:
        if not isinstance(mask_plan, MaskPlan):
            raise TypeError("mask_plan must be a MaskPlan (made by mask_plan())")
        if (mask_plan.B, mask_plan.Sq, mask_plan.Skv) != (B, Sq, Skv):
            raise ValueError(f"mask_plan was made for {mask_plan!r}, not for B={B}, Sq={Sq}, Skv={Skv}")
    if alibi_slopes is not None and alibi_slopes.get_device() != q.get_device():
        _check_same_device(q, alibi_slopes=alibi_slopes)
    if mask_plan is not None and mask_plan.buffer.get_device() != q.get_device():
        _check_same_device(q, mask_plan=mask_plan.buffer)
    return True


def rope_inv_freq(rot_dim: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                  original_len: int = 0, low: float = 1.0, high: float = 32.0,
                  device=None) -> torch.Tensor:
    """The fp64 (rot_dim / 2,) frequencies (radians per position) that rope_fwd takes:
    f[i] = base^(-2 i / rot_dim), and for contexts longer than the trained one by ``factor``

      "linear"  f / factor (every position interpolated),
      "ntk"     the same with base * factor^(rot_dim / (rot_dim - 2)) (the lowest
                frequency interpolated by ``factor``, the highest kept),
      "bands"   by how often a frequency turns over ``original_len`` positions,
                r = original_len * f / (2 pi): kept where r >= high, interpolated where
                r <= low, a linear mix between (the ramp of the YaRN paper, Peng et al.
                2023; its factor on the scores is rope_fwd's mult =
                0.1 ln(factor) + 1 on both queries and keys).

    Made on the host and copied to ``device``: once, outside of a graph's capture.
    """
    if rot_dim <= 0 or rot_dim % 2:
        raise ValueError("rot_dim must be even and positive")
    if not (base > 0.0 and math.isfinite(base)) or not (factor > 0.0 and math.isfinite(factor)):
        raise ValueError("base and factor must be positive finite numbers")
    if scaling not in ("none", "linear", "ntk", "bands"):
        raise ValueError("scaling must be none, linear, ntk or bands")
    if scaling == "ntk":
        if rot_dim < 4:
            raise ValueError("ntk scaling needs rot_dim >= 4")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = float(base) ** (-2.0 * torch.arange(rot_dim // 2, dtype=torch.float64) / rot_dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "bands":
        if original_len <= 0 or not low < high:
            raise ValueError("bands scaling needs original_len > 0 and low < high")
        keep = ((original_len * f / (2.0 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / factor)
    return f.to(torch.device("cuda") if device is None else device)


def rope_axes(sections: Sequence[int], *, mixed: bool = False, device=None) -> torch.Tensor:
    """The int32 (sum(sections),) ``axes`` that rope_fwd takes: axis a turns sections[a] pairs,
    one section after another, or with ``mixed`` the axes in turn from pair to pair, each while
    it has pairs left. Copied to ``device``: once, outside of a graph's capture."""
    sizes = [operator.index(n) for n in sections]
    if not sizes or len(sizes) > _MAX_AXES or min(sizes) < 0 or sum(sizes) == 0:
        raise ValueError(f"sections are 1 to {_MAX_AXES} numbers of pairs, not all 0")
    if mixed:
        order = [a for turn in range(max(sizes)) for a, n in enumerate(sizes) if turn < n]
    else:
        order = [a for a, n in enumerate(sizes) for _ in range(n)]
    return torch.tensor(order, dtype=torch.int32).to(torch.device("cuda") if device is None else device)


def _check_axes(axes, positions, pairs, B, S):
    """Names what is wrong with a call's axes and their positions."""
    if positions is None:
        raise ValueError("axes need positions, (n_axes, S) or (n_axes, B, S)")
    _check_int32("axes", axes, ((pairs,),))
    if not isinstance(positions, torch.Tensor) or positions.dim() not in (2, 3) or not 1 <= positions.shape[0] <= _MAX_AXES:
        raise ValueError(f"positions must be (n_axes, S) or (n_axes, B, S) with axes, n_axes from 1 to {_MAX_AXES}")
    n = positions.shape[0]
    _check_int32("positions", positions, ((n, S), (n, B, S)))


def _check_rope_args(q, k, inv_freq, positions, offset, q_out, k_out, axes=None):
    """Names what is wrong with a rope call's arguments."""
    io = _io_dtype(q)
    if q.dim() != 4:
        raise ValueError("q must be (B, H, S, D)")
    B, _, S, D = q.shape
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    if k is not None and (not isinstance(k, torch.Tensor) or k.dim() != 4):
        raise ValueError("k must be a (B, H, S, D) tensor")
    for name, t, like in (("q", q, q), ("k", k, k), ("q_out", q_out, q), ("k_out", k_out, k)):
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype != io or not t.is_cuda:
            raise ValueError(f"{name} must be a {io} CUDA tensor")
        shape = (B, like.shape[1], S, D)
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
        if t.stride(3) != 1 and D > 1:
            raise ValueError(f"{name} must have contiguous columns (stride 1 in its last dimension)")
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dtype != torch.float64 or not inv_freq.is_cuda \
            or not inv_freq.is_contiguous() or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be a contiguous fp64 CUDA vector (rope_inv_freq)")
    rot = 2 * inv_freq.numel()
    if rot == 0 or rot > D:
        raise ValueError(f"inv_freq rotates {rot} columns of {D}")
    if axes is not None:
        _check_axes(axes, positions, rot // 2, B, S)
    if positions is not None:
        if axes is None:
            _check_int32("positions", positions, ((S,), (B, S)))
        if offset != 0:
            raise ValueError("offset counts from position 0 where no positions are given")
    _check_same_device(q, k=k, inv_freq=inv_freq, positions=positions, q_out=q_out, k_out=k_out, axes=axes)


_strides = struct.Struct("12q").pack  # (0.1 us on the Arm host, against 1.1 for a ctypes array)


def _rope(q, k, inv_freq, mult, positions, offset, interleaved, inverse, q_out, k_out, stream, axes=None):
    lib = load()
    new = torch.empty if stream is None else functools.partial(_empty, stream=stream)
    try:
        shape, sq = q.shape, q.stride()
        B, Hq, S, D = shape
        io, dev, Hkv = q.dtype, q.get_device(), 0
        good = q.is_cuda and io in _IO_CODES and sq[3] == 1
        # (Outputs made here need no checks.)
        if q_out is None:
            q_out, so = new(shape, dtype=io, device=q.device), (Hq * S * D, S * D, D)
        else:
            so = q_out.stride()
            good = good and q_out.dtype is io and q_out.get_device() == dev and q_out.shape == shape and so[3] == 1
        if k is None:
            sk = sl = sq
            good = good and k_out is None
        else:
            shape, sk = k.shape, k.stride()
            Hkv = shape[1]
            good = good and k.dtype is io and k.get_device() == dev and shape == (B, Hkv, S, D) and sk[3] == 1
            if k_out is None:
                k_out, sl = new(shape, dtype=io, device=q.device), (Hkv * S * D, S * D, D)
            else:
                sl = k_out.stride()
                good = good and k_out.dtype is io and k_out.get_device() == dev and k_out.shape == shape and sl[3] == 1
        rot = 2 * inv_freq.shape[0]
        good = good and 0 < rot <= D and _is(inv_freq, torch.float64, dev, (rot // 2,)) \
            and (positions is None or offset == 0 and (_is(positions, torch.int32, dev, (B, S))
                                                       or _is(positions, torch.int32, dev, (S,)))
                 if axes is None else
                 offset == 0 and _is(axes, torch.int32, dev, (rot // 2,)) and 1 <= positions.shape[0] <= _MAX_AXES
                 and (_is(positions, torch.int32, dev, (positions.shape[0], B, S))
                      or _is(positions, torch.int32, dev, (positions.shape[0], S))))
    except (AttributeError, IndexError, TypeError, ValueError):  # not tensors, or of other dimensions
        good = False
    if not good:
        _check_rope_args(q, k, inv_freq, positions, offset, q_out, k_out, axes)
        B, Hq, S, D = q.shape
        sq, so, Hkv, rot = q.stride(), q_out.stride(), 0, 2 * inv_freq.numel()
        sk, sl = sq, so
        if k is not None:
            sk, sl, Hkv = k.stride(), k_out.stride(), k.shape[1]
    _check_launch_device(q)
    if not 0 <= offset <= _INT32 - S:
        raise ValueError("offset must be at least 0, and offset + S at most 2^31")
    if B > 0 and Hq + Hkv > 0:
        x, z, x_out, z_out = q, k, q_out, k_out
        if Hq == 0:  # the keys alone, as the C call's first tensor
            x, z, x_out, z_out, sq, so, Hq, Hkv = k, None, k_out, None, sk, sl, Hkv, 0
        at = _strides(sq[0], sq[1], sq[2], so[0], so[1], so[2], sk[0], sk[1], sk[2], sl[0], sl[1], sl[2])
        if axes is not None:
            rc = lib.sdpa_rope_axes(_IO_CODES[x.dtype], x.data_ptr(), _addr(z), x_out.data_ptr(), _addr(z_out), B, Hq,
                                    Hkv, S, D, at, inv_freq.data_ptr(), rot, float(mult), positions.data_ptr(),
                                    positions.dim() - 2, positions.shape[0], axes.data_ptr(), bool(interleaved), inverse,
                                    _stream_handle(stream))
            if rc != 0:
                raise SdpaError(rc, "sdpa_rope_axes")
            return q_out, k_out
        rc = lib.sdpa_rope(_IO_CODES[x.dtype], x.data_ptr(), _addr(z), x_out.data_ptr(), _addr(z_out), B, Hq, Hkv, S, D,
                           at, inv_freq.data_ptr(), rot, float(mult), _addr(positions),
                           0 if positions is None else positions.dim() - 1, operator.index(offset), bool(interleaved),
                           inverse, _stream_handle(stream))
        if rc != 0:
            raise SdpaError(rc, "sdpa_rope")
    return q_out, k_out


def rope_fwd(q: torch.Tensor, k: Optional[torch.Tensor], inv_freq: torch.Tensor, *, mult: float = 1.0,
             positions: Optional[torch.Tensor] = None, offset: int = 0, interleaved: bool = False,
             q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
             axes: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """Rotary embedding of q (B,Hq,S,D) and k (B,Hkv,S,D) (or of q alone, k None): the
    first 2 * inv_freq.numel() columns turn pair by pair by position * inv_freq and are
    multiplied by ``mult``, the others are copied (sdpa_rope in include/sdpa_bwd.h).

    bf16 or fp16, any strides of batch, head and position with contiguous columns: a
    projection's (B,S,H,D) output goes in as a transposed view and comes out contiguous
    (B,H,S,D) for sdpa_fwd. ``inv_freq``: fp64 CUDA vector (rope_inv_freq).
    ``positions``: int32 (S,) or (B,S), else offset .. offset + S - 1. Pairs are columns
    (i, i + rot/2), or (2i, 2i+1) when ``interleaved``. With ``axes`` (int32 (rot/2,), the axis of
    each pair: rope_axes) positions are (n_axes,S) or (n_axes,B,S), and pair i turns by that of
    its axis (tokens of images and videos; sdpa_rope_axes). Returns (q_out, k_out). An
    output may be its own input (the same tensor: in place) and overlaps nothing else.
    """
    return _rope(q, k, inv_freq, mult, positions, offset, interleaved, False, q_out, k_out, stream, axes)


def rope_bwd(dq: torch.Tensor, dk: Optional[torch.Tensor], inv_freq: torch.Tensor, *, mult: float = 1.0,
             positions: Optional[torch.Tensor] = None, offset: int = 0, interleaved: bool = False,
             q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
             axes: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """The gradients of rope_fwd's inputs from those of its outputs (dq, dk of sdpa_bwd):
    the transposed rotation, with rope_fwd's other arguments."""
    return _rope(dq, dk, inv_freq, mult, positions, offset, interleaved, True, q_out, k_out, stream, axes)


class KVCache(NamedTuple):
    """A paged cache: keys and values (n_pages, Hkv, page_size, D), bf16, fp16 or float8_e4m3fn, and in 8
    bits the scale of every page and head, fp32 (n_pages, Hkv): a code stands for code * scale.
    Position j of a sequence is slot j % page_size of the page that its page table names at
    j // page_size. page_size is 16, 32, 64, 128 or 256; D a multiple of 16 up to 128."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None


def kv_cache(n_pages: int, Hkv: int, page_size: int, D: int, dtype: torch.dtype = torch.bfloat16,
             device=None) -> KVCache:
    """An empty cache of that many pages."""
    if dtype not in _CACHE_CODES:
        raise ValueError("a cache is bfloat16, float16 or float8_e4m3fn")
    if page_size not in (16, 32, 64, 128, 256) or D <= 0 or D % 16 or D > 128 or n_pages <= 0 or Hkv <= 0:
        raise ValueError("page_size must be 16, 32, 64, 128 or 256, D a multiple of 16 up to 128, n_pages and Hkv positive")
    dev = torch.device("cuda") if device is None else device
    k, v = (torch.zeros(n_pages, Hkv, page_size, D, dtype=torch.uint8 if dtype == torch.float8_e4m3fn else dtype, device=dev)
            for _ in range(2))
    if dtype != torch.float8_e4m3fn:
        return KVCache(k, v)
    scales = [torch.ones(n_pages, Hkv, dtype=torch.float32, device=dev) for _ in range(2)]
    return KVCache(k.view(dtype), v.view(dtype), *scales)


# Element types of a cache (sdpa_dtype).
_CACHE_CODES = {torch.bfloat16: 0, torch.float16: 2, torch.float8_e4m3fn: 3}


def _check_cache(cache, page_table, seq_kv_lens, B, io, ref):
    """Names what is wrong with a cache call's cache, table and lengths."""
    if not isinstance(cache, tuple) or len(cache) != 4:
        raise TypeError("cache must be a KVCache")
    k, v, ks, vs = cache
    for name, t in (("cache.k", k), ("cache.v", v)):
        if not isinstance(t, torch.Tensor) or t.dim() != 4 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous (n_pages, Hkv, page_size, D) CUDA tensor")
        if t.dtype not in (io, torch.float8_e4m3fn) or t.dtype != k.dtype:
            raise ValueError(f"the cache must be {io} or float8_e4m3fn, keys and values alike")
    if k.shape != v.shape:
        raise ValueError("cache.k and cache.v must have one shape")
    for name, t in (("cache.k_scale", ks), ("cache.v_scale", vs)):
        if (t is not None) != (k.dtype == torch.float8_e4m3fn):
            raise ValueError(f"{name} goes with a float8_e4m3fn cache, and only with one")
        if t is not None and (not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or not t.is_cuda
                              or not t.is_contiguous() or t.shape != k.shape[:2]):
            raise ValueError(f"{name} must be a contiguous fp32 CUDA tensor of shape (n_pages, Hkv)")
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be an int32 (B, max_pages) CUDA tensor")
    _check_int32("page_table", page_table, ((B, page_table.shape[1]),))
    _check_int32("seq_kv_lens", seq_kv_lens, ((B,),))
    _check_same_device(ref, k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, page_table=page_table, seq_kv_lens=seq_kv_lens)


def _cache_fits(cache, page_table, seq_kv_lens, B, io, dev) -> bool:
    """The same in one test: whether all is as it has to be."""
    try:
        k, v, ks, vs = cache
        shape, t, table = k.shape, k.dtype, page_table.shape
        good = (k.get_device() == dev == v.get_device() == page_table.get_device() == seq_kv_lens.get_device()
                and len(shape) == 4 and v.shape == shape and v.dtype is t and k.is_contiguous() and v.is_contiguous()
                and len(table) == 2 and table[0] == B and page_table.dtype is torch.int32 is seq_kv_lens.dtype
                and page_table.is_contiguous() and seq_kv_lens.shape == (B,) and seq_kv_lens.is_contiguous())
        if t is torch.float8_e4m3fn:
            return good and _is(ks, torch.float32, dev, shape[:2]) and _is(vs, torch.float32, dev, shape[:2])
        return good and t is io and ks is None and vs is None
    except (AttributeError, IndexError, TypeError, ValueError):
        return False


def _check_append_args(k, v, cache, seq_q_lens, q, inv_freq, positions, axes, q_out):
    """Names what is wrong with an append's arguments other than its cache, table and lengths."""
    io = _io_dtype(k)
    if k.dim() != 4:
        raise ValueError("k must be (B, H, S, D)")
    B, Hkv, S, D = k.shape
    if q is None and q_out is not None:
        raise ValueError("q_out without q")
    if q is not None and (not isinstance(q, torch.Tensor) or q.dim() != 4):
        raise ValueError("q must be a (B, H, S, D) tensor")
    for name, t, H in (("k", k, Hkv), ("v", v, Hkv), ("q", q, 0 if q is None else q.shape[1]),
                       ("q_out", q_out, 0 if q is None else q.shape[1])):
        if t is None and name in ("q", "q_out"):
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype != io or not t.is_cuda:
            raise ValueError(f"{name} must be a {io} CUDA tensor")
        if tuple(t.shape) != (B, H, S, D):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(B, H, S, D)}")
        if t.stride(3) != 1 and D > 1:
            raise ValueError(f"{name} must have contiguous columns (stride 1 in its last dimension)")
    if cache[0].shape[1] != Hkv or cache[0].shape[3] != D:
        raise ValueError(f"the cache holds {cache[0].shape[1]} heads of {cache[0].shape[3]} columns, k has {Hkv} of {D}")
    if seq_q_lens is not None:
        _check_int32("seq_q_lens", seq_q_lens, ((B,),))
    if inv_freq is not None:
        if not isinstance(inv_freq, torch.Tensor) or inv_freq.dtype != torch.float64 or not inv_freq.is_cuda \
                or not inv_freq.is_contiguous() or inv_freq.dim() != 1:
            raise ValueError("inv_freq must be a contiguous fp64 CUDA vector (rope_inv_freq)")
        rot = 2 * inv_freq.numel()
        if rot == 0 or rot > D:
            raise ValueError(f"inv_freq rotates {rot} columns of {D}")
        if axes is not None:
            _check_axes(axes, positions, rot // 2, B, S)
        elif positions is not None:
            _check_int32("positions", positions, ((S,), (B, S)))
    elif positions is not None or axes is not None:
        raise ValueError("positions and axes go with inv_freq")
    _check_same_device(k, _ref="k", v=v, q=q, q_out=q_out, seq_q_lens=seq_q_lens, inv_freq=inv_freq, positions=positions,
                       axes=axes, k_cache=cache[0])


def kv_append(k: torch.Tensor, v: torch.Tensor, cache: KVCache, page_table: torch.Tensor, seq_kv_lens: torch.Tensor, *,
              seq_q_lens: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
              inv_freq: Optional[torch.Tensor] = None, mult: float = 1.0, positions: Optional[torch.Tensor] = None,
              axes: Optional[torch.Tensor] = None, interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> Optional[torch.Tensor]:
    """Appends the rows of k and v (B,Hkv,S,D) to the cache, in place, and rotates keys and queries
    on the way (sdpa_kv_append in include/sdpa_bwd.h).

    ``page_table`` int32 (B,max_pages), ``seq_kv_lens`` int32 (B,): the lengths with the new rows,
    which sdpa_fwd_cached then takes as they are. Row t of the first n = ``seq_q_lens``[b] rows (default: all S)
    goes to position seq_kv_lens[b] - n + t. With ``inv_freq`` (rope_inv_freq) keys and queries turn as in rope_fwd, by
    the positions in the cache or by ``positions`` ((S,), (B,S), or with ``axes`` (n_axes,S), (n_axes,B,S)).
    bf16 or fp16, any strides of batch, head and position with contiguous columns. Returns the rotated
    ``q`` (B,Hq,S,D), contiguous unless ``q_out`` is given (it may be q itself); None without q.
    """
    lib = load()
    new = torch.empty if stream is None else functools.partial(_empty, stream=stream)
    io = _io_dtype(k)
    rot = good = Hq = 0
    try:
        B, Hkv, S, D = shape = k.shape
        dev, st, sv = k.get_device(), k.stride(), v.stride()
        sq = so = st
        good = (k.is_cuda and v.dtype is io and v.get_device() == dev and v.shape == shape and st[3] == 1 == sv[3]
                and (seq_q_lens is None or _is(seq_q_lens, torch.int32, dev, (B,))))
        if q is None:
            good = good and q_out is None
        else:
            Hq, sq = q.shape[1], q.stride()
            good = good and q.dtype is io and q.get_device() == dev and q.shape == (B, Hq, S, D) and sq[3] == 1
            if q_out is None:
                q_out, so = new((B, Hq, S, D), dtype=io, device=k.device), (Hq * S * D, S * D, D)
            else:
                so = q_out.stride()
                good = good and q_out.dtype is io and q_out.get_device() == dev and q_out.shape == q.shape and so[3] == 1
        if inv_freq is not None:
            rot = 2 * inv_freq.shape[0]
            good = good and 0 < rot <= D and _is(inv_freq, torch.float64, dev, (rot // 2,))
        if positions is not None or axes is not None:
            good = good and rot > 0
            if axes is None:
                good = good and (_is(positions, torch.int32, dev, (B, S)) or _is(positions, torch.int32, dev, (S,)))
            else:
                n = positions.shape[0]
                good = good and 1 <= n <= _MAX_AXES and _is(axes, torch.int32, dev, (rot // 2,)) \
                    and (_is(positions, torch.int32, dev, (n, B, S)) or _is(positions, torch.int32, dev, (n, S)))
    except (AttributeError, IndexError, TypeError, ValueError):  # not tensors, or of other dimensions
        good = False
    if not good or not _cache_fits(cache, page_table, seq_kv_lens, B, io, dev):
        if k.dim() != 4:
            raise ValueError("k must be (B, H, S, D)")
        _check_cache(cache, page_table, seq_kv_lens, k.shape[0], io, k)
        _check_append_args(k, v, cache, seq_q_lens, q, inv_freq, positions, axes, q_out)
    kc, vc, ks, vs = cache
    n_pages, heads, P, columns = kc.shape
    if heads != Hkv or columns != D:
        raise ValueError(f"the cache holds {heads} heads of {columns} columns, k has {Hkv} of {D}")
    _check_launch_device(k)
    rc = lib.sdpa_kv_append(
        _IO_CODES[io], _CACHE_CODES[kc.dtype], _addr(q), _addr(q_out), k.data_ptr(), v.data_ptr(), kc.data_ptr(),
        vc.data_ptr(), _addr(ks), _addr(vs), page_table.data_ptr(), seq_kv_lens.data_ptr(), _addr(seq_q_lens), B, Hq,
        Hkv, S, D, n_pages, P, page_table.shape[1],
        _strides(sq[0], sq[1], sq[2], so[0], so[1], so[2], st[0], st[1], st[2], sv[0], sv[1], sv[2]),
        _addr(inv_freq), rot, float(mult), _addr(positions),
        0 if positions is None else positions.dim() - (1 if axes is None else 2),
        1 if axes is None else positions.shape[0], _addr(axes), bool(interleaved), _stream_handle(stream))
    if rc != 0:
        raise SdpaError(rc, "sdpa_kv_append")
    return q_out


def kv_gather(cache: KVCache, page_table: torch.Tensor, seq_kv_lens: torch.Tensor, S: Optional[int] = None, *,
              dtype: Optional[torch.dtype] = None, k_out: Optional[torch.Tensor] = None,
              v_out: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The cached keys and values of the first ``S`` positions (default: all that the page table has) of
    every sequence as contiguous (B,Hkv,S,D) tensors, zeros past the lengths (sdpa_kv_gather), for
    sdpa_fwd, say. ``dtype`` is bf16 or fp16; a 16-bit cache has its own (the default), an 8-bit one bf16."""
    lib = load()
    kc = cache[0] if isinstance(cache, tuple) and len(cache) == 4 else None
    if not isinstance(kc, torch.Tensor) or kc.dim() != 4 or not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("cache must be a KVCache and page_table an int32 (B, max_pages) CUDA tensor")
    io = dtype if dtype is not None else torch.bfloat16 if kc.dtype == torch.float8_e4m3fn else kc.dtype
    if io not in _IO_CODES:
        raise ValueError("dtype must be bfloat16 or float16")
    B, dev = page_table.shape[0], kc.get_device()
    if not _cache_fits(cache, page_table, seq_kv_lens, B, io, dev):
        _check_cache(cache, page_table, seq_kv_lens, B, io, kc)
    n_pages, Hkv, P, D = kc.shape
    most = page_table.shape[1] * P
    S = most if S is None else operator.index(S)
    if not 0 <= S <= most:
        raise ValueError(f"S must be from 0 to {most}, what the page table has")
    new = torch.empty if stream is None else functools.partial(_empty, stream=stream)
    shape, device = (B, Hkv, S, D), kc.device
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t is not None and not _is(t, io, dev, shape):
            _check_bf16(name, t, shape, io)
            _check_same_device(kc, _ref="the cache", **{name: t})
    k_out = new(shape, dtype=io, device=device) if k_out is None else k_out
    v_out = new(shape, dtype=io, device=device) if v_out is None else v_out
    _check_launch_device(kc)
    rc = lib.sdpa_kv_gather(_IO_CODES[io], _CACHE_CODES[kc.dtype], kc.data_ptr(), cache[1].data_ptr(), _addr(cache[2]),
                            _addr(cache[3]), page_table.data_ptr(), seq_kv_lens.data_ptr(), k_out.data_ptr(),
                            v_out.data_ptr(), B, Hkv, S, D, n_pages, P, page_table.shape[1], _stream_handle(stream))
    if rc != 0:
        raise SdpaError(rc, "sdpa_kv_gather")
    return k_out, v_out


def sdpa_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, scale: Optional[float] = None,
             causal: bool = False, bottom_right: bool = False, window_left: int = -1,
             window_right: int = -1, seq_q_lens: Optional[torch.Tensor] = None,
             seq_kv_lens: Optional[torch.Tensor] = None, sink: Optional[torch.Tensor] = None,
             bias: Optional[torch.Tensor] = None,
             o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
             softcap: float = 0.0, alibi_slopes: Optional[torch.Tensor] = None,
             mask_plan: Optional["MaskPlan"] = None,
             stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """O (bf16, (B,Hq,Sq,Dv)) and natural-log LSE (fp32, (B,Hq,Sq)) of the masked
    softmax attention (see include/sdpa_bwd.h); the inputs of sdpa_bwd. ``bias``
    ((1|B, Hq, Sq, Skv) bf16, fp16 or fp32 CUDA, contiguous) is added to the scaled
    scores (sdpa_fwd_bias). ``softcap`` (> 0) caps the scaled scores at
    softcap * tanh(. / softcap); ``alibi_slopes`` (fp32 (Hq,) CUDA) subtracts slope[h] *
    |q + diag - k|; ``mask_plan`` (see mask_plan()) limits each row to its range of
    keys, for document and prefix masks (sdpa_fwd_scored; not together with ``bias``)."""
    lib = load()
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be (B, H, S, D)")
    io = _io_dtype(q)
    B, Hq, Sq, Dqk = q.shape
    Hkv, Skv = k.shape[1], k.shape[2]
    Dv = v.shape[3]
    fresh = o is None and lse is None  # (outputs made here need no checks)
    new = torch.empty if stream is None else functools.partial(_empty, stream=stream)
    o = new((B, Hq, Sq, Dv), dtype=io, device=q.device) if o is None else o
    lse = new((B, Hq, Sq), dtype=torch.float32, device=q.device) if lse is None else lse
    dev = q.get_device()
    if not (q.is_cuda and _is(q, io, dev, (B, Hq, Sq, Dqk)) and _is(k, io, dev, (B, Hkv, Skv, Dqk))
            and _is(v, io, dev, (B, Hkv, Skv, Dv))
            and (fresh or _is(o, io, dev, (B, Hq, Sq, Dv)) and _optional(lse, torch.float32, dev, B * Hq * Sq))
            and (seq_q_lens is None or _optional(seq_q_lens, torch.int32, dev, B))
            and (seq_kv_lens is None or _optional(seq_kv_lens, torch.int32, dev, B))
            and (sink is None or _optional(sink, torch.float32, dev, Hq)) and bias is None):
        _check_bf16("q", q, (B, Hq, Sq, Dqk), io)
        _check_bf16("k", k, (B, Hkv, Skv, Dqk), io)
        _check_bf16("v", v, (B, Hkv, Skv, Dv), io)
        _check_lens(B, seq_q_lens, seq_kv_lens)
        if sink is not None and (sink.dtype != torch.float32 or not sink.is_cuda
                                 or not sink.is_contiguous() or sink.numel() != Hq):
            raise ValueError("sink must be a contiguous fp32 CUDA tensor of Hq elements")
        _check_bf16("o", o, (B, Hq, Sq, Dv), io)
        _check_lse(lse, B, Hq, Sq)
        _check_same_device(q, k=k, v=v, o=o, lse=lse, seq_q_lens=seq_q_lens, seq_kv_lens=seq_kv_lens,
                           sink=sink, bias=bias)
    scored = _check_score_mods(q, B, Hq, Sq, Skv, softcap, alibi_slopes, mask_plan, bias, window_left, window_right)
    _check_launch_device(q)
    sc = 0.0 if scale is None else float(scale)
    if scored:
        rc = lib.sdpa_fwd_scored(_IO_CODES[io], q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                 B, Hq, Hkv, Sq, Skv, Dqk, Dv, sc, int(causal), int(bottom_right), int(window_left),
                                 int(window_right), _addr(seq_q_lens), _addr(seq_kv_lens), _addr(sink),
                                 float(softcap), _addr(alibi_slopes),
                                 None if mask_plan is None else mask_plan._on(stream), _stream_handle(stream))
        if rc != 0:
            raise SdpaError(rc, "sdpa_fwd_scored")
        return o, lse
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Sq, Skv, Dqk, Dv, sc,
            int(causal), int(bottom_right), int(window_left), int(window_right),
            _ptr(seq_q_lens), _ptr(seq_kv_lens), _ptr(sink))
    if io == torch.float16:
        bias_dtype = _check_bias(bias, B, Hq, Sq, Skv) if bias is not None else 0
        rc = lib.sdpa_fwd_typed(_IO_CODES[io], *args, _ptr(bias), bias_dtype,
                                0 if bias is None else int(bias.shape[0]), _stream_handle(stream))
    elif bias is None:
        rc = lib.sdpa_fwd(*args, _stream_handle(stream))
    else:
        dt = _check_bias(bias, B, Hq, Sq, Skv)
        rc = lib.sdpa_fwd_bias(*args, _ptr(bias), dt, int(bias.shape[0]), _stream_handle(stream))
    if rc != 0:
        raise SdpaError(rc, "sdpa_fwd_bias" if bias is not None else "sdpa_fwd")
    return o, lse


def cached_workspace_size(B, Hq, Hkv, Sq, D, cache_dtype, page_size, max_pages) -> int:
    """Workspace bytes of sdpa_fwd_cached for these sizes (cache_dtype: the cache's torch dtype)."""
    return int(load().sdpa_fwd_cached_workspace_size(B, Hq, Hkv, Sq, D, _CACHE_CODES[cache_dtype], page_size, max_pages))


@functools.lru_cache(maxsize=4096)
def _cached_workspace(lib, *sizes) -> int:
    return int(lib.sdpa_fwd_cached_workspace_size(*sizes))


def sdpa_fwd_cached(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor, seq_kv_lens: torch.Tensor, *,
                    scale: Optional[float] = None, causal: bool = True, window_left: int = -1, first_keys: int = 0,
                    seq_q_lens: Optional[torch.Tensor] = None, sink: Optional[torch.Tensor] = None,
                    softcap: float = 0.0, alibi_slopes: Optional[torch.Tensor] = None,
                    o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """O (as q) and natural-log LSE (fp32 (B,Hq,Sq)) of queries q (B,Hq,Sq,D) over a paged cache (sdpa_fwd_cached in
    include/sdpa_bwd.h): one token, a few, or a chunk of a prompt.

    ``page_table`` int32 (B,max_pages), ``seq_kv_lens`` int32 (B,): what kv_append took, so the queries are the last
    positions: query i of the first n = ``seq_q_lens``[b] (default Sq) stands at seq_kv_lens[b] - n + i. It sees the
    keys up to its own (``causal``), from ``window_left`` before it on, and under a window the ``first_keys`` first
    ones too. ``sink``, ``softcap`` and ``alibi_slopes`` as in sdpa_fwd.
    """
    lib = load()
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be (B, H, S, D)")
    io = _io_dtype(q)
    B, Hq, Sq, D = shape = q.shape
    dev, fresh = q.get_device(), o is None and lse is None  # (outputs made here need no checks)
    if not (q.is_cuda and q.is_contiguous() and _cache_fits(cache, page_table, seq_kv_lens, B, io, dev)
            and (fresh or _is(o, io, dev, shape) and _optional(lse, torch.float32, dev, B * Hq * Sq))
            and (seq_q_lens is None or _optional(seq_q_lens, torch.int32, dev, B))
            and (sink is None or _optional(sink, torch.float32, dev, Hq)) and workspace is None):
        _check_cache(cache, page_table, seq_kv_lens, B, io, q)
        _check_bf16("q", q, shape, io)
        _check_lens(B, seq_q_lens, None)
        if sink is not None and (sink.dtype != torch.float32 or not sink.is_cuda
                                 or not sink.is_contiguous() or sink.numel() != Hq):
            raise ValueError("sink must be a contiguous fp32 CUDA tensor of Hq elements")
        if o is not None:
            _check_bf16("o", o, shape, io)
        if lse is not None:
            _check_lse(lse, B, Hq, Sq)
        _check_workspace(workspace)
        _check_same_device(q, o=o, lse=lse, seq_q_lens=seq_q_lens, sink=sink, workspace=workspace)
    kc, vc, ks, vs = cache
    n_pages, Hkv, P, columns = kc.shape
    max_pages, cache_code = page_table.shape[1], _CACHE_CODES[kc.dtype]
    if columns != D:
        raise ValueError(f"the cache holds {columns} columns, q has {D}")
    if softcap != 0.0 or alibi_slopes is not None:
        _check_score_mods(q, B, Hq, Sq, 0, softcap, alibi_slopes, None, None, -1, -1)
    window_left, first_keys = operator.index(window_left), operator.index(first_keys)
    if not (-_INT32 <= window_left < _INT32 and 0 <= first_keys < _INT32):
        raise ValueError("window_left and first_keys are 32-bit numbers of keys, first_keys not negative")
    _check_launch_device(q)
    o = _empty_like(q, stream) if o is None else o
    if lse is None:
        lse = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device) if stream is None \
            else _empty((B, Hq, Sq), torch.float32, q.device, stream)
    if workspace is not None:
        ws_bytes = _check_workspace(workspace)
    else:
        ws_bytes = _cached_workspace(lib, B, Hq, Hkv, Sq, D, cache_code, P, max_pages)
        if ws_bytes and stream is None:  # (a call on a stream given to it leaves this to the library, as sdpa_bwd)
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    rc = lib.sdpa_fwd_cached(
        _IO_CODES[io], cache_code, q.data_ptr(), kc.data_ptr(), vc.data_ptr(), _addr(ks), _addr(vs),
        page_table.data_ptr(), seq_kv_lens.data_ptr(), _addr(seq_q_lens), o.data_ptr(), lse.data_ptr(), B, Hq, Hkv, Sq, D,
        n_pages, P, max_pages, 0.0 if scale is None else float(scale), int(causal), window_left, first_keys,
        _addr(sink), float(softcap), _addr(alibi_slopes), _addr(workspace), ws_bytes, _stream_handle(stream))
    if rc != 0:
        raise SdpaError(rc, "sdpa_fwd_cached")
    return o, lse


def nvfp4_fake_quant(x: torch.Tensor, out: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """NVFP4 fake quantization of a contiguous bf16 CUDA tensor in blocks of 16
    consecutive values (sdpa_nvfp4_fake_quant); numel must be a multiple of 16."""
    lib = load()
    if not isinstance(x, torch.Tensor) or x.dtype != torch.bfloat16 or not x.is_cuda \
            or not x.is_contiguous():
        raise ValueError("x must be a contiguous bf16 CUDA tensor")
    out = _empty_like(x, stream) if out is None else out
    _check_bf16("out", out, x.shape)
    _check_same_device(x, out=out)
    _check_launch_device(x)
    rc = lib.sdpa_nvfp4_fake_quant(_ptr(x), _ptr(out), x.numel(), _stream_handle(stream))
    if rc != 0:
        raise SdpaError(rc, "sdpa_nvfp4_fake_quant")
    return out


def sdpa_fwd_nvfp4_qat(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, **kw):
    """The QAT forward statistics the QAT backward takes: sdpa_fwd() of the
    fake-quantized q, k, v, i.e. (O_hp, LSE) with O_hp = softmax(scale q^ k^^T) v^."""
    stream = kw.get("stream")
    return sdpa_fwd(nvfp4_fake_quant(q, stream=stream), nvfp4_fake_quant(k, stream=stream),
                    nvfp4_fake_quant(v, stream=stream), **kw)


def sdpa_bwd_nvfp4_qat(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o_hp: torch.Tensor,
                       do: torch.Tensor, lse: torch.Tensor, *, scale: Optional[float] = None,
                       causal: bool = False, bottom_right: bool = False, window_left: int = -1,
                       window_right: int = -1, seq_q_lens: Optional[torch.Tensor] = None,
                       seq_kv_lens: Optional[torch.Tensor] = None, dq: Optional[torch.Tensor] = None,
                       dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None):
    """dQ, dK, dV of NVFP4 QAT attention (sdpa_bwd_nvfp4_qat): q, k, v unquantized,
    o_hp / lse from sdpa_fwd_nvfp4_qat. D = 128."""
    lib = load()
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be (B, H, S, D) tensors")
    B, Hq, Sq, Dqk = q.shape
    Hkv, Skv, Dv = k.shape[1], k.shape[2], v.shape[3]
    for name, t, shape in (("q", q, (B, Hq, Sq, Dqk)), ("k", k, (B, Hkv, Skv, Dqk)),
                           ("v", v, (B, Hkv, Skv, Dv)), ("o_hp", o_hp, (B, Hq, Sq, Dv)),
                           ("do", do, (B, Hq, Sq, Dv))):
        _check_bf16(name, t, shape)
    _check_lse(lse, B, Hq, Sq)
    _check_lens(B, seq_q_lens, seq_kv_lens)
    dq = _empty_like(q, stream) if dq is None else dq
    dk = _empty_like(k, stream) if dk is None else dk
    dv = _empty_like(v, stream) if dv is None else dv
    _check_bf16("dq", dq, q.shape)
    _check_bf16("dk", dk, k.shape)
    _check_bf16("dv", dv, v.shape)
    ws_bytes = _check_workspace(workspace)
    _check_same_device(q, k=k, v=v, o_hp=o_hp, do=do, lse=lse, seq_q_lens=seq_q_lens,
                       seq_kv_lens=seq_kv_lens, dq=dq, dk=dk, dv=dv, workspace=workspace)
    _check_launch_device(q)
    rc = lib.sdpa_bwd_nvfp4_qat(_ptr(q), _ptr(k), _ptr(v), _ptr(o_hp), _ptr(do), _ptr(lse), _ptr(dq),
                                _ptr(dk), _ptr(dv), B, Hq, Hkv, Sq, Skv, Dqk, Dv,
                                0.0 if scale is None else float(scale), int(causal),
                                int(bottom_right), int(window_left), int(window_right),
                                _ptr(seq_q_lens), _ptr(seq_kv_lens), _ptr(workspace), ws_bytes,
                                _stream_handle(stream))
    if rc != 0:
        raise SdpaError(rc, "sdpa_bwd_nvfp4_qat")
    return dq, dk, dv


def nvfp4_qat_workspace_size(B, Hq, Hkv, Sq, Skv, Dqk, Dv) -> int:
    return int(load().sdpa_bwd_nvfp4_qat_workspace_size(B, Hq, Hkv, Sq, Skv, Dqk, Dv))


def debug_relay(wait_limit_ns: int = 0, turn_skew: int = 0) -> None:
    """Sets the ordered relay's wait limit (0: the 4 s default) and turn skew (0:
    normal use) for later calls; see sdpa_bwd_debug_relay in the header."""
    load().sdpa_bwd_debug_relay(int(wait_limit_ns), int(turn_skew))


def check_device_status(stream: Optional[torch.cuda.Stream] = None) -> None:
    """Synchronizes the stream and raises if a kernel reported a timed-out wait."""
    rc = load().sdpa_bwd_check_device_status(_stream_handle(stream))
    if rc != 0:
        raise SdpaError(rc, "device status")


def profile_enable(on: bool = True) -> None:
    load().sdpa_bwd_profile_enable(int(on))


def profile_read():
    """{kernel name: (total ms, launches)} accumulated since profile_enable()."""
    ms = (ctypes.c_float * len(KERNEL_NAMES))()
    n = (ctypes.c_int * len(KERNEL_NAMES))()
    load().sdpa_bwd_profile_read(ms, n, len(KERNEL_NAMES))
    return {name: (float(ms[i]), int(n[i])) for i, name in enumerate(KERNEL_NAMES)}
