"""B200 (sm_100a) Kimi Delta Attention prefill -- Python binding of ``libkda.so``.

This module only marshals arguments: it checks torch tensors, allocates
outputs with torch (device memory), and calls the C ABI declared in
``include/kda.h`` on the current CUDA stream. Every step of the computation
runs in the library's CUDA kernels; there is no fallback. Importing the
module fails loudly if ``libkda.so`` has not been built.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional, Tuple

import torch

__all__ = ["kda_fwd", "kda_fwd_fused", "kda_decode", "kda_bwd", "kda_conv_fwd", "kda_conv_decode", "kda_conv_bwd",
           "kda_ssm_fwd", "kda_ssm_decode", "kda_ssm_bwd", "library_path", "wait_timeouts", "device_status", "set_slice_columns", "set_path",
           "set_time_split", "set_schedule", "describe", "KDAError", "HEAD_DIM"]

HEAD_DIM = 128
_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libkda.so")

if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"{_LIB_PATH} is missing: build the CUDA library first "
        "(python kimi_delta_attention_26_b200/build.py or __graft_entry__.build())")

_lib = ctypes.CDLL(_LIB_PATH)

KDA_BF16, KDA_F32, KDA_I32, KDA_F16 = 1, 2, 3, 4
_DTYPE = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32, torch.int32: KDA_I32, torch.float16: KDA_F16}


class TensorDesc(ctypes.Structure):
    """``kda_tensor_t``: data pointer, ndim, dtype, shape[4], stride[4] (elements)."""
    _fields_ = [("data", ctypes.c_void_p), ("ndim", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


def describe(t: Optional[torch.Tensor]):
    """A ``kda_tensor_t`` for a torch tensor (None -> NULL)."""
    if t is None:
        return None
    if t.dim() > 4:
        raise ValueError("at most 4 dimensions")
    d = TensorDesc()
    d.data = t.data_ptr() if t.numel() else None
    d.ndim = t.dim()
    d.dtype = _DTYPE.get(t.dtype, 0)
    for i, (n, st) in enumerate(zip(t.shape, t.stride())):
        d.shape[i] = n
        d.stride[i] = st
    return ctypes.byref(d), d  # keep d alive with the reference


_P = ctypes.c_void_p
_T = ctypes.POINTER(TensorDesc)
_FWD_ARGS = [_T, _T, _T, _T, _T, ctypes.c_float, _P, ctypes.c_int32, _T, _T, _T, _P]
_lib.kda_fwd.argtypes = _FWD_ARGS
_lib.kda_fwd.restype = ctypes.c_int
_lib.kda_fwd_noalloc.argtypes = _FWD_ARGS
_lib.kda_fwd_noalloc.restype = ctypes.c_int
_lib.kda_status_string.argtypes = [ctypes.c_int]
_lib.kda_status_string.restype = ctypes.c_char_p
_lib.kda_last_cuda_error.argtypes = []
_lib.kda_last_cuda_error.restype = ctypes.c_char_p
_lib.kda_abi_version.argtypes = []
_lib.kda_abi_version.restype = ctypes.c_int32
_lib.kda_wait_timeouts.argtypes = [ctypes.POINTER(ctypes.c_uint32), ctypes.c_int32]
_lib.kda_wait_timeouts.restype = ctypes.c_int
_lib.kda_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint32), ctypes.c_int32]
_lib.kda_device_status.restype = ctypes.c_int
_lib.kda_set_slice_columns.argtypes = [ctypes.c_int32]
_lib.kda_set_slice_columns.restype = ctypes.c_int
_lib.kda_set_path.argtypes = [ctypes.c_int32]
_lib.kda_set_path.restype = ctypes.c_int
_lib.kda_set_time_split.argtypes = [ctypes.c_int32]
_lib.kda_set_time_split.restype = ctypes.c_int
_lib.kda_set_schedule.argtypes = [ctypes.c_int32, ctypes.c_int32]
_lib.kda_set_schedule.restype = ctypes.c_int
_lib.kda_fwd_fused.argtypes = [_T, _T, _T, _T, _T, ctypes.c_float, ctypes.c_float, _P, ctypes.c_int32, _T, _T, _T, _P]
_lib.kda_fwd_fused.restype = ctypes.c_int
_lib.kda_bwd.argtypes = [_T, _T, _T, _T, _T, ctypes.c_float, _P, ctypes.c_int32, _T, _T, _T, _T, _T, _T, _T, _T, _T, _P]
_lib.kda_bwd.restype = ctypes.c_int
_lib.kda_decode.argtypes = [_T, _T, _T, _T, _T, ctypes.c_float, _T, _P, _T, _P]
_lib.kda_decode.restype = ctypes.c_int
# The convolution and the scan take their descriptors packed (bytes), see _pack.
_I = ctypes.c_int32
_lib.kda_conv_fwd.argtypes = [_P, _P, _P, _I, _P, _I, _P, _P, _P, _P]
_lib.kda_conv_decode.argtypes = [_P, _P, _P, _I, _P, _P, _P, _P]
_lib.kda_conv_bwd.argtypes = [_P, _P, _P, _I, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P]
_lib.kda_ssm_fwd.argtypes = [_P] * 8 + [_I, _P, _I] + [_P] * 4
_lib.kda_ssm_decode.argtypes = [_P] * 8 + [_I] + [_P] * 4
_lib.kda_ssm_bwd.argtypes = [_P] * 8 + [_I, _P, _I] + [_P] * 13
for _f in ("kda_conv_fwd", "kda_conv_decode", "kda_conv_bwd", "kda_ssm_fwd", "kda_ssm_decode", "kda_ssm_bwd"):
    getattr(_lib, _f).restype = ctypes.c_int


class KDAError(RuntimeError):
    def __init__(self, code: int):
        msg = _lib.kda_status_string(code).decode()
        cuda = _lib.kda_last_cuda_error().decode()
        super().__init__(f"KDA call failed ({code}): {msg}" + (f" [{cuda}]" if cuda else ""))
        self.code = code


def library_path() -> str:
    return _LIB_PATH


def wait_timeouts(reset: bool = True) -> int:
    """Bounded in-kernel waits that ran out of budget on the current device
    since the last reset (0 for a healthy run); synchronises with the device."""
    n = ctypes.c_uint32(0)
    rc = _lib.kda_wait_timeouts(ctypes.byref(n), 1 if reset else 0)
    if rc != 0:
        raise KDAError(rc)
    return int(n.value)


def set_slice_columns(columns: int) -> None:
    """Value columns per CTA of the 16-token path for later calls: 0 chooses per
    call (default), 16 or 32 forces that variant. Process-wide."""
    rc = _lib.kda_set_slice_columns(int(columns))
    if rc != 0:
        raise KDAError(rc)


def set_path(path: int) -> None:
    """Kernel for later calls: 16 (16-token chunks on mma.sync), 64 (64-token
    chunks on tcgen05) or 0 (the library's default). Process-wide."""
    rc = _lib.kda_set_path(int(path))
    if rc != 0:
        raise KDAError(rc)


def set_time_split(mode: int) -> None:
    """Time-split prefill of one long sequence (16-token path), and the time split
    of the selective scan and its gradients: 0 automatic (default), 1 never, 2
    whenever possible. Process-wide."""
    rc = _lib.kda_set_time_split(int(mode))
    if rc != 0:
        raise KDAError(rc)


def set_schedule(mode: int, clusters: int = 0) -> None:
    """Mapping of (sequence, head) pairs onto clusters (16-token path): 0
    automatic (default), 1 one cluster per pair, 2 persistent clusters taking
    the pairs round robin (at most `clusters` of them when > 0). Process-wide;
    results are bitwise the same."""
    rc = _lib.kda_set_schedule(int(mode), int(clusters))
    if rc != 0:
        raise KDAError(rc)


def device_status(reset: bool = True) -> int:
    """The device status word (bit 0: a bad cu_seqlens was seen, bit 1: a
    bounded in-kernel wait ran out, bit 2: a decode call met a state index out
    of range); synchronises with the device."""
    n = ctypes.c_uint32(0)
    rc = _lib.kda_device_status(ctypes.byref(n), 1 if reset else 0)
    if rc not in (0, 9):
        raise KDAError(rc)
    return int(n.value)


def _check(t: torch.Tensor, name: str, dtype: torch.dtype, shape: Tuple[int, ...], device,
           contiguous: bool = False) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def kda_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
            scale: Optional[float] = None, cu_seqlens: Optional[torch.Tensor] = None,
            initial_state: Optional[torch.Tensor] = None, output_final_state: bool = True,
            out: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
            stream: Optional[torch.cuda.Stream] = None, noalloc: bool = False,
            fused_lower_bound: Optional[float] = None):
    """Chunked KDA forward on packed sequences (see ``include/kda.h``).

    q, k, v: bf16 [T, H, 128]; g: fp32 [T, H, 128] (log decay, in [-5, 0]);
    beta: fp32 [T, H]; cu_seqlens: int32 [N + 1] on the device (None: one
    sequence); initial_state: fp32 [N, H, 128, 128] or None.
    Returns ``(out, final_state)``; ``final_state`` is None unless requested.
    With ``fused_lower_bound`` set, calls ``kda_fwd_fused``: q and k are raw
    projections, g and beta are logits (see ``kda_fwd_fused``).
    """
    if q.dim() != 3:
        raise ValueError("q must be [T, H, 128]")
    T, H, d = q.shape
    if d != HEAD_DIM:
        raise ValueError(f"head dimension must be {HEAD_DIM}")
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("kda_fwd runs on CUDA tensors only")
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    _check(q, "q", torch.bfloat16, (T, H, d), dev)
    _check(k, "k", torch.bfloat16, (T, H, d), dev)
    _check(v, "v", torch.bfloat16, (T, H, d), dev)
    _check(g, "g", torch.float32, (T, H, d), dev)
    _check(beta, "beta", torch.float32, (T, H), dev)
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), dev, contiguous=True)
    if initial_state is not None:
        _check(initial_state, "initial_state", torch.float32, (N, H, d, d), dev, contiguous=True)
    if out is None:
        out = torch.empty((T, H, d), dtype=torch.bfloat16, device=dev)
    _check(out, "out", torch.bfloat16, (T, H, d), dev)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, H, d, d), dtype=torch.float32, device=dev)
    if final_state is not None:
        _check(final_state, "final_state", torch.float32, (N, H, d, d), dev, contiguous=True)
    if scale is None:
        scale = d ** -0.5
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    descs = [describe(t) for t in (q, k, v, g, beta, initial_state, out, final_state)]
    ref = [None if d is None else d[0] for d in descs]
    with torch.cuda.device(dev):
        if fused_lower_bound is not None:
            if noalloc:
                raise ValueError("the fused preprocessing has no allocation-free entry point")
            rc = _lib.kda_fwd_fused(ref[0], ref[1], ref[2], ref[3], ref[4], ctypes.c_float(scale),
                                    ctypes.c_float(fused_lower_bound), _ptr(cu_seqlens), N, ref[5], ref[6], ref[7],
                                    ctypes.c_void_p(stream.cuda_stream))
        else:
            fn = _lib.kda_fwd_noalloc if noalloc else _lib.kda_fwd
            rc = fn(ref[0], ref[1], ref[2], ref[3], ref[4], ctypes.c_float(scale), _ptr(cu_seqlens), N,
                    ref[5], ref[6], ref[7], ctypes.c_void_p(stream.cuda_stream))
    if rc != 0:
        raise KDAError(rc)
    return out, final_state


def kda_fwd_fused(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g_logit: torch.Tensor,
                  beta_logit: torch.Tensor, scale: Optional[float] = None, lower_bound: float = -5.0, **kw):
    """``kda_fwd`` with the gate preprocessing fused (see ``include/kda.h``):
    q, k raw bf16 projections (L2-normalised in the kernel), g_logit fp32
    gate logits (decay max(log sigmoid(x), lower_bound)), beta_logit fp32
    (write strength sigmoid(b)). Other arguments as for ``kda_fwd``."""
    return kda_fwd(q, k, v, g_logit, beta_logit, scale, fused_lower_bound=float(lower_bound), **kw)


def kda_decode(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
               state: torch.Tensor, scale: Optional[float] = None, state_indices: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One decode step for B requests (see ``include/kda.h``): advances each
    request's state by its token, in place, and returns the outputs.

    q, k, v: bf16 [B, H, 128]; g: fp32 [B, H, 128] (log decay, in [-5, 0]);
    beta: fp32 [B, H]; state: fp32 [P, H, 128, 128], updated in place;
    state_indices: int32 [B] on the device (distinct slots), or None for slot b.
    """
    if q.dim() != 3:
        raise ValueError("q must be [B, H, 128]")
    B, H, d = q.shape
    if d != HEAD_DIM:
        raise ValueError(f"head dimension must be {HEAD_DIM}")
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("kda_decode runs on CUDA tensors only")
    _check(q, "q", torch.bfloat16, (B, H, d), dev)
    _check(k, "k", torch.bfloat16, (B, H, d), dev)
    _check(v, "v", torch.bfloat16, (B, H, d), dev)
    _check(g, "g", torch.float32, (B, H, d), dev)
    _check(beta, "beta", torch.float32, (B, H), dev)
    if state.dim() != 4:
        raise ValueError("state must be [P, H, 128, 128]")
    _check(state, "state", torch.float32, (state.shape[0], H, d, d), dev, contiguous=True)
    if state_indices is not None:
        _check(state_indices, "state_indices", torch.int32, (B,), dev, contiguous=True)
    if out is None:
        out = torch.empty((B, H, d), dtype=torch.bfloat16, device=dev)
    _check(out, "out", torch.bfloat16, (B, H, d), dev)
    if scale is None:
        scale = d ** -0.5
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    descs = [describe(t) for t in (q, k, v, g, beta, state, out)]
    ref = [x[0] for x in descs]
    with torch.cuda.device(dev):
        rc = _lib.kda_decode(ref[0], ref[1], ref[2], ref[3], ref[4], ctypes.c_float(scale), ref[5],
                             _ptr(state_indices), ref[6], ctypes.c_void_p(stream.cuda_stream))
    if rc != 0:
        raise KDAError(rc)
    return out


def kda_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
            dout: torch.Tensor, scale: Optional[float] = None, cu_seqlens: Optional[torch.Tensor] = None,
            initial_state: Optional[torch.Tensor] = None, dfinal_state: Optional[torch.Tensor] = None,
            stream: Optional[torch.cuda.Stream] = None):
    """Gradients of the prefill (see ``include/kda.h``): returns a dict of fp32
    tensors ``dq, dk, dv, dg`` [T, H, 128], ``dbeta`` [T, H] and
    ``dinitial_state`` [N, H, 128, 128], for the output gradient ``dout``
    (bf16 [T, H, 128]) and the final-state gradient ``dfinal_state``
    (fp32 [N, H, 128, 128] or None)."""
    if q.dim() != 3:
        raise ValueError("q must be [T, H, 128]")
    T, H, d = q.shape
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("kda_bwd runs on CUDA tensors only")
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    _check(dout, "dout", torch.bfloat16, (T, H, d), dev)
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), dev, contiguous=True)
    if initial_state is not None:
        _check(initial_state, "initial_state", torch.float32, (N, H, d, d), dev, contiguous=True)
    if dfinal_state is not None:
        _check(dfinal_state, "dfinal_state", torch.float32, (N, H, d, d), dev, contiguous=True)
    grads = {n: torch.empty((T, H, d), dtype=torch.float32, device=dev) for n in ("dq", "dk", "dv", "dg")}
    grads["dbeta"] = torch.empty((T, H), dtype=torch.float32, device=dev)
    grads["dinitial_state"] = torch.empty((N, H, d, d), dtype=torch.float32, device=dev)
    if scale is None:
        scale = d ** -0.5
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    ts = (q, k, v, g, beta, initial_state, dout, dfinal_state, grads["dq"], grads["dk"], grads["dv"], grads["dg"],
          grads["dbeta"], grads["dinitial_state"])
    descs = [describe(t) for t in ts]
    r = [None if x is None else x[0] for x in descs]
    with torch.cuda.device(dev):
        rc = _lib.kda_bwd(r[0], r[1], r[2], r[3], r[4], ctypes.c_float(scale), _ptr(cu_seqlens), N, r[5], r[6], r[7],
                          r[8], r[9], r[10], r[11], r[12], r[13], ctypes.c_void_p(stream.cuda_stream))
    if rc != 0:
        raise KDAError(rc)
    return grads


# ------------------------------------------------- short convolution and scan
_ACTIVATION = {None: 0, "silu": 1}
_desc = struct.Struct("@Pii4q4q").pack


def _pack(t: Optional[torch.Tensor], name: str, index: int):
    """``kda_tensor_t`` of a tensor on CUDA device `index`, as bytes (None -> NULL)."""
    if t is None:
        return None
    try:
        on, n, code = t.get_device(), t.dim(), _DTYPE.get(t.dtype, 0)
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if on != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if n == 2:
        (a, b), (p, q) = t.shape, t.stride()
        return _desc(t.data_ptr(), 2, code, a, b, 0, 0, p, q, 0, 0)
    if n == 3:
        (a, b, c), (p, q, r) = t.shape, t.stride()
        return _desc(t.data_ptr(), 3, code, a, b, c, 0, p, q, r, 0)
    if n > 4:
        raise ValueError(f"{name} has more than 4 dimensions")
    pad = (0,) * (4 - n)
    return _desc(t.data_ptr(), n, code, *t.shape, *pad, *t.stride(), *pad)


def _dims(t: torch.Tensor, name: str, dims: int) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions")


def _device_of(t: torch.Tensor, name: str, dims: int, fn: str) -> int:
    _dims(t, name, dims)
    if not t.is_cuda:
        raise ValueError(f"{fn} runs on CUDA tensors only")
    return t.get_device()


def _int32_ptr(t: Optional[torch.Tensor], name: str, index: int, n: Optional[int] = None):
    """Address of a contiguous int32 vector (of n elements) on the device."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32:
        raise TypeError(f"{name} must be a torch.int32 tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.dim() != 1 or not t.is_contiguous() or (t.numel() < 2 if n is None else t.numel() != n):
        raise ValueError(f"{name} must be a contiguous vector" + ("" if n is None else f" of {n} elements"))
    return t.data_ptr()


class _On:
    """The device and stream of a call: outputs are allocated for that stream,
    and tensors of another stream are kept until its work is done."""

    def __init__(self, index: int, stream: Optional[torch.cuda.Stream], tensors):
        if stream.device_index != index:
            raise ValueError(f"stream is on {stream.device}, expected cuda:{index}")
        self.stream, self.tensors = stream, tensors

    def __enter__(self):
        self.context = torch.cuda.stream(self.stream)
        self.context.__enter__()

    def __exit__(self, *exc):
        self.context.__exit__(*exc)
        for t in self.tensors:
            if t is not None and exc[0] is None:
                t.record_stream(self.stream)


class _Here:
    """The current stream of the current device: nothing to switch."""

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return None


_HERE = _Here()


def _on(index: int, stream: Optional[torch.cuda.Stream], tensors):
    if stream is not None and (stream.device_index != index or stream != torch.cuda.current_stream(index)):
        return _On(index, stream, tensors)
    return _HERE if torch._C._cuda_getDevice() == index else torch.cuda.device(index)


def _rows_like(t: torch.Tensor) -> torch.Tensor:
    """New contiguous rows of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _raise(code: int, checks) -> None:
    """The error of a refused call: what is wrong with a tensor, where the checks find it, else the status."""
    error = KDAError(code)
    for t, name, dtype, shape, contiguous in checks:
        if t is not None:
            _check(t, name, dtype, shape, t.device, contiguous)
    raise error


def _activation(name: Optional[str]) -> int:
    if name not in _ACTIVATION:
        raise ValueError(f"activation must be None or 'silu', got {name!r}")
    return _ACTIVATION[name]


def kda_conv_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                 activation: Optional[str] = "silu", cu_seqlens: Optional[torch.Tensor] = None,
                 initial_state: Optional[torch.Tensor] = None, output_final_state: bool = True,
                 out: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None):
    """Short causal depthwise convolution of packed sequences (see ``include/kda.h``).

    x: [T, C] bf16, fp16 or fp32; weight: fp32 [C, W], W in 2..4; bias: fp32 [C]
    or None; activation: "silu" or None; cu_seqlens: int32 [N + 1] on the device
    (None: one sequence; tokens behind the last sequence are left as they were);
    initial_state: [N, W - 1, C] of x's type (the inputs before each sequence,
    oldest first) or None. Returns ``(out, final_state)``; ``final_state`` is
    None unless requested.
    """
    dev = _device_of(x, "x", 2, "kda_conv_fwd")
    act = _activation(activation)
    cu = _int32_ptr(cu_seqlens, "cu_seqlens", dev)
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    _dims(weight, "weight", 2)
    (T, C), W = x.shape, weight.shape[1]
    with _on(dev, stream, (x, weight, bias, cu_seqlens, initial_state, out, final_state)):
        if out is None:
            out = _rows_like(x)
        if final_state is None and output_final_state:
            final_state = torch.empty((N, max(W - 1, 0), C), dtype=x.dtype, device=x.device)
        rc = _lib.kda_conv_fwd(_pack(x, "x", dev), _pack(weight, "weight", dev), _pack(bias, "bias", dev), act, cu, N,
                               _pack(initial_state, "initial_state", dev), _pack(out, "out", dev),
                               _pack(final_state, "final_state", dev), torch._C._cuda_getCurrentRawStream(dev))
    if rc != 0:
        t = x.dtype
        _raise(rc, [(weight, "weight", torch.float32, (C, W), True), (bias, "bias", torch.float32, (C,), True),
                    (initial_state, "initial_state", t, (N, W - 1, C), True), (out, "out", t, (T, C), False),
                    (final_state, "final_state", t, (N, W - 1, C), True)])
    return out, final_state


def kda_conv_decode(x: torch.Tensor, weight: torch.Tensor, state: torch.Tensor, bias: Optional[torch.Tensor] = None,
                    activation: Optional[str] = "silu", state_indices: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One token of the convolution for B requests (see ``include/kda.h``):
    returns the outputs and moves each request's state on, in place.

    x: [B, C]; state: [P, W - 1, C] of x's type; state_indices: int32 [B] on the
    device (distinct slots), or None for slot b; out may be x.
    """
    dev = _device_of(x, "x", 2, "kda_conv_decode")
    act = _activation(activation)
    _dims(weight, "weight", 2)
    _dims(state, "state", 3)
    B, C = x.shape
    idx = _int32_ptr(state_indices, "state_indices", dev, B)
    with _on(dev, stream, (x, weight, bias, state, state_indices, out)):
        if out is None:
            out = _rows_like(x)
        rc = _lib.kda_conv_decode(_pack(x, "x", dev), _pack(weight, "weight", dev), _pack(bias, "bias", dev), act,
                                  _pack(state, "state", dev), idx, _pack(out, "out", dev),
                                  torch._C._cuda_getCurrentRawStream(dev))
    if rc != 0:
        W = weight.shape[-1]
        _raise(rc, [(weight, "weight", torch.float32, (C, W), True), (bias, "bias", torch.float32, (C,), True),
                    (state, "state", x.dtype, (state.shape[0], W - 1, C), True), (out, "out", x.dtype, (B, C), False)])
    return out


def kda_conv_bwd(x: torch.Tensor, weight: torch.Tensor, dout: torch.Tensor, bias: Optional[torch.Tensor] = None,
                 activation: Optional[str] = "silu", cu_seqlens: Optional[torch.Tensor] = None,
                 initial_state: Optional[torch.Tensor] = None, dfinal_state: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None):
    """Gradients of ``kda_conv_fwd`` (see ``include/kda.h``): a dict of ``dx``
    [T, C] and ``dinitial_state`` [N, W - 1, C] of x's type, ``dweight`` fp32
    [C, W] and ``dbias`` fp32 [C] (None without a bias), for the output's
    gradient ``dout`` and the final state's (or None)."""
    dev = _device_of(x, "x", 2, "kda_conv_bwd")
    act = _activation(activation)
    cu = _int32_ptr(cu_seqlens, "cu_seqlens", dev)
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    _dims(weight, "weight", 2)
    (T, C), W = x.shape, weight.shape[1]
    with _on(dev, stream, (x, weight, bias, cu_seqlens, initial_state, dout, dfinal_state)):
        dx = _rows_like(x)
        dw = torch.empty((C, W), dtype=torch.float32, device=x.device)
        db = None if bias is None else torch.empty((C,), dtype=torch.float32, device=x.device)
        di = torch.empty((N, max(W - 1, 0), C), dtype=x.dtype, device=x.device)
        rc = _lib.kda_conv_bwd(_pack(x, "x", dev), _pack(weight, "weight", dev), _pack(bias, "bias", dev), act, cu, N,
                               _pack(initial_state, "initial_state", dev), _pack(dout, "dout", dev),
                               _pack(dfinal_state, "dfinal_state", dev), _pack(dx, "dx", dev),
                               _pack(dw, "dweight", dev), _pack(db, "dbias", dev), _pack(di, "dinitial_state", dev),
                               torch._C._cuda_getCurrentRawStream(dev))
    if rc != 0:
        t = x.dtype
        _raise(rc, [(weight, "weight", torch.float32, (C, W), True), (bias, "bias", torch.float32, (C,), True),
                    (initial_state, "initial_state", t, (N, W - 1, C), True), (dout, "dout", t, (T, C), False),
                    (dfinal_state, "dfinal_state", t, (N, W - 1, C), True)])
    return {"dx": dx, "dweight": dw, "dbias": db, "dinitial_state": di}


def _ssm_checks(u, dt, A, B, C, D, z, dt_bias):
    t, (T, c) = u.dtype, u.shape
    n, g = A.shape[1], B.shape[1]
    return [(dt, "dt", t, (T, c), False), (A, "A", torch.float32, (c, n), True), (B, "B", t, (T, g, n), False),
            (C, "C", t, (T, g, n), False), (D, "D", torch.float32, (c,), True), (z, "z", t, (T, c), False),
            (dt_bias, "dt_bias", torch.float32, (c,), True)]


def kda_ssm_fwd(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = True,
                cu_seqlens: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
                output_final_state: bool = True, out: Optional[torch.Tensor] = None,
                final_state: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """Selective state space scan of packed sequences (see ``include/kda.h``).

    u, dt: [T, C] bf16, fp16 or fp32; A: fp32 [C, S]; B, C: [T, G, S] of u's
    type; D, dt_bias: fp32 [C] or None; z: the gate, [T, C] of u's type, or None;
    dt_softplus: whether the step is log(1 + exp(dt + dt_bias)); cu_seqlens:
    int32 [N + 1] on the device (None: one sequence; tokens behind the last
    sequence are left as they were); initial_state: fp32 [N, C, S] or None.
    Returns ``(out, final_state)``; ``final_state`` is None unless requested and
    may be the initial state's tensor.
    """
    dev = _device_of(u, "u", 2, "kda_ssm_fwd")
    cu = _int32_ptr(cu_seqlens, "cu_seqlens", dev)
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    _dims(A, "A", 2)
    _dims(B, "B", 3)
    T, c = u.shape
    with _on(dev, stream, (u, dt, A, B, C, D, z, dt_bias, cu_seqlens, initial_state, out, final_state)):
        if out is None:
            out = _rows_like(u)
        if final_state is None and output_final_state:
            final_state = torch.empty((N, c, A.shape[1]), dtype=torch.float32, device=u.device)
        rc = _lib.kda_ssm_fwd(_pack(u, "u", dev), _pack(dt, "dt", dev), _pack(A, "A", dev), _pack(B, "B", dev),
                              _pack(C, "C", dev), _pack(D, "D", dev), _pack(z, "z", dev),
                              _pack(dt_bias, "dt_bias", dev), bool(dt_softplus), cu, N,
                              _pack(initial_state, "initial_state", dev), _pack(out, "out", dev),
                              _pack(final_state, "final_state", dev), torch._C._cuda_getCurrentRawStream(dev))
    if rc != 0:
        state = (N, c, A.shape[1])
        _raise(rc, _ssm_checks(u, dt, A, B, C, D, z, dt_bias) +
               [(initial_state, "initial_state", torch.float32, state, True), (out, "out", u.dtype, (T, c), False),
                (final_state, "final_state", torch.float32, state, True)])
    return out, final_state


def kda_ssm_decode(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                   state: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                   dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = True,
                   state_indices: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One token of the scan for R requests (see ``include/kda.h``): returns the
    outputs and moves each request's state on, in place.

    u, dt, z: [R, C]; B, C: [R, G, S]; state: fp32 [P, C, S]; state_indices:
    int32 [R] on the device (distinct slots), or None for slot r.
    """
    dev = _device_of(u, "u", 2, "kda_ssm_decode")
    _dims(A, "A", 2)
    _dims(B, "B", 3)
    _dims(state, "state", 3)
    R, c = u.shape
    idx = _int32_ptr(state_indices, "state_indices", dev, R)
    with _on(dev, stream, (u, dt, A, B, C, D, z, dt_bias, state, state_indices, out)):
        if out is None:
            out = _rows_like(u)
        rc = _lib.kda_ssm_decode(_pack(u, "u", dev), _pack(dt, "dt", dev), _pack(A, "A", dev), _pack(B, "B", dev),
                                 _pack(C, "C", dev), _pack(D, "D", dev), _pack(z, "z", dev),
                                 _pack(dt_bias, "dt_bias", dev), bool(dt_softplus), _pack(state, "state", dev), idx,
                                 _pack(out, "out", dev), torch._C._cuda_getCurrentRawStream(dev))
    if rc != 0:
        _raise(rc, _ssm_checks(u, dt, A, B, C, D, z, dt_bias) +
               [(state, "state", torch.float32, (state.shape[0], c, A.shape[1]), True),
                (out, "out", u.dtype, (R, c), False)])
    return out


def kda_ssm_bwd(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                dout: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = True,
                cu_seqlens: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
                dfinal_state: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """Gradients of ``kda_ssm_fwd`` (see ``include/kda.h``) for the output's
    gradient ``dout`` and the final state's (or None): a dict of ``du``, ``ddt``,
    ``dz`` [T, C], ``dB``, ``dC`` [T, G, S] of u's type and fp32 ``dA`` [C, S],
    ``dD``, ``ddt_bias`` [C], ``dinitial_state`` [N, C, S]; None for ``dz``,
    ``dD`` and ``ddt_bias`` whose input is None."""
    dev = _device_of(u, "u", 2, "kda_ssm_bwd")
    cu = _int32_ptr(cu_seqlens, "cu_seqlens", dev)
    N = 1 if cu_seqlens is None else cu_seqlens.numel() - 1
    (T, c), f32 = u.shape, torch.float32
    _dims(A, "A", 2)
    _dims(B, "B", 3)
    with _on(dev, stream, (u, dt, A, B, C, D, z, dt_bias, cu_seqlens, initial_state, dout, dfinal_state)):
        def new(shape, dtype=u.dtype, of=u):
            return None if of is None else torch.empty(shape, dtype=dtype, device=u.device)

        gr = {"du": new((T, c)), "ddt": new((T, c)), "dA": new(A.shape, f32), "dB": new(B.shape), "dC": new(B.shape),
              "dD": new((c,), f32, D), "dz": new((T, c), u.dtype, z), "ddt_bias": new((c,), f32, dt_bias),
              "dinitial_state": new((N, c, A.shape[1]), f32)}
        rc = _lib.kda_ssm_bwd(_pack(u, "u", dev), _pack(dt, "dt", dev), _pack(A, "A", dev), _pack(B, "B", dev),
                              _pack(C, "C", dev), _pack(D, "D", dev), _pack(z, "z", dev),
                              _pack(dt_bias, "dt_bias", dev), bool(dt_softplus), cu, N,
                              _pack(initial_state, "initial_state", dev), _pack(dout, "dout", dev),
                              _pack(dfinal_state, "dfinal_state", dev), *(_pack(t, n, dev) for n, t in gr.items()),
                              torch._C._cuda_getCurrentRawStream(dev))
    if rc != 0:
        state = (N, c, A.shape[1])
        _raise(rc, _ssm_checks(u, dt, A, B, C, D, z, dt_bias) +
               [(initial_state, "initial_state", f32, state, True), (dout, "dout", u.dtype, (T, c), False),
                (dfinal_state, "dfinal_state", f32, state, True)])
    return gr
