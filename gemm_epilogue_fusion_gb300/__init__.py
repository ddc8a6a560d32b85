"""Python binding of the GB300 fused GEMM-epilogue library (``include/coda.h``).

Argument marshalling only: every function here takes torch tensors, checks
that they are contiguous CUDA tensors, passes their device pointers, sizes and
the current CUDA stream to the C ABI function of the same name, and raises
``CodaError`` on a non-OK status.  All arithmetic runs in the library's
kernels; PyTorch only provides device memory and streams.  Outputs can be
passed in (pre-allocated) or are allocated with ``torch.empty``, on the
current stream: a call given another ``stream`` has to be ordered with the
current one, as for any tensor that two streams use.  A workspace that the call
itself makes and drops is the given stream's.

The library is ``libcoda_gb300.so`` next to this file, compiled for sm_103a
by ``_build.build()``.  There is no fallback: if it cannot be built or
loaded, importing a function raises.

Hot path (the CODA write-up, section "CODA: the treasure hidden in the
epilogue"):

    h, P = coda_gemm_residual_partial_rms(X, W1t, R)   # h = R + X W1, partial sums of h^2
    r    = coda_rms_reduce(P, N, eps)                  # r = 1/sqrt(mean h^2 + eps)
    Z    = coda_gemm_rowscale(h, W2t_folded, r)        # diag(r) h diag(gamma) W2
    act  = coda_gemm_swiglu(h, Wgt_folded, Wut_folded, r)
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
import warnings
from typing import Optional

import torch

from . import _build

CODA_OK, CODA_ERR_INVALID_ARG, CODA_ERR_UNSUPPORTED, CODA_ERR_CUDA, CODA_ERR_TIMEOUT = range(5)
CODA_F32, CODA_BF16, CODA_E4M3 = 0, 1, 2
CODA_K_MAJOR, CODA_MN_MAJOR = 0, 1

_STATUS_NAMES = {0: "CODA_OK", 1: "CODA_ERR_INVALID_ARG", 2: "CODA_ERR_UNSUPPORTED", 3: "CODA_ERR_CUDA",
                 4: "CODA_ERR_TIMEOUT"}

# Every symbol include/coda.h declares, with (restype, argtypes).
_vp, _fp, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
SIGNATURES = {
    "coda_version": (_i32, []),
    "coda_status_string": (ctypes.c_char_p, [_i32]),
    "coda_last_error": (ctypes.c_char_p, []),
    "coda_partial_cols": (_i64, [_i64]),
    "coda_fold_gamma": (_i32, [_vp, _fp, _vp, _i64, _i64, _i32, _vp]),
    "coda_gemm_residual_partial_rms": (_i32, [_vp, _vp, _vp, _vp, _fp, _i64, _i64, _i64, _i32, _fp, _fp, _fp, _vp]),
    "coda_rms_reduce": (_i32, [_fp, _i64, _i64, _f32, _fp, _vp]),
    "coda_gemm_rowscale": (_i32, [_vp, _vp, _fp, _vp, _i64, _i64, _i64, _i32, _fp, _fp, _vp]),
    "coda_gemm_swiglu": (_i32, [_vp, _vp, _vp, _fp, _vp, _i64, _i64, _i64, _i32, _fp, _fp, _fp, _fp, _vp]),
    "coda_gemm_rowscale_fused_rms": (_i32, [_vp, _vp, _fp, _f32, _fp, _vp, _i64, _i64, _i64, _i32, _fp, _fp, _vp]),
    "coda_gemm_swiglu_fused_rms": (_i32, [_vp, _vp, _vp, _fp, _f32, _fp, _vp, _i64, _i64, _i64, _i32, _fp, _fp, _fp,
                                          _fp, _vp]),
    "coda_block_workspace_bytes": (_i64, [_i64]),
    "coda_block_rowscale": (_i32, [_vp, _vp, _vp, _vp, _f32, _vp, _fp, _fp, _vp, _i64, _i64, _i64, _i64, _i32, _vp,
                                   _vp]),
    "coda_block_swiglu": (_i32, [_vp, _vp, _vp, _vp, _vp, _f32, _vp, _fp, _fp, _vp, _i64, _i64, _i64, _i64, _i32, _vp,
                                 _vp]),
    "coda_block_rowscale_rope": (_i32, [_vp, _vp, _vp, _vp, _f32, _vp, _fp, _fp, _vp, _i64, _i64, _i64, _i64, _i32,
                                        _i64, _i64, ctypes.c_double, _i64, _vp, _vp, _vp]),
    "coda_block_swiglu_noalloc": (_i32, [_vp, _vp, _vp, _vp, _vp, _f32, _vp, _fp, _fp, _vp, _i64, _i64, _i64, _i64,
                                         _i32, _vp]),
    "coda_gemm_rowscale_rope": (_i32, [_vp, _vp, _fp, _fp, _f32, _fp, _vp, _i64, _i64, _i64, _i32, _fp, _fp, _i64,
                                       _i64, ctypes.c_double, _i64, _vp, _vp]),
    "coda_gemm": (_i32, [_vp, _i32, _vp, _i32, _vp, _i64, _i64, _i64, _i32, _fp, _fp, _vp]),
    "coda_gemm_grad_norm": (_i32, [_vp, _vp, _vp, _fp, _vp, _fp, _i64, _i64, _i64, _i32, _vp]),
    "coda_rmsnorm_backward_workspace_bytes": (_i64, [_i64, _i64]),
    "coda_rmsnorm_backward": (_i32, [_vp, _vp, _fp, _fp, _fp, _vp, _vp, _vp, _fp, _fp, _i64, _i64, _vp]),
    "coda_gemm_swiglu_backward": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp]),
    "coda_gemm_swiglu_save": (_i32, [_vp, _vp, _vp, _fp, _fp, _f32, _fp, _vp, _vp, _i64, _i64, _i64, _i32, _vp]),
    "coda_block_fp8_workspace_bytes": (_i64, [_i64]),
    "coda_block_swiglu_fp8": (_i32, [_vp, _fp, _vp, _fp, _vp, _fp, _vp, _vp, _fp, _vp, _fp, _f32, _vp, _fp, _fp, _fp,
                                     _vp, _fp, _vp, _fp, _i64, _i64, _i64, _i64, _vp, _vp]),
    "coda_block_rowscale_fp8": (_i32, [_vp, _fp, _vp, _fp, _vp, _fp, _vp, _vp, _fp, _f32, _vp, _fp, _fp, _fp, _vp, _fp,
                                       _vp, _i64, _i64, _i64, _i64, _vp, _vp]),
    "coda_paged_append": (_i32, [_vp] * 7 + [_i64] * 8 + [ctypes.c_double, _i32, _i32, _fp, _fp, _vp]),
    "coda_paged_attention_workspace_bytes": (_i64, [_i64, _i64, _i64]),
    "coda_paged_attention": (_i32, [_vp, _i64] + [_vp] * 7 + [_i64] * 8 + [_f32, _i32, _i32, _fp, _fp, _vp, _vp]),
    "coda_logprobs": (_i32, [_vp, _i64, _vp, _fp, _fp, _fp, _fp, _vp, _i64, _i64, _i64, _i32, _vp]),
    "coda_logprobs_backward": (_i32, [_vp, _i64, _vp, _fp, _fp, _fp, _fp, _vp, _i64, _i64, _i64, _i32, _vp]),
    "coda_add_rmsnorm": (_i32, [_vp, _i64, _vp, _i64, _fp, _f32, _vp, _vp, _vp, _fp, _fp, _i64, _i64, _i32, _vp]),
    "coda_quantize_rows_e4m3": (_i32, [_vp, _i64, _vp, _fp, _i64, _i64, _i32, _vp]),
    "coda_add_rmsnorm_backward_workspace_bytes": (_i64, [_i64, _i64]),
    "coda_add_rmsnorm_backward": (_i32, [_vp, _vp, _fp, _fp, _vp, _vp, _fp, _fp, _i64, _i64, _i32, _vp]),
    "coda_route_workspace_bytes": (_i64, [_i64, _i64, _i64]),
    "coda_route": (_i32, [_vp, _i64, _i64, _i32, _vp, _fp, _vp, _vp, _vp, _i64, _i64, _i32, _vp]),
    "coda_route_backward": (_i32, [_vp, _i64, _vp, _fp, _fp, _i32, _vp, _i64, _i64, _i64, _i64, _i32, _vp]),
    "coda_expert_dispatch": (_i32, [_vp, _fp, _vp, _vp, _fp, _i64, _i64, _i64, _i64, _i32, _vp]),
    "coda_expert_combine": (_i32, [_vp, _vp, _fp, _vp, _vp, _fp, _i64, _i64, _i64, _i64, _i32, _vp]),
    "coda_expert_combine_backward": (_i32, [_vp, _vp, _vp, _fp, _vp, _fp, _i64, _i64, _i64, _i64, _i32, _vp]),
    "coda_grouped_gemm": (_i32, [_vp, _vp, _i32, _vp, _fp, _fp, _vp, _i64, _i64, _i64, _i64, _i32, _vp]),
    "coda_grouped_gemm_swiglu": (_i32, [_vp, _vp, _vp, _fp, _fp, _vp, _vp, _i64, _i64, _i64, _i64, _i32, _vp]),
    "coda_grouped_gemm_swiglu_backward": (_i32, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i32, _vp]),
    "coda_grouped_gemm_wgrad": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i32, _vp]),
    "coda_amax": (_i32, [_vp, _i64, _i32, _fp, _vp]),
    "coda_quantize_e4m3": (_i32, [_vp, _i64, _i32, _fp, _vp, _fp, _vp]),
    "coda_selftest_wait_timeout": (_i32, [_i64, _vp]),
    "coda_get_device_status": (_i32, []),
}

# The mixture-of-experts calls in the order that the C marshalling keeps them.
_EXPERT_CALLS = ("coda_add_rmsnorm", "coda_quantize_rows_e4m3", "coda_add_rmsnorm_backward",
                 "coda_add_rmsnorm_backward_workspace_bytes", "coda_route", "coda_route_workspace_bytes",
                 "coda_route_backward", "coda_expert_dispatch", "coda_expert_combine", "coda_expert_combine_backward",
                 "coda_grouped_gemm", "coda_grouped_gemm_swiglu", "coda_grouped_gemm_swiglu_backward",
                 "coda_grouped_gemm_wgrad")

_lock = threading.Lock()
_lib = None
_fast = None  # _coda_marshal once the library is loaded
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class CodaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def library_path() -> str:
    return _build.LIB


def load_library(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libcoda_gb300.so (compiling it first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.build() if build_if_missing else _build.LIB
            if not os.path.exists(path):
                raise RuntimeError(f"CUDA library {path} is missing: run __graft_entry__.build()")
            lib = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype, fn.argtypes = res, args
            _load_marshal(lib)
            _lib = lib
    return _lib


def _load_marshal(lib) -> None:
    """The C marshalling of the short calls (coda_marshal.c), given the library's own entry points."""
    global _fast
    if _raw_stream is None or not os.path.exists(_build.MARSHAL):
        return  # a PyTorch without CUDA, or a module that was not built: the checks in Python serve
    try:
        from . import _coda_marshal as m
    except ImportError as e:
        warnings.warn(f"{_build.MARSHAL} cannot be loaded, the decode, scoring and experts' calls take longer on the host: {e}",
                      RuntimeWarning, stacklevel=3)
        return
    names = ("coda_paged_append", "coda_paged_attention", "coda_paged_attention_workspace_bytes", "coda_logprobs",
             "coda_logprobs_backward")
    m.init(torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.uint8, torch.int32, torch.cuda.current_device,
           _raw_stream, *(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names))
    m.init_experts(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _EXPERT_CALLS))
    _fast = m


def _check(status: int):
    if status != CODA_OK:
        raise CodaError(status, load_library().coda_last_error().decode())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return CODA_F32
    if t.dtype == torch.bfloat16:
        return CODA_BF16
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return CODA_E4M3
    raise TypeError(f"unsupported operand dtype {t.dtype}")


def _out_dtype(code: int) -> torch.dtype:
    return torch.float32 if code == CODA_F32 else torch.bfloat16


_F32 = (torch.float32,)
_BYTE = (torch.uint8, torch.float8_e4m3fn)


def _want(t: Optional[torch.Tensor], name: str, shape=None, dtypes=None, numel=None, nbytes=None):
    """Checks that a given tensor matches the sizes the call passes to the
    library (the kernels read and write exactly those extents): its shape,
    its dtype, at least `numel` elements (scalars) or `nbytes` bytes
    (workspaces).  None passes (a NULL argument, which the library checks)."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected at least {numel}")
    if nbytes is not None and t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes, expected at least {nbytes}")


def _operand_dtypes(code: int):
    return {CODA_F32: (torch.float32,), CODA_BF16: (torch.bfloat16,), CODA_E4M3: _BYTE}[code]


def _want_scalars(**scalars):
    """Per-tensor scales and amax outputs: one fp32 each."""
    for name, t in scalars.items():
        _want(t, name, dtypes=_F32, numel=1)


def _want_block(X, W1t, R, Wb, Wb2, H, P, out, r_out, workspace, n_out, code, out_name, wb_name):
    """The tensors of a one-launch block: X [M, K], W1t [N, K], R and h [M, N],
    the consumer's weights [n_out, N], P [M, T], the output [M, n_out]."""
    M, K = X.shape
    N = W1t.shape[0]
    ops, od = _operand_dtypes(code), (_out_dtype(code),)
    _want(W1t, "W1t", (N, K), ops)
    _want(R, "R", (M, N), od)
    _want(Wb, wb_name, (n_out, N), ops)
    _want(Wb2, "Wut", (n_out, N), ops)
    _want(H, "H", (M, N), od)
    _want(P, "P", (M, coda_partial_cols(N)), _F32)
    _want(out, out_name, (M, n_out), od)
    _want(r_out, "r_out", (M,), _F32)
    _want(workspace, "workspace", nbytes=coda_block_workspace_bytes(M))


def _want_fp8_block(A, amax_a, Aq, scale_a, W1t, scale_w1, R, Wb, scale_wb, Wb2, scale_wb2, H, P, r_out, amax_h, Hq,
                    scale_h, out, amax_out, workspace, M, N, K, n_out, out_name, wb_name):
    """The tensors of an FP8 one-launch block (e4m3 operands as uint8 bytes)."""
    bf = (torch.bfloat16,)
    _want(A, "A", (M, K), bf)
    _want(Aq, "Aq", (M, K), _BYTE)
    _want(W1t, "W1t", (N, K), _BYTE)
    _want(R, "R", (M, N), bf)
    _want(Wb, wb_name, (n_out, N), _BYTE)
    _want(Wb2, "Wut", (n_out, N), _BYTE)
    _want(H, "H", (M, N), bf)
    _want(P, "P", (M, coda_partial_cols(N)), _F32)
    _want(r_out, "r_out", (M,), _F32)
    _want(Hq, "Hq", (M, N), _BYTE)
    _want(out, out_name, (M, n_out), bf)
    _want_scalars(amax_a=amax_a, scale_a=scale_a, scale_w1=scale_w1, scale_w=scale_wb, scale_wu=scale_wb2,
                  amax_h=amax_h, scale_h=scale_h, amax_act=amax_out)
    _want(workspace, "workspace", nbytes=coda_block_fp8_workspace_bytes(M))


def _dev(t: Optional[torch.Tensor], name: str):
    """Device pointer of a contiguous CUDA tensor on the current device (None -> NULL)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device.index is not None and t.device.index != torch.cuda.current_device():
        # the library launches on the current device
        raise ValueError(f"{name} is on {t.device} but the current device is cuda:{torch.cuda.current_device()}")
    return t.data_ptr() or None


def _stream(t: torch.Tensor, stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(t.device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _stream_object(stream, device):
    """The torch stream behind a ``stream`` argument: one of torch's, or anything with an address."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    address = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    # the default stream goes by 0 and by 1 (cudaStreamLegacy)
    return torch.cuda.default_stream(device) if address in (0, 1) else torch.cuda.ExternalStream(address, device=device)


def _made_on(stream, device, make):
    """A call's own workspace, make(), from the pool of the stream it launches on.  The call drops it on return: from the
    current stream's pool it could be given out again there, or still be in use there, while the kernels on `stream` have
    it."""
    if stream is None:
        return make()
    with torch.cuda.stream(_stream_object(stream, device)):
        return make()


def coda_partial_cols(N: int) -> int:
    return int(load_library().coda_partial_cols(N))


def coda_fold_gamma(Wt: torch.Tensor, gamma: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None):
    """W'^T = W^T diag(gamma): out[n, k] = Wt[n, k] * gamma[k]."""
    lib = load_library()
    N_out, K = Wt.shape
    out = torch.empty_like(Wt) if out is None else out
    _want(Wt, "Wt", dtypes=(torch.float32, torch.bfloat16))
    _want(gamma, "gamma", (K,), _F32)
    _want(out, "out", (N_out, K), (Wt.dtype,))
    _check(lib.coda_fold_gamma(_dev(Wt, "Wt"), _dev(gamma, "gamma"), _dev(out, "out"), N_out, K, _dtype_code(Wt),
                               _stream(Wt, stream)))
    return out


def coda_gemm_residual_partial_rms(X, W1t, R, H=None, P=None, *, scale_x=None, scale_w=None, amax_h=None,
                                   stream=None):
    """h = R + X W1 (W1t = W1^T) and P[i, g] = sum of h[i, j]^2 over 128-column group g.  Returns (h, P)."""
    lib = load_library()
    M, K = X.shape
    N = W1t.shape[0]
    code = _dtype_code(X)
    if H is None:
        H = torch.empty(M, N, dtype=_out_dtype(code), device=X.device)
    if P is None:
        P = torch.empty(M, max(coda_partial_cols(N), 0), dtype=torch.float32, device=X.device)
    ops, od = _operand_dtypes(code), (_out_dtype(code),)
    _want(W1t, "W1t", (N, K), ops)
    _want(R, "R", (M, N), od)
    _want(H, "H", (M, N), od)
    _want(P, "P", (M, coda_partial_cols(N)), _F32)
    _want_scalars(scale_x=scale_x, scale_w=scale_w, amax_h=amax_h)
    _check(lib.coda_gemm_residual_partial_rms(_dev(X, "X"), _dev(W1t, "W1t"), _dev(R, "R"), _dev(H, "H"),
                                              _dev(P, "P"), M, N, K, code, _dev(scale_x, "scale_x"),
                                              _dev(scale_w, "scale_w"), _dev(amax_h, "amax_h"), _stream(X, stream)))
    return H, P


def coda_rms_reduce(P, N: int, eps: float, r=None, stream=None):
    """r[i] = 1 / sqrt(sum_g P[i, g] / N + eps)."""
    lib = load_library()
    M = P.shape[0]
    if r is None:
        r = torch.empty(M, dtype=torch.float32, device=P.device)
    _want(P, "P", (M, coda_partial_cols(N)), _F32)
    _want(r, "r", (M,), _F32)
    _check(lib.coda_rms_reduce(_dev(P, "P"), M, N, float(eps), _dev(r, "r"), _stream(P, stream)))
    return r


def coda_gemm_rowscale(H, W2t, r, Z=None, *, scale_h=None, scale_w=None, stream=None):
    """Z = diag(r) H W2 (W2t = W2^T, gamma already folded in)."""
    lib = load_library()
    M, K = H.shape
    N2 = W2t.shape[0]
    code = _dtype_code(H)
    if Z is None:
        Z = torch.empty(M, N2, dtype=_out_dtype(code), device=H.device)
    _want(W2t, "W2t", (N2, K), _operand_dtypes(code))
    _want(r, "r", (M,), _F32)
    _want(Z, "Z", (M, N2), (_out_dtype(code),))
    _want_scalars(scale_h=scale_h, scale_w=scale_w)
    _check(lib.coda_gemm_rowscale(_dev(H, "H"), _dev(W2t, "W2t"), _dev(r, "r"), _dev(Z, "Z"), M, N2, K, code,
                                  _dev(scale_h, "scale_h"), _dev(scale_w, "scale_w"), _stream(H, stream)))
    return Z


def coda_gemm_swiglu(H, Wgt, Wut, r=None, Act=None, *, scale_h=None, scale_wg=None, scale_wu=None, amax_act=None,
                     stream=None):
    """Act = silu(diag(r) H Wg) * (diag(r) H Wu)."""
    lib = load_library()
    M, K = H.shape
    I = Wgt.shape[0]
    code = _dtype_code(H)
    if Act is None:
        Act = torch.empty(M, I, dtype=_out_dtype(code), device=H.device)
    _want(Wgt, "Wgt", (I, K), _operand_dtypes(code))
    _want(Wut, "Wut", (I, K), _operand_dtypes(code))
    _want(r, "r", (M,), _F32)
    _want(Act, "Act", (M, I), (_out_dtype(code),))
    _want_scalars(scale_h=scale_h, scale_wg=scale_wg, scale_wu=scale_wu, amax_act=amax_act)
    _check(lib.coda_gemm_swiglu(_dev(H, "H"), _dev(Wgt, "Wgt"), _dev(Wut, "Wut"), _dev(r, "r"), _dev(Act, "Act"),
                                M, I, K, code, _dev(scale_h, "scale_h"), _dev(scale_wg, "scale_wg"),
                                _dev(scale_wu, "scale_wu"), _dev(amax_act, "amax_act"), _stream(H, stream)))
    return Act


def coda_gemm_rowscale_fused_rms(H, W2t, P, eps: float, Z=None, r_out=None, *, scale_h=None, scale_w=None,
                                 stream=None):
    """Z = diag(r) H W2 with r reduced from the partials P inside the epilogue."""
    lib = load_library()
    M, K = H.shape
    N2 = W2t.shape[0]
    code = _dtype_code(H)
    if Z is None:
        Z = torch.empty(M, N2, dtype=_out_dtype(code), device=H.device)
    _want(W2t, "W2t", (N2, K), _operand_dtypes(code))
    _want(P, "P", (M, coda_partial_cols(K)), _F32)
    _want(r_out, "r_out", (M,), _F32)
    _want(Z, "Z", (M, N2), (_out_dtype(code),))
    _want_scalars(scale_h=scale_h, scale_w=scale_w)
    _check(lib.coda_gemm_rowscale_fused_rms(_dev(H, "H"), _dev(W2t, "W2t"), _dev(P, "P"), float(eps),
                                            _dev(r_out, "r_out"), _dev(Z, "Z"), M, N2, K, code,
                                            _dev(scale_h, "scale_h"), _dev(scale_w, "scale_w"), _stream(H, stream)))
    return Z


def coda_gemm_swiglu_fused_rms(H, Wgt, Wut, P, eps: float, Act=None, r_out=None, *, scale_h=None, scale_wg=None,
                               scale_wu=None, amax_act=None, stream=None):
    """Act = silu(diag(r) H Wg) * (diag(r) H Wu) with r reduced from P inside the epilogue."""
    lib = load_library()
    M, K = H.shape
    I = Wgt.shape[0]
    code = _dtype_code(H)
    if Act is None:
        Act = torch.empty(M, I, dtype=_out_dtype(code), device=H.device)
    _want(Wgt, "Wgt", (I, K), _operand_dtypes(code))
    _want(Wut, "Wut", (I, K), _operand_dtypes(code))
    _want(P, "P", (M, coda_partial_cols(K)), _F32)
    _want(r_out, "r_out", (M,), _F32)
    _want(Act, "Act", (M, I), (_out_dtype(code),))
    _want_scalars(scale_h=scale_h, scale_wg=scale_wg, scale_wu=scale_wu, amax_act=amax_act)
    _check(lib.coda_gemm_swiglu_fused_rms(_dev(H, "H"), _dev(Wgt, "Wgt"), _dev(Wut, "Wut"), _dev(P, "P"),
                                          float(eps), _dev(r_out, "r_out"), _dev(Act, "Act"), M, I, K, code,
                                          _dev(scale_h, "scale_h"), _dev(scale_wg, "scale_wg"),
                                          _dev(scale_wu, "scale_wu"), _dev(amax_act, "amax_act"),
                                          _stream(H, stream)))
    return Act


def coda_gemm_rowscale_rope(H, W2t, head_dim: int, rope_cols: int, base: float, *, seq_len: int = 0, positions=None,
                            r=None, P=None, eps: float = 0.0, r_out=None, Z=None, scale_h=None, scale_w=None,
                            stream=None):
    """Z = RoPE(diag(r) H W2) on the first rope_cols columns; r given, or reduced from P inside the epilogue.
    Positions: ``positions`` [M] int32, else row mod ``seq_len``."""
    lib = load_library()
    M, K = H.shape
    N2 = W2t.shape[0]
    code = _dtype_code(H)
    if Z is None:
        Z = torch.empty(M, N2, dtype=_out_dtype(code), device=H.device)
    _want(W2t, "W2t", (N2, K), _operand_dtypes(code))
    _want(r, "r", (M,), _F32)
    _want(P, "P", (M, coda_partial_cols(K)), _F32)
    _want(r_out, "r_out", (M,), _F32)
    _want(Z, "Z", (M, N2), (_out_dtype(code),))
    _want(positions, "positions", (M,), (torch.int32,))
    _want_scalars(scale_h=scale_h, scale_w=scale_w)
    _check(lib.coda_gemm_rowscale_rope(_dev(H, "H"), _dev(W2t, "W2t"), _dev(r, "r"), _dev(P, "P"), float(eps),
                                       _dev(r_out, "r_out"), _dev(Z, "Z"), M, N2, K, code, _dev(scale_h, "scale_h"),
                                       _dev(scale_w, "scale_w"), head_dim, rope_cols, float(base), seq_len,
                                       _dev(positions, "positions"), _stream(H, stream)))
    return Z


def coda_gemm(A, B, *, a_mn: bool = False, b_mn: bool = False, row_scale=None, col_scale=None, D=None,
              stream=None):
    """D = diag(row_scale) opA(A) opB(B)^T diag(col_scale), with opA(A) = A [M, K] or A^T for A [K, M]
    (a_mn) and opB(B) = B [N, K] or B^T for B [K, N] (b_mn)."""
    lib = load_library()
    M, K = (A.shape[1], A.shape[0]) if a_mn else (A.shape[0], A.shape[1])
    N = B.shape[1] if b_mn else B.shape[0]
    if (B.shape[0] if b_mn else B.shape[1]) != K:
        raise ValueError("inner dimensions differ")
    code = _dtype_code(A)
    if D is None:
        D = torch.empty(M, N, dtype=_out_dtype(code), device=A.device)
    _want(B, "B", dtypes=(A.dtype,))
    _want(D, "D", (M, N), (_out_dtype(code),))
    _want(row_scale, "row_scale", (M,), _F32)
    _want(col_scale, "col_scale", (N,), _F32)
    _check(lib.coda_gemm(_dev(A, "A"), int(a_mn), _dev(B, "B"), int(b_mn), _dev(D, "D"), M, N, K, code,
                         _dev(row_scale, "row_scale"), _dev(col_scale, "col_scale"), _stream(A, stream)))
    return D


def coda_gemm_grad_norm(dOut, Wt, H, gamma, dY=None, S=None, stream=None):
    """dY = dOut . Wt (Wt [K, N] as the forward stores it) and S = per-group sums of gamma dY H.  Returns (dY, S)."""
    lib = load_library()
    M, K = dOut.shape
    N = Wt.shape[1]
    if dY is None:
        dY = torch.empty(M, N, dtype=torch.bfloat16, device=dOut.device)
    if S is None:
        S = torch.empty(M, coda_partial_cols(N), dtype=torch.float32, device=dOut.device)
    bf = (torch.bfloat16,)
    _want(dOut, "dOut", dtypes=bf)
    _want(Wt, "Wt", (K, N), bf)
    _want(H, "H", (M, N), bf)
    _want(gamma, "gamma", (N,), _F32)
    _want(dY, "dY", (M, N), bf)
    _want(S, "S", (M, coda_partial_cols(N)), _F32)
    _check(lib.coda_gemm_grad_norm(_dev(dOut, "dOut"), _dev(Wt, "Wt"), _dev(H, "H"), _dev(gamma, "gamma"),
                                   _dev(dY, "dY"), _dev(S, "S"), M, N, K, _dtype_code(dOut), _stream(dOut, stream)))
    return dY, S


def coda_rmsnorm_backward(dY, H, r, gamma, S, dH_in=None, dH=None, Yt=None, dgamma=None, workspace=None,
                          stream=None):
    """dH = r gamma dY - c H (+ dH_in), Yt = r H, dgamma.  Returns (dH, Yt, dgamma)."""
    lib = load_library()
    M, N = dY.shape
    dH = torch.empty_like(dY) if dH is None else dH
    Yt = torch.empty_like(dY) if Yt is None else Yt
    if dgamma is None:
        dgamma = torch.empty(N, dtype=torch.float32, device=dY.device)
    if workspace is None:
        n = max(lib.coda_rmsnorm_backward_workspace_bytes(M, N) // 4, 1)
        workspace = _made_on(stream, dY.device, lambda: torch.empty(n, dtype=torch.float32, device=dY.device))
    bf = (torch.bfloat16,)
    for t, name in ((dY, "dY"), (H, "H"), (dH_in, "dH_in"), (dH, "dH"), (Yt, "Yt")):
        _want(t, name, (M, N), bf)
    _want(r, "r", (M,), _F32)
    _want(gamma, "gamma", (N,), _F32)
    _want(S, "S", (M, coda_partial_cols(N)), _F32)
    _want(dgamma, "dgamma", (N,), _F32)
    _want(workspace, "workspace", nbytes=lib.coda_rmsnorm_backward_workspace_bytes(M, N))
    _check(lib.coda_rmsnorm_backward(_dev(dY, "dY"), _dev(H, "H"), _dev(r, "r"), _dev(gamma, "gamma"), _dev(S, "S"),
                                     _dev(dH_in, "dH_in"), _dev(dH, "dH"), _dev(Yt, "Yt"), _dev(dgamma, "dgamma"),
                                     _dev(workspace, "workspace"), M, N, _stream(dY, stream)))
    return dH, Yt, dgamma


def coda_gemm_swiglu_save(H, Wgt, Wut, *, r=None, P=None, eps: float = 0.0, r_out=None, Act=None, GU=None,
                          stream=None):
    """SwiGLU GEMM that also returns the pre-activations G || U [M, 2I].  Returns (Act, GU)."""
    lib = load_library()
    M, K = H.shape
    I = Wgt.shape[0]
    if Act is None:
        Act = torch.empty(M, I, dtype=torch.bfloat16, device=H.device)
    if GU is None:
        GU = torch.empty(M, 2 * I, dtype=torch.bfloat16, device=H.device)
    bf = (torch.bfloat16,)
    _want(H, "H", dtypes=bf)
    _want(Wgt, "Wgt", (I, K), bf)
    _want(Wut, "Wut", (I, K), bf)
    _want(r, "r", (M,), _F32)
    _want(P, "P", (M, coda_partial_cols(K)), _F32)
    _want(r_out, "r_out", (M,), _F32)
    _want(Act, "Act", (M, I), bf)
    _want(GU, "GU", (M, 2 * I), bf)
    _check(lib.coda_gemm_swiglu_save(_dev(H, "H"), _dev(Wgt, "Wgt"), _dev(Wut, "Wut"), _dev(r, "r"), _dev(P, "P"),
                                     float(eps), _dev(r_out, "r_out"), _dev(Act, "Act"), _dev(GU, "GU"), M, I, K,
                                     _dtype_code(H), _stream(H, stream)))
    return Act, GU


def coda_gemm_swiglu_backward(dOut, Wt, GU, dGU=None, stream=None):
    """dG || dU from dAct = dOut . Wt (Wt [K, I]) and the saved G || U [M, 2I]."""
    lib = load_library()
    M, K = dOut.shape
    I = Wt.shape[1]
    if dGU is None:
        dGU = torch.empty(M, 2 * I, dtype=torch.bfloat16, device=dOut.device)
    bf = (torch.bfloat16,)
    _want(dOut, "dOut", dtypes=bf)
    _want(Wt, "Wt", (K, I), bf)
    _want(GU, "GU", (M, 2 * I), bf)
    _want(dGU, "dGU", (M, 2 * I), bf)
    _check(lib.coda_gemm_swiglu_backward(_dev(dOut, "dOut"), _dev(Wt, "Wt"), _dev(GU, "GU"), _dev(dGU, "dGU"), M, I,
                                         K, _dtype_code(dOut), _stream(dOut, stream)))
    return dGU


def coda_block_workspace_bytes(M: int) -> int:
    return int(load_library().coda_block_workspace_bytes(M))


def block_workspace(M: int, device) -> torch.Tensor:
    """A zeroed workspace for the one-launch blocks (calls leave it zeroed)."""
    n = coda_block_workspace_bytes(M)
    return torch.zeros((n + 3) // 4, dtype=torch.int32, device=device)


def _block_outputs(X, R, N, n_out, H, P, out, code):
    M = X.shape[0]
    if H is None:
        H = torch.empty(M, N, dtype=_out_dtype(code), device=X.device)
    if P is None:
        P = torch.empty(M, max(coda_partial_cols(N), 0), dtype=torch.float32, device=X.device)
    if out is None:
        out = torch.empty(M, n_out, dtype=_out_dtype(code), device=X.device)
    return H, P, out


def coda_block_rowscale(X, W1t, R, W2t, eps: float, workspace, H=None, P=None, Z=None, r_out=None, stream=None):
    """One launch: h = R + X W1, P, r, Z = diag(r) h W2 (W2t gamma-folded).  Returns (h, P, Z)."""
    lib = load_library()
    M, K = X.shape
    N, N2 = W1t.shape[0], W2t.shape[0]
    code = _dtype_code(X)
    H, P, Z = _block_outputs(X, R, N, N2, H, P, Z, code)
    _want_block(X, W1t, R, W2t, None, H, P, Z, r_out, workspace, N2, code, "Z", "W2t")
    _check(lib.coda_block_rowscale(_dev(X, "X"), _dev(W1t, "W1t"), _dev(R, "R"), _dev(W2t, "W2t"), float(eps),
                                   _dev(H, "H"), _dev(P, "P"), _dev(r_out, "r_out"), _dev(Z, "Z"), M, N, K, N2, code,
                                   _dev(workspace, "workspace"), _stream(X, stream)))
    return H, P, Z


def coda_block_rowscale_rope(X, W1t, R, W2t, eps: float, workspace, head_dim: int, rope_cols: int, base: float, *,
                             seq_len: int = 0, positions=None, H=None, P=None, Z=None, r_out=None, stream=None):
    """One launch: h = R + X W1, P, r, Z = RoPE(diag(r) h W2) on the first rope_cols columns.
    Positions: ``positions`` [M] int32, else row mod ``seq_len``.  Returns (h, P, Z)."""
    lib = load_library()
    M, K = X.shape
    N, N2 = W1t.shape[0], W2t.shape[0]
    code = _dtype_code(X)
    H, P, Z = _block_outputs(X, R, N, N2, H, P, Z, code)
    _want_block(X, W1t, R, W2t, None, H, P, Z, r_out, workspace, N2, code, "Z", "W2t")
    _want(positions, "positions", (M,), (torch.int32,))
    _check(lib.coda_block_rowscale_rope(_dev(X, "X"), _dev(W1t, "W1t"), _dev(R, "R"), _dev(W2t, "W2t"), float(eps),
                                        _dev(H, "H"), _dev(P, "P"), _dev(r_out, "r_out"), _dev(Z, "Z"), M, N, K, N2,
                                        code, head_dim, rope_cols, float(base), seq_len, _dev(positions, "positions"),
                                        _dev(workspace, "workspace"), _stream(X, stream)))
    return H, P, Z


def coda_block_swiglu(X, W1t, R, Wgt, Wut, eps: float, workspace, H=None, P=None, Act=None, r_out=None,
                      stream=None):
    """One launch: h = R + X W1, P, r, Act = silu(r h Wg) * (r h Wu).  Returns (h, P, Act)."""
    lib = load_library()
    M, K = X.shape
    N, I = W1t.shape[0], Wgt.shape[0]
    code = _dtype_code(X)
    H, P, Act = _block_outputs(X, R, N, I, H, P, Act, code)
    _want_block(X, W1t, R, Wgt, Wut, H, P, Act, r_out, workspace, I, code, "Act", "Wgt")
    _check(lib.coda_block_swiglu(_dev(X, "X"), _dev(W1t, "W1t"), _dev(R, "R"), _dev(Wgt, "Wgt"), _dev(Wut, "Wut"),
                                 float(eps), _dev(H, "H"), _dev(P, "P"), _dev(r_out, "r_out"), _dev(Act, "Act"), M, N,
                                 K, I, code, _dev(workspace, "workspace"), _stream(X, stream)))
    return H, P, Act


def coda_block_swiglu_noalloc(X, W1t, R, Wgt, Wut, eps: float, H=None, P=None, Act=None, r_out=None, stream=None):
    """coda_block_swiglu without a workspace, for callers that cannot allocate
    device memory (the library keeps the counters itself; M <= 131072; calls
    must not overlap on the GPU).  Returns (h, P, Act)."""
    lib = load_library()
    M, K = X.shape
    N, I = W1t.shape[0], Wgt.shape[0]
    code = _dtype_code(X)
    H, P, Act = _block_outputs(X, R, N, I, H, P, Act, code)
    _want_block(X, W1t, R, Wgt, Wut, H, P, Act, r_out, None, I, code, "Act", "Wgt")
    _check(lib.coda_block_swiglu_noalloc(_dev(X, "X"), _dev(W1t, "W1t"), _dev(R, "R"), _dev(Wgt, "Wgt"),
                                         _dev(Wut, "Wut"), float(eps), _dev(H, "H"), _dev(P, "P"), _dev(r_out, "r_out"),
                                         _dev(Act, "Act"), M, N, K, I, code, _stream(X, stream)))
    return H, P, Act


def coda_block_fp8_workspace_bytes(M: int) -> int:
    return int(load_library().coda_block_fp8_workspace_bytes(M))


def block_fp8_workspace(M: int, device) -> torch.Tensor:
    """A zeroed workspace for the FP8 one-launch blocks (calls leave it zeroed)."""
    n = coda_block_fp8_workspace_bytes(M)
    return torch.zeros((n + 3) // 4, dtype=torch.int32, device=device)


def _fp8_block_buffers(M, N, K, n_out, dev, A, Aq, scale_a, H, P, amax_h, Hq, scale_h, out):
    f32, bf, u8 = torch.float32, torch.bfloat16, torch.uint8
    e = lambda *shape, dt: torch.empty(*shape, dtype=dt, device=dev)  # noqa: E731
    if A is not None:  # the launch quantises A: it writes Aq and scale_a
        Aq = e(M, K, dt=u8) if Aq is None else Aq
        scale_a = e(1, dt=f32) if scale_a is None else scale_a
    elif Aq is None or scale_a is None:
        raise ValueError("without A, Aq and scale_a (the e4m3 operand and its scale) must be given")
    return (Aq, scale_a, e(M, N, dt=bf) if H is None else H,
            e(M, max(coda_partial_cols(N), 0), dt=f32) if P is None else P, e(1, dt=f32) if amax_h is None else amax_h,
            e(M, N, dt=u8) if Hq is None else Hq, e(1, dt=f32) if scale_h is None else scale_h,
            e(M, n_out, dt=bf) if out is None else out)


def coda_block_swiglu_fp8(A, amax_a, W1t, scale_w1, R, Wgt, scale_wg, Wut, scale_wu, eps: float, workspace,
                          Aq=None, scale_a=None, H=None, P=None, r_out=None, amax_h=None, Hq=None, scale_h=None,
                          Act=None, amax_act=None, M=None, stream=None):
    """FP8 one-launch block: [Aq = e4m3(A)], h = R + Aq W1, Hq = e4m3(h), Act =
    silu(r Hq Wg) * (r Hq Wu).  A (bf16) may be None when Aq and scale_a are
    given.  Returns a dict of the outputs (Aq, scale_a, h, P, amax_h, Hq,
    scale_h, act, amax_act)."""
    lib = load_library()
    src = A if A is not None else Aq
    M, K = src.shape
    N, I = W1t.shape[0], Wgt.shape[0]
    dev = src.device
    Aq, scale_a, H, P, amax_h, Hq, scale_h, Act = _fp8_block_buffers(M, N, K, I, dev, A, Aq, scale_a, H, P, amax_h,
                                                                      Hq, scale_h, Act)
    _want_fp8_block(A, amax_a, Aq, scale_a, W1t, scale_w1, R, Wgt, scale_wg, Wut, scale_wu, H, P, r_out, amax_h,
                    Hq, scale_h, Act, amax_act, workspace, M, N, K, I, "Act", "Wgt")
    _check(lib.coda_block_swiglu_fp8(_dev(A, "A"), _dev(amax_a, "amax_a"), _dev(Aq, "Aq"), _dev(scale_a, "scale_a"),
                                     _dev(W1t, "W1t"), _dev(scale_w1, "scale_w1"), _dev(R, "R"), _dev(Wgt, "Wgt"),
                                     _dev(scale_wg, "scale_wg"), _dev(Wut, "Wut"), _dev(scale_wu, "scale_wu"),
                                     float(eps), _dev(H, "H"), _dev(P, "P"), _dev(r_out, "r_out"),
                                     _dev(amax_h, "amax_h"), _dev(Hq, "Hq"), _dev(scale_h, "scale_h"), _dev(Act, "Act"),
                                     _dev(amax_act, "amax_act"), M, N, K, I, _dev(workspace, "workspace"),
                                     _stream(src, stream)))
    return {"Aq": Aq, "scale_a": scale_a, "h": H, "P": P, "amax_h": amax_h, "Hq": Hq, "scale_h": scale_h,
            "act": Act, "amax_act": amax_act}


def coda_block_rowscale_fp8(A, amax_a, W1t, scale_w1, R, W2t, scale_w2, eps: float, workspace, Aq=None,
                            scale_a=None, H=None, P=None, r_out=None, amax_h=None, Hq=None, scale_h=None, Z=None,
                            stream=None):
    """FP8 one-launch block: [Aq = e4m3(A)], h = R + Aq W1, Hq = e4m3(h), Z =
    diag(r) Hq W2.  Returns a dict of the outputs (Aq, scale_a, h, P, amax_h,
    Hq, scale_h, Z)."""
    lib = load_library()
    src = A if A is not None else Aq
    M, K = src.shape
    N, N2 = W1t.shape[0], W2t.shape[0]
    dev = src.device
    Aq, scale_a, H, P, amax_h, Hq, scale_h, Z = _fp8_block_buffers(M, N, K, N2, dev, A, Aq, scale_a, H, P, amax_h,
                                                                    Hq, scale_h, Z)
    _want_fp8_block(A, amax_a, Aq, scale_a, W1t, scale_w1, R, W2t, scale_w2, None, None, H, P, r_out, amax_h,
                    Hq, scale_h, Z, None, workspace, M, N, K, N2, "Z", "W2t")
    _check(lib.coda_block_rowscale_fp8(_dev(A, "A"), _dev(amax_a, "amax_a"), _dev(Aq, "Aq"), _dev(scale_a, "scale_a"),
                                       _dev(W1t, "W1t"), _dev(scale_w1, "scale_w1"), _dev(R, "R"), _dev(W2t, "W2t"),
                                       _dev(scale_w2, "scale_w2"), float(eps), _dev(H, "H"), _dev(P, "P"),
                                       _dev(r_out, "r_out"), _dev(amax_h, "amax_h"), _dev(Hq, "Hq"),
                                       _dev(scale_h, "scale_h"), _dev(Z, "Z"), M, N, K, N2,
                                       _dev(workspace, "workspace"), _stream(src, stream)))
    return {"Aq": Aq, "scale_a": scale_a, "h": H, "P": P, "amax_h": amax_h, "Hq": Hq, "scale_h": scale_h, "Z": Z}


# The decode, scoring and experts' calls are short on the GPU (a few microseconds), so a good call is marshalled in C
# (coda_marshal.c: the same checks, half the time); it hands back what it does not take, and the checks here say what
# is wrong.

def _pointers(specs):
    """Device pointers of (tensor or None, name, shape or None for one or more elements, dtype): contiguous CUDA tensors
    on the current device, checked by _want and _dev."""
    for t, name, shape, dtype in specs:
        _want(t, name, shape, (dtype,), numel=None if shape is not None else 1)
    return [_dev(t, name) for t, name, _, _ in specs]


def _stream_arg(stream):
    """A stream argument for the C marshalling: None (the current one) or its address."""
    return stream if stream is None else stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _done(status):
    """Whether the C marshalling made the call; raises if the library refused it."""
    if status is None:
        return False
    if status:
        _check(status)
    return True


def _cache_shape(k_cache, v_cache, dtype):
    """(num_pages, kv_heads, page_size, head_dim, cache dtype code) of a pair of caches for rows of `dtype`."""
    if k_cache.dim() != 4:
        raise ValueError(f"k_cache has {k_cache.dim()} dimensions, expected [num_pages, kv_heads, page_size, head_dim]")
    if k_cache.dtype is not dtype:
        _want(k_cache, "k_cache", dtypes=(dtype,) + (_BYTE if dtype == torch.bfloat16 else ()))
    return (*k_cache.shape, CODA_E4M3 if k_cache.dtype is not dtype else _dtype_code(k_cache))


def _table_shape(page_table):
    if page_table.dim() != 2:
        raise ValueError(f"page_table has {page_table.dim()} dimensions, expected [num_seqs, max_pages]")
    return page_table.shape


def _rows(t: torch.Tensor, name: str):
    """(device pointer, row stride in elements) of a CUDA matrix [M, N], or
    [M, heads, head_dim] with contiguous heads, whose rows may lie further
    apart than they are wide."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device})")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device} but the current device is cuda:{torch.cuda.current_device()}")
    shape, stride, inner = t.shape, t.stride(), 1
    for i in range(len(shape) - 1, 0, -1):
        if shape[i] != 1 and stride[i] != inner:
            raise ValueError(f"{name}'s rows must be contiguous")
        inner *= shape[i]
    return t.data_ptr() or None, stride[0] if shape[0] > 1 else inner


def coda_paged_append(Z, positions, page_table, k_cache, v_cache, q_heads: int, *, row_seq=None, base: float = 0.0,
                      Q=None, want_q: bool = True, scale_k=None, scale_v=None, stream=None):
    """Writes K (rotated) and V of the QKV rows Z [M, (q_heads + 2 kv_heads) head_dim] to the paged caches
    [num_pages, kv_heads, page_size, head_dim] (changed in place) at ``positions`` [M] int32 of the rows' sequences
    (``row_seq`` [M] int32, else row i is sequence i of ``page_table`` [num_seqs, max_pages] int32).  ``base`` 0: Z is
    already rotated.  Rows with a negative position are left out.  Returns the rotated queries [M, q_heads, head_dim],
    or None with ``want_q=False``."""
    lib = load_library()
    if Q is None and want_q and k_cache.dim() == 4:
        Q = torch.empty(Z.shape[0], q_heads, k_cache.shape[3], dtype=Z.dtype, device=Z.device)
    if _fast is not None and _done(_fast.paged_append(Z, positions, row_seq, page_table, Q, k_cache, v_cache, scale_k,
                                                      scale_v, q_heads, base, _stream_arg(stream))):
        return Q
    M, dt = Z.shape[0], Z.dtype
    code = _dtype_code(Z)
    pages, kv_heads, page_size, D, ccode = _cache_shape(k_cache, v_cache, dt)
    seqs, max_pages = _table_shape(page_table)
    ptr = _pointers(((Z, "Z", (M, (q_heads + 2 * kv_heads) * D), dt), (positions, "positions", (M,), torch.int32),
                     (row_seq, "row_seq", (M,), torch.int32), (page_table, "page_table", page_table.shape, torch.int32),
                     (Q, "Q", (M, q_heads, D), dt), (k_cache, "k_cache", k_cache.shape, k_cache.dtype),
                     (v_cache, "v_cache", k_cache.shape, k_cache.dtype), (scale_k, "scale_k", None, torch.float32),
                     (scale_v, "scale_v", None, torch.float32)))
    _check(lib.coda_paged_append(*ptr[:7], M, seqs, max_pages, q_heads, kv_heads, D, pages, page_size, base, code, ccode,
                                 ptr[7], ptr[8], _stream(Z, stream)))
    return Q


@functools.lru_cache(maxsize=None)
def coda_paged_attention_workspace_bytes(q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(load_library().coda_paged_attention_workspace_bytes(q_heads, kv_heads, head_dim))


def paged_attention_workspace(q_heads: int, kv_heads: int, head_dim: int, device) -> torch.Tensor:
    """A zeroed workspace for coda_paged_attention, for any number of rows (calls leave it ready for the next)."""
    n = coda_paged_attention_workspace_bytes(q_heads, kv_heads, head_dim)
    if n < 0:
        raise ValueError(f"q_heads = {q_heads}, kv_heads = {kv_heads}, head_dim = {head_dim} out of range")
    return torch.zeros((n + 3) // 4, dtype=torch.int32, device=device)


def coda_paged_attention(Q, k_cache, v_cache, page_table, lengths, workspace, *, row_seq=None, scale=None, O=None,
                         lse=None, scale_k=None, scale_v=None, stream=None):
    """o = softmax(scale q K^T) V of one new token per row over its sequence's first ``lengths`` [M] int32 cached
    keys.  Q [M, q_heads, head_dim], possibly a strided view of a QKV product's rows; caches, page_table and row_seq as
    for coda_paged_append; ``scale`` defaults to 1 / sqrt(head_dim); ``lse`` [M, q_heads] fp32 is written when given.
    Returns O [M, q_heads * head_dim]."""
    lib = load_library()
    if Q.dim() != 3:
        raise ValueError(f"Q has {Q.dim()} dimensions, expected [M, q_heads, head_dim]")
    M, q_heads, D = Q.shape
    scale = D ** -0.5 if scale is None else scale
    if O is None:
        O = torch.empty(M, q_heads * D, dtype=Q.dtype, device=Q.device)
    if _fast is not None and _done(_fast.paged_attention(Q, k_cache, v_cache, page_table, lengths, workspace, row_seq,
                                                         scale, O, lse, scale_k, scale_v, _stream_arg(stream))):
        return O
    dt, code = Q.dtype, _dtype_code(Q)
    pages, kv_heads, page_size, Dk, ccode = _cache_shape(k_cache, v_cache, dt)
    if Dk != D:
        raise ValueError(f"Q has head_dim {D}, the caches {Dk}")
    seqs, max_pages = _table_shape(page_table)
    _want(workspace, "workspace", nbytes=coda_paged_attention_workspace_bytes(q_heads, kv_heads, D))
    ptr = _pointers(((O, "O", (M, q_heads * D), dt), (k_cache, "k_cache", k_cache.shape, k_cache.dtype),
                     (v_cache, "v_cache", k_cache.shape, k_cache.dtype),
                     (page_table, "page_table", page_table.shape, torch.int32), (lengths, "lengths", (M,), torch.int32),
                     (row_seq, "row_seq", (M,), torch.int32), (lse, "lse", (M, q_heads), torch.float32),
                     (scale_k, "scale_k", None, torch.float32), (scale_v, "scale_v", None, torch.float32),
                     (workspace, "workspace", workspace.shape, workspace.dtype)))
    q_ptr, ldq = _rows(Q, "Q")
    _check(lib.coda_paged_attention(q_ptr, ldq, *ptr[1:6], ptr[0], ptr[6], M, seqs, max_pages, q_heads, kv_heads, D,
                                    pages, page_size, scale, code, ccode, ptr[7],
                                    ptr[8], ptr[9], _stream(Q, stream)))
    return O


def _logits_rows(t, name):
    """(pointer, row stride) of a logits matrix [M, V]; a single row's stride is rounded up to whole 16 bytes."""
    ptr, ld = _rows(t, name)
    if t.shape[0] <= 1:
        step = 16 // t.element_size()
        ld = -(-t.shape[1] // step) * step
    return ptr, ld


def coda_logprobs(logits, targets, top: int = 0, *, logp=None, entropy=None, lse=None, top_logp=None, top_ids=None,
                  stream=None):
    """Log probabilities of ``targets`` [M] int32 (negative: not scored) under softmax of ``logits`` [M, V] (rows may be
    a strided view), with entropy, lse and the ``top`` best alternatives.  Returns a dict (logp, entropy, lse [M] fp32;
    with top > 0 top_logp [M, top] fp32 and top_ids [M, top] int32)."""
    lib = load_library()
    if logits.dim() != 2:
        raise ValueError(f"logits has {logits.dim()} dimensions, expected [M, V]")
    M, V = logits.shape
    f32, e = torch.float32, lambda *shape, dt=torch.float32: torch.empty(*shape, dtype=dt, device=logits.device)
    out = {"logp": e(M) if logp is None else logp, "entropy": e(M) if entropy is None else entropy,
           "lse": e(M) if lse is None else lse}
    if top > 0:
        top_logp = out["top_logp"] = e(M, top) if top_logp is None else top_logp
        top_ids = out["top_ids"] = e(M, top, dt=torch.int32) if top_ids is None else top_ids
    else:
        top_logp = top_ids = None
    if _fast is not None and _done(_fast.logprobs(logits, targets, top, out["logp"], out["entropy"], out["lse"],
                                                  top_logp, top_ids, _stream_arg(stream))):
        return out
    _want(logits, "logits", dtypes=(torch.float32, torch.bfloat16))
    ptr = _pointers(((targets, "targets", (M,), torch.int32), (out["logp"], "logp", (M,), f32),
                     (out["entropy"], "entropy", (M,), f32), (out["lse"], "lse", (M,), f32),
                     (top_logp, "top_logp", (M, top), f32), (top_ids, "top_ids", (M, top), torch.int32)))
    row, ld = _logits_rows(logits, "logits")
    _check(lib.coda_logprobs(row, ld, *ptr, M, V, top, _dtype_code(logits), _stream(logits, stream)))
    return out


def coda_logprobs_backward(logits, targets, lse, entropy=None, dlogp=None, dentropy=None, dlogits=None, stream=None):
    """dlogits = dlogp ([j = t] - p) - dentropy p (log p + entropy), from coda_logprobs' lse and entropy; dlogp and
    dentropy [M] fp32 may be None (= 0).  ``dlogits`` [M, V] may be a strided view.  Returns dlogits."""
    lib = load_library()
    if logits.dim() != 2:
        raise ValueError(f"logits has {logits.dim()} dimensions, expected [M, V]")
    M, V = logits.shape
    if dlogits is None:  # rows on 16-byte boundaries, as the logits' own
        step = 16 // logits.element_size()
        dlogits = torch.empty(M, -(-V // step) * step, dtype=logits.dtype, device=logits.device)[:, :V]
    if _fast is not None and _done(_fast.logprobs_backward(logits, targets, lse, entropy, dlogp, dentropy, dlogits,
                                                           _stream_arg(stream))):
        return dlogits
    f32 = torch.float32
    _want(logits, "logits", dtypes=(f32, torch.bfloat16))
    _want(dlogits, "dlogits", (M, V), (logits.dtype,))
    ptr = _pointers(((targets, "targets", (M,), torch.int32), (lse, "lse", (M,), f32), (entropy, "entropy", (M,), f32),
                     (dlogp, "dlogp", (M,), f32), (dentropy, "dentropy", (M,), f32)))
    row, ld = _logits_rows(logits, "logits")
    drow, ldd = _logits_rows(dlogits, "dlogits")
    _check(lib.coda_logprobs_backward(row, ld, *ptr, drow, ldd, M, V, _dtype_code(logits), _stream(logits, stream)))
    return dlogits


# ------------------------------------------------------ mixture of experts ----

_REAL = (torch.float32, torch.bfloat16)


def _alloc(t, shape, dtype, like):
    return torch.empty(shape, dtype=dtype, device=like.device) if t is None else t


def _matrix(t, name, dims=2):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} has {t.dim()} dimensions, expected {dims}")
    return t.shape


def coda_add_rmsnorm(X, gamma, eps: float, R=None, *, H=None, Y=None, Yq=None, scale=None, r=None,
                     want_y: Optional[bool] = None, want_q: bool = False, stream=None):
    """h = X + R, r = 1 / sqrt(mean h^2 + eps), y = h r gamma, in X's type (``want_y`` or a given ``Y``), in e4m3 with a
    scale for each row (``want_q`` or a given ``Yq``), or both; without ``want_y``, y is wanted unless a ``Yq`` is given.
    X and R [M, N] may be strided views of rows.  Returns a dict: h (X itself without R, unless ``H`` is given), y, q,
    scale [M] (with q alone), r [M]; what was not asked for is None."""
    lib = load_library()
    if Y is None and (Yq is None if want_y is None else want_y):
        Y = torch.empty(_matrix(X, "X"), dtype=X.dtype, device=X.device)
    if Yq is None and want_q:
        Yq = torch.empty(_matrix(X, "X"), dtype=torch.uint8, device=X.device)
    if Yq is None:
        scale = None  # it is written with the codes alone
    elif scale is None:
        scale = torch.empty(_matrix(X, "X")[0], dtype=torch.float32, device=X.device)
    if H is None and R is not None:
        H = torch.empty(_matrix(X, "X"), dtype=X.dtype, device=X.device)
    if r is None:
        r = torch.empty(_matrix(X, "X")[0], dtype=torch.float32, device=X.device)
    out = {"h": X if H is None else H, "y": Y, "q": Yq, "scale": scale, "r": r}
    if _fast is not None and _done(_fast.add_rmsnorm(X, R, gamma, H, Y, Yq, scale, r, eps, _stream_arg(stream))):
        return out
    M, N = _matrix(X, "X")
    _want(X, "X", dtypes=_REAL)
    _want(R, "R", (M, N), (X.dtype,))
    _want(H, "H", (M, N), (X.dtype,))
    _want(Y, "Y", (M, N), (X.dtype,))
    _want(Yq, "Yq", (M, N), _BYTE)
    _want(gamma, "gamma", (N,), _F32)
    _want(scale, "scale", (M,), _F32)
    _want(r, "r", (M,), _F32)
    x, ldx = _logits_rows(X, "X")
    res, ldr = (None, 0) if R is None else _logits_rows(R, "R")
    _check(lib.coda_add_rmsnorm(x, ldx, res, ldr, _dev(gamma, "gamma"), float(eps), _dev(H, "H"), _dev(Y, "Y"),
                                _dev(Yq, "Yq"), _dev(scale, "scale"), _dev(r, "r"), M, N, _dtype_code(X),
                                _stream(X, stream)))
    return out


def coda_quantize_rows_e4m3(X, q=None, scale=None, stream=None):
    """q = e4m3(X / s) with a scale s = max |x| / 448 for each row of X [M, N] (possibly a strided view of rows).
    Returns (q as uint8, scale [M])."""
    lib = load_library()
    M, N = _matrix(X, "X")
    q = _alloc(q, (M, N), torch.uint8, X)
    scale = _alloc(scale, (M,), torch.float32, X)
    if _fast is not None and _done(_fast.quantize_rows(X, q, scale, _stream_arg(stream))):
        return q, scale
    _want(X, "X", dtypes=_REAL)
    _want(q, "q", (M, N), _BYTE)
    _want(scale, "scale", (M,), _F32)
    x, ldx = _logits_rows(X, "X")
    _check(lib.coda_quantize_rows_e4m3(x, ldx, _dev(q, "q"), _dev(scale, "scale"), M, N, _dtype_code(X),
                                       _stream(X, stream)))
    return q, scale


def _workspace(nbytes, what, device):
    if nbytes < 0:
        raise ValueError(f"{what} out of range")
    return torch.empty(max(nbytes, 4) // 4, dtype=torch.float32, device=device)


def add_rmsnorm_backward_workspace(M: int, N: int, device) -> torch.Tensor:
    """A workspace for coda_add_rmsnorm_backward on [M, N] (any contents)."""
    return _workspace(int(load_library().coda_add_rmsnorm_backward_workspace_bytes(M, N)), f"M = {M}, N = {N}", device)


def coda_add_rmsnorm_backward(dY, H, r, gamma, dH_in=None, *, dH=None, dgamma=None, workspace=None, stream=None):
    """Gradient of coda_add_rmsnorm from its h and r: dH = r gamma dY - (r^3 / N) (sum gamma dY h) h + dH_in (the
    gradient of X and of R), dgamma [N].  Returns (dH, dgamma)."""
    lib = load_library()
    M, N = _matrix(H, "H")
    dH = _alloc(dH, (M, N), H.dtype, H)
    dgamma = _alloc(dgamma, (N,), torch.float32, H)
    if workspace is None:
        workspace = _made_on(stream, H.device, lambda: add_rmsnorm_backward_workspace(M, N, H.device))
    if _fast is not None and _done(_fast.add_rmsnorm_backward(dY, H, r, gamma, dH_in, dH, dgamma, workspace,
                                                              _stream_arg(stream))):
        return dH, dgamma
    _want(H, "H", dtypes=_REAL)
    _want(dY, "dY", (M, N), (H.dtype,))
    _want(dH_in, "dH_in", (M, N), (H.dtype,))
    _want(dH, "dH", (M, N), (H.dtype,))
    _want(r, "r", (M,), _F32)
    _want(gamma, "gamma", (N,), _F32)
    _want(dgamma, "dgamma", (N,), _F32)
    _want(workspace, "workspace", nbytes=int(lib.coda_add_rmsnorm_backward_workspace_bytes(M, N)))
    _check(lib.coda_add_rmsnorm_backward(_dev(dY, "dY"), _dev(H, "H"), _dev(r, "r"), _dev(gamma, "gamma"),
                                         _dev(dH_in, "dH_in"), _dev(dH, "dH"), _dev(dgamma, "dgamma"),
                                         _dev(workspace, "workspace"), M, N, _dtype_code(H), _stream(H, stream)))
    return dH, dgamma


def route_workspace(M: int, E: int, top_k: int, device) -> torch.Tensor:
    """A workspace for coda_route of M rows (any contents)."""
    return _workspace(int(load_library().coda_route_workspace_bytes(M, E, top_k)), f"M = {M}, E = {E}, top_k = {top_k}",
                      device)


def coda_route(logits, top_k: int, *, renormalize: bool = True, ids=None, weights=None, slots=None, offsets=None,
               workspace=None, stream=None):
    """The ``top_k`` largest of each row of ``logits`` [M, E] (rows may be a strided view; -inf is never chosen) and
    where the (row, choice) pairs lie when they are sorted by expert.  Returns a dict: ids [M, top_k] int32 (-1: none
    left), weights [M, top_k] fp32 (softmax over the chosen, or with ``renormalize=False`` over all experts), slots
    [M, top_k] int32, offsets [E + 1] int32."""
    lib = load_library()
    M, E = _matrix(logits, "logits")
    ids = _alloc(ids, (M, top_k), torch.int32, logits)
    weights = _alloc(weights, (M, top_k), torch.float32, logits)
    slots = _alloc(slots, (M, top_k), torch.int32, logits)
    offsets = _alloc(offsets, (E + 1,), torch.int32, logits)
    out = {"ids": ids, "weights": weights, "slots": slots, "offsets": offsets}
    if workspace is None:
        workspace = _made_on(stream, logits.device, lambda: route_workspace(M, E, top_k, logits.device))
    if _fast is not None and _done(_fast.route(logits, ids, weights, slots, offsets, workspace, top_k, renormalize,
                                               _stream_arg(stream))):
        return out
    _want(logits, "logits", dtypes=_REAL)
    _want(workspace, "workspace", nbytes=int(lib.coda_route_workspace_bytes(M, E, top_k)))
    ptr = _pointers(((ids, "ids", (M, top_k), torch.int32), (weights, "weights", (M, top_k), torch.float32),
                     (slots, "slots", (M, top_k), torch.int32), (offsets, "offsets", (E + 1,), torch.int32)))
    row, ld = _logits_rows(logits, "logits")
    _check(lib.coda_route(row, ld, top_k, int(renormalize), *ptr, _dev(workspace, "workspace"), M, E,
                          _dtype_code(logits), _stream(logits, stream)))
    return out


def coda_route_backward(logits, ids, weights, dweights, *, renormalize: bool = True, dlogits=None, stream=None):
    """dlogits [M, E] from the gradient of coda_route's weights (``renormalize`` as there).  Returns dlogits."""
    lib = load_library()
    M, E = _matrix(logits, "logits")
    k = _matrix(ids, "ids")[1]
    if dlogits is None:  # rows on 16-byte boundaries, as the logits' own
        step = 16 // logits.element_size()
        dlogits = torch.empty(M, -(-E // step) * step, dtype=logits.dtype, device=logits.device)[:, :E]
    if _fast is not None and _done(_fast.route_backward(logits, dlogits, ids, weights, dweights, renormalize,
                                                        _stream_arg(stream))):
        return dlogits
    _want(logits, "logits", dtypes=_REAL)
    _want(dlogits, "dlogits", (M, E), (logits.dtype,))
    ptr = _pointers(((ids, "ids", (M, k), torch.int32), (weights, "weights", (M, k), torch.float32),
                     (dweights, "dweights", (M, k), torch.float32)))
    row, ld = _logits_rows(logits, "logits")
    drow, ldd = _logits_rows(dlogits, "dlogits")
    _check(lib.coda_route_backward(row, ld, *ptr, int(renormalize), drow, ldd, M, E, k, _dtype_code(logits),
                                   _stream(logits, stream)))
    return dlogits


def coda_expert_dispatch(X, slots, *, scale=None, Xs=None, scale_s=None, T: Optional[int] = None, stream=None):
    """Xs[slots[i, j]] = X[i] for X [M, N] (fp32, bf16 or e4m3 bytes), and scale_s[slots[i, j]] = scale[i] when ``scale``
    [M] is given.  ``T``: rows of Xs, M top_k unless given (or Xs is).  Returns (Xs [T, N], scale_s [T], or None without
    ``scale``: a given ``scale_s`` is then left as it is)."""
    lib = load_library()
    M, N = _matrix(X, "X")
    k = _matrix(slots, "slots")[1]
    if Xs is not None:
        T = _matrix(Xs, "Xs")[0]
    elif T is None:
        T = M * k
    Xs = _alloc(Xs, (T, N), X.dtype, X)
    scale_s = None if scale is None else _alloc(scale_s, (T,), torch.float32, X)  # without scale it is not written
    if _fast is not None and _done(_fast.expert_dispatch(X, slots, scale, Xs, scale_s, _stream_arg(stream))):
        return Xs, scale_s
    code = _dtype_code(X)
    _want(Xs, "Xs", (T, N), _operand_dtypes(code))
    _want(slots, "slots", (M, k), (torch.int32,))
    _want(scale, "scale", (M,), _F32)
    _want(scale_s, "scale_s", (T,), _F32)
    _check(lib.coda_expert_dispatch(_dev(X, "X"), _dev(scale, "scale"), _dev(slots, "slots"), _dev(Xs, "Xs"),
                                    _dev(scale_s, "scale_s"), M, N, k, T, code, _stream(X, stream)))
    return Xs, scale_s


def coda_expert_combine(Y, slots, weights=None, R=None, *, H=None, P=None, want_p: bool = False, stream=None):
    """H[i] = R[i] + sum_j weights[i, j] Y[slots[i, j]] for Y [T, N]; with ``want_p`` (or a given ``P``) also the stored
    rows' partial sums of squares, as coda_gemm_residual_partial_rms writes them.  R and weights may be None (0 and 1).
    Returns (H [M, N], P or None)."""
    lib = load_library()
    T, N = _matrix(Y, "Y")
    M, k = _matrix(slots, "slots")
    H = _alloc(H, (M, N), Y.dtype, Y)
    T_p = -(-N // 128)  # coda_partial_cols(N)
    if want_p:
        P = _alloc(P, (M, T_p), torch.float32, Y)
    if _fast is not None and _done(_fast.expert_combine(Y, slots, weights, R, H, P, _stream_arg(stream))):
        return H, P
    _want(Y, "Y", dtypes=_REAL)
    _want(slots, "slots", (M, k), (torch.int32,))
    _want(weights, "weights", (M, k), _F32)
    _want(R, "R", (M, N), (Y.dtype,))
    _want(H, "H", (M, N), (Y.dtype,))
    _want(P, "P", (M, T_p), _F32)
    _check(lib.coda_expert_combine(_dev(Y, "Y"), _dev(slots, "slots"), _dev(weights, "weights"), _dev(R, "R"),
                                   _dev(H, "H"), _dev(P, "P"), M, N, k, T, _dtype_code(Y), _stream(Y, stream)))
    return H, P


def coda_expert_combine_backward(dH, Y, slots, weights, *, dY=None, dweights=None, stream=None):
    """Gradient of coda_expert_combine: dY[slots[i, j]] = weights[i, j] dH[i] and dweights[i, j] = <dH[i],
    Y[slots[i, j]]>.  Returns (dY [T, N], dweights [M, top_k])."""
    lib = load_library()
    T, N = _matrix(Y, "Y")
    M, k = _matrix(slots, "slots")
    dY = _alloc(dY, (T, N), Y.dtype, Y)
    dweights = _alloc(dweights, (M, k), torch.float32, Y)
    if _fast is not None and _done(_fast.expert_combine_backward(dH, Y, slots, weights, dY, dweights,
                                                                 _stream_arg(stream))):
        return dY, dweights
    _want(Y, "Y", dtypes=_REAL)
    _want(dH, "dH", (M, N), (Y.dtype,))
    _want(slots, "slots", (M, k), (torch.int32,))
    _want(weights, "weights", (M, k), _F32)
    _want(dY, "dY", (T, N), (Y.dtype,))
    _want(dweights, "dweights", (M, k), _F32)
    _check(lib.coda_expert_combine_backward(_dev(dH, "dH"), _dev(Y, "Y"), _dev(slots, "slots"),
                                            _dev(weights, "weights"), _dev(dY, "dY"), _dev(dweights, "dweights"), M, N,
                                            k, T, _dtype_code(Y), _stream(Y, stream)))
    return dY, dweights


def _want_group(X, W, w_name, w_shape, offsets, E, row_scale, w_scale, code):
    _want(X, "X", dtypes=(torch.bfloat16,) + _BYTE)
    _want(W, w_name, w_shape, _operand_dtypes(code))
    _want(offsets, "offsets", (E + 1,), (torch.int32,))
    _want(row_scale, "row_scale", (X.shape[0],), _F32)
    _want(w_scale, "w_scale", (E,), _F32)


def coda_grouped_gemm(X, W, offsets, *, b_mn: bool = False, row_scale=None, w_scale=None, Y=None, stream=None):
    """Y[t] = s_t X[t] W_e for the rows t in [offsets[e], offsets[e + 1]) of X [T, K]; W [E, N, K], or [E, K, N] with
    ``b_mn`` (bf16).  s_t = row_scale[t] w_scale[e]: both for e4m3 operands, an optional row_scale for bf16.  Rows of no
    expert are left as they are.  Returns Y [T, N] bf16."""
    lib = load_library()
    T, K = _matrix(X, "X")
    E = _matrix(W, "W", 3)[0]
    N = W.shape[2] if b_mn else W.shape[1]
    code = _dtype_code(X)
    Y = _alloc(Y, (T, N), torch.bfloat16, X)
    if _fast is not None and _done(_fast.grouped_gemm(X, W, offsets, row_scale, w_scale, Y, b_mn,
                                                      _stream_arg(stream))):
        return Y
    _want_group(X, W, "W", (E, K, N) if b_mn else (E, N, K), offsets, E, row_scale, w_scale, code)
    _want(Y, "Y", (T, N), (torch.bfloat16,))
    _check(lib.coda_grouped_gemm(_dev(X, "X"), _dev(W, "W"), CODA_MN_MAJOR if b_mn else CODA_K_MAJOR,
                                 _dev(offsets, "offsets"), _dev(row_scale, "row_scale"), _dev(w_scale, "w_scale"),
                                 _dev(Y, "Y"), T, E, N, K, code, _stream(X, stream)))
    return Y


def coda_grouped_gemm_swiglu(X, Wgu, offsets, *, row_scale=None, w_scale=None, Act=None, GU=None, save: bool = False,
                             stream=None):
    """Act[t] = silu(s_t X[t] Wg_e) * (s_t X[t] Wu_e) for Wgu [E, 2 I, K] (gate rows, then up rows); scales as for
    coda_grouped_gemm.  With ``save`` (or a given ``GU``) the pre-activations G || U [T, 2 I] are stored too.  Returns
    (Act [T, I] bf16, GU or None)."""
    lib = load_library()
    T, K = _matrix(X, "X")
    E, two_i, _ = _matrix(Wgu, "Wgu", 3)
    if two_i % 2:
        raise ValueError(f"Wgu has {two_i} rows an expert, expected gate rows and as many up rows")
    I, code = two_i // 2, _dtype_code(X)
    Act = _alloc(Act, (T, I), torch.bfloat16, X)
    if save:
        GU = _alloc(GU, (T, 2 * I), torch.bfloat16, X)
    if _fast is not None and _done(_fast.grouped_swiglu(X, Wgu, offsets, row_scale, w_scale, Act, GU,
                                                        _stream_arg(stream))):
        return Act, GU
    _want_group(X, Wgu, "Wgu", (E, 2 * I, K), offsets, E, row_scale, w_scale, code)
    _want(Act, "Act", (T, I), (torch.bfloat16,))
    _want(GU, "GU", (T, 2 * I), (torch.bfloat16,))
    _check(lib.coda_grouped_gemm_swiglu(_dev(X, "X"), _dev(Wgu, "Wgu"), _dev(offsets, "offsets"),
                                        _dev(row_scale, "row_scale"), _dev(w_scale, "w_scale"), _dev(Act, "Act"),
                                        _dev(GU, "GU"), T, E, I, K, code, _stream(X, stream)))
    return Act, GU


def coda_grouped_gemm_swiglu_backward(dY, Wd, GU, offsets, dGU=None, stream=None):
    """dG || dU [T, 2 I] from dAct = dY Wd_e (dY [T, K], Wd [E, K, I]) and the saved G || U.  Returns dGU."""
    lib = load_library()
    T, K = _matrix(dY, "dY")
    E, _, I = _matrix(Wd, "Wd", 3)
    bf = (torch.bfloat16,)
    dGU = _alloc(dGU, (T, 2 * I), torch.bfloat16, dY)
    if _fast is not None and _done(_fast.grouped_swiglu_backward(dY, Wd, GU, offsets, dGU, _stream_arg(stream))):
        return dGU
    _want(dY, "dY", dtypes=bf)
    _want(Wd, "Wd", (E, K, I), bf)
    _want(GU, "GU", (T, 2 * I), bf)
    _want(offsets, "offsets", (E + 1,), (torch.int32,))
    _want(dGU, "dGU", (T, 2 * I), bf)
    _check(lib.coda_grouped_gemm_swiglu_backward(_dev(dY, "dY"), _dev(Wd, "Wd"), _dev(GU, "GU"),
                                                 _dev(offsets, "offsets"), _dev(dGU, "dGU"), T, E, I, K, CODA_BF16,
                                                 _stream(dY, stream)))
    return dGU


def coda_grouped_gemm_wgrad(dY, X, offsets, dW=None, stream=None):
    """dW[e] = dY[rows of e]^T X[rows of e] for dY [T, N] and X [T, K] (bf16).  Returns dW [E, N, K]."""
    lib = load_library()
    T, N = _matrix(dY, "dY")
    K = _matrix(X, "X")[1]
    E = _matrix(offsets, "offsets", 1)[0] - 1
    bf = (torch.bfloat16,)
    dW = _alloc(dW, (E, N, K), torch.bfloat16, dY)
    if _fast is not None and _done(_fast.grouped_wgrad(dY, X, offsets, dW, _stream_arg(stream))):
        return dW
    _want(dY, "dY", dtypes=bf)
    _want(X, "X", (T, K), bf)
    _want(offsets, "offsets", (E + 1,), (torch.int32,))
    _want(dW, "dW", (E, N, K), bf)
    _check(lib.coda_grouped_gemm_wgrad(_dev(dY, "dY"), _dev(X, "X"), _dev(offsets, "offsets"), _dev(dW, "dW"), T, E, N,
                                       K, CODA_BF16, _stream(dY, stream)))
    return dW


def coda_amax(x, amax=None, stream=None):
    """amax = max |x| (fp32 scalar tensor)."""
    lib = load_library()
    if amax is None:
        amax = torch.empty(1, dtype=torch.float32, device=x.device)
    _want(x, "x", dtypes=(torch.float32, torch.bfloat16))
    _want(amax, "amax", dtypes=_F32, numel=1)
    _check(lib.coda_amax(_dev(x, "x"), x.numel(), _dtype_code(x), _dev(amax, "amax"), _stream(x, stream)))
    return amax


def coda_quantize_e4m3(x, amax, q=None, scale=None, stream=None):
    """q = e4m3(x / s) with s = amax / 448; returns (q as uint8, s)."""
    lib = load_library()
    if q is None:
        q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    if scale is None:
        scale = torch.empty(1, dtype=torch.float32, device=x.device)
    _want(x, "x", dtypes=(torch.float32, torch.bfloat16))
    _want(amax, "amax", dtypes=_F32, numel=1)
    _want(q, "q", dtypes=_BYTE, numel=x.numel())
    _want(scale, "scale", dtypes=_F32, numel=1)
    _check(lib.coda_quantize_e4m3(_dev(x, "x"), x.numel(), _dtype_code(x), _dev(amax, "amax"), _dev(q, "q"),
                                  _dev(scale, "scale"), _stream(x, stream)))
    return q, scale


def coda_selftest_wait_timeout(timeout_ns: int, stream=None):
    """Enqueue the failure-path self-test: a bounded wait on an mbarrier that
    nothing signals gives up after timeout_ns and raises the timeout bit, so
    the next coda_get_device_status() raises CodaError(CODA_ERR_TIMEOUT)."""
    lib = load_library()
    if stream is None:
        stream = torch.cuda.current_stream()
    s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    _check(lib.coda_selftest_wait_timeout(int(timeout_ns), s))


def coda_get_device_status() -> int:
    """Synchronise and read/clear the device status words; raises CodaError on a timeout or (next) a bad index."""
    st = load_library().coda_get_device_status()
    _check(st)
    return st
