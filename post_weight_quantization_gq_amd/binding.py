"""Python binding of libgq.so (C ABI in include/gq.h).

Argument marshalling only: torch tensors supply device memory and the HIP
stream; every step of the computation runs in the library's kernels.  Each
function has the name of the C entry point it calls.  A non-OK status raises
GQError(status, message).  If the built library is missing, loading raises.
GQ_LIBRARY=<path> loads another build of the same library instead (for instance the
host-sanitized libgq_asan.so, see build.py).
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_LIB_PATH = os.environ.get("GQ_LIBRARY") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "_lib", "libgq.so")

GQ_OK, GQ_EINVAL, GQ_ESHAPE, GQ_EDTYPE, GQ_ENOMEM, GQ_EHIP = 0, 1, 2, 3, 4, 5
GQ_ENOTPD, GQ_ENONFINITE, GQ_ENOTIMPL, GQ_ECHECK = 6, 7, 8, 9
GQ_F32, GQ_BF16 = 0, 1
GQ_INIT_QUANTILE, GQ_INIT_GIVEN, GQ_INIT_UNIFORM = 0, 1, 2
GQ_GRAM_AUTO, GQ_GRAM_DENSE = 0, 1
GQ_FISHER_CHECK_FINITE = 2
ABI_VERSION = 8
DEFAULT_BLOCK = 512

# every symbol include/gq.h declares
EXPORTS = (
    "gq_abi_version", "gq_last_error", "gq_lnq_options_default", "lnq_options_default",
    "gq_fisher_workspace_size", "gq_fisher_accumulate", "gq_lnq_workspace_size",
    "lnq_workspace_size", "lnq_codebook_update", "lnq_assign_sweep",
    "lnq_objective", "lnq_quantize", "lnq_quantize_static", "lnq_static_scratch_bytes",
    "grid_quantize", "lut_packed_row_words", "lut_pack_codes",
    "lut_gemv", "gq_fisher_stream_workspace_size", "gq_fisher_accumulate_host",
    "ganq_workspace_size", "ganq_quantize", "ganq_factor_damped",
    "mxfp4_row_bytes", "mxfp4_row_scales", "mxfp4_quantize", "mxfp4_dequantize",
    "mxfp4_gemm_workspace_size", "mxfp4_gemm", "mxfp4_gemm_mx_workspace_size", "mxfp4_gemm_mx",
    "mxfp4_gemm_dx_workspace_size", "mxfp4_gemm_dx", "mxfp4_plan",
    "gq_timing_enable", "gq_timing_read", "gq_timing_read_mxfp4", "gq_stage_name",
)
STAGE_COUNT, MXFP4_STAGE_COUNT = 18, 2


class GQError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"libgq status {status}: {message}")
        self.status = status
        self.message = message


class lnq_options(ctypes.Structure):
    """gq_lnq_options (block, ridge_rel, init, gram_update, ridge_abs, check_finite,
    check_residual)."""
    _fields_ = [("block", ctypes.c_int32), ("ridge_rel", ctypes.c_float),
                ("init", ctypes.c_int32), ("gram_update", ctypes.c_int32),
                ("ridge_abs", ctypes.c_float), ("check_finite", ctypes.c_int32),
                ("check_residual", ctypes.c_int32)]


_vp, _i32, _i64, _sz, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float

_SIGS = {
    "gq_abi_version": (ctypes.c_int, []),
    "gq_last_error": (ctypes.c_char_p, []),
    "gq_lnq_options_default": (None, [ctypes.POINTER(lnq_options)]),
    "lnq_options_default": (None, [ctypes.POINTER(lnq_options)]),
    "gq_fisher_workspace_size": (_sz, [_i64, _i64, _i64, _i32, _i32]),
    "gq_fisher_accumulate": (ctypes.c_int, [_vp, _i32, _i64, _i64, _vp, _i32, _i64, _i32, _vp,
                                            _i32, _vp, _sz, _vp]),
    "gq_lnq_workspace_size": (_sz, [_i64, _i64, _i32, _i32, _i32]),
    "lnq_workspace_size": (_sz, [_i64, _i64, _i32, _i32, _i32]),
    "lnq_codebook_update": (ctypes.c_int, [_vp, _i32, _i64, _vp, _i32, _i64, _vp, _i32, _vp, _f32,
                                           _vp, _vp, _sz, _vp]),
    "lnq_assign_sweep": (ctypes.c_int, [_vp, _i32, _i64, _vp, _i32, _i64, _vp, _i32, _vp, _f32,
                                        _i32, _vp, _vp, _sz, _vp]),
    "lnq_objective": (ctypes.c_int, [_vp, _i32, _i64, _vp, _i32, _i64, _vp, _vp, _i32, _f32, _vp,
                                     _vp, _vp, _sz, _vp]),
    "lnq_quantize": (ctypes.c_int, [_vp, _i32, _i64, _i64, _vp, _i32, _i32, _i32,
                                    ctypes.POINTER(lnq_options), _vp, _vp, _vp, _vp, _vp, _sz,
                                    _vp]),
    "lnq_quantize_static": (ctypes.c_int, [_vp, _i32, _i64, _i64, _vp, _i32, _i32, _i32,
                                           ctypes.POINTER(lnq_options), _vp, _vp, _vp, _vp,
                                           _vp]),
    "lnq_static_scratch_bytes": (_sz, []),
    "grid_quantize": (ctypes.c_int, [_vp, _i32, _i64, _i64, _vp, _i32, _i32, _i32,
                                     ctypes.POINTER(lnq_options), _vp, _vp, _vp, _vp, _vp, _sz,
                                     _vp]),
    "lut_packed_row_words": (_i64, [_i64, _i32]),
    "lut_pack_codes": (ctypes.c_int, [_vp, _i64, _i64, _i32, _vp, _vp]),
    "lut_gemv": (ctypes.c_int, [_vp, _vp, _i64, _i64, _i32, _vp, _i32, _i32, _vp, _vp]),
    "gq_fisher_stream_workspace_size": (_sz, [_i64, _i64, _i64, _i32, _i32]),
    "gq_fisher_accumulate_host": (ctypes.c_int, [_vp, _i32, _i64, _i64, _vp, _i32, _i64, _i32,
                                                 _vp, _i32, _i64, _vp, _sz, _vp]),
    "ganq_workspace_size": (_sz, [_i64, _i64, _i32, _i32, _i32]),
    "ganq_quantize": (ctypes.c_int, [_vp, _i32, _i64, _i64, _vp, _i32, _i32, _i32,
                                     ctypes.POINTER(lnq_options), _vp, _vp, _vp, _vp, _vp, _vp,
                                     _sz, _vp]),
    "ganq_factor_damped": (ctypes.c_int, [_vp, _i32, _i64, _f32, _vp, _vp, _vp, _sz, _vp]),
    "mxfp4_row_bytes": (_i64, [_i64]),
    "mxfp4_row_scales": (_i64, [_i64]),
    "mxfp4_quantize": (ctypes.c_int, [_vp, _i32, _i64, _i64, _vp, _vp, _vp]),
    "mxfp4_dequantize": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _i32, _vp]),
    "mxfp4_gemm_workspace_size": (_sz, [_i64, _i64, _i64, _i32, _i32]),
    "mxfp4_gemm": (ctypes.c_int, [_vp, _i32, _i64, _i64, _vp, _vp, _i64, _i32, _vp, _vp, _i32,
                                  _vp, _sz, _vp]),
    "mxfp4_gemm_mx_workspace_size": (_sz, [_i64, _i64, _i64, _i32]),
    "mxfp4_gemm_mx": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _i32, _vp, _vp, _i32,
                                     _vp, _sz, _vp]),
    "mxfp4_gemm_dx_workspace_size": (_sz, [_i64, _i64, _i64, _i32, _i32]),
    "mxfp4_gemm_dx": (ctypes.c_int, [_vp, _i32, _i64, _i64, _vp, _vp, _i64, _i32, _vp, _vp, _i32,
                                     _vp, _sz, _vp]),
    "mxfp4_plan": (ctypes.c_int, [_i32, _i32, _i64, _i64, _i64, _i32, _i32, ctypes.POINTER(_i32),
                                  ctypes.POINTER(_i64)]),
    "gq_timing_enable": (None, [ctypes.c_int]),
    "gq_timing_read": (ctypes.c_int, [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_i64)]),
    "gq_timing_read_mxfp4": (ctypes.c_int, [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_i64)]),
    "gq_stage_name": (ctypes.c_char_p, [ctypes.c_int]),
}

_lib = None


def library(path: str | None = None) -> ctypes.CDLL:
    """Load libgq.so once (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or _LIB_PATH
    if not os.path.exists(p):
        raise GQError(GQ_ENOTIMPL, f"{p} is missing: build it with "
                                   "`python -m post_weight_quantization_gq_amd.build`")
    lib = ctypes.CDLL(p)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if lib.gq_abi_version() != ABI_VERSION:
        raise GQError(GQ_ENOTIMPL, "libgq ABI version mismatch")
    _lib = lib
    return lib


def _check(status: int):
    if status != GQ_OK:
        raise GQError(status, library().gq_last_error().decode(errors="replace"))


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return GQ_F32
    if t.dtype == torch.bfloat16:
        return GQ_BF16
    raise GQError(GQ_EDTYPE, f"unsupported dtype {t.dtype}")


def _dev(t: torch.Tensor, name: str, dtype=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise GQError(GQ_EINVAL, f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise GQError(GQ_EINVAL, f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise GQError(GQ_EDTYPE, f"{name} must be {dtype}, got {t.dtype}")
    return t


def _shape(t, shape, name):
    """GQ_ESHAPE unless tensor t has exactly this shape (checked before any launch: the
    C ABI sees only pointers, so a mis-shaped buffer would be read or written out of
    bounds on the device)."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise GQError(GQ_ESHAPE, f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _counter(t, name, n=1):
    """Optional device counter: int64 with at least n elements (its device is checked
    with the other tensors)."""
    if t is None:
        return
    if t.dtype != torch.int64 or t.numel() < n:
        raise GQError(GQ_ESHAPE, f"{name} must be an int64 tensor of at least {n} element(s)")


def _same_device(*ts):
    devs = {t.device for t in ts if t is not None}
    if len(devs) > 1:
        raise GQError(GQ_EINVAL, f"tensors on different devices: {sorted(map(str, devs))}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ws(nbytes: int, device):
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _ws_arg(ws):
    """(pointer, bytes) of a workspace tensor; ws=False passes NULL, which makes the
    library allocate its scratch stream-ordered (hipMallocAsync / hipFreeAsync)."""
    if ws is False or ws is None:
        return None, 0
    return _ptr(ws), ws.numel()


def abi_version() -> int:
    return library().gq_abi_version()


def options(block: int = DEFAULT_BLOCK, ridge_rel: float = 1e-6, init: int = GQ_INIT_QUANTILE,
            gram_update: int = GQ_GRAM_AUTO, ridge_abs: float = 0.0,
            check_finite: bool = False, check_residual: bool = False) -> lnq_options:
    o = lnq_options()
    library().gq_lnq_options_default(ctypes.byref(o))
    o.block, o.ridge_rel, o.init, o.gram_update = block, ridge_rel, init, gram_update
    o.ridge_abs, o.check_finite = ridge_abs, int(bool(check_finite))
    o.check_residual = int(bool(check_residual))
    return o


def fisher_workspace_size(n, d_in, d_out, groups, dtype=GQ_BF16) -> int:
    return int(library().gq_fisher_workspace_size(n, d_in, d_out, groups, dtype))


def lnq_workspace_size(d_out, d_in, groups, bits, w_dtype=GQ_BF16) -> int:
    return int(library().gq_lnq_workspace_size(d_out, d_in, groups, bits, w_dtype))


def gq_fisher_accumulate(X, G, groups: int, F=None, accumulate: bool = False, ws=None,
                         stream=None, check_finite: bool = False) -> torch.Tensor:
    """F[g] (=|+=) X^T diag(s_g) X; X [n][d_in], G [n][d_out] (float32 or bfloat16).
    check_finite: scan X and G for NaN / Inf first (GQError GQ_ENONFINITE, F untouched;
    the call then synchronises the stream)."""
    lib = library()
    if X.dim() != 2 or G.dim() != 2:
        raise GQError(GQ_ESHAPE, "X and G must be 2-D")
    n, d_in = X.shape
    d_out = G.shape[1]
    if G.shape[0] != n:
        raise GQError(GQ_ESHAPE, "X and G need the same number of tokens")
    _shape(F, (groups, d_in, d_in), "F")
    _dev(X, "X")
    _dev(G, "G")
    if F is None:
        F = torch.empty((groups, d_in, d_in), dtype=torch.float32, device=X.device)
        if accumulate:
            raise GQError(GQ_EINVAL, "accumulate needs an existing F")
    _dev(F, "F", torch.float32)
    _same_device(X, G, F, ws if isinstance(ws, torch.Tensor) else None)
    if ws is None:
        ws = _ws(fisher_workspace_size(n, d_in, d_out, groups, _dt(X)), X.device)
    wp, wn = _ws_arg(ws)
    flags = int(bool(accumulate)) | (GQ_FISHER_CHECK_FINITE if check_finite else 0)
    _check(lib.gq_fisher_accumulate(_ptr(X), _dt(X), n, d_in, _ptr(G), _dt(G), d_out, groups,
                                    _ptr(F), flags, wp, wn, _stream(stream)))
    return F


fisher = gq_fisher_accumulate


def _lnq_common(F, W, groups, bits=None, C=None, P=None):
    """Shapes first (no device needed), then device, dtype and contiguity."""
    if W.dim() != 2 or F.dim() != 3:
        raise GQError(GQ_ESHAPE, "W must be 2-D and F 3-D")
    d_out, d_in = W.shape
    _shape(F, (groups, d_in, d_in), "F")
    if bits is not None:
        _shape(C, (d_out, 1 << bits), "C")
        _shape(P, (d_out, d_in), "P")
    _dev(F, "F", torch.float32)
    _dev(W, "W")
    if C is not None:
        _dev(C, "C", torch.float32)
    if P is not None:
        _dev(P, "P", torch.uint8)
    _same_device(F, W, C, P)
    return d_out, d_in


def _lnq_ws(ws, d_out, d_in, groups, bits, W):
    if ws is None:
        ws = _ws(lnq_workspace_size(d_out, d_in, groups, bits, _dt(W)), W.device)
    elif ws is not False:
        _same_device(W, ws)
    return _ws_arg(ws)


def lnq_codebook_update(F, W, P, C, bits: int, ridge_rel: float = 1e-6, n_not_pd=None,
                        ws=None, stream=None) -> torch.Tensor:
    """One codebook step; C [d_out][2^bits] float32 is updated in place."""
    lib = library()
    groups = F.shape[0]
    _counter(n_not_pd, "n_not_pd")
    d_out, d_in = _lnq_common(F, W, groups, bits, C, P)
    if n_not_pd is not None:
        _dev(n_not_pd, "n_not_pd")
        _same_device(W, n_not_pd)
    wp, nb = _lnq_ws(ws, d_out, d_in, groups, bits, W)
    _check(lib.lnq_codebook_update(_ptr(F), groups, d_in, _ptr(W), _dt(W), d_out, _ptr(P), bits,
                                   _ptr(C), ridge_rel, _ptr(n_not_pd), wp, nb,
                                   _stream(stream)))
    return C


def lnq_assign_sweep(F, W, C, P, bits: int, ridge_rel: float = 1e-6,
                     block: int = DEFAULT_BLOCK, n_changed=None, ws=None,
                     stream=None) -> torch.Tensor:
    """One assignment pass; P [d_out][d_in] uint8 is updated in place."""
    lib = library()
    groups = F.shape[0]
    _counter(n_changed, "n_changed")
    d_out, d_in = _lnq_common(F, W, groups, bits, C, P)
    if n_changed is not None:
        _dev(n_changed, "n_changed")
        _same_device(W, n_changed)
    wp, nb = _lnq_ws(ws, d_out, d_in, groups, bits, W)
    _check(lib.lnq_assign_sweep(_ptr(F), groups, d_in, _ptr(W), _dt(W), d_out, _ptr(C), bits,
                                _ptr(P), ridge_rel, block, _ptr(n_changed), wp, nb,
                                _stream(stream)))
    return P


def lnq_objective(F, W, C, P, bits: int, ridge_rel: float = 1e-6, obj_total=None, ws=None,
                  stream=None) -> torch.Tensor:
    """Per-row objectives e_j^T F' e_j (float64 [d_out])."""
    lib = library()
    groups = F.shape[0]
    if obj_total is not None and (obj_total.dtype != torch.float64 or obj_total.numel() < 1):
        raise GQError(GQ_ESHAPE, "obj_total must be a float64 tensor of at least one element")
    d_out, d_in = _lnq_common(F, W, groups, bits, C, P)
    if obj_total is not None:
        _dev(obj_total, "obj_total")
        _same_device(W, obj_total)
    rows = torch.empty(d_out, dtype=torch.float64, device=W.device)
    wp, nb = _lnq_ws(ws, d_out, d_in, groups, bits, W)
    _check(lib.lnq_objective(_ptr(F), groups, d_in, _ptr(W), _dt(W), d_out, _ptr(C), _ptr(P),
                             bits, ridge_rel, _ptr(rows), _ptr(obj_total), wp, nb,
                             _stream(stream)))
    return rows


def _outputs(W, d_out, d_in, bits, C, P):
    m = 1 << bits
    if C is None:
        C = torch.empty((d_out, m), dtype=torch.float32, device=W.device)
    if P is None:
        P = torch.empty((d_out, d_in), dtype=torch.uint8, device=W.device)
    return C, P


def lnq_quantize(W, F, bits: int, iters: int, block: int = DEFAULT_BLOCK,
                 ridge_rel: float = 1e-6, C=None, P=None, init: int | None = None,
                 trace: bool = True, ws=None, stream=None, gram_update: int = GQ_GRAM_AUTO,
                 ridge_abs: float = 0.0, check_finite: bool = False,
                 check_residual: bool = False):
    """Whole LNQ on a layer.  Returns (C, P, obj_trace or None, n_changed).

    With C and P given and init unset, starts from them (GQ_INIT_GIVEN).
    ridge_abs: fixed ridge added to ridge_rel * mean(diag F_g).  check_finite: a checked
    call (GQ_ENONFINITE for NaN / Inf in W or F before anything is written, GQ_ENOTPD
    after the run if a codebook system was not positive definite).  ws=False lets the
    library allocate its scratch.  check_residual: the debug check of every assignment
    pass against a fresh F'(C[P] - W) (GQError GQ_ECHECK on a mismatch).
    """
    lib = library()
    groups = F.shape[0]
    if init is None:
        init = GQ_INIT_GIVEN if (C is not None and P is not None) else GQ_INIT_QUANTILE
    d_out, d_in = _lnq_common(F, W, groups, bits, C, P)
    C, P = _outputs(W, d_out, d_in, bits, C, P)
    tr = torch.empty(2 * iters + 1, dtype=torch.float64, device=W.device) if trace else None
    nch = torch.zeros(max(iters, 1), dtype=torch.int64, device=W.device)
    opt = options(block, ridge_rel, init, gram_update, ridge_abs, check_finite, check_residual)
    wp, nb = _lnq_ws(ws, d_out, d_in, groups, bits, W)
    _check(lib.lnq_quantize(_ptr(W), _dt(W), d_out, d_in, _ptr(F), groups, bits, iters,
                            ctypes.byref(opt), _ptr(C), _ptr(P), _ptr(tr), _ptr(nch), wp,
                            nb, _stream(stream)))
    return C, P, tr, nch[:iters]


def lnq_quantize_static(W, F, bits: int, iters: int, block: int = DEFAULT_BLOCK,
                        ridge_rel: float = 1e-6, C=None, P=None, init: int | None = None,
                        trace: bool = True, stream=None, gram_update: int = GQ_GRAM_AUTO,
                        ridge_abs: float = 0.0, check_finite: bool = False,
                        check_residual: bool = False):
    """lnq_quantize on the library's fixed per-device scratch (no workspace, nothing
    allocated by the library; the outputs are still the caller's).  Calls that overlap
    on one device race.  Returns (C, P, obj_trace or None, n_changed)."""
    lib = library()
    groups = F.shape[0]
    if init is None:
        init = GQ_INIT_GIVEN if (C is not None and P is not None) else GQ_INIT_QUANTILE
    d_out, d_in = _lnq_common(F, W, groups, bits, C, P)
    C, P = _outputs(W, d_out, d_in, bits, C, P)
    tr = torch.empty(2 * iters + 1, dtype=torch.float64, device=W.device) if trace else None
    nch = torch.zeros(max(iters, 1), dtype=torch.int64, device=W.device)
    opt = options(block, ridge_rel, init, gram_update, ridge_abs, check_finite, check_residual)
    _check(lib.lnq_quantize_static(_ptr(W), _dt(W), d_out, d_in, _ptr(F), groups, bits, iters,
                                   ctypes.byref(opt), _ptr(C), _ptr(P), _ptr(tr), _ptr(nch),
                                   _stream(stream)))
    return C, P, tr, nch[:iters]


def lnq_static_scratch_bytes() -> int:
    return int(library().lnq_static_scratch_bytes())


def grid_quantize(W, F, bits: int, iters: int, block: int = DEFAULT_BLOCK,
                  ridge_rel: float = 1e-6, C=None, P=None, init: int | None = None,
                  trace: bool = True, ws=None, stream=None, ridge_abs: float = 0.0,
                  check_finite: bool = False, check_residual: bool = False):
    """Fixed-grid backend: uniform grid per row, `iters` assignment passes.

    Returns (C, P, obj_trace [iters+1] or None, n_changed [iters]).  With C and P
    given and init unset, starts from them (GQ_INIT_GIVEN).
    """
    lib = library()
    groups = F.shape[0]
    if init is None:
        init = GQ_INIT_GIVEN if (C is not None and P is not None) else GQ_INIT_UNIFORM
    d_out, d_in = _lnq_common(F, W, groups, bits, C, P)
    C, P = _outputs(W, d_out, d_in, bits, C, P)
    tr = torch.empty(iters + 1, dtype=torch.float64, device=W.device) if trace else None
    nch = torch.zeros(max(iters, 1), dtype=torch.int64, device=W.device)
    opt = options(block, ridge_rel, init, GQ_GRAM_AUTO, ridge_abs, check_finite, check_residual)
    wp, nb = _lnq_ws(ws, d_out, d_in, groups, bits, W)
    _check(lib.grid_quantize(_ptr(W), _dt(W), d_out, d_in, _ptr(F), groups, bits, iters,
                             ctypes.byref(opt), _ptr(C), _ptr(P), _ptr(tr), _ptr(nch), wp,
                             nb, _stream(stream)))
    return C, P, tr, nch[:iters]


def fisher_stream_workspace_size(chunk_tokens, d_in, d_out, groups, dtype=GQ_BF16) -> int:
    return int(library().gq_fisher_stream_workspace_size(chunk_tokens, d_in, d_out, groups,
                                                          dtype))


def gq_fisher_accumulate_host(X, G, groups: int, F=None, accumulate: bool = False,
                              chunk_tokens: int = 16384, ws=None, stream=None,
                              device=None) -> torch.Tensor:
    """F[g] (=|+=) X^T diag(s_g) X with X [n][d_in], G [n][d_out] in HOST memory (CPU
    tensors, pinned for asynchronous copies), streamed to the GPU in chunks of tokens."""
    lib = library()
    for t, name in ((X, "X"), (G, "G")):
        if t.device.type != "cpu" or not t.is_contiguous():
            raise GQError(GQ_EINVAL, f"{name} must be a contiguous host (CPU) tensor")
    n, d_in = X.shape
    d_out = G.shape[1]
    if G.shape[0] != n:
        raise GQError(GQ_ESHAPE, "X and G need the same number of tokens")
    if X.dtype != G.dtype:
        raise GQError(GQ_EDTYPE, "X and G must share a dtype")
    _shape(F, (groups, d_in, d_in), "F")
    dev = F.device if F is not None else (device or torch.device("cuda", torch.cuda.current_device()))
    if F is None:
        F = torch.empty((groups, d_in, d_in), dtype=torch.float32, device=dev)
        if accumulate:
            F.zero_()
    _dev(F, "F", torch.float32)
    if ws is not None:
        _same_device(F, ws)
    if ws is None:
        nb = fisher_stream_workspace_size(min(chunk_tokens, n), d_in, d_out, groups, _dt(X))
        ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=dev)
    _check(lib.gq_fisher_accumulate_host(ctypes.c_void_p(X.data_ptr()), _dt(X), n, d_in,
                                         ctypes.c_void_p(G.data_ptr()), _dt(G), d_out, groups,
                                         _ptr(F), int(accumulate), chunk_tokens, _ptr(ws),
                                         ws.numel(), _stream(stream)))
    return F


def ganq_workspace_size(d_out, d_in, groups, bits, w_dtype=GQ_BF16) -> int:
    return int(library().ganq_workspace_size(d_out, d_in, groups, bits, w_dtype))


def ganq_quantize(W, F, bits: int, iters: int, ridge_rel: float = 1e-6, C=None, P=None,
                  init: int | None = None, trace: bool = True, ws=None, stream=None,
                  ridge_abs: float = 0.0, check_finite: bool = False):
    """GANQ-style alternation.  Returns (C, P, obj_trace [2 iters + 1] or None,
    n_changed [iters], not_pd [groups] int32)."""
    lib = library()
    groups = F.shape[0]
    if init is None:
        init = GQ_INIT_GIVEN if (C is not None and P is not None) else GQ_INIT_QUANTILE
    d_out, d_in = _lnq_common(F, W, groups, bits, C, P)
    C, P = _outputs(W, d_out, d_in, bits, C, P)
    tr = torch.empty(2 * iters + 1, dtype=torch.float64, device=W.device) if trace else None
    nch = torch.zeros(max(iters, 1), dtype=torch.int64, device=W.device)
    npd = torch.zeros(groups, dtype=torch.int32, device=W.device)
    opt = options(DEFAULT_BLOCK, ridge_rel, init, GQ_GRAM_AUTO, ridge_abs, check_finite)
    if ws is None:
        ws = torch.empty(max(ganq_workspace_size(d_out, d_in, groups, bits, _dt(W)), 1),
                         dtype=torch.uint8, device=W.device)
    wp, nb = _ws_arg(ws)
    _check(lib.ganq_quantize(_ptr(W), _dt(W), d_out, d_in, _ptr(F), groups, bits, iters,
                             ctypes.byref(opt), _ptr(C), _ptr(P), _ptr(tr), _ptr(nch), _ptr(npd),
                             wp, nb, _stream(stream)))
    return C, P, tr, nch[:iters], npd


def ganq_factor_damped(F, ridge_rel: float = 1e-6, ws=None, stream=None):
    """(L [groups][d][d] float32 lower, not_pd [groups] int32) of F' = F + lambda I."""
    lib = library()
    if F.dim() != 3 or F.shape[1] != F.shape[2]:
        raise GQError(GQ_ESHAPE, "F must be [groups][d_in][d_in]")
    _dev(F, "F", torch.float32)
    groups, d_in = F.shape[0], F.shape[1]
    L = torch.empty_like(F)
    npd = torch.zeros(groups, dtype=torch.int32, device=F.device)
    if ws is None:
        ws = torch.empty(max(ganq_workspace_size(groups, d_in, groups, 1), 1), dtype=torch.uint8,
                         device=F.device)
    _check(lib.ganq_factor_damped(_ptr(F), groups, d_in, ridge_rel, _ptr(L), _ptr(npd), _ptr(ws),
                                  ws.numel(), _stream(stream)))
    return L, npd


def lut_packed_row_words(d_in: int, bits: int) -> int:
    return int(library().lut_packed_row_words(d_in, bits))


def lut_pack_codes(P, bits: int, Q=None, stream=None) -> torch.Tensor:
    """P [d_out][d_in] uint8 -> packed codes Q [d_out][row words] (int32 storage of the
    uint32 words)."""
    lib = library()
    if P.dim() != 2:
        raise GQError(GQ_ESHAPE, "P must be [d_out][d_in]")
    d_out, d_in = P.shape
    rw = lut_packed_row_words(d_in, bits)
    _shape(Q, (d_out, max(rw, 1)), "Q")
    _dev(P, "P", torch.uint8)
    if Q is None:
        Q = torch.empty((d_out, max(rw, 1)), dtype=torch.int32, device=P.device)
    _dev(Q, "Q", torch.int32)
    _same_device(P, Q)
    _check(lib.lut_pack_codes(_ptr(P), d_out, d_in, bits, _ptr(Q), _stream(stream)))
    return Q


def lut_gemv(Q, C, x, bits: int, d_in: int | None = None, y=None, stream=None) -> torch.Tensor:
    """y [batch][d_out] = sum_i C[j][code_ji] x[b][i]; x [batch][d_in] or [d_in]
    (d_in, if given, must be x's last dimension)."""
    lib = library()
    if x.dim() not in (1, 2) or C.dim() != 2:
        raise GQError(GQ_ESHAPE, "x must be [batch][d_in] or [d_in] and C [d_out][2^bits]")
    xx = x if x.dim() == 2 else x.unsqueeze(0)
    batch, dx = xx.shape
    if d_in is not None and d_in != dx:
        raise GQError(GQ_ESHAPE, f"d_in={d_in} differs from the activations' {dx}")
    d_in = dx
    d_out = C.shape[0]
    _shape(C, (d_out, 1 << bits), "C")
    _shape(Q, (d_out, max(lut_packed_row_words(d_in, bits), 1)), "Q")
    _shape(y, (batch, d_out), "y")
    _dev(Q, "Q", torch.int32)
    _dev(C, "C", torch.float32)
    _dev(x, "x")
    if y is None:
        y = torch.empty((batch, d_out), dtype=torch.float32, device=x.device)
    _dev(y, "y", torch.float32)
    _same_device(Q, C, x, y)
    _check(lib.lut_gemv(_ptr(Q), _ptr(C), d_out, d_in, bits, _ptr(xx), _dt(xx), batch, _ptr(y),
                        _stream(stream)))
    return y if x.dim() == 2 else y[0]


def mxfp4_row_bytes(d: int) -> int:
    return int(library().mxfp4_row_bytes(d))


def mxfp4_row_scales(d: int) -> int:
    return int(library().mxfp4_row_scales(d))


@contextlib.contextmanager
def _other_place(device, stream):
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


def _place(t, stream):
    """(context, stream pointer) of a call on t's device: inside the context that device is
    current, and what the call allocates belongs to the stream it runs on (its memory is reused
    in that stream's order).  Without a device or stream to change to, the context does nothing."""
    index = t.get_device()
    if stream is None:
        if index == torch._C._cuda_getDevice():
            return _NOWHERE, torch._C._cuda_getCurrentRawStream(index)
        stream = torch.cuda.current_stream(index)
    elif stream.device != t.device:
        raise GQError(GQ_EINVAL, f"stream of {stream.device} for tensors on {t.device}")
    return _other_place(t.device, stream), stream.cuda_stream


_NOWHERE = contextlib.nullcontext()
_MX_DTYPES = {torch.float32: GQ_F32, torch.bfloat16: GQ_BF16}


def _mx_shape(t, shape, name):
    if t.shape != shape:
        raise GQError(GQ_ESHAPE, f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _mx_tensor(t, name, index, dtypes=_MX_DTYPES):
    """A contiguous GPU tensor of an allowed dtype, on GPU `index`."""
    if t.get_device() == index and index >= 0 and t.is_contiguous() and t.dtype in dtypes:
        return
    if not t.is_cuda:
        raise GQError(GQ_EINVAL, f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise GQError(GQ_EINVAL, f"{name} must be contiguous")
    if t.dtype not in dtypes:
        raise GQError(GQ_EDTYPE, f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    raise GQError(GQ_EINVAL, f"{name} is on {t.device}, the call's first tensor is not")


_U8, _I64 = (torch.uint8,), (torch.int64,)
_MX_MAX_D = 1 << 20


def _mx_width(d):
    """(bytes of codes, bytes of scales) of a packed row of d values."""
    if d < 1 or d > _MX_MAX_D:
        raise GQError(GQ_ESHAPE if d < 1 else GQ_ENOTIMPL, f"rows of {d} values: 1 to 2^20")
    groups = -(-d // 128)
    return 64 * groups, 4 * groups


def mxfp4_quantize(x, Q=None, S=None, stream=None):
    """x [..][d] float32 or bfloat16 -> (Q [..][64 ceil(d / 128)], S [..][4 ceil(d / 128)])
    uint8: 4-bit codes and a scale byte for each block of 32 along the last dimension."""
    lib = _lib or library()
    if x.dim() < 1:
        raise GQError(GQ_ESHAPE, "x needs a last dimension to quantise along")
    lead, d = x.shape[:-1], x.shape[-1]
    rb, rs = _mx_width(d)
    index = x.get_device()
    for t, width, name in ((Q, rb, "Q"), (S, rs, "S")):
        if t is not None:
            _mx_shape(t, (*lead, width), name)
            _mx_tensor(t, name, index, _U8)
    _mx_tensor(x, "x", index)
    where, st = _place(x, stream)
    with where:
        if Q is None:
            Q = x.new_empty((*lead, rb), dtype=torch.uint8)
        if S is None:
            S = x.new_empty((*lead, rs), dtype=torch.uint8)
        status = lib.mxfp4_quantize(x.data_ptr(), _MX_DTYPES[x.dtype], x.numel() // d, d, Q.data_ptr(),
                                    S.data_ptr(), st)
    if status:
        _check(status)
    return Q, S


def mxfp4_dequantize(Q, S, d: int, dtype=torch.bfloat16, y=None, stream=None) -> torch.Tensor:
    """The values [..][d] that packed rows stand for, in float32 or bfloat16."""
    lib = _lib or library()
    lead = Q.shape[:-1]
    rb, rs = _mx_width(d)
    if dtype not in _MX_DTYPES:
        raise GQError(GQ_EDTYPE, f"unsupported dtype {dtype}")
    index = Q.get_device()
    _mx_shape(Q, (*lead, rb), "Q")
    _mx_shape(S, (*lead, rs), "S")
    if y is not None:
        _mx_shape(y, (*lead, d), "y")
        _mx_tensor(y, "y", index, (dtype,))
    _mx_tensor(Q, "Q", index, _U8)
    _mx_tensor(S, "S", index, _U8)
    where, st = _place(Q, stream)
    with where:
        if y is None:
            y = Q.new_empty((*lead, d), dtype=dtype)
        status = lib.mxfp4_dequantize(Q.data_ptr(), S.data_ptr(), y.numel() // d, d, y.data_ptr(),
                                      _MX_DTYPES[dtype], st)
    if status:
        _check(status)
    return y


def mxfp4_gemm_workspace_size(n, d_in, d_out, experts=1, dtype=GQ_BF16) -> int:
    return int(library().mxfp4_gemm_workspace_size(n, d_in, d_out, experts, dtype))


def mxfp4_gemm_mx_workspace_size(n, d_in, d_out, experts=1) -> int:
    return int(library().mxfp4_gemm_mx_workspace_size(n, d_in, d_out, experts))


def mxfp4_gemm_dx_workspace_size(n, d_in, d_out, experts=1, dtype=GQ_BF16) -> int:
    return int(library().mxfp4_gemm_dx_workspace_size(n, d_in, d_out, experts, dtype))


def mxfp4_plan(op: str, n, d_in, d_out, experts=None, dtype=GQ_BF16) -> dict:
    """How a product ("gemm", "gemm_mx" or "gemm_dx") of these sizes is done: planes, streamed,
    rows and cols of a tile, waves of a block, split; first_rows < n where a call is divided in
    two products (the plan is the first's).  experts: None for one weight, else their number."""
    plan, first = (_i32 * 6)(), _i64()
    _check(library().mxfp4_plan(("gemm", "gemm_mx", "gemm_dx").index(op), dtype, n, d_in, d_out,
                                experts or 1, experts is not None, plan, ctypes.byref(first)))
    names = ("planes", "streamed", "rows", "cols", "waves", "split")
    return dict(zip(names, plan), first_rows=first.value)


def _mx_weight(Q, S, d_in, offsets, index):
    """(experts, d_out) of a packed weight, one ([d_out][..]) or, with offsets, several
    ([experts][d_out][..])."""
    rb, rs = _mx_width(d_in)
    lead = Q.shape[:-1]
    if len(lead) != (1 if offsets is None else 2):
        raise GQError(GQ_ESHAPE, "Q must be [d_out][row bytes], or [experts][d_out][row bytes] "
                                 "with offsets")
    _mx_shape(Q, (*lead, rb), "Q")
    _mx_shape(S, (*lead, rs), "S")
    if offsets is not None:
        _mx_shape(offsets, (lead[0] + 1,), "offsets")
        _mx_tensor(offsets, "offsets", index, _I64)
    _mx_tensor(Q, "Q", index, _U8)
    _mx_tensor(S, "S", index, _U8)
    return (1, lead[0]) if offsets is None else lead


def _mx_product(fn, size, x, first, size_args, n, width, Q, S, last, experts, offsets, y, out_dtype,
                ws, stream):
    """What the three products share: output, workspace and the call itself.  A grouped
    product's own output has zeros in the rows past the last expert's."""
    index = x.get_device()
    if y is not None:
        if out_dtype is not None and y.dtype != out_dtype:
            raise GQError(GQ_EDTYPE, f"y is {y.dtype}, out_dtype {out_dtype}")
        _mx_shape(y, (n, width), "y")
        _mx_tensor(y, "y", index)
    elif out_dtype not in _MX_DTYPES:
        raise GQError(GQ_EDTYPE, f"unsupported dtype {out_dtype}")
    wp, wn = None, 0
    if ws is not None and ws is not False:
        _mx_tensor(ws, "ws", index, _U8)
        wp, wn = ws.data_ptr(), ws.numel()
    where, st = _place(x, stream)
    with where:
        if y is None:
            y = (x.new_empty if offsets is None else x.new_zeros)((n, width), dtype=out_dtype)
        if ws is None:
            wn = size(*size_args)
            if wn:
                ws = x.new_empty(wn, dtype=torch.uint8)
                wp = ws.data_ptr()
        status = fn(*first, Q.data_ptr(), S.data_ptr(), last, experts,
                    None if offsets is None else offsets.data_ptr(), y.data_ptr(),
                    _MX_DTYPES[y.dtype], wp, wn, st)
    if status:
        _check(status)
    return y


class _MxProduct(torch.autograd.Function):
    """mxfp4_gemm as a function of x or, with `back`, mxfp4_gemm_dx as one of g: the weight is
    fixed and both are linear, so each one's gradient is the other."""

    @staticmethod
    def forward(ctx, a, Q, S, d_in, offsets, out_dtype, ws, back):
        ctx.save_for_backward(Q, S, offsets)
        ctx.d_in, ctx.dtype, ctx.back = d_in, a.dtype, back
        if back:
            return mxfp4_gemm_dx(a, Q, S, d_in, offsets=offsets, out_dtype=out_dtype, ws=ws)
        return mxfp4_gemm(a, Q, S, offsets=offsets, out_dtype=out_dtype, ws=ws)

    @staticmethod
    def backward(ctx, grad):
        Q, S, offsets = ctx.saved_tensors
        grad = grad.contiguous()
        if grad.data_ptr() & 15:           # a part of a larger gradient, off the rows' alignment
            grad = grad.clone()
        if ctx.back:
            d = mxfp4_gemm(grad, Q, S, offsets=offsets, out_dtype=ctx.dtype)
        else:
            d = mxfp4_gemm_dx(grad, Q, S, ctx.d_in, offsets=offsets, out_dtype=ctx.dtype)
        return d, None, None, None, None, None, None, None


def _mx_recorded(a, name, Q, S, d_in, offsets, y, out_dtype, ws, stream, back):
    """A product of activations that require a gradient, as autograd records it: its backward
    pass runs on the stream of the call."""
    if y is not None:
        raise GQError(GQ_EINVAL, f"{name} requires a gradient, which a given y would not carry: "
                                 "call without y, or under torch.no_grad()")
    _mx_tensor(a, name, a.get_device())
    where, _ = _place(a, stream)
    with where:
        return _MxProduct.apply(a, Q, S, d_in, offsets, out_dtype, ws, back)


def mxfp4_gemm(x, Q, S, offsets=None, y=None, out_dtype=None, ws=None, stream=None) -> torch.Tensor:
    """y [n][d_out] = x W^T for x [n][d_in] (float32 or bfloat16) and the packed weight (Q, S)
    of mxfp4_quantize.  With offsets (int64 [experts + 1] on the device) rows offsets[e] ..
    offsets[e + 1] - 1 of x are multiplied by weight e of Q [experts][d_out][row bytes], and
    the other rows of a given y keep their values (of a new one: zeros).
    out_dtype: float32 or bfloat16, x's unless given.
    Where x requires a gradient, autograd gets it by mxfp4_gemm_dx (and y cannot be given)."""
    lib = _lib or library()
    if x.dim() != 2:
        raise GQError(GQ_ESHAPE, "x must be [n][d_in]")
    n, d_in = x.shape
    if x.requires_grad and torch.is_grad_enabled():
        return _mx_recorded(x, "x", Q, S, d_in, offsets, y, out_dtype, ws, stream, False)
    index = x.get_device()
    experts, d_out = _mx_weight(Q, S, d_in, offsets, index)
    _mx_tensor(x, "x", index)
    dt = _MX_DTYPES[x.dtype]
    if y is None and out_dtype is None:
        out_dtype = x.dtype
    return _mx_product(lib.mxfp4_gemm, lib.mxfp4_gemm_workspace_size, x, (x.data_ptr(), dt, n, d_in),
                       (n, d_in, d_out, experts, dt), n, d_out, Q, S, d_out, experts, offsets, y,
                       out_dtype, ws, stream)


def mxfp4_gemm_mx(XQ, XS, Q, S, d_in: int, offsets=None, y=None, out_dtype=None, ws=None,
                  stream=None) -> torch.Tensor:
    """mxfp4_gemm with the activations packed by mxfp4_quantize as well: XQ [n][row bytes],
    XS [n][row scales].  out_dtype: bfloat16 unless given.  Bytes carry no gradient: autograd
    does not reach what they were packed from (mxfp4_gemm_dx is the product's part of it)."""
    lib = _lib or library()
    if XQ.dim() != 2:
        raise GQError(GQ_ESHAPE, "XQ must be [n][row bytes]")
    n = XQ.shape[0]
    rb, rs = _mx_width(d_in)
    index = XQ.get_device()
    _mx_shape(XQ, (n, rb), "XQ")
    _mx_shape(XS, (n, rs), "XS")
    experts, d_out = _mx_weight(Q, S, d_in, offsets, index)
    _mx_tensor(XQ, "XQ", index, _U8)
    _mx_tensor(XS, "XS", index, _U8)
    if y is None and out_dtype is None:
        out_dtype = torch.bfloat16
    return _mx_product(lib.mxfp4_gemm_mx, lib.mxfp4_gemm_mx_workspace_size, XQ,
                       (XQ.data_ptr(), XS.data_ptr(), n, d_in), (n, d_in, d_out, experts), n, d_out,
                       Q, S, d_out, experts, offsets, y, out_dtype, ws, stream)


def mxfp4_gemm_dx(g, Q, S, d_in: int, offsets=None, y=None, out_dtype=None, ws=None,
                  stream=None) -> torch.Tensor:
    """dx [n][d_in] = g W for the output's gradient g [n][d_out] (float32 or bfloat16): the
    gradient of mxfp4_gemm's x (and, straight through the rounding, of the values that
    mxfp4_gemm_mx's were packed from).  Grouped by offsets like mxfp4_gemm.
    Where g requires a gradient, autograd gets it by mxfp4_gemm (and y cannot be given)."""
    lib = _lib or library()
    if g.dim() != 2:
        raise GQError(GQ_ESHAPE, "g must be [n][d_out]")
    if g.requires_grad and torch.is_grad_enabled():
        return _mx_recorded(g, "g", Q, S, d_in, offsets, y, out_dtype, ws, stream, True)
    n = g.shape[0]
    index = g.get_device()
    experts, d_out = _mx_weight(Q, S, d_in, offsets, index)
    _mx_shape(g, (n, d_out), "g")
    _mx_tensor(g, "g", index)
    dt = _MX_DTYPES[g.dtype]
    if y is None and out_dtype is None:
        out_dtype = g.dtype
    return _mx_product(lib.mxfp4_gemm_dx, lib.mxfp4_gemm_dx_workspace_size, g,
                       (g.data_ptr(), dt, n, d_out), (n, d_in, d_out, experts, dt), n, d_in, Q, S,
                       d_in, experts, offsets, y, out_dtype, ws, stream)


STAGES = ("group_scale", "fisher_mfma", "fisher_finalize", "fisher_plain", "lnq_prepare",
          "lnq_resid", "lnq_init", "lnq_gram", "lnq_solve", "lnq_sweep", "lnq_small",
          "fisher_pack", "lnq_delta", "lut_pack", "lut_gemv", "fisher_h2d", "ganq_chol",
          "ganq_pass", "mxfp4_pack", "mxfp4_gemm")     # the last two are read on their own


def gq_timing_enable(on=True) -> None:
    """Bracket later launch sequences with HIP events on their stream (diagnostics).

    on: True (every stage), False (off), a stage name, or an iterable of names.
    """
    if on is True:
        mask = -1
    elif on is False or on is None:
        mask = 0
    else:
        names = [on] if isinstance(on, str) else list(on)
        mask = 0
        for n in names:
            mask |= 1 << STAGES.index(n)
    library().gq_timing_enable(mask)


def gq_timing_read() -> dict:
    """{stage name: (milliseconds, launch sequences)} since the last read; clears.  The MXFP4
    stages (mxfp4_pack, mxfp4_gemm) are in it where they were timed."""
    lib = library()
    ms = (ctypes.c_double * STAGE_COUNT)()
    cnt = (_i64 * STAGE_COUNT)()
    _check(lib.gq_timing_read(ms, cnt))
    times = {lib.gq_stage_name(i).decode(): (ms[i], cnt[i]) for i in range(STAGE_COUNT)}
    ms = (ctypes.c_double * MXFP4_STAGE_COUNT)()
    cnt = (_i64 * MXFP4_STAGE_COUNT)()
    _check(lib.gq_timing_read_mxfp4(ms, cnt))
    times.update((name, (ms[i], cnt[i])) for i, name in enumerate(STAGES[STAGE_COUNT:]) if cnt[i])
    return times
