"""ctypes binding of libpsgd.so: the C ABI of include/psgd.h, under the same names.

Argument marshalling only. Every step of the PowerSGD path runs in the HIP kernels of the
library; torch tensors are used for device memory and streams. If the library is missing the
import of this module's functions raises: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Iterable, List, Optional, Sequence

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpsgd.so")

PSGD_OK, PSGD_EINVAL, PSGD_EDTYPE, PSGD_ENOMEM, PSGD_EHIP, PSGD_EUNSUPPORTED = range(6)
PSGD_F16, PSGD_BF16, PSGD_F32 = 1, 2, 3
PSGD_NS_FAST, PSGD_NS_ACCURATE = 0, 1
PSGD_I32, PSGD_I64 = 4, 8
STATUS_NAMES = {0: "PSGD_OK", 1: "PSGD_EINVAL", 2: "PSGD_EDTYPE", 3: "PSGD_ENOMEM",
                4: "PSGD_EHIP", 5: "PSGD_EUNSUPPORTED"}

# Names of the profiling slots (order of psgd_profile_events).
PROFILE_SLOTS = ("zero_flags", "ef_mq", "gs_gram", "gs_factor", "gs_apply", "mtp",
                 "zero_skip", "check_finite", "decompress", "gs_reduce", "split3",
                 "gs_second_pass", "adam_norm", "decompress_adam", "adam_passthrough")


class psgd_matrix(ctypes.Structure):
    _fields_ = [
        ("grad", ctypes.c_void_p), ("ld_grad", ctypes.c_int64),
        ("err", ctypes.c_void_p), ("ld_err", ctypes.c_int64),
        ("q", ctypes.c_void_p),
        ("q_next", ctypes.c_void_p),
        ("p", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("ld_out", ctypes.c_int64),
        ("m", ctypes.c_int64), ("n", ctypes.c_int64),
        ("block", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]


class psgd_tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("numel", ctypes.c_int64)]


class psgd_adam_hparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float)]


class psgd_adam_matrix(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("ld_param", ctypes.c_int64),
                ("m1", ctypes.c_void_p), ("m2", ctypes.c_void_p)]


class psgd_adam_tensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("m1", ctypes.c_void_p), ("m2", ctypes.c_void_p),
                ("grad", ctypes.c_void_p), ("numel", ctypes.c_int64)]


class psgd_ns_hparams(ctypes.Structure):
    _fields_ = [("a", ctypes.c_float), ("b", ctypes.c_float), ("c", ctypes.c_float), ("eps", ctypes.c_float),
                ("steps", ctypes.c_int32)]


class psgd_ns_matrix(ctypes.Structure):
    # the C field is named `in`, a Python keyword: reach it with getattr
    _fields_ = [("in", ctypes.c_void_p), ("ld_in", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("ld_out", ctypes.c_int64),
                ("m", ctypes.c_int64), ("n", ctypes.c_int64)]


class psgd_muon_hparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("nesterov", ctypes.c_int32), ("adjust", ctypes.c_int32), ("ns", psgd_ns_hparams)]


class psgd_muon_matrix(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("ld_param", ctypes.c_int64), ("momentum", ctypes.c_void_p)]


class PsgdError(RuntimeError):
    def __init__(self, call: str, status: int, message: str):
        super().__init__(f"{call} failed: {STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


_lib = None


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libpsgd.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or os.environ.get("PSGD_LIBRARY") or LIB_PATH
    # torch first: its HIP runtime is then the one libpsgd.so binds to (same soname), so the
    # streams and events torch hands out are valid inside the library.
    import torch  # noqa: F401
    if not os.path.exists(p):
        raise ImportError(
            f"{p} is missing: build it with `python -m rank_gradient_compression_powersgd_amd.build` "
            "(there is no CPU fallback for the PowerSGD kernels)")
    lib = ctypes.CDLL(p)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.psgd_version.restype = ctypes.c_int
    lib.psgd_create.argtypes = [ctypes.POINTER(vp), ctypes.c_int, ctypes.c_int]
    lib.psgd_destroy.argtypes = [vp]
    lib.psgd_plan_create.argtypes = [vp, ctypes.POINTER(psgd_matrix), ctypes.c_int, ctypes.c_int,
                                     ctypes.c_int, ctypes.POINTER(vp)]
    lib.psgd_plan_destroy.argtypes = [vp]
    lib.psgd_compress.argtypes = [vp, vp, vp, vp, vp]
    lib.psgd_check_finite.argtypes = [vp, vp, vp, ctypes.POINTER(psgd_tensor), ctypes.c_int, vp, vp,
                                      ctypes.POINTER(i32), vp]
    lib.psgd_decompress_update.argtypes = [vp, vp, vp, vp, vp]
    lib.psgd_last_error.argtypes = [vp]
    lib.psgd_last_error.restype = ctypes.c_char_p
    lib.psgd_debug_buffer.argtypes = [vp, ctypes.c_int, ctypes.c_int, ctypes.POINTER(vp),
                                      ctypes.POINTER(i64), ctypes.POINTER(i32)]
    lib.psgd_profile_events.argtypes = [vp, ctypes.POINTER(vp), ctypes.c_int]
    lib.psgd_compress_p.argtypes = [vp, vp, vp, vp, vp]
    lib.psgd_orthogonalize.argtypes = [vp, vp, vp]
    lib.psgd_compress_q.argtypes = [vp, vp, vp, vp]
    lib.psgd_refresh_q.argtypes = [vp, vp, vp]
    lib.psgd_factor_buffer.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(i64), ctypes.POINTER(i32)]
    lib.psgd_reset_errors.argtypes = [vp, vp, vp]
    lib.psgd_step_noalloc.argtypes = [vp, ctypes.POINTER(psgd_matrix), ctypes.c_int, ctypes.c_int, vp,
                                      ctypes.c_int, ctypes.POINTER(psgd_tensor), ctypes.c_int, vp, vp, vp]
    lib.psgd_plan_counters.argtypes = [vp, ctypes.POINTER(vp)]
    lib.psgd_adam_attach.argtypes = [vp, vp, ctypes.POINTER(psgd_adam_matrix), ctypes.c_int]
    lib.psgd_adam_prepare.argtypes = [vp, vp, ctypes.POINTER(psgd_adam_tensor), ctypes.c_int, ctypes.c_float,
                                      vp, vp, vp, vp]
    lib.psgd_decompress_adam.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.POINTER(psgd_adam_hparams), vp]
    lib.psgd_adam_update.argtypes = [vp, ctypes.POINTER(psgd_adam_tensor), ctypes.c_int, vp, vp, vp,
                                     ctypes.POINTER(psgd_adam_hparams), vp]
    lib.psgd_block_grad_enter.argtypes = [vp, vp, i64, vp, vp, ctypes.c_int, vp]
    lib.psgd_block_grad_exit.argtypes = [vp, vp, vp, i64, vp, ctypes.c_int, vp, vp]
    lib.psgd_block_grad_exit_enter.argtypes = [vp, vp, vp, i64, vp, vp, vp, ctypes.c_int, vp, vp]
    lib.psgd_ns_plan_create.argtypes = [vp, ctypes.POINTER(psgd_ns_matrix), ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_int, ctypes.POINTER(vp)]
    lib.psgd_ns_plan_destroy.argtypes = [vp]
    lib.psgd_newton_schulz.argtypes = [vp, vp, ctypes.POINTER(psgd_ns_hparams), vp]
    lib.psgd_muon_attach.argtypes = [vp, vp, ctypes.POINTER(psgd_muon_matrix), ctypes.c_int, ctypes.c_int]
    lib.psgd_muon_update.argtypes = [vp, vp, vp, vp, ctypes.POINTER(psgd_muon_hparams), vp]
    lib.psgd_embed_lookup.argtypes = [vp, vp, i64, i64, i64, ctypes.c_int, vp, ctypes.c_int, i64, ctypes.c_float,
                                      vp, i64, ctypes.c_int, vp]
    lib.psgd_embed_grad_workspace.argtypes = [i64, i64, i64, ctypes.POINTER(i64)]
    lib.psgd_embed_grad.argtypes = [vp, vp, i64, ctypes.c_int, vp, ctypes.c_int, i64, i64, i64, ctypes.c_float,
                                    vp, i64, ctypes.c_int, vp, i64, vp]
    for name in ("psgd_ns_plan_create", "psgd_ns_plan_destroy", "psgd_newton_schulz", "psgd_muon_attach",
                 "psgd_muon_update", "psgd_embed_lookup", "psgd_embed_grad_workspace", "psgd_embed_grad",
                 "psgd_create", "psgd_destroy", "psgd_plan_create", "psgd_plan_destroy",
                 "psgd_compress", "psgd_check_finite", "psgd_decompress_update",
                 "psgd_debug_buffer", "psgd_profile_events", "psgd_compress_p", "psgd_orthogonalize",
                 "psgd_compress_q", "psgd_refresh_q", "psgd_factor_buffer", "psgd_reset_errors",
                 "psgd_step_noalloc", "psgd_plan_counters", "psgd_adam_attach", "psgd_adam_prepare", "psgd_decompress_adam",
                 "psgd_adam_update", "psgd_block_grad_enter",
                 "psgd_block_grad_exit", "psgd_block_grad_exit_enter"):
        getattr(lib, name).restype = ctypes.c_int
    if path is None:
        _lib = lib
    return lib


def _check(ctx, call: str, status: int):
    if status != PSGD_OK:
        msg = ""
        if ctx:
            raw = load_library().psgd_last_error(ctx)
            msg = raw.decode() if raw else ""
        raise PsgdError(call, status, msg)


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _stream(stream, device=None) -> int:
    if stream is None:
        import torch
        return int(torch.cuda.current_stream(device).cuda_stream)
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


# --------------------------------------------------------------------------------------
# the C ABI, one function per entry point
# --------------------------------------------------------------------------------------
def psgd_version() -> int:
    return int(load_library().psgd_version())


_ctx_device = {}                             # device of every context made here


def psgd_create(device: int, rank: int) -> int:
    h = ctypes.c_void_p()
    _check(None, "psgd_create", load_library().psgd_create(ctypes.byref(h), device, rank))
    _ctx_device[h.value] = device
    return h.value


def psgd_destroy(ctx: int) -> None:
    _ctx_device.pop(ctx, None)
    load_library().psgd_destroy(ctx)


def dtype_code(torch_dtype) -> int:
    import torch
    return {torch.float16: PSGD_F16, torch.bfloat16: PSGD_BF16, torch.float32: PSGD_F32}[torch_dtype]


def make_matrix(grad, err, q, q_next, p, block: int, out=None) -> psgd_matrix:
    """psgd_matrix over torch tensors (row-major; leading dimensions from the strides).
    grad=None describes an in-place matrix: err already holds M = s_b G + E."""
    m, n = (grad if grad is not None else err).shape
    for name, t, shape in (("err", err, (m, n)), ("q", q, None), ("q_next", q_next, None),
                           ("p", p, None), ("out", out, (m, n))):
        if t is None:
            continue
        if shape is not None and tuple(t.shape) != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
        if t.stride(-1) != 1:
            raise ValueError(f"{name} must have unit stride along rows")
    for name, t in (("q", q), ("q_next", q_next), ("p", p)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    return psgd_matrix(
        grad=_ptr(grad), ld_grad=grad.stride(0) if grad is not None else 0,
        err=_ptr(err), ld_err=err.stride(0),
        q=_ptr(q), q_next=_ptr(q_next), p=_ptr(p),
        out=_ptr(out), ld_out=out.stride(0) if out is not None else 0,
        m=m, n=n, block=block, reserved=0)


def psgd_plan_create(ctx: int, mats: Sequence[psgd_matrix], grad_dtype: int, n_blocks: int) -> int:
    arr = (psgd_matrix * len(mats))(*mats)
    h = ctypes.c_void_p()
    _check(ctx, "psgd_plan_create",
           load_library().psgd_plan_create(ctx, arr, len(mats), grad_dtype, n_blocks, ctypes.byref(h)))
    return h.value


def psgd_plan_destroy(plan: int) -> None:
    load_library().psgd_plan_destroy(plan)


def psgd_compress(ctx: int, plan: int, scale, flags, stream=None) -> None:
    _check(ctx, "psgd_compress",
           load_library().psgd_compress(ctx, plan, _ptr(scale), _ptr(flags), _stream(stream)))


def psgd_compress_p(ctx: int, plan: int, scale, flags, stream=None) -> None:
    _check(ctx, "psgd_compress_p",
           load_library().psgd_compress_p(ctx, plan, _ptr(scale), _ptr(flags), _stream(stream)))


def psgd_orthogonalize(ctx: int, plan: int, stream=None) -> None:
    _check(ctx, "psgd_orthogonalize", load_library().psgd_orthogonalize(ctx, plan, _stream(stream)))


def psgd_compress_q(ctx: int, plan: int, scale, stream=None) -> None:
    _check(ctx, "psgd_compress_q",
           load_library().psgd_compress_q(ctx, plan, _ptr(scale), _stream(stream)))


def psgd_refresh_q(ctx: int, plan: int, stream=None) -> None:
    _check(ctx, "psgd_refresh_q", load_library().psgd_refresh_q(ctx, plan, _stream(stream)))


def psgd_plan_counters(plan: int) -> int:
    """Device address of the plan's two int64 step counters (steps decompressed, steps skipped)."""
    ptr = ctypes.c_void_p()
    _check(None, "psgd_plan_counters", load_library().psgd_plan_counters(plan, ctypes.byref(ptr)))
    return ptr.value


def psgd_factor_buffer(plan: int):
    """(device address, float count, rpad) of the plan's contiguous raw-factor buffer."""
    ptr, count, rpad = ctypes.c_void_p(), ctypes.c_int64(), ctypes.c_int32()
    _check(None, "psgd_factor_buffer",
           load_library().psgd_factor_buffer(plan, ctypes.byref(ptr), ctypes.byref(count),
                                             ctypes.byref(rpad)))
    return ptr.value, count.value, rpad.value


def psgd_check_finite(ctx: int, plan: int, flags, passthrough: Iterable, scale, skip_dev,
                      host: bool = False, stream=None) -> Optional[int]:
    pts = [t for t in passthrough]
    arr = (psgd_tensor * max(1, len(pts)))(*[psgd_tensor(_ptr(t), t.numel()) for t in pts])
    skip_host = ctypes.c_int32(-1)
    _check(ctx, "psgd_check_finite",
           load_library().psgd_check_finite(ctx, plan, _ptr(flags), arr, len(pts), _ptr(scale),
                                            _ptr(skip_dev), ctypes.byref(skip_host) if host else None,
                                            _stream(stream)))
    return int(skip_host.value) if host else None


def psgd_decompress_update(ctx: int, plan: int, scale, skip_dev, stream=None) -> None:
    _check(ctx, "psgd_decompress_update",
           load_library().psgd_decompress_update(ctx, plan, _ptr(scale), _ptr(skip_dev), _stream(stream)))


def psgd_reset_errors(ctx: int, plan: int, stream=None) -> None:
    """Zero every error buffer of the plan (restart from a checkpoint)."""
    _check(ctx, "psgd_reset_errors", load_library().psgd_reset_errors(ctx, plan, _stream(stream)))


def psgd_step_noalloc(ctx: int, mats: Sequence[psgd_matrix], grad_dtype: int, scale, flags,
                      skip_dev, passthrough: Iterable = (), stream=None) -> None:
    """One whole step on a group without a plan or any device allocation (the library's static
    scratch array holds the workspace); calls overlapping on one device race."""
    arr = (psgd_matrix * len(mats))(*mats)
    pts = [t for t in passthrough]
    parr = (psgd_tensor * max(1, len(pts)))(*[psgd_tensor(_ptr(t), t.numel()) for t in pts])
    _check(ctx, "psgd_step_noalloc",
           load_library().psgd_step_noalloc(ctx, arr, len(mats), grad_dtype, _ptr(scale), int(scale.numel()),
                                            parr, len(pts), _ptr(flags), _ptr(skip_dev), _stream(stream)))


def make_adam_matrix(param, m1, m2) -> psgd_adam_matrix:
    """psgd_adam_matrix over torch tensors: param m x n (unit row stride), m1 and m2 contiguous
    m x n 16-bit tensors (any 2-byte dtype: their bits are the stored codes)."""
    if param.stride(-1) != 1 or not m1.is_contiguous() or not m2.is_contiguous():
        raise PsgdError("psgd_adam_attach", PSGD_EINVAL, "param needs unit row stride, m1 and m2 contiguity")
    if m1.element_size() != 2 or m2.element_size() != 2:
        raise PsgdError("psgd_adam_attach", PSGD_EDTYPE, "m1 and m2 must be 16-bit tensors")
    if tuple(m1.shape) != tuple(param.shape) or tuple(m2.shape) != tuple(param.shape):
        raise PsgdError("psgd_adam_attach", PSGD_EINVAL, "param, m1 and m2 must have the same shape")
    return psgd_adam_matrix(_ptr(param), param.stride(0), _ptr(m1), _ptr(m2))


def make_adam_tensor(param, m1, m2, grad) -> psgd_adam_tensor:
    """psgd_adam_tensor over contiguous fp32 torch tensors of one size (param, m1, m2 may be
    None for psgd_adam_prepare, which reads the gradient only)."""
    for t in (param, m1, m2, grad):
        if t is not None and (not t.is_contiguous() or t.numel() != grad.numel() or t.element_size() != 4):
            raise PsgdError("psgd_adam_update", PSGD_EINVAL, "pass-through tensors must be contiguous fp32 of one size")
    return psgd_adam_tensor(_ptr(param), _ptr(m1), _ptr(m2), _ptr(grad), grad.numel())


def _hparams(hp) -> psgd_adam_hparams:
    if isinstance(hp, psgd_adam_hparams):
        return hp
    return psgd_adam_hparams(float(hp.lr), float(hp.beta1), float(hp.beta2), float(hp.eps),
                             float(hp.weight_decay))


def psgd_adam_attach(ctx: int, plan: int, opt: Sequence[psgd_adam_matrix], param_dtype: int) -> None:
    arr = (psgd_adam_matrix * len(opt))(*opt)
    _check(ctx, "psgd_adam_attach", load_library().psgd_adam_attach(ctx, plan, arr, param_dtype))


def psgd_adam_prepare(ctx: int, plan: int, passthrough: Sequence[psgd_adam_tensor], max_norm: float,
                      skip_dev, step_dev, norm_dev, stream=None) -> None:
    arr = (psgd_adam_tensor * max(1, len(passthrough)))(*passthrough)
    _check(ctx, "psgd_adam_prepare",
           load_library().psgd_adam_prepare(ctx, plan, arr, len(passthrough), float(max_norm), _ptr(skip_dev),
                                            _ptr(step_dev), _ptr(norm_dev), _stream(stream)))


def psgd_decompress_adam(ctx: int, plan: int, scale, skip_dev, step_dev, norm_dev, hp, stream=None) -> None:
    h = _hparams(hp)
    _check(ctx, "psgd_decompress_adam",
           load_library().psgd_decompress_adam(ctx, plan, _ptr(scale), _ptr(skip_dev), _ptr(step_dev),
                                               _ptr(norm_dev), ctypes.byref(h), _stream(stream)))


def psgd_adam_update(ctx: int, passthrough: Sequence[psgd_adam_tensor], skip_dev, step_dev, norm_dev, hp,
                     stream=None) -> None:
    arr = (psgd_adam_tensor * max(1, len(passthrough)))(*passthrough)
    h = _hparams(hp)
    _check(ctx, "psgd_adam_update",
           load_library().psgd_adam_update(ctx, arr, len(passthrough), _ptr(skip_dev), _ptr(step_dev),
                                           _ptr(norm_dev), ctypes.byref(h), _stream(stream)))


def _block_dtype(t, call: str) -> int:
    import torch
    if t.dtype == torch.float16:
        return PSGD_F16
    if t.dtype == torch.bfloat16:
        return PSGD_BF16
    raise PsgdError(call, PSGD_EDTYPE, f"block gradients must be float16 or bfloat16, got {t.dtype}")


def psgd_block_grad_enter(ctx: int, dx, scale, out, stream=None) -> None:
    """out = to16(S_b * dx): a contiguous fp32 gradient entering a resblock, scaled by the
    block's factor (scale: one-element fp32 device tensor) into the 16-bit tensor out."""
    if dx.numel() != out.numel() or not dx.is_contiguous() or not out.is_contiguous():
        raise PsgdError("psgd_block_grad_enter", PSGD_EINVAL,
                        "dx and out must be contiguous with the same number of elements")
    _check(ctx, "psgd_block_grad_enter",
           load_library().psgd_block_grad_enter(ctx, _ptr(dx), dx.numel(), _ptr(scale), _ptr(out),
                                                _block_dtype(out, "psgd_block_grad_enter"), _stream(stream)))


def psgd_block_grad_exit(ctx: int, dx, g, scale, flag=None, stream=None) -> None:
    """dx += g / S_b over the finite elements of the 16-bit block output g (Inf/NaN add 0);
    flag (one-element uint8 device tensor, or None) is set to 1 if g held Inf/NaN."""
    if dx.numel() != g.numel() or not dx.is_contiguous() or not g.is_contiguous():
        raise PsgdError("psgd_block_grad_exit", PSGD_EINVAL,
                        "dx and g must be contiguous with the same number of elements")
    _check(ctx, "psgd_block_grad_exit",
           load_library().psgd_block_grad_exit(ctx, _ptr(dx), _ptr(g), dx.numel(), _ptr(scale),
                                               _block_dtype(g, "psgd_block_grad_exit"), None if flag is None else _ptr(flag),
                                               _stream(stream)))


def psgd_block_grad_exit_enter(ctx: int, dx, g, scale_exit, scale_enter, out, flag=None, stream=None) -> None:
    """Leave block b (dx += g / S_b over finite g) and enter block b - 1 (out = to16(S_{b-1} dx))
    in one pass; g and out are 16-bit tensors of the same dtype."""
    if not (dx.numel() == g.numel() == out.numel()) or not (dx.is_contiguous() and g.is_contiguous() and out.is_contiguous()):
        raise PsgdError("psgd_block_grad_exit_enter", PSGD_EINVAL,
                        "dx, g and out must be contiguous with the same number of elements")
    if g.dtype != out.dtype:
        raise PsgdError("psgd_block_grad_exit_enter", PSGD_EDTYPE, "g and out must have the same 16-bit dtype")
    _check(ctx, "psgd_block_grad_exit_enter",
           load_library().psgd_block_grad_exit_enter(ctx, _ptr(dx), _ptr(g), dx.numel(), _ptr(scale_exit),
                                                     _ptr(scale_enter), _ptr(out),
                                                     _block_dtype(g, "psgd_block_grad_exit_enter"),
                                                     _ptr(flag), _stream(stream)))


def ns_hparams(a: float = 3.4445, b: float = -4.7750, c: float = 2.0315, steps: int = 5,
               eps: float = 1e-20) -> psgd_ns_hparams:
    """Newton-Schulz coefficients of X <- a X + (b A + c A A) X, A = X X^T, and the smallest norm
    an update is divided by."""
    return psgd_ns_hparams(a, b, c, eps, steps)


def muon_hparams(lr: float, momentum: float = 0.95, weight_decay: float = 0.0, nesterov: bool = True, adjust: int = 1,
                 **ns) -> psgd_muon_hparams:
    """Scalars of psgd_muon_update; further keywords go to ns_hparams."""
    return psgd_muon_hparams(lr, momentum, weight_decay, int(nesterov), adjust, ns_hparams(**ns))


def make_ns_matrix(update, out) -> psgd_ns_matrix:
    """psgd_ns_matrix over torch tensors of one 2-D shape with unit row stride."""
    call = "psgd_ns_plan_create"
    if update.dim() != 2 or tuple(update.shape) != tuple(out.shape):
        raise PsgdError(call, PSGD_EINVAL, "update and out must be 2-D tensors of one shape")
    return psgd_ns_matrix(_ptr(update), _row_stride(update, call), _ptr(out), _row_stride(out, call), *update.shape)


def make_muon_matrix(param, momentum) -> psgd_muon_matrix:
    """psgd_muon_matrix over torch tensors: param m x n (unit row stride), momentum contiguous fp32."""
    import torch
    call = "psgd_muon_attach"
    if tuple(param.shape) != tuple(momentum.shape) or param.dim() != 2:
        raise PsgdError(call, PSGD_EINVAL, "param and momentum must be 2-D tensors of one shape")
    if momentum.dtype != torch.float32:
        raise PsgdError(call, PSGD_EDTYPE, "momentum must be float32")
    if not momentum.is_contiguous():
        raise PsgdError(call, PSGD_EINVAL, "momentum must be contiguous")
    return psgd_muon_matrix(_ptr(param), _row_stride(param, call), _ptr(momentum))


def _row_stride(t, call: str) -> int:
    """Leading dimension of a 2-D tensor whose rows are contiguous and do not overlap."""
    m, n = t.shape
    ld, one = t.stride()
    if n > 1 and one != 1:
        raise PsgdError(call, PSGD_EINVAL, "tensors need unit stride along rows")
    if m <= 1:
        return max(n, 1)                     # one row: its stride is never used
    if ld < n:
        raise PsgdError(call, PSGD_EINVAL, "the rows of a tensor must not overlap")
    return ld


@functools.lru_cache(maxsize=None)
def _codes():
    """torch dtype -> code, of values and of ids."""
    import torch
    return ({torch.float16: PSGD_F16, torch.bfloat16: PSGD_BF16, torch.float32: PSGD_F32},
            {torch.int32: PSGD_I32, torch.int64: PSGD_I64})


def _dtype(t, call: str) -> int:
    code = _codes()[0].get(t.dtype)
    if code is None:
        raise PsgdError(call, PSGD_EDTYPE, f"tensors must be float16, bfloat16 or float32, got {t.dtype}")
    return code


def psgd_ns_plan_create(ctx: int, mats: Sequence[psgd_ns_matrix], in_dtype: int, out_dtype: int,
                        precision: int = PSGD_NS_FAST) -> int:
    arr = (psgd_ns_matrix * max(1, len(mats)))(*mats)
    h = ctypes.c_void_p()
    _check(ctx, "psgd_ns_plan_create",
           load_library().psgd_ns_plan_create(ctx, arr, len(mats), in_dtype, out_dtype, precision, ctypes.byref(h)))
    return h.value


def psgd_ns_plan_destroy(plan: int) -> None:
    load_library().psgd_ns_plan_destroy(plan)


def psgd_newton_schulz(ctx: int, plan: int, hp: Optional[psgd_ns_hparams] = None, stream=None) -> None:
    """Orthogonalise every matrix of the plan, on the current stream of the context's device by default."""
    _check(ctx, "psgd_newton_schulz",
           load_library().psgd_newton_schulz(ctx, plan, ctypes.byref(hp or ns_hparams()),
                                             _stream(stream, _ctx_device.get(ctx))))


def psgd_muon_attach(ctx: int, plan: int, opt: Sequence[psgd_muon_matrix], param_dtype: int,
                     precision: int = PSGD_NS_FAST) -> None:
    arr = (psgd_muon_matrix * max(1, len(opt)))(*opt)
    _check(ctx, "psgd_muon_attach", load_library().psgd_muon_attach(ctx, plan, arr, param_dtype, precision))


def psgd_muon_update(ctx: int, plan: int, skip_dev, norm_dev, hp: psgd_muon_hparams, stream=None) -> None:
    """One Muon step of every matrix of the plan on its decompressed gradient (norm_dev may be None), on
    the current stream of the context's device by default."""
    _check(ctx, "psgd_muon_update",
           load_library().psgd_muon_update(ctx, plan, _ptr(skip_dev), _ptr(norm_dev), ctypes.byref(hp),
                                           _stream(stream, _ctx_device.get(ctx))))


def _ids(ids, call: str):
    code = _codes()[1].get(ids.dtype)
    if code is None:
        raise PsgdError(call, PSGD_EDTYPE, f"ids must be int32 or int64, got {ids.dtype}")
    if not ids.is_contiguous():
        raise PsgdError(call, PSGD_EINVAL, "ids must be contiguous")
    return code


def _embed_rows(t, n: int, dim: int, name: str, call: str) -> int:
    """Row stride of a tensor that holds one row of dim values per token (2-D, or contiguous with
    the tokens spread over the leading dimensions)."""
    shape = t.shape
    if shape == (n, dim):
        return _row_stride(t, call)
    if len(shape) < 2 or shape[-1] != dim or t.numel() != n * dim:
        raise PsgdError(call, PSGD_EINVAL, f"{name} must hold one row of {dim} values per token")
    if len(shape) > 2:
        if not t.is_contiguous():
            raise PsgdError(call, PSGD_EINVAL, f"{name} with more than two dimensions must be contiguous")
        return dim
    return _row_stride(t, call)


def _same_device(call: str, *tensors, ctx: int = 0):
    """All on one GPU, and on the context's: its device is the one that the kernels are launched on."""
    device = tensors[0].device
    if device.type != "cuda" or any(t.device != device for t in tensors):
        raise PsgdError(call, PSGD_EINVAL, "tensors must live on one GPU")
    if _ctx_device.get(ctx, device.index) != device.index:
        raise PsgdError(call, PSGD_EINVAL, f"tensors live on {device}, the context on device {_ctx_device[ctx]}")


def psgd_embed_lookup(ctx: int, table, ids, out, scale: float = 1.0, stream=None) -> None:
    """out[t] = round(scale * table[ids[t]]) over all tokens of ids (any shape; out has one row per
    token); a row of zeros where the id lies outside the table."""
    call = "psgd_embed_lookup"
    if table.dim() != 2 or table.shape[0] < 1 or table.shape[1] < 1:
        raise PsgdError(call, PSGD_EINVAL, "table must be a vocab x dim tensor")
    vocab, dim = table.shape
    ld_out = _embed_rows(out, ids.numel(), dim, "out", call)
    _same_device(call, table, ids, out, ctx=ctx)
    _check(ctx, call, load_library().psgd_embed_lookup(
        ctx, _ptr(table), _row_stride(table, call), vocab, dim, _dtype(table, call), _ptr(ids), _ids(ids, call),
        ids.numel(), float(scale), _ptr(out), ld_out, _dtype(out, call), _stream(stream, table.device.index)))


def psgd_embed_grad_workspace(n: int, vocab: int, dim: int) -> int:
    """Bytes of device workspace of psgd_embed_grad for up to n tokens."""
    out = ctypes.c_int64()
    _check(None, "psgd_embed_grad_workspace", load_library().psgd_embed_grad_workspace(n, vocab, dim, ctypes.byref(out)))
    return out.value


def psgd_embed_grad(ctx: int, dx, ids, dtable, scale: float = 1.0, accumulate: bool = False, workspace=None,
                    stream=None) -> None:
    """dtable[v] = (accumulate: dtable[v] +) scale * sum of dx[t] over the tokens with ids[t] = v.
    dtable is vocab x dim fp32; workspace is a contiguous device tensor of at least
    psgd_embed_grad_workspace(...) bytes, allocated for the call on its stream when None."""
    import torch
    call = "psgd_embed_grad"
    if dtable.dim() != 2 or dtable.shape[0] < 1 or dtable.shape[1] < 1:
        raise PsgdError(call, PSGD_EINVAL, "dtable must be a vocab x dim tensor")
    if dtable.dtype != torch.float32:
        raise PsgdError(call, PSGD_EDTYPE, "dtable must be float32")
    vocab, dim = dtable.shape
    n = ids.numel()
    ld_dx, ld_dt = _embed_rows(dx, n, dim, "dx", call), _row_stride(dtable, call)
    dt, it = _dtype(dx, call), _ids(ids, call)
    _same_device(call, dx, ids, dtable, *([] if workspace is None else [workspace]), ctx=ctx)
    if workspace is None:
        need = psgd_embed_grad_workspace(n, vocab, dim)
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dtable.device)
        else:
            # allocated on the stream that uses it, so that its memory is not handed out earlier
            s = stream
            if isinstance(stream, int):
                s = torch.cuda.ExternalStream(stream, dtable.device) if stream else torch.cuda.default_stream(dtable.device)
            with torch.cuda.stream(s):
                workspace = torch.empty(need, dtype=torch.uint8, device=dtable.device)
    elif not workspace.is_contiguous():
        raise PsgdError(call, PSGD_EINVAL, "workspace must be contiguous")
    _check(ctx, call, load_library().psgd_embed_grad(
        ctx, _ptr(dx), ld_dx, dt, _ptr(ids), it, n, vocab, dim, float(scale), _ptr(dtable), ld_dt, int(accumulate),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream, dtable.device.index)))


def psgd_last_error(ctx: int) -> str:
    raw = load_library().psgd_last_error(ctx)
    return raw.decode() if raw else ""


def psgd_debug_buffer(plan: int, which: int, mat: int):
    """(device address, bytes, rpad) of an internal buffer of a plan."""
    ptr, nbytes, rpad = ctypes.c_void_p(), ctypes.c_int64(), ctypes.c_int32()
    _check(None, "psgd_debug_buffer",
           load_library().psgd_debug_buffer(plan, which, mat, ctypes.byref(ptr), ctypes.byref(nbytes),
                                            ctypes.byref(rpad)))
    return ptr.value, nbytes.value, rpad.value


def psgd_profile_events(ctx: int, events: Optional[List[int]]) -> None:
    """Install (or with None remove) HIP events recorded around every kernel launch: event
    2*k before and 2*k+1 after the launch of slot k of PROFILE_SLOTS."""
    if events is None:
        _check(ctx, "psgd_profile_events", load_library().psgd_profile_events(ctx, None, 0))
        return
    arr = (ctypes.c_void_p * len(events))(*events)
    _check(ctx, "psgd_profile_events", load_library().psgd_profile_events(ctx, arr, len(events)))
