"""Python binding of the training operators of libzerostep.so (zero_train.h):
8-bit block conversion and product, residual RMS norm, distillation loss.

Argument marshalling only, as in the package's main binding, which re-exports
every name here.  Matrices are 2-D device tensors whose rows are contiguous;
a row stride above the row's length is passed on.  8-bit data are
torch.float8_e4m3fn or torch.float8_e5m2 tensors, scales torch.float8_e8m0fnu
(or uint8) tensors, in the layout of zero_train.h; ``q8_empty`` allocates a
pair.  Calls run on ``stream``, by default the current stream of the tensors'
device, which need not be the current device.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import StepControl, ZeroStepError, _check, _ctl, lib

ZERO_F32, ZERO_F16, ZERO_BF16 = 0, 1, 2
ZERO_E4M3, ZERO_E5M2 = 0, 1
ZERO_Q8_BLOCK = 128
ZERO_Q8_MAX_LD = 8388608
ZERO_NORM_MAX_COLS = 65536
ZERO_NORM_MAX_PARTS = 1024
ZERO_DISTILL_MAX_TOP = 1024

EXPORTED = ("zero_q8_quantize", "zero_q8_quantize_ctl", "zero_q8_gemm", "zero_rmsnorm",
            "zero_rmsnorm_backward_workspace", "zero_rmsnorm_backward", "zero_distill_forward",
            "zero_distill_backward", "zero_distill")

_ELEM = {torch.float32: ZERO_F32, torch.float16: ZERO_F16, torch.bfloat16: ZERO_BF16}
_FP8 = {torch.float8_e4m3fn: ZERO_E4M3, torch.float8_e5m2: ZERO_E5M2}
_SCALE = {torch.float8_e8m0fnu: 0, torch.uint8: 0}
_INDEX = {torch.int32: 4, torch.int64: 8}


class DistillInputs(ctypes.Structure):
    """zero_distill_inputs"""
    _fields_ = [("logits", ctypes.c_void_p), ("top_index", ctypes.c_void_p),
                ("top_logit", ctypes.c_void_p), ("row_weight", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("vocab", ctypes.c_int64),
                ("ld_logits", ctypes.c_int64), ("ld_top", ctypes.c_int64),
                ("logits_dtype", ctypes.c_int32), ("top_dtype", ctypes.c_int32),
                ("index_bytes", ctypes.c_int32), ("top", ctypes.c_int32),
                ("temperature", ctypes.c_float), ("pad_", ctypes.c_int32)]


def _declare() -> None:
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    mat = [vp, i32, i64]
    q8_out = [vp, i64, vp, i64]
    lib.zero_q8_quantize.argtypes = [vp, i32, i64, i64, i64, i32, *q8_out, *q8_out, vp]
    lib.zero_q8_quantize_ctl.argtypes = [ctypes.POINTER(vp), i64, i64, i64, i32, *q8_out, *q8_out,
                                         vp, vp]
    lib.zero_q8_gemm.argtypes = [*mat, vp, i64, *mat, vp, i64, i64, i64, i64, vp, i32, i64, i32,
                                 vp]
    lib.zero_rmsnorm.argtypes = [*mat, *mat, vp, i32, i64, i64, f32, vp, i64, *mat, vp, i32, i64,
                                 vp, i64, vp, vp]
    lib.zero_rmsnorm_backward_workspace.argtypes = [i64, i64]
    lib.zero_rmsnorm_backward.argtypes = [*mat, *mat, vp, i32, vp, *mat, i64, i64, *mat, vp, i32,
                                          vp, i64, vp]
    inputs = ctypes.POINTER(DistillInputs)
    lib.zero_distill_forward.argtypes = [inputs, vp, vp, vp]
    lib.zero_distill_backward.argtypes = [inputs, vp, f32, vp, vp, i64, vp]
    lib.zero_distill.argtypes = [inputs, f32, vp, vp, vp, vp, i64, vp]
    for name in EXPORTED:
        getattr(lib, name).restype = ctypes.c_int
    lib.zero_rmsnorm_backward_workspace.restype = ctypes.c_int64


_declare()


# What a call looks at is written out below rather than wrapped in objects: a
# short call's time is the host's.

def _mat(t: torch.Tensor, kinds: dict, dev: torch.device, name: str) -> Tuple[int, int, int]:
    """(pointer, type code, row stride) of a matrix on dev.  A single row's
    stride says nothing: it counts as the row's length, rounded up to what the
    q8 layout asks of strides."""
    code = kinds.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} has dtype {t.dtype}")
    if t.device != dev:
        raise TypeError(f"{name} is on {t.device}, expected {dev}")
    stride = t.stride()
    if len(stride) != 2:
        raise ValueError(f"{name} has {len(stride)} dimensions, expected 2")
    ld, inner = stride
    rows, cols = t.shape
    if inner != 1 and cols > 1:
        raise ValueError(f"the rows of {name} are not contiguous")
    if rows <= 1:
        ld = (cols + 15) & -16
    return t.data_ptr(), code, ld


def _like(t: torch.Tensor, shape, kinds: dict, dev: torch.device, name: str):
    """_mat of a matrix of this shape."""
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return _mat(t, kinds, dev, name)


def _vec(t: torch.Tensor, n: int, kinds: dict, dev: torch.device, name: str) -> Tuple[int, int]:
    """(pointer, type code) of a contiguous vector of n elements on dev."""
    code = kinds.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} has dtype {t.dtype}")
    if t.device != dev:
        raise TypeError(f"{name} is on {t.device}, expected {dev}")
    if t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} elements, expected {n}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr(), code


def _q8(data: Optional[torch.Tensor], scales: Optional[torch.Tensor], rows: int, cols: int,
        dev: torch.device, name: str, fmt: Optional[int] = None):
    """(data pointer, ld, scale pointer, ld, format) of a q8 matrix."""
    if data is None or scales is None:
        if data is not None or scales is not None:
            raise ValueError(f"{name}: data and scales go together")
        return None, 0, None, 0, fmt
    p, code, ld = _mat(data, _FP8, dev, name)
    if fmt is not None and code != fmt:
        raise TypeError(f"{name} has dtype {data.dtype}, unlike the other output")
    ps, _, lds = _mat(scales, _SCALE, dev, name)
    blocks = -(-cols // ZERO_Q8_BLOCK)
    have, wide = data.shape
    if have != rows or wide < blocks * ZERO_Q8_BLOCK:
        raise ValueError(f"{name} has shape {tuple(data.shape)}, expected {rows} rows of "
                         f"{blocks * ZERO_Q8_BLOCK}")
    have, wide = scales.shape
    if have != rows or wide < -(-blocks // 4) * 4:
        raise ValueError(f"scales of {name} have shape {tuple(scales.shape)}, expected "
                         f"{rows} rows of {-(-blocks // 4) * 4}")
    return p, ld, ps, lds, code


def _device(t: torch.Tensor) -> torch.device:
    dev = t.device
    if dev.type != "cuda":
        raise TypeError("the tensors must be device tensors")
    return dev


def _raw_stream(stream, dev: torch.device) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev.index)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _run(fn, dev: torch.device, *args) -> None:
    """Make the call with dev current, as the library launches there."""
    if dev.index == torch.cuda.current_device():
        rc = fn(*args)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args)
    if rc:
        _check(rc)


_F32 = {torch.float32: ZERO_F32}
_BYTES = {torch.uint8: 0}


def q8_shape(rows: int, cols: int) -> Tuple[Tuple[int, int], Tuple[int, int]]:
    """Shapes of the data and scale tensors of a rows x cols q8 matrix."""
    blocks = -(-cols // ZERO_Q8_BLOCK)
    return (rows, blocks * ZERO_Q8_BLOCK), (rows, -(-blocks // 4) * 4)


def q8_empty(rows: int, cols: int, dtype: torch.dtype = torch.float8_e4m3fn, device="cuda"):
    """Uninitialised (data, scales) of a rows x cols q8 matrix."""
    data, scales = q8_shape(rows, cols)
    return (torch.empty(data, dtype=dtype, device=device),
            torch.empty(scales, dtype=torch.float8_e8m0fnu, device=device))


def zero_q8_quantize(src: torch.Tensor, q: Optional[torch.Tensor] = None,
                     s: Optional[torch.Tensor] = None, qt: Optional[torch.Tensor] = None,
                     st: Optional[torch.Tensor] = None, stream=None) -> None:
    """src [rows, cols] in the q8 layout, by rows into (q, s), transposed into
    (qt, st), or both; the 8-bit format is the outputs' dtype (see
    zero_train.h)."""
    dev = _device(src)
    p, dt, ld = _mat(src, _ELEM, dev, "src")
    rows, cols = src.shape
    pq, ldq, ps, lds, fmt = _q8(q, s, rows, cols, dev, "q")
    pt, ldt, pst, ldst, fmt = _q8(qt, st, cols, rows, dev, "qt", fmt)
    _run(lib.zero_q8_quantize, dev, p, dt, rows, cols, ld, ZERO_E4M3 if fmt is None else fmt, pq,
         ldq, ps, lds, pt, ldt, pst, ldst, _raw_stream(stream, dev))


def zero_q8_quantize_ctl(srcs_fp16, ctl: torch.Tensor, q: Optional[torch.Tensor] = None,
                         s: Optional[torch.Tensor] = None, qt: Optional[torch.Tensor] = None,
                         st: Optional[torch.Tensor] = None, stream=None) -> None:
    """zero_q8_quantize of the copy the control block says is current: srcs_fp16
    are the same fp16 matrix in the two copies of the parameters."""
    first, second = srcs_fp16
    dev = _device(first)
    rows, cols = first.shape
    half = {torch.float16: ZERO_F16}
    p0, _, ld = _mat(first, half, dev, "srcs_fp16[0]")
    p1, _, ld1 = _like(second, (rows, cols), half, dev, "srcs_fp16[1]")
    if ld1 != ld:
        raise ValueError("the two copies have different row strides")
    if ctl.device != dev:
        raise TypeError(f"ctl is on {ctl.device}, expected {dev}")
    pq, ldq, ps, lds, fmt = _q8(q, s, rows, cols, dev, "q")
    pt, ldt, pst, ldst, fmt = _q8(qt, st, cols, rows, dev, "qt", fmt)
    _run(lib.zero_q8_quantize_ctl, dev, (ctypes.c_void_p * 2)(p0, p1), rows, cols, ld,
         ZERO_E4M3 if fmt is None else fmt, pq, ldq, ps, lds, pt, ldt, pst, ldst, _ctl(ctl),
         _raw_stream(stream, dev))


def zero_q8_gemm(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor,
                 c: torch.Tensor, k: Optional[int] = None, accumulate: bool = False,
                 stream=None) -> None:
    """c [m, n] = a b^T of q8 matrices a [m, k] and b [n, k] (added to c with
    ``accumulate``).  k defaults to a's padded row length."""
    dev = _device(c)
    pc, dt, ldc = _mat(c, _ELEM, dev, "c")
    m, n = c.shape
    if k is None:
        k = a.shape[1]
        if b.shape[1] != k:
            raise ValueError(f"a has rows of {k}, b of {b.shape[1]}")
    pa, lda, psa, ldsa, fa = _q8(a, sa, m, k, dev, "a")
    pb, ldb, psb, ldsb, fb = _q8(b, sb, n, k, dev, "b")
    _run(lib.zero_q8_gemm, dev, pa, fa, lda, psa, ldsa, pb, fb, ldb, psb, ldsb, m, n, k, pc, dt,
         ldc, 1 if accumulate else 0, _raw_stream(stream, dev))


def zero_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float, *,
                 residual: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                 y: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                 s: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                 stream=None) -> None:
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight, into y, or in
    the q8 layout into (q, s), or both; rstd and the rounded h for the
    backward pass (see zero_train.h)."""
    dev = _device(x)
    px, dx, ldx = _mat(x, _ELEM, dev, "x")
    rows, cols = shape = x.shape
    pw, dw = _vec(weight, cols, _ELEM, dev, "weight")
    pr, dr, ldr = (None, ZERO_F32, 0) if residual is None else \
        _like(residual, shape, _ELEM, dev, "residual")
    ph, ldh = None, 0
    if h is not None:
        if residual is not None and h.dtype != residual.dtype:
            raise TypeError(f"h has dtype {h.dtype}, residual {residual.dtype}")
        ph, _, ldh = _like(h, shape, _ELEM, dev, "h")
    py, dy, ldy = (None, ZERO_F32, 0) if y is None else _like(y, shape, _ELEM, dev, "y")
    pq, ldq, ps, lds, fmt = _q8(q, s, rows, cols, dev, "q")
    prstd = None if rstd is None else _vec(rstd, rows, _F32, dev, "rstd")[0]
    _run(lib.zero_rmsnorm, dev, px, dx, ldx, pr, dr, ldr, pw, dw, rows, cols, eps, ph, ldh, py, dy,
         ldy, pq, fmt or ZERO_E4M3, ldq, ps, lds, prstd, _raw_stream(stream, dev))


def zero_rmsnorm_backward_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace zero_rmsnorm_backward needs."""
    n = lib.zero_rmsnorm_backward_workspace(int(rows), int(cols))
    if n < 0:
        raise ZeroStepError(-1, lib.zero_last_error_string().decode())
    return n


def zero_rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor,
                          rstd: torch.Tensor, dx: torch.Tensor, dw: Optional[torch.Tensor],
                          workspace: Optional[torch.Tensor], *,
                          dres: Optional[torch.Tensor] = None, stream=None) -> None:
    """dx (of x and of residual, with dres, the gradient at h, added) and dw;
    workspace: uint8, zero_rmsnorm_backward_workspace bytes, not needed when
    dw is None (see zero_train.h)."""
    dev = _device(dy)
    pd, dd, ldd = _mat(dy, _ELEM, dev, "dy")
    rows, cols = shape = dy.shape
    ph, dh, ldh = _like(h, shape, _ELEM, dev, "h")
    pw, dwt = _vec(weight, cols, _ELEM, dev, "weight")
    prstd, _ = _vec(rstd, rows, _F32, dev, "rstd")
    pr, dr, ldr = (None, ZERO_F32, 0) if dres is None else _like(dres, shape, _ELEM, dev, "dres")
    px, dxt, ldx = _like(dx, shape, _ELEM, dev, "dx")
    pdw, ddw = (None, ZERO_F32) if dw is None else _vec(dw, cols, _ELEM, dev, "dw")
    pws, nws = (None, 0) if workspace is None else \
        (_vec(workspace, workspace.numel(), _BYTES, dev, "workspace")[0], workspace.numel())
    _run(lib.zero_rmsnorm_backward, dev, pd, dd, ldd, ph, dh, ldh, pw, dwt, prstd, pr, dr, ldr,
         rows, cols, px, dxt, ldx, pdw, ddw, pws, nws, _raw_stream(stream, dev))


def _distill_inputs(dev: torch.device, logits, index, teacher, temperature, row_weight):
    p, dt, ld = _mat(logits, _ELEM, dev, "logits")
    rows, vocab = logits.shape
    if index.dim() != 2:
        raise ValueError(f"index has {index.dim()} dimensions, expected 2")
    top = index.shape[1]
    pi, ib, ldi = _like(index, (rows, top), _INDEX, dev, "index")
    pt, tt, ldt = _like(teacher, (rows, top), _ELEM, dev, "teacher")
    if ldi != ldt:
        raise ValueError("index and teacher have different row strides")
    pw = None if row_weight is None else _vec(row_weight, rows, _F32, dev, "row_weight")[0]
    return DistillInputs(p, pi, pt, pw, rows, vocab, ld, ldi, dt, tt, ib, top, temperature, 0)


def _distill_scale(dev: torch.device, ctl):
    if ctl is None:
        return None
    if ctl.device != dev:
        raise TypeError(f"ctl is on {ctl.device}, expected {dev}")
    return _ctl(ctl)


def _distill_grad(dev: torch.device, grad, logits):
    if grad.dtype != logits.dtype:
        raise TypeError(f"grad has dtype {grad.dtype}, logits {logits.dtype}")
    p, _, ld = _like(grad, logits.shape, _ELEM, dev, "grad")
    return p, ld


def zero_distill_forward(logits: torch.Tensor, index: torch.Tensor, teacher: torch.Tensor,
                         loss: Optional[torch.Tensor], lse: Optional[torch.Tensor], *,
                         temperature: float = 1.0, row_weight: Optional[torch.Tensor] = None,
                         stream=None) -> None:
    """Per-row loss and lse (fp32[rows]) of the student's logits [rows, vocab]
    against the teacher's entries: vocab indices [rows, top] (-1: no entry) and
    logits [rows, top] (see zero_distill_inputs in zero_train.h)."""
    dev = _device(logits)
    rows = logits.shape[0]
    inputs = _distill_inputs(dev, logits, index, teacher, temperature, row_weight)
    pl = None if loss is None else _vec(loss, rows, _F32, dev, "loss")[0]
    pe = None if lse is None else _vec(lse, rows, _F32, dev, "lse")[0]
    _run(lib.zero_distill_forward, dev, ctypes.byref(inputs), pl, pe, _raw_stream(stream, dev))


def zero_distill_backward(logits: torch.Tensor, index: torch.Tensor, teacher: torch.Tensor,
                          lse: torch.Tensor, grad: torch.Tensor, *, temperature: float = 1.0,
                          row_weight: Optional[torch.Tensor] = None, loss_scale: float = 1.0,
                          ctl: Optional[torch.Tensor] = None, stream=None) -> None:
    """The loss-scaled gradient of the logits, from the forward's lse.  S is
    loss_scale, or the scale of the control block ``ctl``; grad may be logits."""
    dev = _device(logits)
    inputs = _distill_inputs(dev, logits, index, teacher, temperature, row_weight)
    pe = _vec(lse, logits.shape[0], _F32, dev, "lse")[0]
    pg, ldg = _distill_grad(dev, grad, logits)
    _run(lib.zero_distill_backward, dev, ctypes.byref(inputs), pe, loss_scale,
         _distill_scale(dev, ctl), pg, ldg, _raw_stream(stream, dev))


def zero_distill(logits: torch.Tensor, index: torch.Tensor, teacher: torch.Tensor,
                 loss: Optional[torch.Tensor], lse: Optional[torch.Tensor], grad: torch.Tensor, *,
                 temperature: float = 1.0, row_weight: Optional[torch.Tensor] = None,
                 loss_scale: float = 1.0, ctl: Optional[torch.Tensor] = None,
                 stream=None) -> None:
    """zero_distill_forward and zero_distill_backward in one pass."""
    dev = _device(logits)
    rows = logits.shape[0]
    inputs = _distill_inputs(dev, logits, index, teacher, temperature, row_weight)
    pl = None if loss is None else _vec(loss, rows, _F32, dev, "loss")[0]
    pe = None if lse is None else _vec(lse, rows, _F32, dev, "lse")[0]
    pg, ldg = _distill_grad(dev, grad, logits)
    _run(lib.zero_distill, dev, ctypes.byref(inputs), loss_scale, _distill_scale(dev, ctl), pl, pe,
         pg, ldg, _raw_stream(stream, dev))
