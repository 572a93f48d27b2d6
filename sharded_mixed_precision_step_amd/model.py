"""Python binding of zero_model.h's operators in libzerostep.so: embedding,
layer norm, activation with 8-bit checkpoints, log probabilities.

Argument marshalling only, with the training operators' conventions (train.py):
matrices are 2-D device tensors with contiguous rows, 8-bit matrices are (data,
scales) pairs as ``q8_empty`` allocates them, calls run on ``stream``, by default
the current stream of the tensors' device.  The package re-exports every name.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import ZeroStepError, _ctl, _marshal, lib
from .train import (_BYTES, _ELEM, _F32, _INDEX, ZERO_E4M3, ZERO_F16, ZERO_F32, _device,
                    _distill_scale, _like, _mat, _q8, _raw_stream, _run, _vec)

ZERO_EMBED_MAX_TOKENS = 16777216
ZERO_LAYERNORM_MAX_COLS = 65536
ZERO_LOGPROB_MAX_TOP = 128
ZERO_SILU, ZERO_GELU, ZERO_GELU_TANH = 0, 1, 2

EXPORTED = ("zero_embed", "zero_embed_ctl", "zero_embed_backward_workspace",
            "zero_embed_backward", "zero_layernorm", "zero_layernorm_backward_workspace",
            "zero_layernorm_backward", "zero_act", "zero_act_backward", "zero_logprob",
            "zero_logprob_backward")

_KIND = {"silu": ZERO_SILU, "gelu": ZERO_GELU, "gelu_tanh": ZERO_GELU_TANH}
_INT32 = {torch.int32: 4}
_HALF = {torch.float16: ZERO_F16}


def _declare() -> None:
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    mat = [vp, i32, i64]
    out = [vp, i64]
    q8 = [vp, i64, vp, i64]
    lib.zero_embed.argtypes = [vp, i32, i64, i64, i64, vp, i32, i64, f32, *mat, vp]
    lib.zero_embed_ctl.argtypes = [ctypes.POINTER(vp), i64, i64, i64, vp, i32, i64, f32, *mat, vp,
                                   vp]
    lib.zero_embed_backward_workspace.argtypes = [i64, i64, i64]
    lib.zero_embed_backward.argtypes = [*mat, vp, i32, i64, i64, i64, f32, *mat, i32, vp, i64, vp]
    lib.zero_layernorm.argtypes = [*mat, *mat, vp, vp, i32, i64, i64, f32, *out, *mat, vp, i32, i64,
                                   *out, vp, vp, vp]
    lib.zero_layernorm_backward_workspace.argtypes = [i64, i64]
    lib.zero_layernorm_backward.argtypes = [*mat, *mat, vp, i32, vp, vp, *mat, i64, i64, *mat, vp,
                                            vp, i32, vp, i64, vp]
    lib.zero_act.argtypes = [*out, *out, i32, i32, i64, i64, *mat, vp, i32, i64, *out, vp, i32, i64,
                             *out, *q8, vp]
    lib.zero_act_backward.argtypes = [*mat, vp, i32, i64, *out, *q8, i32, i64, i64, *out, *out, i32,
                                      *mat, vp]
    lib.zero_logprob.argtypes = [*mat, i64, i64, vp, i32, f32, vp, vp, vp, vp, vp, i32, i64, vp]
    lib.zero_logprob_backward.argtypes = [*mat, i64, i64, vp, i32, f32, vp, vp, vp, vp, f32, vp,
                                          *out, vp]
    for name in EXPORTED:
        getattr(lib, name).restype = ctypes.c_int
    lib.zero_embed_backward_workspace.restype = i64
    lib.zero_layernorm_backward_workspace.restype = i64


_declare()
# the calls that a program makes often, without ctypes' conversions (csrc/marshal.cpp) where
# that library is there
_calls = lib
if _marshal is not None:
    _marshal.bind({name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
                   for name in EXPORTED})
    _calls = _marshal


def _optional_vec(t: Optional[torch.Tensor], n: int, kinds: dict, dev: torch.device, name: str):
    return None if t is None else _vec(t, n, kinds, dev, name)[0]


def _workspace(t: Optional[torch.Tensor], dev: torch.device):
    if t is None:
        return None, 0
    n = t.numel()
    return _vec(t, n, _BYTES, dev, "workspace")[0], n


def _bytes(n: int) -> int:
    if n < 0:
        raise ZeroStepError(-1, lib.zero_last_error_string().decode())
    return n


def _kind(kind) -> int:
    code = _KIND.get(kind)
    if code is None:
        raise ValueError(f"activation {kind!r}, expected one of {', '.join(_KIND)}")
    return code


def zero_embed(table: torch.Tensor, ids: torch.Tensor, y: torch.Tensor, *, scale: float = 1.0,
               stream=None) -> None:
    """y[r] = scale * table[ids[r]]; ids (int32 or int64) is contiguous, of any
    shape; y is [ids.numel(), cols].  A negative id gives a row of zeros (see
    zero_model.h)."""
    dev = _device(table)
    pt, dt, ldt = _mat(table, _ELEM, dev, "table")
    vocab, cols = table.shape
    tokens = ids.numel()
    pi, ib = _vec(ids, tokens, _INDEX, dev, "ids")
    py, dy, ldy = _like(y, (tokens, cols), _ELEM, dev, "y")
    _run(_calls.zero_embed, dev, pt, dt, vocab, cols, ldt, pi, ib, tokens, scale, py, dy, ldy,
         _raw_stream(stream, dev))


def zero_embed_ctl(tables_fp16, ctl: torch.Tensor, ids: torch.Tensor, y: torch.Tensor, *,
                   scale: float = 1.0, stream=None) -> None:
    """zero_embed from the copy the control block says is current: tables_fp16 are
    the same fp16 table in the two copies of the parameters."""
    first, second = tables_fp16
    dev = _device(first)
    p0, _, ld = _mat(first, _HALF, dev, "tables_fp16[0]")
    vocab, cols = first.shape
    p1, _, ld1 = _like(second, (vocab, cols), _HALF, dev, "tables_fp16[1]")
    if ld1 != ld:
        raise ValueError("the two copies have different row strides")
    if ctl.device != dev:
        raise TypeError(f"ctl is on {ctl.device}, expected {dev}")
    tokens = ids.numel()
    pi, ib = _vec(ids, tokens, _INDEX, dev, "ids")
    py, dy, ldy = _like(y, (tokens, cols), _ELEM, dev, "y")
    _run(lib.zero_embed_ctl, dev, (ctypes.c_void_p * 2)(p0, p1), vocab, cols, ld, pi, ib, tokens,
         scale, py, dy, ldy, _ctl(ctl), _raw_stream(stream, dev))


def zero_embed_backward_workspace(tokens: int, vocab: int, cols: int) -> int:
    """Bytes of workspace zero_embed_backward needs."""
    return _bytes(lib.zero_embed_backward_workspace(int(tokens), int(vocab), int(cols)))


def zero_embed_backward(dy: torch.Tensor, ids: torch.Tensor, dtable: torch.Tensor,
                        workspace: Optional[torch.Tensor], *, scale: float = 1.0,
                        accumulate: bool = False, stream=None) -> None:
    """dtable[v] = scale * sum of dy's rows whose id is v, zeros elsewhere; with
    ``accumulate`` added to the rows that have tokens.  workspace: uint8,
    zero_embed_backward_workspace bytes (see zero_model.h)."""
    dev = _device(dy)
    pd, dd, ldd = _mat(dy, _ELEM, dev, "dy")
    tokens, cols = dy.shape
    pi, ib = _vec(ids, tokens, _INDEX, dev, "ids")
    pt, dt, ldt = _mat(dtable, _ELEM, dev, "dtable")
    vocab, wide = dtable.shape
    if wide != cols:
        raise ValueError(f"dtable has rows of {wide}, dy of {cols}")
    pws, nws = _workspace(workspace, dev)
    _run(_calls.zero_embed_backward, dev, pd, dd, ldd, pi, ib, tokens, vocab, cols, scale, pt, dt,
         ldt, 1 if accumulate else 0, pws, nws, _raw_stream(stream, dev))


def zero_layernorm(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor],
                   eps: float, *, residual: Optional[torch.Tensor] = None,
                   h: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                   q: Optional[torch.Tensor] = None, s: Optional[torch.Tensor] = None,
                   mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                   stream=None) -> None:
    """h = x + residual; y = (h - mean(h)) / sqrt(var(h) + eps) * weight + bias,
    into y, or in the q8 layout into (q, s), or both; mean, rstd and the rounded
    h for the backward pass (see zero_model.h)."""
    dev = _device(x)
    px, dx, ldx = _mat(x, _ELEM, dev, "x")
    rows, cols = shape = x.shape
    pw, dw = _vec(weight, cols, _ELEM, dev, "weight")
    pb = None
    if bias is not None:
        pb, db = _vec(bias, cols, _ELEM, dev, "bias")
        if db != dw:
            raise TypeError(f"bias has dtype {bias.dtype}, weight {weight.dtype}")
    pr, dr, ldr = (None, ZERO_F32, 0) if residual is None else \
        _like(residual, shape, _ELEM, dev, "residual")
    ph, ldh = None, 0
    if h is not None:
        if residual is not None and h.dtype != residual.dtype:
            raise TypeError(f"h has dtype {h.dtype}, residual {residual.dtype}")
        ph, _, ldh = _like(h, shape, _ELEM, dev, "h")
    py, dy, ldy = (None, ZERO_F32, 0) if y is None else _like(y, shape, _ELEM, dev, "y")
    pq, ldq, ps, lds, fmt = _q8(q, s, rows, cols, dev, "q")
    pm = _optional_vec(mean, rows, _F32, dev, "mean")
    prstd = _optional_vec(rstd, rows, _F32, dev, "rstd")
    _run(_calls.zero_layernorm, dev, px, dx, ldx, pr, dr, ldr, pw, pb, dw, rows, cols, eps, ph,
         ldh, py, dy, ldy, pq, fmt or ZERO_E4M3, ldq, ps, lds, pm, prstd, _raw_stream(stream, dev))


def zero_layernorm_backward_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace zero_layernorm_backward needs."""
    return _bytes(lib.zero_layernorm_backward_workspace(int(rows), int(cols)))


def zero_layernorm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor,
                            mean: torch.Tensor, rstd: torch.Tensor, dx: torch.Tensor,
                            dw: Optional[torch.Tensor], db: Optional[torch.Tensor],
                            workspace: Optional[torch.Tensor], *,
                            dres: Optional[torch.Tensor] = None, stream=None) -> None:
    """dx (of x and of residual, with dres, the gradient at h, added), dw and db;
    workspace: uint8, zero_layernorm_backward_workspace bytes, not needed when dw
    and db are None (see zero_model.h)."""
    dev = _device(dy)
    pd, dd, ldd = _mat(dy, _ELEM, dev, "dy")
    rows, cols = shape = dy.shape
    ph, dh, ldh = _like(h, shape, _ELEM, dev, "h")
    pw, dwt = _vec(weight, cols, _ELEM, dev, "weight")
    pm, _ = _vec(mean, rows, _F32, dev, "mean")
    prstd, _ = _vec(rstd, rows, _F32, dev, "rstd")
    pr, dr, ldr = (None, ZERO_F32, 0) if dres is None else _like(dres, shape, _ELEM, dev, "dres")
    px, dxt, ldx = _like(dx, shape, _ELEM, dev, "dx")
    pdw, ddw = (None, None) if dw is None else _vec(dw, cols, _ELEM, dev, "dw")
    pdb, ddb = (None, None) if db is None else _vec(db, cols, _ELEM, dev, "db")
    if dw is not None and db is not None and ddw != ddb:
        raise TypeError(f"dw has dtype {dw.dtype}, db {db.dtype}")
    pws, nws = _workspace(workspace, dev)
    _run(_calls.zero_layernorm_backward, dev, pd, dd, ldd, ph, dh, ldh, pw, dwt, pm, prstd, pr,
         dr, ldr, rows, cols, px, dxt, ldx, pdw, pdb,
         ddw if ddw is not None else ddb if ddb is not None else ZERO_F32, pws, nws,
         _raw_stream(stream, dev))


def zero_act(gate: torch.Tensor, kind: str, *, up: Optional[torch.Tensor] = None,
             y: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
             s: Optional[torch.Tensor] = None, gate_q: Optional[torch.Tensor] = None,
             gate_s: Optional[torch.Tensor] = None, up_q: Optional[torch.Tensor] = None,
             up_s: Optional[torch.Tensor] = None, stream=None) -> None:
    """y = f(gate) * up (or f(gate)), f being ``kind``: "silu", "gelu" or
    "gelu_tanh"; into y, or in the q8 layout into (q, s), or both; gate and up as
    8-bit checkpoints into (gate_q, gate_s) and (up_q, up_s), for
    zero_act_backward (see zero_model.h)."""
    dev = _device(gate)
    code = _kind(kind)
    pg, dt, ldg = _mat(gate, _ELEM, dev, "gate")
    rows, cols = shape = gate.shape
    pu, ldu = None, 0
    if up is not None:
        if up.dtype != gate.dtype:
            raise TypeError(f"up has dtype {up.dtype}, gate {gate.dtype}")
        pu, _, ldu = _like(up, shape, _ELEM, dev, "up")
    py, dy, ldy = (None, ZERO_F32, 0) if y is None else _like(y, shape, _ELEM, dev, "y")
    pq, ldq, ps, lds, fmt = _q8(q, s, rows, cols, dev, "q")
    pgq, ldgq, pgs, ldgs, ck = _q8(gate_q, gate_s, rows, cols, dev, "gate_q")
    puq, lduq, pus, ldus, ck = _q8(up_q, up_s, rows, cols, dev, "up_q", ck)
    _run(_calls.zero_act, dev, pg, ldg, pu, ldu, dt, code, rows, cols, py, dy, ldy, pq,
         fmt or ZERO_E4M3, ldq, ps, lds, pgq, ck or ZERO_E4M3, ldgq, pgs, ldgs, puq, lduq, pus,
         ldus, _raw_stream(stream, dev))


def zero_act_backward(dy: torch.Tensor, gate_q: torch.Tensor, gate_s: torch.Tensor,
                      dgate: torch.Tensor, kind: str, *, up_q: Optional[torch.Tensor] = None,
                      up_s: Optional[torch.Tensor] = None, dup: Optional[torch.Tensor] = None,
                      y: Optional[torch.Tensor] = None, stream=None) -> None:
    """dgate = dy * u * f'(g), dup = dy * f(g) and y = f(g) * u, of the values g
    and u that the checkpoints stand for (see zero_model.h)."""
    dev = _device(dy)
    code = _kind(kind)
    pd, dd, ldd = _mat(dy, _ELEM, dev, "dy")
    rows, cols = shape = dy.shape
    pgq, ldgq, pgs, ldgs, ck = _q8(gate_q, gate_s, rows, cols, dev, "gate_q")
    puq, lduq, pus, ldus, ck = _q8(up_q, up_s, rows, cols, dev, "up_q", ck)
    pg, dx, ldg = _like(dgate, shape, _ELEM, dev, "dgate")
    pu, ldu = None, 0
    if dup is not None:
        if dup.dtype != dgate.dtype:
            raise TypeError(f"dup has dtype {dup.dtype}, dgate {dgate.dtype}")
        pu, _, ldu = _like(dup, shape, _ELEM, dev, "dup")
    py, dyt, ldy = (None, ZERO_F32, 0) if y is None else _like(y, shape, _ELEM, dev, "y")
    _run(_calls.zero_act_backward, dev, pd, dd, ldd, pgq, ck or ZERO_E4M3, ldgq, pgs, ldgs, puq,
         lduq, pus, ldus, code, rows, cols, pg, ldg, pu, ldu, dx, py, dyt, ldy,
         _raw_stream(stream, dev))


def zero_logprob(logits: torch.Tensor, ids: Optional[torch.Tensor],
                 logp: Optional[torch.Tensor], *, entropy: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, top_index: Optional[torch.Tensor] = None,
                 top_logit: Optional[torch.Tensor] = None, temperature: float = 1.0,
                 stream=None) -> None:
    """Per row of logits [rows, vocab]: log probability of ids' token, entropy,
    lse (fp32[rows] each) and the largest logits with their places, top_index
    (int32) and top_logit (the logits' dtype), [rows, top] each, in the form that
    zero_distill takes from a teacher (see zero_model.h)."""
    dev = _device(logits)
    p, dt, ld = _mat(logits, _ELEM, dev, "logits")
    rows, vocab = logits.shape
    pi, ib = (None, 8) if ids is None else _vec(ids, rows, _INDEX, dev, "ids")
    pl = _optional_vec(logp, rows, _F32, dev, "logp")
    pe = _optional_vec(entropy, rows, _F32, dev, "entropy")
    ps = _optional_vec(lse, rows, _F32, dev, "lse")
    pti, ptl, top, ldt = None, None, 0, 0
    if top_index is not None or top_logit is not None:
        if top_index is None or top_logit is None:
            raise ValueError("top_index and top_logit go together")
        if top_index.dim() != 2:
            raise ValueError(f"top_index has {top_index.dim()} dimensions, expected 2")
        top = top_index.shape[1]
        pti, _, ldt = _like(top_index, (rows, top), _INT32, dev, "top_index")
        if top_logit.dtype != logits.dtype:
            raise TypeError(f"top_logit has dtype {top_logit.dtype}, logits {logits.dtype}")
        ptl, _, ldl = _like(top_logit, (rows, top), _ELEM, dev, "top_logit")
        if ldl != ldt:
            raise ValueError("top_index and top_logit have different row strides")
    _run(_calls.zero_logprob, dev, p, dt, ld, rows, vocab, pi, ib, temperature, pl, pe, ps, pti,
         ptl, top, ldt, _raw_stream(stream, dev))


def zero_logprob_backward(logits: torch.Tensor, ids: Optional[torch.Tensor], lse: torch.Tensor,
                          dlogp: Optional[torch.Tensor], grad: torch.Tensor, *,
                          entropy: Optional[torch.Tensor] = None,
                          dentropy: Optional[torch.Tensor] = None, temperature: float = 1.0,
                          loss_scale: float = 1.0, ctl: Optional[torch.Tensor] = None,
                          stream=None) -> None:
    """The loss-scaled gradient of the logits for the gradients dlogp and dentropy
    (fp32[rows]) that arrive at zero_logprob's outputs, from its lse and entropy.
    S is loss_scale, or the scale of the control block ``ctl``; grad may be
    logits (see zero_model.h)."""
    dev = _device(logits)
    p, dt, ld = _mat(logits, _ELEM, dev, "logits")
    rows, vocab = shape = logits.shape
    pi, ib = (None, 8) if ids is None else _vec(ids, rows, _INDEX, dev, "ids")
    ps, _ = _vec(lse, rows, _F32, dev, "lse")
    pl = _optional_vec(dlogp, rows, _F32, dev, "dlogp")
    pe = _optional_vec(entropy, rows, _F32, dev, "entropy")
    pde = _optional_vec(dentropy, rows, _F32, dev, "dentropy")
    if grad.dtype != logits.dtype:
        raise TypeError(f"grad has dtype {grad.dtype}, logits {logits.dtype}")
    pg, _, ldg = _like(grad, shape, _ELEM, dev, "grad")
    _run(_calls.zero_logprob_backward, dev, p, dt, ld, rows, vocab, pi, ib, temperature, ps, pl,
         pe, pde, loss_scale, _distill_scale(dev, ctl), pg, ldg, _raw_stream(stream, dev))
