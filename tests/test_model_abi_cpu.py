"""zero_model.h's C boundary without a GPU: what every call refuses, before
anything is enqueued, and the header against the binding."""
import ctypes
import math
import os
import re

import pytest
import torch

import sharded_mixed_precision_step_amd as zs
from sharded_mixed_precision_step_amd import model

pytestmark = pytest.mark.cpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, EALIGN, ERANGE = -1, -2, -3
P = 1 << 20           # fake device addresses, far apart
A, B, C, D, E, F, G, H, I, J, K = (P * (k + 1) for k in range(11))


def _header():
    text = open(os.path.join(ROOT, "include", "zero_model.h")).read()
    return re.sub(r"/\*.*?\*/", "", text, flags=re.S)


def test_exports_every_declared_symbol():
    names = set(re.findall(r"\b(zero_\w+)\s*\(", _header()))
    assert names == set(model.EXPORTED)
    for nm in names:
        assert hasattr(zs.lib, nm) and hasattr(zs, nm), nm


def test_constants_match_the_header():
    found = re.findall(r"#define (ZERO_\w+) (-?\d+)", _header())
    assert len(found) == 6
    for name, value in found:
        assert getattr(model, name) == int(value) == getattr(zs, name), name


def _refused(rc, code, *words):
    text = zs.lib.zero_last_error_string().decode()
    assert rc == code, (rc, text)
    for w in words:
        assert w in text, text


def _embed(**kw):
    a = dict(table=A, tt=1, vocab=50, cols=40, ldt=40, ids=B, ib=8, tokens=7, scale=1.0, y=C, yt=1,
             ldy=40)
    a.update(kw)
    return zs.lib.zero_embed(*a.values(), None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(tt=3), EINVAL, "t_dtype"), (dict(yt=-1), EINVAL, "y_dtype"),
    (dict(tokens=-1), EINVAL, "tokens"), (dict(vocab=0), EINVAL, "vocab"),
    (dict(vocab=1 << 31), EINVAL, "vocab"), (dict(cols=0), EINVAL, "cols"),
    (dict(cols=1 << 31, ldt=1 << 31, ldy=1 << 31), EINVAL, "cols"), (dict(ib=2), EINVAL, "id_bytes"),
    (dict(scale=math.inf), EINVAL, "scale"), (dict(scale=math.nan), EINVAL, "scale"),
    (dict(table=None), EINVAL, "table"), (dict(ids=None), EINVAL, "ids"), (dict(y=None), EINVAL, "y "),
    (dict(table=A + 1), EALIGN, "table"), (dict(ids=B + 4), EALIGN, "ids"),
    (dict(y=C + 1), EALIGN, "y "), (dict(ldt=39), EINVAL, "table"), (dict(ldy=39), EINVAL, "y "),
    (dict(y=A), EINVAL, "overlaps"), (dict(y=B), EINVAL, "overlaps"),
    (dict(tokens=0x7fffffff, cols=10000, ldt=10000, ldy=10000, table=1 << 60, ids=1 << 61),
     EINVAL, "launches"),
])
def test_embed_refuses(kw, code, word):
    _refused(_embed(**kw), code, word)


def test_embed_ctl_refuses():
    two = (ctypes.c_void_p * 2)(A, B)
    args = (50, 40, 40, C, 8, 7, 1.0, D, 1, 40)
    call = zs.lib.zero_embed_ctl
    _refused(call(None, *args, E, None), EINVAL, "tables_fp16")
    _refused(call(two, *args, None, None), EINVAL, "d_ctl")
    _refused(call(two, *args, E + 4, None), EALIGN, "d_ctl")
    _refused(call((ctypes.c_void_p * 2)(A, None), *args, E, None), EINVAL, "table")
    _refused(call((ctypes.c_void_p * 2)(A, D), *args, E, None), EINVAL, "overlaps")


def _embed_back(**kw):
    a = dict(dy=A, dt=1, ldd=40, ids=B, ib=4, tokens=7, vocab=50, cols=40, scale=1.0, dtable=C, tt=0,
             ldt=40, acc=0, ws=D, nws=1 << 16)
    a.update(kw)
    return zs.lib.zero_embed_backward(*a.values(), None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(dt=4), EINVAL, "dy_dtype"), (dict(tt=4), EINVAL, "dt_dtype"),
    (dict(tokens=-1), EINVAL, "tokens"), (dict(tokens=16777217), ERANGE, "16777216"),
    (dict(vocab=0), EINVAL, "vocab"), (dict(cols=0), EINVAL, "cols"), (dict(ib=1), EINVAL, "id_bytes"),
    (dict(scale=-math.inf), EINVAL, "scale"), (dict(acc=2), EINVAL, "accumulate"),
    (dict(dtable=None), EINVAL, "dtable"), (dict(dy=None), EINVAL, "dy"),
    (dict(ids=None), EINVAL, "ids"), (dict(dtable=C + 2), EALIGN, "dtable"),
    (dict(ldd=39), EINVAL, "dy"), (dict(ldt=39), EINVAL, "dtable"), (dict(nws=100), ERANGE, "needed"),
    (dict(ws=None), EINVAL, "workspace"), (dict(ws=D + 8), EALIGN, "workspace"),
    (dict(dtable=A), EINVAL, "overlaps"), (dict(dtable=B), EINVAL, "overlaps"),
    (dict(ws=A), EINVAL, "overlaps"), (dict(ws=C), EINVAL, "overlaps"),
])
def test_embed_backward_refuses(kw, code, word):
    _refused(_embed_back(**kw), code, word)


@pytest.mark.parametrize("tokens", [0, 1, 31, 33, 4096, 4097, 8192, 100000, 16777216])
@pytest.mark.parametrize("cols", [1, 64, 1001, 4096, 2147483647])
def test_embed_backward_workspace_is_as_documented(tokens, cols):
    n = zs.zero_embed_backward_workspace(tokens, 1000, cols)
    assert 0 <= n <= 20 * tokens + (tokens + 64) * cols / 2 + 65536


def test_workspace_queries_refuse():
    for args in ((-1, 5, 5), (5, 0, 5), (5, 5, 0), (16777217, 5, 5)):
        with pytest.raises(zs.ZeroStepError):
            zs.zero_embed_backward_workspace(*args)
    f = zs.zero_layernorm_backward_workspace
    assert f(0, 100) == 0 and 0 < f(10 ** 9, 65536) <= 8 * 1024 * 65536
    for args in ((-1, 5), (5, 0), (5, 65537)):
        with pytest.raises(zs.ZeroStepError):
            f(*args)


def _norm(**kw):
    a = dict(x=A, xt=1, ldx=200, res=B, rt=0, ldr=200, w=C, b=I, wt=1, rows=4, cols=200, eps=1e-5,
             h=D, ldh=200, y=E, yt=1, ldy=200, q=F, fmt=0, ldq=256, s=G, lds=4, mean=H, rstd=J)
    a.update(kw)
    return zs.lib.zero_layernorm(*a.values(), None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(xt=5), EINVAL, "x"), (dict(rt=5), EINVAL, "residual"), (dict(wt=-1), EINVAL, "weight"),
    (dict(yt=9), EINVAL, "y"), (dict(fmt=3), EINVAL, "fmt"), (dict(rows=-1), EINVAL, "rows"),
    (dict(cols=0), EINVAL, "cols"), (dict(cols=65537, ldx=70000), ERANGE, "65536"),
    (dict(eps=-1.0), EINVAL, "eps"), (dict(eps=math.nan), EINVAL, "eps"),
    (dict(s=None), EINVAL, "together"), (dict(res=None), EINVAL, "residual"),
    (dict(x=None), EINVAL, "x "), (dict(w=None), EINVAL, "weight"), (dict(ldx=199), EINVAL, "x "),
    (dict(x=A + 1), EALIGN, "x "), (dict(res=B + 2), EALIGN, "residual"), (dict(b=I + 1), EALIGN, "bias"),
    (dict(ldq=240), EINVAL, "q "), (dict(rstd=J + 2), EALIGN, "rstd"),
    (dict(mean=H + 1), EALIGN, "mean"), (dict(h=A), EINVAL, "overlaps"),
    (dict(h=B, ldh=201), EINVAL, "overlaps"), (dict(y=A, yt=0), EINVAL, "overlaps"),
    (dict(y=B), EINVAL, "overlaps"), (dict(y=C), EINVAL, "overlaps"), (dict(y=I), EINVAL, "overlaps"),
    (dict(y=D), EINVAL, "overlaps"), (dict(q=A), EINVAL, "overlaps"),
    (dict(mean=J), EINVAL, "overlaps"),
    (dict(h=None, y=None, q=None, s=None, mean=None, rstd=None), EINVAL, "no output"),
])
def test_layernorm_refuses(kw, code, word):
    _refused(_norm(**kw), code, word)


NEED = zs.zero_layernorm_backward_workspace(4, 200)


def _norm_back(**kw):
    a = dict(dy=A, dt=1, ldd=200, h=B, ht=0, ldh=200, w=C, wt=1, mean=D, rstd=I, dr=E, drt=1,
             ldr=200, rows=4, cols=200, dx=F, dxt=1, ldx=200, dw=G, db=J, dwt=1, ws=H,
             nws=NEED)
    a.update(kw)
    return zs.lib.zero_layernorm_backward(*a.values(), None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(dt=4), EINVAL, "dy"), (dict(ht=4), EINVAL, "h"), (dict(wt=4), EINVAL, "weight"),
    (dict(drt=4), EINVAL, "dresidual"), (dict(dxt=4), EINVAL, "dx"), (dict(dwt=4), EINVAL, "dw"),
    (dict(dwt=4, dw=None), EINVAL, "db"), (dict(rows=-2), EINVAL, "rows"),
    (dict(cols=0), EINVAL, "cols"), (dict(cols=70000), ERANGE, "65536"),
    (dict(rstd=None), EINVAL, "rstd"), (dict(mean=None), EINVAL, "mean"),
    (dict(dx=None), EINVAL, "dx"), (dict(ldh=10), EINVAL, "h "), (dict(nws=NEED - 1), ERANGE, str(NEED)),
    (dict(ws=None), EINVAL, "workspace"), (dict(ws=H + 4), EALIGN, "workspace"),
    (dict(dx=A, ldx=201), EINVAL, "overlaps"), (dict(dx=B), EINVAL, "overlaps"),
    (dict(dx=D), EINVAL, "overlaps"), (dict(dx=I), EINVAL, "overlaps"),
    (dict(dw=C), EINVAL, "overlaps"), (dict(ws=A), EINVAL, "overlaps"),
    (dict(db=F), EINVAL, "overlaps"), (dict(db=G), EINVAL, "overlaps"),
])
def test_layernorm_backward_refuses(kw, code, word):
    _refused(_norm_back(**kw), code, word)


def _act(**kw):
    a = dict(gate=A, ldg=300, up=B, ldu=300, xt=1, kind=0, rows=10, cols=300, y=C, yt=1, ldy=300,
             q=D, fmt=0, ldq=384, s=E, lds=4, gq=F, ck=1, ldgq=384, gs=G, ldgs=4, uq=H, lduq=384,
             us=I, ldus=4)
    a.update(kw)
    return zs.lib.zero_act(*a.values(), None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(xt=3), EINVAL, "x_dtype"), (dict(kind=3), EINVAL, "kind"), (dict(kind=-1), EINVAL, "kind"),
    (dict(rows=-1), EINVAL, "rows"), (dict(cols=-1), EINVAL, "cols"), (dict(yt=5), EINVAL, "y"),
    (dict(fmt=2), EINVAL, "fmt"), (dict(ck=2), EINVAL, "ck_fmt"), (dict(s=None), EINVAL, "together"),
    (dict(gq=None), EINVAL, "together"), (dict(us=None), EINVAL, "together"),
    (dict(up=None), EINVAL, "without an up"), (dict(gate=None), EINVAL, "gate"),
    (dict(gate=A + 1), EALIGN, "gate"), (dict(ldu=299), EINVAL, "up"), (dict(ldgq=392), EALIGN, "gate_q"),
    (dict(lduq=256), EINVAL, "up_q"), (dict(ldus=3), EALIGN, "up_s"), (dict(q=D + 8), EALIGN, "q"),
    (dict(y=A, yt=2), EINVAL, "overlaps"), (dict(y=A, ldy=301), EINVAL, "overlaps"),
    (dict(gq=A), EINVAL, "overlaps"), (dict(uq=F), EINVAL, "overlaps"), (dict(q=C), EINVAL, "overlaps"),
    (dict(gs=E), EINVAL, "overlaps"),
    (dict(y=None, q=None, s=None, gq=None, gs=None, uq=None, us=None), EINVAL, "no output"),
    (dict(rows=1 << 40, ldg=1 << 40), EINVAL, "too large"),
    (dict(rows=1 << 40, cols=16, ldg=16, ldu=16, up=1 << 60, y=1 << 61, ldy=16, q=None, s=None,
          gq=None, gs=None, uq=None, us=None), EINVAL, "launches"),
])
def test_act_refuses(kw, code, word):
    _refused(_act(**kw), code, word)


def _act_back(**kw):
    a = dict(dy=A, dt=1, ldd=300, gq=B, ck=0, ldgq=384, gs=C, ldgs=4, uq=D, lduq=384, us=E, ldus=4,
             kind=0, rows=10, cols=300, dg=F, lddg=300, du=G, lddu=300, xt=1, y=H, yt=1, ldy=300)
    a.update(kw)
    return zs.lib.zero_act_backward(*a.values(), None)


@pytest.mark.parametrize("kw,code,word", [
    (dict(dt=3), EINVAL, "dy_dtype"), (dict(xt=3), EINVAL, "dx_dtype"), (dict(yt=3), EINVAL, "y"),
    (dict(ck=2), EINVAL, "ck_fmt"), (dict(kind=7), EINVAL, "kind"), (dict(rows=-1), EINVAL, "rows"),
    (dict(cols=-1), EINVAL, "cols"), (dict(us=None), EINVAL, "together"),
    (dict(du=None), EINVAL, "dup"), (dict(uq=None, us=None), EINVAL, "dup"),
    (dict(gq=None), EINVAL, "gate_q"), (dict(gs=None), EINVAL, "gate_s"), (dict(dy=None), EINVAL, "dy"),
    (dict(dg=None), EINVAL, "dgate"), (dict(ldgq=256), EINVAL, "gate_q"),
    (dict(ldus=2), EALIGN, "up_s"), (dict(dg=F + 1), EALIGN, "dgate"),
    (dict(dg=A, xt=2), EINVAL, "overlaps"), (dict(dg=A, du=A), EINVAL, "overlaps"),
    (dict(dg=B), EINVAL, "overlaps"), (dict(y=E), EINVAL, "overlaps"), (dict(y=G), EINVAL, "overlaps"),
])
def test_act_backward_refuses(kw, code, word):
    _refused(_act_back(**kw), code, word)


def test_column_ranges_of_one_matrix_are_apart():
    """Halves of one product may be inputs and outputs side by side; a range that
    reaches into its neighbour is refused.  (What is asked next, y's alignment,
    shows that the overlap check was passed; nothing is enqueued.)"""
    halves = dict(ldd=300, dg=F, lddg=600, du=F + 600, lddu=600, y=H + 1)
    _refused(_act_back(**halves), EALIGN, "y is not")
    _refused(_act_back(**dict(halves, y=None, du=F + 598)), EINVAL, "overlaps")
    _refused(_act_back(**dict(halves, y=None, du=F + 602)), EINVAL, "overlaps")
    _refused(_act_back(**dict(halves, y=None, lddu=601)), EINVAL, "overlaps")
    _refused(_act(up=A + 600, ldg=600, ldu=600, y=A, ldy=600, gq=A), EINVAL, "overlaps")


def _logprob(**kw):
    a = dict(logits=A, dt=1, ld=100, rows=4, vocab=100, ids=B, ib=8, tau=1.0, logp=C, ent=D, lse=E,
             ti=F, tl=G, top=5, ldt=5)
    a.update(kw)
    return zs.lib.zero_logprob(*a.values(), None)


LOGITS = [
    (dict(dt=3), EINVAL, "dtype"), (dict(rows=-1), EINVAL, "rows"), (dict(vocab=0), EINVAL, "vocab"),
    (dict(vocab=1 << 31, ld=1 << 31), EINVAL, "vocab"), (dict(ib=2), EINVAL, "id_bytes"),
    (dict(tau=0.0), EINVAL, "temperature"), (dict(tau=math.nan), EINVAL, "temperature"),
    (dict(tau=math.inf), EINVAL, "temperature"), (dict(tau=3.5e-39), EINVAL, "temperature"),
    (dict(ld=99), EINVAL, "logits"), (dict(logits=None), EINVAL, "logits"),
    (dict(logits=A + 1), EALIGN, "logits"), (dict(ids=B + 4), EALIGN, "ids"),
]


@pytest.mark.parametrize("kw,code,word", LOGITS + [
    (dict(ti=None), EINVAL, "together"), (dict(top=0), EINVAL, "top"),
    (dict(top=129, ldt=129), ERANGE, "128"), (dict(ldt=4), EINVAL, "top_index"),
    (dict(ids=None), EINVAL, "ids"), (dict(ti=F + 2), EALIGN, "top_index"),
    (dict(tl=G + 1), EALIGN, "top_logit"), (dict(logp=C + 2), EALIGN, "logp"),
    (dict(logp=A), EINVAL, "overlaps"), (dict(lse=B), EINVAL, "overlaps"),
    (dict(tl=F), EINVAL, "overlaps"), (dict(ent=C + 4), EINVAL, "overlaps"),
    (dict(logp=None, ent=None, lse=None, ti=None, tl=None), EINVAL, "no output"),
])
def test_logprob_refuses(kw, code, word):
    _refused(_logprob(**kw), code, word)


def _logprob_back(**kw):
    a = dict(logits=A, dt=1, ld=100, rows=4, vocab=100, ids=B, ib=8, tau=1.0, lse=C, dlogp=D, ent=E,
             dent=F, S=1.0, ctl=None, grad=G, ldg=100)
    a.update(kw)
    return zs.lib.zero_logprob_backward(*a.values(), None)


@pytest.mark.parametrize("kw,code,word", LOGITS + [
    (dict(S=0.0), EINVAL, "loss_scale"), (dict(S=math.inf), EINVAL, "loss_scale"),
    (dict(ctl=H + 4), EALIGN, "d_ctl"), (dict(dlogp=None, dent=None), EINVAL, "neither"),
    (dict(ids=None), EINVAL, "ids"), (dict(ent=None), EINVAL, "entropy"), (dict(lse=None), EINVAL, "lse"),
    (dict(grad=None), EINVAL, "grad"), (dict(ldg=99), EINVAL, "grad"),
    (dict(grad=A, ldg=101), EINVAL, "stride"), (dict(grad=A + 2), EINVAL, "overlaps"),
    (dict(grad=C), EINVAL, "overlaps"), (dict(dent=F + 1), EALIGN, "dentropy"),
])
def test_logprob_backward_refuses(kw, code, word):
    _refused(_logprob_back(**kw), code, word)


def test_empty_calls_are_accepted_without_pointers():
    assert _embed(tokens=0, table=None, ids=None, y=None) == 0
    assert _norm(rows=0, x=None, w=None, b=None, res=None, h=None, y=None, q=None, s=None,
                 mean=None, rstd=None) == 0
    assert _act(rows=0, gate=None, up=None, y=None, q=None, s=None, gq=None, gs=None, uq=None,
                us=None) == 0
    assert _act(cols=0, gate=None, up=None) == 0
    assert _act_back(rows=0, dy=None, gq=None, gs=None, uq=None, us=None, dg=None, du=None) == 0
    assert _logprob(rows=0, logits=None, ids=None, logp=None) == 0
    assert _logprob_back(rows=0, logits=None, grad=None) == 0
    assert _norm_back(rows=0, dy=None, h=None, w=None, mean=None, rstd=None, dr=None, dx=None,
                      dw=None, db=None, ws=None, nws=0) == 0
    assert _embed_back(tokens=0, acc=1, dy=None, ids=None, ws=None, nws=0) == 0


def test_the_binding_refuses_host_and_mismatched_tensors():
    x, w = torch.zeros(4, 200), torch.ones(200)
    ids = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: zs.zero_layernorm(x, w, w, 1e-5, y=torch.empty_like(x)),
                 lambda: zs.zero_embed(x, ids, x), lambda: zs.zero_act(x, "silu", y=x),
                 lambda: zs.zero_logprob(x, ids, w[:4]),
                 lambda: zs.zero_embed_backward(x, ids, x, None)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="gelu_tanh"):
        model._kind("relu")
