"""Plain 64-bit definitions of the training operators, for the tests: written
from the formulas, with torch double tensors on whatever device the inputs
are on, and the error bounds the tests hold the kernels to.

u = 2^-24 is half a step of fp32 relative to the value.  Each bound counts the
fp32 roundings on the longest path into a value (a sum of n terms in any order
is off by at most n u times the sum of magnitudes) and adds half a step of the
output's type."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
FMT = {torch.float8_e4m3fn: (448.0, 3, -6), torch.float8_e5m2: (57344.0, 2, -14)}


def half_step(dtype, ref):
    """Half a step of dtype at ref: relative, and below the smallest normal
    number half the subnormal spacing."""
    fi = torch.finfo(dtype)
    return (fi.eps / 2) * ref.abs().clamp_min(fi.smallest_normal)


def pow2(e):
    return torch.ldexp(torch.ones((), dtype=torch.float64), e.cpu().to(torch.int32)).to(e.device)


def scale_exponent(amax, fp8):
    """min e with amax <= max * 2^e, e >= -127; 0 for a block of zeros."""
    big = FMT[fp8][0]
    m, e = torch.frexp(amax.cpu() / big)          # in [0.5, 1) * 2^e
    e = torch.where(m == 0.5, e - 1, e).to(torch.int64).clamp_min(-127)
    return torch.where(amax.cpu() == 0, 0, e).to(amax.device)


def round8(v, fp8):
    """v rounded half to even to the 8-bit type's grid."""
    _, bits, low = FMT[fp8]
    _, e = torch.frexp(v.cpu())
    step = pow2((e.to(torch.int64) - 1).clamp_min(low) - bits).to(v.device)
    return torch.round(v / step) * step


def to_blocks(x, fp8):
    """x (double, [rows, cols]) -> (8-bit values, scale exponents) as double and
    int64, in the padded layout; NaN exponent marker 128 for a non-finite block."""
    rows, cols = x.shape
    blocks = -(-cols // 128)
    xb = torch.zeros(rows, blocks * 128, dtype=torch.float64, device=x.device)
    xb[:, :cols] = x
    xb = xb.view(rows, blocks, 128)
    amax = xb.abs().amax(-1)
    bad = ~torch.isfinite(xb).all(-1)
    e = scale_exponent(torch.where(bad, 0.0, amax), fp8)
    q = round8(torch.where(bad[..., None], 0.0, xb) / pow2(e)[..., None], fp8)
    q = torch.where(bad[..., None], math.nan, q)
    ex = torch.zeros(rows, -(-blocks // 4) * 4, dtype=torch.int64, device=x.device)
    ex[:, :blocks] = torch.where(bad, 128, e)
    return q.view(rows, blocks * 128), ex


def from_blocks(q, s):
    """The values a q8 pair stands for, in double."""
    blocks = q.shape[1] // 128
    e = s[:, :blocks].view(torch.uint8).to(torch.int64) - 127
    v = q.to(torch.float32).double().view(q.shape[0], blocks, 128) * pow2(e)[..., None]
    return torch.where((e == 128)[..., None], math.nan, v).reshape(q.shape)


def rmsnorm(x, residual, w, eps):
    h = x.double() if residual is None else x.double() + residual.double()
    rstd = 1 / torch.sqrt((h * h).mean(-1) + eps)
    return h, rstd, h * rstd[:, None] * w.double()


def rmsnorm_backward(dy, h, w, rstd, dres):
    dy, h, r = dy.double(), h.double(), rstd.double()[:, None]
    g, xhat = dy * w.double(), h * r
    dx = r * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    if dres is not None:
        dx = dx + dres.double()
    return dx, (dy * xhat).sum(0)


def distill(logits, index, teacher, tau, weight, S):
    """loss, lse, gradient (double), by rows, with every special case spelled
    out."""
    rows, vocab = logits.shape
    z = logits.double() / tau
    idx, t = index.long(), teacher.double() / tau
    w = torch.ones(rows, dtype=torch.float64, device=z.device) if weight is None \
        else weight.double()
    bad = (idx >= vocab).any(1)
    valid = (idx >= 0) & (idx < vocab)
    bad |= (valid & ~(t < math.inf)).any(1)
    bad |= ~(logits.double() < math.inf).all(1) | (logits.double() == -math.inf).all(1)
    have = valid & (t > -math.inf)
    empty = ~have.any(1)
    tt = torch.where(have, t, -math.inf)
    top = torch.where(empty, 0.0, tt.amax(1).nan_to_num(0.0, 0.0, 0.0))
    e = torch.where(have, torch.exp(tt - top[:, None]), 0.0)
    p = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    lse = torch.logsumexp(z, 1)
    at = idx.clamp(0, vocab - 1)
    logq = z.gather(1, at) - lse[:, None]
    logp = tt - top[:, None] - torch.log(e.sum(1, keepdim=True).clamp_min(1e-300))
    kl = torch.where(p > 0, p * (logp - logq), 0.0).sum(1)
    q = torch.exp(z - lse[:, None])
    grad = q.scatter_add(1, at, -torch.where(have, p, 0.0))
    coef = S * w * tau
    loss, grad = w * tau * tau * kl, coef[:, None] * grad
    loss = torch.where(empty, 0.0, loss)
    grad = torch.where(empty[:, None], 0.0, grad)
    loss, lse = torch.where(bad, math.nan, loss), torch.where(bad, math.nan, lse)
    grad = torch.where(bad[:, None], math.nan, grad)
    off = w == 0
    return (torch.where(off, 0.0, loss), torch.where(off, 0.0, lse),
            torch.where(off[:, None], 0.0, grad))


def assert_close(got, want, tol, name):
    """|got - want| <= tol elementwise; the same NaN and inf places."""
    got = got.to(torch.float32).double() if got.dtype != torch.float64 else got
    assert got.shape == want.shape, (name, got.shape, want.shape)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{name}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{name}: inf in other places"
    live = ~(nan | inf)
    err = (got - want).abs()
    tol = torch.as_tensor(tol, dtype=torch.float64, device=got.device).expand_as(err)
    over = live & ~(err <= tol)
    if over.any():
        i = tuple(torch.nonzero(over)[0].tolist())
        raise AssertionError(f"{name}: {int(over.sum())} of {over.numel()} outside; first at {i}: "
                             f"{float(got[i])!r}, want {float(want[i])!r}, tol {float(tol[i]):.3g}")
