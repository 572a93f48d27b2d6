"""Plain 64-bit definitions of zero_model.h's operators, for the tests, and the
error bounds the tests hold the kernels to (see train_ref.py for u and how
roundings are counted)."""
from __future__ import annotations

import math

import torch

from train_ref import FMT, U, assert_close, half_step, pow2, scale_exponent

# ---- embedding ---------------------------------------------------------------


def embed(table, ids, scale):
    ids = ids.reshape(-1)
    vocab = table.shape[0]
    y = scale * table.double()[ids.clamp(0, vocab - 1)]
    y = torch.where((ids < 0)[:, None], 0.0, y)
    return torch.where((ids >= vocab)[:, None], math.nan, y)


def embed_backward(dy, ids, vocab, scale):
    """(sum, bound of its fp32 error): a row of n tokens has n - 1 additions and
    the product with scale, which is off by half a step itself."""
    ids = ids.reshape(-1)
    live = (ids >= 0) & (ids < vocab)
    at, d = ids[live], dy.double()[live]
    zeros = torch.zeros(vocab, dy.shape[1], dtype=torch.float64, device=dy.device)
    total = zeros.index_add(0, at, d) * scale
    mag = zeros.index_add(0, at, d.abs()) * abs(scale)
    n = torch.zeros(vocab, dtype=torch.float64, device=dy.device).index_add(
        0, at, torch.ones_like(at, dtype=torch.float64))
    return total, (n[:, None] + 2) * U * mag


# ---- layer norm --------------------------------------------------------------


def layernorm(x, residual, w, b, eps):
    h = x.double() if residual is None else x.double() + residual.double()
    mean = h.mean(-1)
    rstd = 1 / torch.sqrt((h - mean[:, None]).square().mean(-1) + eps)
    y = (h - mean[:, None]) * rstd[:, None] * w.double()
    return h, mean, rstd, y if b is None else y + b.double()


def layernorm_bounds(x, residual, w, b, eps):
    """Bounds of the fp32 errors of mean, rstd and y.  h has one rounding.  A sum
    over the row: at most 64 terms a lane, 6 + 16 joins, and its division; the
    sum of squares, about a mean off by dm, gains dm^2 n and loses nothing to
    first order, as the differences add up to 0."""
    h, mean, rstd, y = layernorm(x, residual, w, b, eps)
    d = (h - mean[:, None]).abs()
    inv = rstd.square()                               # 1 / (var + eps)
    dm = 90 * U * h.abs().mean(-1)
    rel = 60 * U + dm.square() * inv + U * (d * h.abs()).mean(-1) * inv
    w = w.double().abs()
    wide = d * rstd[:, None] * w
    tol = (rel + 4 * U)[:, None] * wide + w * rstd[:, None] * (dm[:, None] + U * h.abs())
    if b is not None:
        tol = tol + U * b.double().abs()
    return dm + U * mean.abs(), rel * rstd, tol + U * y.abs()


def layernorm_backward(dy, h, w, mean, rstd, dres):
    """dx, dw, db and the bounds of their fp32 errors.  dx: the products have 4
    roundings, a sum at most max(64, cols / 256) terms a lane and 22 joins, what
    follows 10.  dw, db: a workgroup's rows one after another (at least 128
    workgroups share them where there are that many), at most 1,024 partial rows
    in 16 groups, then the groups."""
    rows, cols = dy.shape
    dy, h, r = dy.double(), h.double(), rstd.double()[:, None]
    g, xhat = dy * w.double(), (h - mean.double()[:, None]) * r
    dx = r * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
    mag = r * (g.abs() + g.abs().mean(-1, keepdim=True)
               + xhat.abs() * (g * xhat).abs().mean(-1, keepdim=True))
    if dres is not None:
        dx, mag = dx + dres.double(), mag + dres.double().abs()
    n = -(-rows // 128) + 90
    return (dx, (dy * xhat).sum(0), dy.sum(0), (max(64, cols // 256) + 40) * U * mag,
            n * U * (dy * xhat).abs().sum(0), n * U * dy.abs().sum(0))


# ---- activation --------------------------------------------------------------

K2, CUBE = math.sqrt(8 / math.pi), 0.044715


def activation(kind, g):
    """f, f' and the bounds of their errors.  With v the argument of the sigmoid:
    exp2's argument is off by 2 u |v| and by what v is off, the instruction and
    the reciprocal by a step each.  GELU: of exp(-g^2 / 2) the three roundings of the
    exponent are 1.5 g^2 u, the instruction a step; t = 1 / (1 + |g| / 4) is off by 3 u,
    which t P(t) takes up to 3.2 times, the fit by u, the polynomial's and the other
    products by less than 25 u."""
    g = g.double()
    if kind == "gelu":
        phi = torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
        s, d, rel = 0.5 * torch.special.erfc(-g * math.sqrt(0.5)), phi, (2 * g * g + 40) * U
    else:
        if kind == "silu":
            v, dv, rel = g, torch.ones_like(g), (4 * g.abs() + 20) * U
        else:
            v, dv = K2 * g * (1 + CUBE * g * g), K2 * (1 + 3 * CUBE * g * g)
            rel = (8 * v.abs() + 30) * U
        s = torch.special.expit(v)
        d = s * torch.special.expit(-v) * dv
    # below exp(-80) the hardware's results leave the normal range
    rel = torch.where(s < 1e-34, 1.0, rel)
    return g * s, s + g * d, rel * (g * s).abs() + 1e-34, rel * (s + (g * d).abs()) + 1e-34


def act(kind, gate, up):
    f, _, tol, _ = activation(kind, gate)
    if up is None:
        return f, tol
    u = up.double()
    return f * u, (tol + 2 * U * f.abs()) * u.abs()


def act_backward(kind, dy, g, u):
    """dgate, dup, y and their bounds, from the checkpoints' values (double)."""
    f, slope, tf, ts = activation(kind, g)
    dy = dy.double()
    if u is None:
        return ((dy * slope, None, f), (dy.abs() * (ts + 2 * U * slope.abs()), None, tf))
    return ((dy * u * slope, dy * f, f * u),
            ((dy * u).abs() * (ts + 4 * U * slope.abs()), dy.abs() * (tf + 2 * U * f.abs()),
             u.abs() * (tf + 2 * U * f.abs())))


def check_q8(q, s, want, tol, fp8, name):
    """A q8 matrix of values that are off by at most tol: the definition's scale
    for a largest magnitude within tol of the true one, values within half a step
    at that scale; zeros and ones in the padding."""
    rows, cols = want.shape
    blocks = q.shape[1] // 128
    pad = torch.zeros(2, rows, q.shape[1], dtype=torch.float64, device=want.device)
    pad[0, :, :cols], pad[1, :, :cols] = want, tol
    mag = pad[0].abs().view(rows, blocks, 128)
    off = pad[1].view(rows, blocks, 128)
    e = s.view(torch.uint8).to(torch.int64) - 127
    assert (e[:, blocks:] == 0).all(), name
    lo = scale_exponent((mag - off).clamp_min(0).amax(-1), fp8)
    hi = scale_exponent((mag + off).amax(-1), fp8)
    e = e[:, :blocks]
    live = mag.amax(-1) > off.amax(-1)      # a block that may round to zeros has scale 1
    assert ((e >= lo) & (e <= hi))[live].all(), name
    scale = pow2(e).repeat_interleave(128, 1)
    got = q.to(torch.float32).double() * scale
    assert (got[:, cols:] == 0).all(), name
    assert_close(got, pad[0], half_step(fp8, pad[0] / scale) * scale + pad[1], name)
    assert FMT[fp8][0] >= q.to(torch.float32).abs().max()


# ---- log probabilities -------------------------------------------------------


def logprob(logits, ids, tau, top):
    """logp, entropy, lse, top_index, top_logit and bounds of the first three.

    A term of the sums: its exponent d (in powers of two) is off by 3 u |d|, the
    instruction by a step; rescaling on the way to the row's maximum adds as much
    for the maxima's distance, and a few for each of at most 64 packs a lane and
    10 joins, and eight terms add up one after another.  Beyond 200 a term is 0."""
    rows, vocab = logits.shape
    x = logits.double()
    on = torch.ones(rows, dtype=torch.bool, device=x.device) if ids is None else ids >= 0
    at = torch.zeros(rows, dtype=torch.int64, device=x.device) if ids is None else ids.long()
    bad = on & ((at >= vocab) | ~(x < math.inf).all(1) | (x == -math.inf).all(1))
    fine = torch.where((on & ~bad)[:, None], x, 0.0)
    z = fine / tau
    m = z.amax(1)
    d = z - m[:, None]
    e = torch.exp(d)
    s = e.sum(1)
    p = e / s[:, None]
    dist = torch.where(p > 0, -d, 0.0)
    lse = m + torch.log(s)
    entropy = torch.log(s) + (p * dist).sum(1)
    z_id = z.gather(1, at.clamp(0, vocab - 1)[:, None])[:, 0]
    logp = (z_id - m) - torch.log(s)     # large maxima take nothing away

    def fp32_range(v):                   # what fp32 cannot hold is inf there
        return torch.where(v.abs() > torch.finfo(torch.float32).max, torch.sign(v) * math.inf, v)

    lse, logp = fp32_range(lse), fp32_range(logp)
    reach = torch.where(d > -math.inf, -d, 0.0).amax(1).clamp_max(140.0) / math.log(2)
    rel = U * (6 * reach + 300)
    far = (z_id - m).abs()
    far = torch.where(torch.isinf(far), 0.0, far)
    t_lse = rel + 4 * U * (m.abs() + torch.log(s).abs())
    t_logp = rel + 4 * U * (far + torch.log(s).abs())
    t_ent = rel * (1 + 2 * (p * dist).sum(1)) + 4 * U * (entropy + torch.log(s).abs())

    def placed(v):
        return torch.where(on, torch.where(bad, math.nan, v), 0.0)

    out = [placed(logp), placed(entropy), placed(lse)]
    if top:
        v, i = torch.sort(logits.float(), dim=1, descending=True, stable=True)
        v, i = v[:, :top], i[:, :top].to(torch.int32)
        short = top - v.shape[1]
        if short > 0:
            v = torch.nn.functional.pad(v, (0, short), value=-math.inf)
            i = torch.nn.functional.pad(i, (0, short), value=-1)
        gone = (v == -math.inf) | ~on[:, None]
        i, v = torch.where(gone, -1, i), torch.where(gone, -math.inf, v)
        i = torch.where(bad[:, None], 0, i)
        v = torch.where(bad[:, None], math.nan, v)
        out += [i, v.to(logits.dtype)]
    return out, (t_logp, t_ent, t_lse)


def logprob_backward(logits, ids, tau, lse, dlogp, entropy, dentropy, S):
    """grad and the bound of its fp32 error: log p is off by u |z| and 2 u |log p|,
    p by that and 6 u."""
    rows, vocab = logits.shape
    zero = torch.zeros(rows, dtype=torch.float64, device=logits.device)
    a = zero if dlogp is None else dlogp.double()
    b = zero if dentropy is None else dentropy.double()
    h = zero if dentropy is None else entropy.double()
    at = torch.zeros(rows, dtype=torch.int64, device=logits.device) if ids is None else ids.long()
    off = (at < 0) | ((a == 0) & (b == 0))
    bad = ~off & (torch.isnan(lse) | (at >= vocab))
    z = torch.where((off | bad)[:, None], 0.0, logits.double() / tau)
    logq = z - torch.where(off | bad, 0.0, lse.double())[:, None]
    q = torch.exp(logq)
    q = torch.where(logq < -100, torch.where(q < 1e-37, 0.0, q), q)
    safe = torch.where(q > 0, logq, 0.0)
    rest = a[:, None] + b[:, None] * (safe + h[:, None])
    hot = torch.zeros_like(z).scatter(1, at.clamp(0, vocab - 1)[:, None], 1.0)
    k = S / tau
    grad = k * (hot * a[:, None] - q * rest)
    zabs = torch.where(q > 0, z.abs(), 0.0)
    off_log = U * (2 * zabs + 4 * safe.abs() + 8)
    mag = a.abs()[:, None] + b.abs()[:, None] * (safe.abs() + h.abs()[:, None])
    tol = k * (q * (off_log * mag + b.abs()[:, None] * off_log) + 6 * U * hot * a.abs()[:, None])
    tol = tol + 1e-36 * k * (mag + 1)
    grad = torch.where(off[:, None], 0.0, torch.where(bad[:, None], math.nan, grad))
    return grad, tol
