"""The activation's gradients at every 8-bit code under every scale: the far ends,
where the sigmoid or the normal distribution is 0 or 1 and x^2 leaves fp32's range,
subnormal values, scale bytes 0 and 254."""
import math

import pytest
import torch

import model_ref as ref
import sharded_mixed_precision_step_amd as zs
import train_ref
from gpu_util import device
from train_ref import U

pytestmark = pytest.mark.gpu

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
TINY = 2.0 ** -149          # fp32's smallest step


def _every_code(fp8, dev):
    """A q8 matrix of 255 rows, scale byte r in row r, each code in a column; what is
    no finite number, or stands for 1e37 and more, is 0."""
    codes = torch.arange(256, device=dev, dtype=torch.int32).to(torch.uint8)
    q = codes.repeat(255, 1)
    s = torch.full((255, 4), 127, device=dev, dtype=torch.uint8)
    s[:, :2] = torch.arange(255, device=dev, dtype=torch.int32).to(torch.uint8)[:, None]
    v = train_ref.from_blocks(q.view(fp8), s)
    q = torch.where(v.abs() < 1e37, q, 0)       # NaN compares as false
    return q.view(fp8), s.view(torch.float8_e8m0fnu)


def _bounds(kind, g):
    """f, f' and bounds of their fp32 errors, tight at the far ends.

    A sigmoid's exponential e = exp(-|v|): the exponent's product is off by 2 u |v|, the
    instruction and the reciprocal by a step each, the sum and the product by u; the
    derivative has two such factors, of which the larger is off by e's share only.  Of the
    tanh form v is off by 5 u |v| itself.  GELU: -x^2 / 2 log2 e has three roundings, 1.5
    u x^2 of the exponential; t, the polynomial, its fit and the products less than 40 u.
    Behind |v| = 100, or |x| = 15, e is below 1e-43 (and the smaller end below that):
    the larger end is 1, the products with it have a rounding each.  Where the smaller
    end is below fp32's normal range it may be 0: |v| e is under 1e-34 there."""
    if kind == "gelu":
        x = g.abs()
        s = 0.5 * torch.special.erfc(-g * math.sqrt(0.5))
        d = torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
        rel, far = (2 * g * g + 40) * U, x > 15
        end = torch.minimum(s, d)
    else:
        if kind == "silu":
            v, dv, n = g, torch.ones_like(g), 4
        else:
            v, dv, n = ref.K2 * g * (1 + ref.CUBE * g * g), ref.K2 * (1 + 3 * ref.CUBE * g * g), 8
        s, other = torch.special.expit(v), torch.special.expit(-v)
        d = torch.where(v.abs() > 800, 0.0, s * other * dv)     # dv leaves fp64 with g^2
        rel, far = (n * v.abs() + 30) * U, v.abs() > 100
        end = torch.minimum(s, other)
    rel = torch.where(far, 30 * U, rel)
    low = torch.where(end < 1e-34, 1e-34, TINY)
    gd = torch.where(d > 0, g * d, 0.0)
    return g * s, s + gd, rel * (g * s).abs() + low, rel * (s + gd.abs()) + low


def _check(kind, dy, g, u, dgate, dup, y):
    f, slope, tf, ts = _bounds(kind, g)
    dy = dy.double()
    one = torch.ones_like(g) if u is None else u
    for got, want, tol, name in (
            (dgate, dy * one * slope, (dy * one).abs() * (ts + 4 * U * slope.abs()), "dgate"),
            (dup, dy * f, dy.abs() * (tf + 2 * U * f.abs()), "dup"),
            (y, f * one, one.abs() * (tf + 2 * U * f.abs()), "y")):
        if got is not None:
            # each product on the way may end below the normal range, and its step is TINY
            # there, times what it is multiplied with after
            step = TINY * (2 + dy.abs() + one.abs())
            ref.assert_close(got, want, ref.half_step(torch.float32, want) + tol + step, name)


@pytest.mark.parametrize("fp8", [E4, E5])
@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
def test_backward_of_every_gate_code(kind, fp8, gated):
    dev = device()
    print(f"case: act backward of every code, {kind} {fp8} {gated}", flush=True)
    gq = _every_code(fp8, dev)
    g, u, uq = train_ref.from_blocks(*gq), None, (None, None)
    rows, cols = g.shape
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    if gated:
        uq = zs.q8_empty(rows, cols, fp8)
        # up to 2, so that no product leaves fp32's range
        zs.zero_q8_quantize(torch.rand(rows, cols, generator=gen, device=dev) * 4 - 2, *uq)
        u = train_ref.from_blocks(*uq)
    dy = torch.rand(rows, cols, generator=gen, device=dev) * 4 - 2
    dgate, y = torch.empty_like(dy), torch.empty_like(dy)
    dup = torch.empty_like(dy) if gated else None
    zs.zero_act_backward(dy, *gq, dgate, kind, up_q=uq[0], up_s=uq[1], dup=dup, y=y)
    _check(kind, dy, g, u, dgate, dup, y)


@pytest.mark.parametrize("fp8", [E4, E5])
@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
def test_backward_of_every_up_code(kind, fp8):
    dev = device()
    print(f"case: act backward of every up code, {kind} {fp8}", flush=True)
    uq = _every_code(fp8, dev)
    u = train_ref.from_blocks(*uq)
    rows, cols = u.shape
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    gq = zs.q8_empty(rows, cols, fp8)
    zs.zero_q8_quantize(torch.rand(rows, cols, generator=gen, device=dev) * 16 - 8, *gq)
    g = train_ref.from_blocks(*gq)
    dy = torch.rand(rows, cols, generator=gen, device=dev) * 2 - 1
    dgate, dup, y = (torch.empty_like(dy) for _ in range(3))
    zs.zero_act_backward(dy, *gq, dgate, kind, up_q=uq[0], up_s=uq[1], dup=dup, y=y)
    _check(kind, dy, g, u, dgate, dup, y)


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
def test_forward_and_backward_agree_on_checkpoints_values(kind):
    """y of the forward, of the values that a checkpoint stands for, and y once more of
    the backward: SiLU's come by different forms, each within its bound."""
    dev = device()
    gq = _every_code(E4, dev)
    g = train_ref.from_blocks(*gq)
    y, again = (torch.empty(g.shape, device=dev) for _ in range(2))
    zs.zero_act(g.float(), kind, y=y)
    zs.zero_act_backward(torch.ones_like(y), *gq, torch.empty_like(y), kind, y=again)
    f, _, tf, _ = _bounds(kind, g)
    tol = tf + 2 * U * f.abs() + ref.half_step(torch.float32, f) + 3 * TINY
    ref.assert_close(y, f, tol, "y")
    ref.assert_close(again, f, tol, "again")
