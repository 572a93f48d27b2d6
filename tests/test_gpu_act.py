"""Activations with 8-bit checkpoints, and their gradients from them, against the
64-bit definitions."""
import math

import pytest
import torch

import model_ref as ref
import sharded_mixed_precision_step_amd as zs
import train_ref
from gpu_util import device

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
KINDS = ["silu", "gelu", "gelu_tanh"]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(seed, *shape, dtype=F32):
    return torch.randn(*shape, generator=_gen(seed), device="cuda").to(dtype)


def _same8(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


SHAPES = [(1, 1), (3, 7), (70, 64), (5, 128), (4, 129), (33, 255), (7, 500), (6, 1025), (17, 2048),
          (16, 2049), (3, 5001), (4, 14336)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("x_dtype,fp8,gated", [(F16, E4, True), (BF16, E5, True), (F32, E4, False),
                                               (F16, E5, False), (F32, E5, True)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_act_is_the_definition(rows, cols, x_dtype, fp8, gated, kind):
    dev = device()
    print(f"case: act {kind} {rows}x{cols} {x_dtype} {gated}", flush=True)
    gate = (2.5 * _randn(1, rows, cols)).to(x_dtype)
    up = _randn(2, rows, cols, dtype=x_dtype) if gated else None
    y = torch.empty(rows, cols, dtype=x_dtype, device=dev)
    q, gq = zs.q8_empty(rows, cols, fp8), zs.q8_empty(rows, cols, E4 if fp8 == E5 else E5)
    uq = zs.q8_empty(rows, cols, gq[0].dtype) if gated else (None, None)
    zs.zero_act(gate, kind, up=up, y=y, q=q[0], s=q[1], gate_q=gq[0], gate_s=gq[1], up_q=uq[0],
                up_s=uq[1])
    want, tol = ref.act(kind, gate, up)
    ref.assert_close(y, want, ref.half_step(x_dtype, want) + tol, "y")
    ref.check_q8(*q, want, tol, fp8, "q")
    own = zs.q8_empty(rows, cols, gq[0].dtype)
    for t, kept in ((gate, gq), (up, uq)):
        if t is not None:
            zs.zero_q8_quantize(t, *own)
            assert _same8(own, kept)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt,dx,fp8,gated", [(F16, F16, E4, True), (BF16, BF16, E5, False),
                                             (F32, F32, E5, True), (BF16, F32, E4, False),
                                             (F32, F16, E4, True)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward_is_the_formula(rows, cols, dt, dx, fp8, gated, kind):
    dev = device()
    print(f"case: act backward {kind} {rows}x{cols} {dt} {dx} {gated}", flush=True)
    gq, uq = zs.q8_empty(rows, cols, fp8), (None, None)
    zs.zero_q8_quantize(2.5 * _randn(1, rows, cols), *gq)
    g, u = train_ref.from_blocks(*gq)[:, :cols], None
    if gated:
        uq = zs.q8_empty(rows, cols, fp8)
        zs.zero_q8_quantize(_randn(2, rows, cols), *uq)
        u = train_ref.from_blocks(*uq)[:, :cols]
    dy = _randn(3, rows, cols, dtype=dt)
    dgate = torch.empty(rows, cols, dtype=dx, device=dev)
    dup = torch.empty_like(dgate) if gated else None
    y = torch.empty(rows, cols, dtype=dt, device=dev)
    zs.zero_act_backward(dy, *gq, dgate, kind, up_q=uq[0], up_s=uq[1], dup=dup, y=y)
    want, tol = ref.act_backward(kind, dy, g, u)
    for got, w, t, name in zip((dgate, dup, y), want, tol, ("dgate", "dup", "y")):
        if got is not None:
            ref.assert_close(got, w, ref.half_step(got.dtype, w) + t, name)
    alone = torch.empty_like(dgate)
    zs.zero_act_backward(dy, *gq, alone, kind, up_q=uq[0], up_s=uq[1],
                         dup=None if dup is None else torch.empty_like(dup))
    assert torch.equal(alone, dgate)


@pytest.mark.parametrize("kind", KINDS)
def test_every_sixteen_bit_gate(kind):
    """All finite fp16 and bf16 gates, y in fp32: the far ends, zeros of both signs
    and subnormals included."""
    dev = device()
    for dtype in (F16, BF16):
        gate = torch.arange(65536, device=dev, dtype=torch.int32).to(torch.int16).view(dtype)
        gate = gate[torch.isfinite(gate)].view(1, -1)
        if dtype == BF16:                       # beyond, f(g) g leaves fp32
            gate = gate[gate.abs() < 1e30].view(1, -1)
        y = torch.empty(gate.shape, device=dev)
        zs.zero_act(gate, kind, y=y)
        want, tol = ref.act(kind, gate, None)
        ref.assert_close(y, want, ref.half_step(F32, want) + tol, f"{kind} {dtype}")


def test_column_halves_of_one_product_and_of_its_gradient():
    """gate and up as the halves of one matrix, dgate and dup as the halves of its
    gradient; what lies beside stays; y in gate's place."""
    dev = device()
    rows, cols = 37, 200
    both = _randn(1, rows, 2 * cols + 16, dtype=F16)
    gate, up = both[:, 3:3 + cols], both[:, 3 + cols:3 + 2 * cols]
    y = torch.empty(rows, cols, dtype=F16, device=dev)
    gq, uq = zs.q8_empty(rows, cols, E4), zs.q8_empty(rows, cols, E4)
    zs.zero_act(gate, "silu", up=up, y=y, gate_q=gq[0], gate_s=gq[1], up_q=uq[0], up_s=uq[1])
    apart = torch.empty_like(y)
    gq2, uq2 = zs.q8_empty(rows, cols, E4), zs.q8_empty(rows, cols, E4)
    zs.zero_act(gate.contiguous(), "silu", up=up.contiguous(), y=apart, gate_q=gq2[0],
                gate_s=gq2[1], up_q=uq2[0], up_s=uq2[1])
    assert torch.equal(y, apart) and _same8(gq, gq2) and _same8(uq, uq2)
    dy = _randn(2, rows, cols, dtype=F16)
    d = torch.full((rows, 2 * cols + 16), 7.0, dtype=F16, device=dev)
    zs.zero_act_backward(dy, *gq, d[:, 3:3 + cols], "silu", up_q=uq[0], up_s=uq[1],
                         dup=d[:, 3 + cols:3 + 2 * cols])
    one, two = torch.empty_like(dy), torch.empty_like(dy)
    zs.zero_act_backward(dy, *gq, one, "silu", up_q=uq[0], up_s=uq[1], dup=two)
    assert torch.equal(d[:, 3:3 + cols], one) and torch.equal(d[:, 3 + cols:3 + 2 * cols], two)
    assert (d[:, :3] == 7).all() and (d[:, 3 + 2 * cols:] == 7).all()
    for which in range(3):                      # each output in dy's place
        t = dy.clone()
        outs = [torch.empty_like(dy) for _ in range(3)]
        outs[which] = t
        zs.zero_act_backward(t, *gq, outs[0], "silu", up_q=uq[0], up_s=uq[1], dup=outs[1],
                             y=outs[2])
        assert torch.equal(outs[0], one) and torch.equal(outs[1], two)
    kept = both.clone()
    zs.zero_act(gate, "silu", up=up, y=gate)
    assert torch.equal(gate, y)
    both[:, 3:3 + cols] = kept[:, 3:3 + cols]
    assert torch.equal(both, kept)
    zs.zero_act(gate, "silu", up=up, y=up)
    assert torch.equal(up, y)


@pytest.mark.parametrize("kind", KINDS)
def test_non_finite_and_zero_blocks(kind):
    """An infinite or NaN element spoils its checkpoint's block, from which the
    backward is NaN; y is the formula's; rows of zeros have scale 1."""
    dev = device()
    rows, cols = 4, 300
    gate, up = _randn(1, rows, cols), _randn(2, rows, cols)
    gate[0, 5], gate[1, 130], gate[2, 299], gate[3] = math.nan, math.inf, -math.inf, 0.0
    y = torch.empty_like(gate)
    gq, uq, q = (zs.q8_empty(rows, cols) for _ in range(3))
    zs.zero_act(gate, kind, up=up, y=y, q=q[0], s=q[1], gate_q=gq[0], gate_s=gq[1], up_q=uq[0],
                up_s=uq[1])
    assert torch.isnan(y[0, 5]) and torch.isinf(y[1, 130]) and torch.isnan(y[2, 299])
    assert int(torch.isfinite(y).sum()) == rows * cols - 3 and (y[3] == 0).all()
    assert gq[1].view(torch.uint8).tolist() == [[255, 127 + _e(gate[0, 128:256]), 127 + _e(
        gate[0, 256:]), 127], [127 + _e(gate[1, :128]), 255, 127 + _e(gate[1, 256:]), 127],
        [127 + _e(gate[2, :128]), 127 + _e(gate[2, 128:256]), 255, 127], [127] * 4]
    dy = torch.ones_like(gate)
    dgate, dup = torch.empty_like(dy), torch.empty_like(dy)
    zs.zero_act_backward(dy, *gq, dgate, kind, up_q=uq[0], up_s=uq[1], dup=dup)
    nan = torch.zeros(rows, cols, dtype=torch.bool, device=dev)
    nan[0, :128], nan[1, 128:256], nan[2, 256:] = True, True, True
    assert torch.equal(torch.isnan(dgate), nan) and torch.equal(torch.isnan(dup), nan)
    u = train_ref.from_blocks(*uq)[3, :cols]
    assert (dup[3] == 0).all() and torch.equal(dgate[3].double(), 0.5 * u)


def _e(block):
    return int(train_ref.scale_exponent(block.double().abs().amax().view(1), E4))


@pytest.mark.parametrize("kind", KINDS)
def test_backward_is_the_derivative(kind):
    """Against central differences of the 64-bit forward at the checkpoints' values."""
    dev = device()
    rows, cols = 20, 130
    gq, uq = zs.q8_empty(rows, cols), zs.q8_empty(rows, cols)
    zs.zero_q8_quantize(2 * _randn(1, rows, cols), *gq)
    zs.zero_q8_quantize(_randn(2, rows, cols), *uq)
    g, u = (train_ref.from_blocks(*t)[:, :cols] for t in (gq, uq))
    dy = _randn(3, rows, cols)
    dgate, dup = torch.empty_like(dy), torch.empty_like(dy)
    zs.zero_act_backward(dy, *gq, dgate, kind, up_q=uq[0], up_s=uq[1], dup=dup)
    vg, vu = _randn(4, rows, cols).double(), _randn(5, rows, cols).double()
    step = 1e-4
    up, down = (ref.act(kind, g + t * vg, u + t * vu)[0] for t in (step, -step))
    slope = (dy.double() * (up - down)).sum() / (2 * step)
    parts = torch.stack([(dgate.double() * vg), (dup.double() * vu)])
    assert abs(slope - parts.sum()) <= 1e-5 * parts.abs().sum()
    assert dev.type == "cuda"


def test_rows_without_outputs_and_empty_matrices():
    dev = device()
    e = torch.empty(0, 40, dtype=F16, device=dev)
    zs.zero_act(e, "gelu", y=torch.empty_like(e))
    e = torch.empty(5, 0, dtype=F16, device=dev)
    zs.zero_act(e, "gelu", y=torch.empty_like(e))
    with pytest.raises(ValueError):
        zs.zero_act(e, "relu", y=e)
    with pytest.raises(zs.ZeroStepError):
        zs.zero_act(torch.empty(5, 3, device=dev), "gelu")


def test_in_a_graph():
    dev = device()
    rows, cols = 300, 700
    gate, up, dy = (_randn(k, rows, cols, dtype=BF16) for k in (1, 2, 3))
    gq, uq, q = (zs.q8_empty(rows, cols) for _ in range(3))
    dgate, dup, y = (torch.empty_like(dy) for _ in range(3))

    def call():
        zs.zero_act(gate, "gelu_tanh", up=up, q=q[0], s=q[1], gate_q=gq[0], gate_s=gq[1],
                    up_q=uq[0], up_s=uq[1])
        zs.zero_act_backward(dy, *gq, dgate, "gelu_tanh", up_q=uq[0], up_s=uq[1], dup=dup, y=y)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    outs = (*q, *gq, *uq, dgate, dup, y)
    for k in range(3):
        gate.copy_(_randn(10 + k, rows, cols))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        call()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
                   for a, b in zip(got, outs))
    assert dev.type == "cuda"
