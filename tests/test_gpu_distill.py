"""Distillation loss and gradient against the 64-bit definition."""
import math

import pytest
import torch

import sharded_mixed_precision_step_amd as zs
import train_ref as ref
from gpu_util import device

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
U = ref.U


def _case(rows, vocab, top, dtype, tdtype, idtype=torch.int32, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + rows + vocab)
    logits = (2.5 * torch.randn(rows, vocab, generator=g, device="cuda")).to(dtype)
    index = torch.randint(0, vocab, (rows, top), generator=g, device="cuda").to(idtype)
    teacher = (4 + 1.5 * torch.randn(rows, top, generator=g, device="cuda")).to(tdtype)
    weight = torch.rand(rows, generator=g, device="cuda") / rows
    return logits, index, teacher, weight


def _tols(logits, index, teacher, tau, weight, S, loss, lse, grad):
    """Bounds for (loss, lse, grad).  A lane sums vocab / 256 exponentials at
    most (256 lanes or more share a row), 30 joins follow; each exponential is
    off by two steps of exp2 and by the rounding of its argument, at most
    range * log2(e) * 2u; lse adds roundings at the size of its terms."""
    rows, vocab = logits.shape
    z = logits.double() / tau
    zmax = z.nan_to_num(0, 0, 0).abs().amax(1)
    t = teacher.double().nan_to_num(0, 0, 0).abs().amax(1) / tau
    rel = U * (vocab / 256 + 40 + 6 * zmax)
    tol_lse = rel + U * 4 * (zmax + lse.abs().nan_to_num(0))
    w = torch.ones(rows, device=z.device).double() if weight is None else weight.double()
    tol_loss = (w * tau * tau).abs() * (tol_lse * 2 + U * (64 + 6 * t + 6 * zmax + 1100)) \
        + 4 * U * loss.abs().nan_to_num(0)
    coef = (S * w * tau).abs()
    q = torch.exp(z - lse[:, None]).nan_to_num(0, 0, 0)
    taken = (q - grad.nan_to_num(0, 0, 0) / coef.clamp_min(1e-300)[:, None]).abs()
    relg = tol_lse * 2 + U * (64 + 6 * t + 6 * zmax + 1100)
    tol_grad = ref.half_step(grad_dtype(logits), grad.nan_to_num(0, 0, 0)) + \
        coef[:, None] * (q + taken) * relg[:, None] * 1.01
    return tol_loss, tol_lse, tol_grad


def grad_dtype(logits):
    return logits.dtype


def _run(logits, index, teacher, tau, weight, S, two=False, ctl=None):
    rows = logits.shape[0]
    loss, lse = (torch.full((rows,), 7.0, device="cuda") for _ in range(2))
    grad = torch.full_like(logits, 7.0)
    if two:
        zs.zero_distill_forward(logits, index, teacher, loss, lse, temperature=tau,
                                row_weight=weight)
        zs.zero_distill_backward(logits, index, teacher, lse, grad, temperature=tau,
                                 row_weight=weight, loss_scale=S, ctl=ctl)
    else:
        zs.zero_distill(logits, index, teacher, loss, lse, grad, temperature=tau,
                        row_weight=weight, loss_scale=S, ctl=ctl)
    return loss, lse, grad


def _check(logits, index, teacher, tau, weight, S, two=False):
    loss, lse, grad = _run(logits, index, teacher, tau, weight, S, two)
    want = ref.distill(logits, index, teacher, tau, weight, S)
    tl, te, tg = _tols(logits, index, teacher, tau, weight, S, *want)
    ref.assert_close(lse, want[1], te, "lse")
    ref.assert_close(loss, want[0], tl, "loss")
    ref.assert_close(grad, want[2], tg, "grad")


SHAPES = [(1, 1, 1), (3, 2, 4), (5, 7, 3), (4, 100, 1), (7, 1000, 33), (3, 8191, 64),
          (5, 8193, 100), (2, 32001, 20), (37, 5000, 1024), (2, 65536, 64), (3, 131071, 64),
          (2, 131072, 16), (2, 151001, 50), (1, 300007, 128)]


@pytest.mark.parametrize("two", [False, True])
@pytest.mark.parametrize("dtype,tdtype,tau", [(F16, F32, 1.0), (BF16, BF16, 2.0),
                                              (F32, F16, 0.7)])
@pytest.mark.parametrize("rows,vocab,top", SHAPES)
def test_distill_is_the_definition(rows, vocab, top, dtype, tdtype, tau, two):
    device()
    print(f"case: distill {rows}x{vocab} top {top} {dtype} {tdtype} tau {tau} two {two}",
          flush=True)
    idt = torch.int64 if rows % 2 else torch.int32
    logits, index, teacher, weight = _case(rows, vocab, top, dtype, tdtype, idt)
    _check(logits, index, teacher, tau, weight, 1024.0, two)
    _check(logits, index, teacher, tau, None, 1.0, two)


@pytest.mark.parametrize("two", [False, True])
@pytest.mark.parametrize("vocab", [333, 9000, 140_000])
@pytest.mark.parametrize("dtype", [F16, F32])
def test_distill_special_rows(dtype, vocab, two):
    """One kind of row each: masked with anything in it, no entries, all
    teacher logits -inf, an index out of range, NaN or inf logits and entries,
    -inf and lowest-value masks, a repeated index, an entry of no mass on a
    masked logit, negative indices in between."""
    device()
    rows, top = 16, 5
    logits, index, teacher, weight = _case(rows, vocab, top, dtype, F32, seed=5)
    low = torch.finfo(dtype).min
    logits[0], teacher[0], index[0], weight[0] = math.nan, math.nan, vocab + 5, 0.0
    index[1] = -1
    teacher[2] = -math.inf
    index[3, 2] = vocab
    logits[4, vocab // 2] = math.nan
    logits[5, vocab - 1] = math.inf
    teacher[6, 1] = math.nan
    teacher[7, 4] = math.inf
    logits[8, : vocab // 2] = -math.inf
    index[8] = torch.arange(vocab - top, vocab, device="cuda")
    logits[9] = -math.inf
    logits[10] = low
    logits[11, 1:] = low
    index[11] = 0
    index[12] = 17
    teacher[13, 0], logits[13, 50] = -math.inf, -math.inf
    index[13, 0], index[13, 1:] = 50, torch.arange(1, top, device="cuda", dtype=torch.int32)
    index[14, 0::2] = -1
    index[15, 1:] = -7
    _check(logits, index, teacher, 1.0, weight, 8.0, two)
    loss, lse, grad = _run(logits, index, teacher, 1.0, weight, 8.0, two)
    assert (grad[:3][[0, 1, 2]] == 0).all() and (loss[:3] == 0).all() and lse[0] == 0
    for r in (3, 4, 5, 6, 7, 9):
        assert torch.isnan(grad[r]).all() and torch.isnan(loss[r]) and torch.isnan(lse[r]), r


def test_distill_mass_on_a_masked_logit_is_an_infinite_loss():
    device()
    logits, index, teacher, weight = _case(2, 100, 3, F32, F32)
    index[0] = torch.tensor([4, 5, 6], device="cuda")
    logits[0, 5] = -math.inf
    loss, lse, grad = _run(logits, index, teacher, 1.0, weight, 1.0)
    assert loss[0] == math.inf and torch.isfinite(grad).all() and torch.isfinite(loss[1])


@pytest.mark.parametrize("two", [False, True])
@pytest.mark.parametrize("vocab", [1000, 20001, 131072, 200000])
def test_distill_in_place_and_strided(vocab, two):
    """The gradient over the logits; rows with any stride and alignment; what
    lies beside the gradient stays."""
    dev = device()
    rows, top, tau, S = 6, 9, 2.0, 64.0
    logits, index, teacher, weight = _case(rows, vocab, top, F16, F32)
    loss, lse, grad = _run(logits, index, teacher, tau, weight, S, two)
    base = torch.full((rows, vocab + 11), 7.0, dtype=F16, device=dev)
    base[:, 3:3 + vocab] = logits
    x = base[:, 3:3 + vocab]
    wide = torch.full((rows, vocab + 5), 9.0, dtype=F16, device=dev)
    g = wide[:, 1:1 + vocab]
    l2, e2 = torch.empty_like(loss), torch.empty_like(lse)
    for out in (g, x):
        if two:
            zs.zero_distill_forward(x, index, teacher, l2, e2, temperature=tau, row_weight=weight)
            zs.zero_distill_backward(x, index, teacher, e2, out, temperature=tau,
                                     row_weight=weight, loss_scale=S)
        else:
            zs.zero_distill(x, index, teacher, l2, e2, out, temperature=tau, row_weight=weight,
                            loss_scale=S)
        want = ref.distill(logits, index, teacher, tau, weight, S)
        tl, te, tg = _tols(logits, index, teacher, tau, weight, S, *want)
        ref.assert_close(e2, want[1], te, "lse")
        ref.assert_close(l2, want[0], tl, "loss")
        ref.assert_close(out, want[2], tg, "grad")
    assert (wide[:, 0] == 9).all() and (wide[:, 1 + vocab:] == 9).all()
    assert (base[:, :3] == 7).all() and (base[:, 3 + vocab:] == 7).all()


def test_distill_takes_the_control_blocks_scale():
    dev = device()
    logits, index, teacher, weight = _case(5, 2000, 8, F16, F32)
    ctl = zs.control_new(zs.LossScaler.create(scale=512.0), 1, dev)
    for two in (False, True):
        a = _run(logits, index, teacher, 1.0, weight, 512.0, two)
        b = _run(logits, index, teacher, 1.0, weight, 3.0, two, ctl=ctl)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_gradient_against_differences():
    """Directional central difference of the 64-bit loss, weighted by the
    rows, along a random direction."""
    device()
    rows, vocab, top, tau = 6, 700, 12, 1.7
    logits, index, teacher, weight = _case(rows, vocab, top, F32, F32)
    _, _, grad = _run(logits, index, teacher, tau, weight, 1.0)
    v = torch.randn(rows, vocab, device="cuda").double()
    f = lambda t: ref.distill(logits.double() + t * v, index, teacher, tau, weight,  # noqa: E731
                              1.0)[0].sum()
    step = 1e-5
    want = (f(step) - f(-step)) / (2 * step)
    got, size = (grad.double() * v).sum(), (grad.double() * v).abs().sum()
    assert abs(float(got - want)) <= 2e-6 * float(size)


def test_distill_repeats_bit_for_bit_on_streams_and_in_graphs():
    device()
    cases = [_case(33, 5001, 40, F16, F32), _case(9, 131072, 64, BF16, F32),
             _case(3, 140_001, 64, F16, F16)]
    want = [_run(*c[:3], 2.0, c[3], 256.0) for c in cases]
    bufs = [tuple(torch.empty_like(t) for t in w) for w in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for st, c, b in zip(streams, cases, bufs):
        zs.zero_distill(*c[:3], b[0], b[1], b[2], temperature=2.0, row_weight=c[3],
                        loss_scale=256.0, stream=st)
    torch.cuda.synchronize()
    for w, b in zip(want, bufs):
        assert all(torch.equal(x, y) for x, y in zip(w, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c, b in zip(cases, bufs):
            zs.zero_distill(*c[:3], b[0], b[1], b[2], temperature=2.0, row_weight=c[3],
                            loss_scale=256.0)
    for k in range(3):
        for b in bufs:
            for t in b:
                t.fill_(k)
        graph.replay()
        torch.cuda.synchronize()
        for c, w, b in zip(cases, want, bufs):
            assert all(torch.equal(x, y) for x, y in zip(w, b)), k
            _run(*c[:3], 2.0, c[3], 256.0)


@pytest.mark.slow
def test_distill_past_2_31_elements():
    dev = device()
    rows, vocab, top = 17_000, 131_072, 4
    logits = torch.zeros(rows, vocab, dtype=F16, device=dev)
    index = torch.arange(top, device=dev, dtype=torch.int32).expand(rows, top).contiguous()
    teacher = torch.zeros(rows, top, device=dev)
    grad = torch.full_like(logits, 7.0)
    loss, lse = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
    zs.zero_distill(logits, index, teacher, loss, lse, grad, loss_scale=1024.0)
    # uniform student: lse = ln vocab, q = 1 / vocab, loss = ln(vocab / top)
    assert abs(float(lse.min()) - math.log(vocab)) < 1e-5 and float(lse.min()) == float(lse.max())
    assert abs(float(loss.max()) - math.log(vocab / top)) < 2e-5
    assert float(loss.min()) == float(loss.max())
    assert (grad[:, :top] == 1024.0 * (1 / vocab - 0.25)).all()
    assert (grad[-1, top:] == 1024.0 / vocab).all() and (grad[:, top:] == 1024.0 / vocab).all()


@pytest.mark.parametrize("two", [False, True])
@pytest.mark.parametrize("tdtype", [F32, BF16, F16])
@pytest.mark.parametrize("tau", [0.25, 3.0])
def test_distill_teacher_logits_of_the_lowest_value(tau, tdtype, two):
    """Masks of the type's lowest value: beside others, no mass, as -inf (fp16's
    lowest is 65504 / 3 below anything here, of no mass in fp32 either); a row
    of nothing else is uniform, as any row of equal logits.  Divided by a
    temperature below 1 they leave fp32's range."""
    device()
    logits, index, teacher, weight = _case(6, 700, 9, F16, tdtype)
    lowest = torch.finfo(tdtype).min
    teacher[1], teacher[2, ::2], teacher[3, 1:] = lowest, lowest, lowest
    teacher[4] = torch.finfo(tdtype).max
    same = teacher.clone()
    same[1], same[2, ::2], same[3, 1:], same[4] = 0, -math.inf, -math.inf, 0
    got = _run(logits, index, teacher, tau, weight, 64.0, two)
    want = _run(logits, index, same, tau, weight, 64.0, two)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    _check(logits, index, same, tau, weight, 64.0, two)


@pytest.mark.parametrize("two", [False, True])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,vocab,top", [(19, 8200, 70), (3, 12345, 1000), (5, 16384, 3),
                                            (4, 16385, 600)])
def test_distill_of_rows_that_512_lanes_hold(rows, vocab, top, dtype, two):
    """And the first that they do not; in the logits' place too, at an odd
    address."""
    device()
    logits, index, teacher, weight = _case(rows, vocab, top, dtype, F32, torch.int64)
    _check(logits, index, teacher, 1.5, weight, 512.0, two)
    base = torch.empty(rows, vocab + 3, dtype=dtype, device="cuda")
    base[:, 1:1 + vocab] = logits
    want = _run(logits, index, teacher, 1.5, weight, 512.0, two)
    own = base[:, 1:1 + vocab]
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    zs.zero_distill(own, index, teacher, loss, lse, own, temperature=1.5, row_weight=weight,
                    loss_scale=512.0)
    tl, te, tg = _tols(logits, index, teacher, 1.5, weight, 512.0,
                       *(x.double() for x in want))
    ref.assert_close(own, want[2].double(), 2 * tg, "grad in place")
    ref.assert_close(loss, want[0].double(), 2 * tl, "loss")


@pytest.mark.parametrize("tau", [1e-19, 3e-22, 2.0 ** -100])
def test_temperatures_whose_square_is_below_the_range(tau):
    """One entry, p = 1, and a student whose softmax is one-hot, sum = 1: the loss
    is w tau^2 (m - z) / tau.  1 / tau, the quotient, tau times it and the two
    factors round, each by half a step: six roundings."""
    logits, index, teacher, weight = _case(9, 3000, 1, F32, F32)
    tau = float(torch.tensor(tau, dtype=F32))
    loss = torch.full((9,), 7.0, device="cuda")
    zs.zero_distill_forward(logits, index, teacher, loss, None, temperature=tau, row_weight=weight)
    z = logits.double()
    want = weight.double() * tau * (z.amax(1) - z.gather(1, index.long())[:, 0])
    assert (want > 2.0 ** -120).all()
    ref.assert_close(loss, want, 6.1 * U * want, "loss")
