"""Log probabilities, entropy, top alternatives and their gradient, against the
64-bit definitions."""
import math

import pytest
import torch

import model_ref as ref
import sharded_mixed_precision_step_amd as zs
from gpu_util import device

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
U = ref.U


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(seed, *shape, dtype=F32):
    return torch.randn(*shape, generator=_gen(seed), device="cuda").to(dtype)


def _ids(seed, rows, vocab):
    ids = torch.randint(0, vocab, (rows,), generator=_gen(seed), device="cuda")
    return torch.where(torch.rand(rows, generator=_gen(seed + 1), device="cuda") < 0.2, -1, ids)


def _outputs(rows, top, dtype):
    out = [torch.full((rows,), 7.0, device="cuda") for _ in range(3)]
    if top:
        out += [torch.full((rows, top), 7, dtype=torch.int32, device="cuda"),
                torch.full((rows, top), 7.0, dtype=dtype, device="cuda")]
    return out


def _call(logits, ids, out, tau=1.0):
    zs.zero_logprob(logits, ids, out[0], entropy=out[1], lse=out[2], temperature=tau,
                    **(dict(top_index=out[3], top_logit=out[4]) if len(out) > 3 else {}))


def _check(logits, ids, top, tau=1.0):
    out = _outputs(logits.shape[0], top, logits.dtype)
    _call(logits, ids, out, tau)
    want, tol = ref.logprob(logits, ids, torch.tensor(tau, dtype=F32).double().item(), top)
    for got, w, t, name in zip(out, want, tol, ("logp", "entropy", "lse")):
        ref.assert_close(got, w, t + ref.half_step(F32, w.nan_to_num(0, 0, 0)), name)
    if top:
        assert torch.equal(out[3], want[3])
        assert torch.equal(out[4].float().nan_to_num(9e9), want[4].float().nan_to_num(9e9))
    return out


SHAPES = [(1, 1), (3, 2), (5, 7), (9, 100), (7, 129), (4, 1000), (6, 2049), (5, 8192), (5, 8193),
          (4, 16385), (3, 32001), (2, 32777), (3, 50001), (2, 131072)]


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_logprob_is_the_definition(rows, vocab, dtype):
    device()
    print(f"case: logprob {rows}x{vocab} {dtype}", flush=True)
    logits = (3 * _randn(1, rows, vocab)).to(dtype)
    ids = _ids(2, rows, vocab)
    for top, tau in ((0, 1.0), (1, 0.7), (5, 1.0), (64, 2.5), (128, 1.0)):
        _check(logits, ids, top, tau)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("vocab", [40, 300, 3001, 9000, 40001, 70000])
def test_ties_take_the_lowest_places(dtype, vocab):
    """Rows of few values: the border lies inside a run of equal logits, up to all
    of a row; rising and falling rows; zeros of both signs."""
    device()
    i = torch.arange(vocab, device="cuda")
    rows = torch.stack([torch.zeros(vocab, device="cuda"), (i % 3).float(), (i % 50).float(),
                        -(i % 7 == 3).float(), i.float() / vocab, -i.float() / vocab,
                        torch.where(i % 2 == 0, 0.0, -0.0), (i == vocab // 2).float(),
                        (i >= vocab - 20).float() + (i < 5) * 2.0]).to(dtype)
    ids = torch.full((rows.shape[0],), vocab - 1, device="cuda")
    for top in (1, 3, 20, 100, 128):
        print(f"case: ties {vocab} top {top}", flush=True)
        _check(rows, ids, top)


def test_masked_vocabularies_and_rows_without_an_answer():
    device()
    rows, vocab = 11, 3000
    logits = 3 * _randn(1, rows, vocab)
    ids = torch.arange(rows, device="cuda") * 7
    logits[0, 10:] = -math.inf                  # ten alternatives left
    logits[1] = -math.inf                       # none
    logits[2] = -math.inf
    logits[2, 14] = -5.0                        # one, the token itself
    logits[3, 100] = math.nan
    logits[4, 100] = math.inf
    ids[5] = vocab                              # no such token
    ids[6] = -1
    logits[6] = math.nan                        # left out
    logits[7, 49] = -math.inf                   # the token itself is masked
    logits[8] = torch.finfo(F32).min            # all of the type's lowest value
    logits[9, 5:] = torch.finfo(F32).min
    ids[10] = 2 ** 40
    out = _check(logits, ids, 20)
    assert out[3][0, 10:].eq(-1).all() and out[4][0, 10:].eq(-math.inf).all()
    assert out[0][7] == -math.inf and math.isfinite(float(out[1][7]))
    bad = [1, 3, 4, 5, 10]
    for k in range(3):
        assert torch.isnan(out[k][bad]).all() and out[k][6] == 0
    assert out[3][bad].eq(0).all() and torch.isnan(out[4][bad]).all()
    assert out[3][6].eq(-1).all() and out[0][2] == 0 and out[1][2] == 0
    assert abs(float(out[1][8]) - math.log(vocab)) < 1e-5
    for dtype in (F16, BF16):
        low = logits.to(dtype)
        low[8], low[9, 5:] = torch.finfo(dtype).min, torch.finfo(dtype).min
        _check(low, ids, 20)
        _check(low, ids, 20, 0.5)


def test_large_logits_and_small_temperatures():
    device()
    logits = torch.tensor([[3e38, 1e38, -3e38, 0.0], [65504.0, 65503.0, -65504.0, 0.0],
                           [1e-30, 0.0, -1e-30, 2e-30]], device="cuda")
    ids = torch.tensor([0, 1, 3], device="cuda")
    for tau in (1.0, 0.5, 1e-6, 1e6):
        out = _check(logits, ids, 3, tau)
        # the row's largest over tau may leave fp32, its own log probability not
        assert math.isfinite(float(out[0][0])) and math.isfinite(float(out[1][0]))


def test_outputs_alone_strided_and_without_ids():
    """Each output by itself has the bits it has among the others; strided rows at
    odd addresses; no ids; 32-bit ids; what lies beside stays."""
    dev = device()
    rows, vocab, top = 13, 5003, 9
    base = (3 * _randn(1, rows, vocab + 20)).half()
    logits = base[:, 3:3 + vocab]
    ids = _ids(4, rows, vocab)
    whole = _check(logits, ids, top)
    ti = torch.full((rows, top + 4), 7, dtype=torch.int32, device=dev)
    tl = torch.full((rows, top + 4), 7.0, dtype=F16, device=dev)
    zs.zero_logprob(logits, ids.int(), None, top_index=ti[:, :top], top_logit=tl[:, :top])
    assert torch.equal(ti[:, :top], whole[3]) and torch.equal(tl[:, :top], whole[4])
    assert (ti[:, top:] == 7).all() and (tl[:, top:] == 7).all()
    one = torch.empty(rows, device=dev)
    zs.zero_logprob(logits, ids, one)
    assert torch.equal(one, whole[0])
    zs.zero_logprob(logits, ids, None, entropy=one)
    assert torch.equal(one, whole[1])
    zs.zero_logprob(logits, ids, None, lse=one)
    assert torch.equal(one, whole[2])
    out = _outputs(rows, top, F16)
    zs.zero_logprob(logits, None, None, entropy=out[1], lse=out[2], top_index=out[3],
                    top_logit=out[4])
    on = ids >= 0
    for k in (1, 2, 3, 4):
        assert torch.equal(out[k][on], whole[k][on])
    assert (out[3][~on] >= 0).all() and (out[2][~on] != 0).all()


@pytest.mark.parametrize("vocab", [31, 5003, 40001, 140001])
def test_each_alignment(vocab):
    """Rows that start at every multiple of an element within 16 bytes."""
    device()
    for dtype in (F16, F32):
        flat = (3 * _randn(1, 3 * (vocab + 16))).to(dtype)
        for start in range(16 // flat.element_size()):
            row = flat[start:start + 2 * vocab].view(2, vocab)
            _check(row, torch.tensor([0, vocab - 1], device="cuda"), 6)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_backward_is_the_formula(rows, vocab, dtype):
    dev = device()
    print(f"case: logprob backward {rows}x{vocab} {dtype}", flush=True)
    logits = (3 * _randn(1, rows, vocab)).to(dtype)
    ids = _ids(2, rows, vocab)
    a, b = _randn(3, rows), 0.1 * _randn(4, rows)
    if rows > 2:
        a[2], b[2] = 0.0, 0.0
    for tau, use in ((1.0, "a"), (0.7, "ab"), (1.0, "b")):
        t = torch.tensor(tau, dtype=F32).double().item()
        out = _outputs(rows, 0, dtype)
        _call(logits, ids, out, tau)
        kw = dict(entropy=out[1], dentropy=b) if "b" in use else {}
        grad = torch.full_like(logits, 7.0)
        zs.zero_logprob_backward(logits, ids, out[2], a if "a" in use else None, grad,
                                 temperature=tau, loss_scale=64.0, **kw)
        want, tol = ref.logprob_backward(logits, ids, t, out[2], a if "a" in use else None,
                                         out[1], b if "b" in use else None, 64.0)
        ref.assert_close(grad, want, ref.half_step(dtype, want) + tol, f"grad {use}")
        if "a" not in use:                      # needs no token
            again = torch.empty_like(grad)
            lse2, ent2 = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
            zs.zero_logprob(logits, None, None, entropy=ent2, lse=lse2, temperature=tau)
            zs.zero_logprob_backward(logits, None, lse2, None, again, entropy=ent2, dentropy=b,
                                     temperature=tau, loss_scale=64.0)
            on = ids >= 0
            assert torch.equal(again[on], grad[on])
        inplace = logits.clone()
        zs.zero_logprob_backward(inplace, ids, out[2], a if "a" in use else None, inplace,
                                 temperature=tau, loss_scale=64.0, **kw)
        assert torch.equal(inplace, grad)


def test_backward_rows_without_an_answer():
    dev = device()
    rows, vocab = 8, 300
    logits = 3 * _randn(1, rows, vocab)
    ids = torch.arange(rows, device=dev)
    a, b = _randn(2, rows), _randn(3, rows)
    logits[0, 7] = math.nan
    ids[1] = -1
    logits[1] = math.nan
    a[2], b[2] = 0.0, 0.0
    logits[2, 9] = math.inf
    ids[3] = vocab
    logits[4, 50:] = -math.inf
    logits[5, 5] = -math.inf                    # the token itself
    ids[6], a[6], b[6] = vocab, 0.0, 0.0
    out = _outputs(rows, 0, F32)
    _call(logits, ids, out)
    grad = torch.full_like(logits, 7.0)
    zs.zero_logprob_backward(logits, ids, out[2], a, grad, entropy=out[1], dentropy=b)
    assert torch.isnan(grad[[0, 3]]).all() and (grad[[1, 2, 6]] == 0).all()
    live = [4, 5, 7]
    want, tol = ref.logprob_backward(logits[live], ids[live], 1.0, out[2][live], a[live],
                                     out[1][live], b[live], 1.0)
    ref.assert_close(grad[live], want, ref.half_step(F32, want) + tol, "grad")
    assert (grad[4, 50:] == 0).all()


def test_backward_takes_the_control_blocks_scale():
    dev = device()
    logits, ids = 3 * _randn(1, 6, 500), torch.arange(6, device=dev)
    ctl = zs.control_new(zs.LossScaler.create(scale=256.0), 1, dev)
    out = _outputs(6, 0, F32)
    _call(logits, ids, out)
    one, two, a = torch.empty_like(logits), torch.empty_like(logits), _randn(2, 6)
    zs.zero_logprob_backward(logits, ids, out[2], a, one, loss_scale=256.0)
    stepper = zs.DeviceStepper(ctl, zs.AdamWParams(1e-3, 0.9, 0.999, 1e-8, 0.01, 1, 1, 1))
    stepper.logprob_backward(logits, ids, out[2], a, two)
    assert torch.equal(one, two)


def test_backward_is_the_derivative():
    """Against central differences of the 64-bit logp and entropy."""
    dev = device()
    rows, vocab, tau = 12, 200, 0.7
    t = torch.tensor(tau, dtype=F32).double().item()
    logits, ids = 3 * _randn(1, rows, vocab), torch.arange(rows, device=dev)
    a, b = _randn(2, rows), _randn(3, rows)
    out = _outputs(rows, 0, F32)
    _call(logits, ids, out, tau)
    grad = torch.empty_like(logits)
    zs.zero_logprob_backward(logits, ids, out[2], a, grad, entropy=out[1], dentropy=b,
                             temperature=tau)
    v = _randn(4, rows, vocab).double()

    def f(step):
        (logp, ent, _), _ = ref.logprob(logits.double() + step * v, ids, t, 0)
        return (a.double() * logp + b.double() * ent).sum()

    slope = (f(1e-4) - f(-1e-4)) / 2e-4
    terms = grad.double() * v
    assert abs(slope - terms.sum()) <= 1e-4 * terms.abs().sum()


def test_alternatives_are_what_the_distillation_takes():
    """A teacher's alternatives go straight into zero_distill: a student with the
    same logits, over a vocabulary that they fill, has a loss of 0; a row that the
    teacher leaves out, or has no answer for, is one."""
    dev = device()
    rows, vocab = 6, 40
    teacher = 3 * _randn(1, rows, vocab)
    ids = torch.tensor([0, 1, -1, 3, 4, 5], device=dev)
    teacher[3, 2] = math.nan
    out = _outputs(rows, vocab, F32)
    _call(teacher, ids, out)
    student = torch.where(torch.isnan(teacher), 0.0, teacher)
    loss, grad = torch.empty(rows, device=dev), torch.empty_like(student)
    zs.zero_distill(student, out[3], out[4], loss, None, grad)
    ok = [0, 1, 4, 5]
    assert (loss[ok].abs() < 1e-5).all() and (grad[ok].abs() < 1e-6).all()
    assert loss[2] == 0 and (grad[2] == 0).all() and torch.isnan(loss[3])
    assert torch.isnan(grad[3]).all()


def test_in_a_graph():
    dev = device()
    rows, vocab, top = 40, 9000, 10
    logits, ids = (3 * _randn(1, rows, vocab)).half(), _ids(2, rows, vocab)
    out, a, grad = _outputs(rows, top, F16), _randn(3, rows), torch.empty_like(logits)

    def call():
        _call(logits, ids, out)
        zs.zero_logprob_backward(logits, ids, out[2], a, grad, entropy=out[1], dentropy=a)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(3):
        logits.copy_(3 * _randn(10 + k, rows, vocab))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*out, grad)]
        call()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, (*out, grad)))
    assert dev.type == "cuda"


@pytest.mark.slow
def test_offsets_past_32_bits():
    device()
    rows, vocab = 33000, 131072
    print(f"case: logprob {rows}x{vocab}", flush=True)
    logits = torch.zeros(rows, vocab, dtype=F16, device="cuda")
    last = (3 * _randn(1, 40, vocab)).half()
    logits[-40:] = last
    ids = torch.full((rows,), -1, device="cuda")
    ids[-40:] = torch.arange(40, device="cuda")
    out, part = _outputs(rows, 5, F16), _outputs(40, 5, F16)
    _call(logits, ids, out)
    _call(last, ids[-40:], part)
    # few rows are summed in another order than many: both within the bounds of the sums
    want, tol = ref.logprob(last, ids[-40:], 1.0, 5)
    for got in ([p[-40:] for p in out], part):
        for g, w, t in zip(got, want, tol):
            ref.assert_close(g, w, t + ref.half_step(F32, w), "few and many rows")
        assert torch.equal(got[3], want[3]) and torch.equal(got[4].float(), want[4].float())
    out[2][-40:] = part[2]
    a = torch.zeros(rows, device="cuda")
    a[-40:] = 1.0
    grad = torch.empty_like(last)
    zs.zero_logprob_backward(last, ids[-40:], part[2], a[-40:], grad)
    zs.zero_logprob_backward(logits, ids, out[2], a, logits)
    assert torch.equal(logits[-40:], grad) and not logits[:-40].any()
