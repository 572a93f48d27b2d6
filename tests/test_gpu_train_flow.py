"""The training operators together, as one rank's program runs them around the
shard step: parameters to 8 bits, norm, product, distillation loss under the
control block's scale, the products of the backward pass, the norm's backward,
bucket flatten, and the step.  Every stage is checked against its 64-bit
definition on what the stage before it left, the step against the oracle."""
import numpy as np
import pytest
import torch

import oracle.zero_step as ozs
import sharded_mixed_precision_step_amd as zs
import train_ref as ref
import workloads as wl
from gpu_util import device
from test_gpu_distill import _tols
from test_gpu_norm import NORM, U, _assert_backward, _check_q
from test_gpu_q8 import _check_q8, _gemm_tol

pytestmark = pytest.mark.gpu

E4 = torch.float8_e4m3fn
EPS = 1e-5
TOKENS, WIDTH, VOCAB, TOP = 203, 384, 1000, 16
N_PARAMS = VOCAB * WIDTH + WIDTH


class Program:
    """A norm, a projection to the vocabulary and the loss, with their gradients
    flattened into one bucket, over parameters [projection, norm weight]."""

    def __init__(self, dev, scale):
        g = torch.Generator(device=dev)
        g.manual_seed(3)
        rnd = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
        self.x, self.res = rnd(TOKENS, WIDTH).half(), rnd(TOKENS, WIDTH)
        self.index = torch.randint(0, VOCAB, (TOKENS, TOP), generator=g, device=dev)
        self.teacher = 3 + rnd(TOKENS, TOP)
        self.weight = (torch.rand(TOKENS, generator=g, device=dev) < 0.9).float() / TOKENS
        self.dres = (0.01 * rnd(TOKENS, WIDTH)).half()
        self.bucket = torch.zeros(-(-N_PARAMS // 256) * 256, dtype=torch.float16, device=dev)
        n = self.bucket.numel()
        master = torch.zeros(n, device=dev)
        master[:VOCAB * WIDTH] = 0.05 * rnd(VOCAB * WIDTH)
        master[VOCAB * WIDTH:N_PARAMS] = 1 + 0.1 * rnd(WIDTH)
        self.state = [master, torch.zeros(n, device=dev), torch.zeros(n, device=dev),
                      master.half()]
        self.ctl = zs.control_new(zs.LossScaler.create(scale=scale), 1, dev)
        self.hyper = wl.AdamWHyper()
        self.stepper = zs.DeviceStepper(self.ctl, zs.adamw_params(self.hyper))
        e = torch.empty
        self.q = {k: zs.q8_empty(r, c, E4, dev) for k, (r, c) in dict(
            w=(VOCAB, WIDTH), wt=(WIDTH, VOCAB), y=(TOKENS, WIDTH), yt=(WIDTH, TOKENS),
            d=(TOKENS, VOCAB), dt=(VOCAB, TOKENS)).items()}
        self.h, self.rstd = e(TOKENS, WIDTH, device=dev), e(TOKENS, device=dev)
        self.y = e(TOKENS, WIDTH, dtype=torch.float16, device=dev)
        self.logits = e(TOKENS, VOCAB, dtype=torch.float16, device=dev)
        self.dlogits = torch.empty_like(self.logits)
        self.loss, self.lse = e(TOKENS, device=dev), e(TOKENS, device=dev)
        self.dy, self.dx = torch.empty_like(self.y), torch.empty_like(self.y)
        self.dw = e(VOCAB, WIDTH, dtype=torch.float16, device=dev)
        self.dnorm = e(WIDTH, dtype=torch.float16, device=dev)
        self.work = e(zs.zero_rmsnorm_backward_workspace(TOKENS, WIDTH), dtype=torch.uint8,
                      device=dev)

    def params(self):
        p16 = self.state[3]
        return p16[:VOCAB * WIDTH].view(VOCAB, WIDTH), p16[VOCAB * WIDTH:N_PARAMS]

    def gradients(self):
        w, norm_w = self.params()
        q = self.q
        zs.zero_q8_quantize(w, *q["w"], *q["wt"])
        zs.zero_rmsnorm(self.x, norm_w, EPS, residual=self.res, h=self.h, y=self.y, q=q["y"][0],
                        s=q["y"][1], rstd=self.rstd)
        zs.zero_q8_quantize(self.y, qt=q["yt"][0], st=q["yt"][1])
        zs.zero_q8_gemm(*q["y"], *q["w"], self.logits)
        self.stepper.distill(self.logits, self.index, self.teacher, self.loss, self.lse,
                             self.dlogits, temperature=2.0, row_weight=self.weight)
        zs.zero_q8_quantize(self.dlogits, *q["d"], *q["dt"])
        zs.zero_q8_gemm(*q["d"], *q["wt"], self.dy)
        zs.zero_q8_gemm(*q["dt"], *q["yt"], self.dw)
        zs.zero_rmsnorm_backward(self.dy, self.h, norm_w, self.rstd, self.dx, self.dnorm,
                                 self.work, dres=self.dres)
        zs.zero_bucket_flatten([self.dw, self.dnorm], self.bucket)

    def step(self):
        self.gradients()
        self.stepper.two_pass([self.bucket], *self.state)

    def outputs(self):
        return [t.clone() for t in (self.logits, self.loss, self.dlogits, self.dx, self.bucket,
                                    *self.state)]


def _check_gradients(p, S):
    w, norm_w = p.params()
    q = p.q
    val = {k: ref.from_blocks(*q[k]) for k in q}
    _check_q8(w, *q["w"], E4, "w")
    _check_q8(w.t(), *q["wt"], E4, "w transposed")
    h, rstd, y = ref.rmsnorm(p.x, p.res, norm_w, EPS)
    ref.assert_close(p.h, h, ref.half_step(torch.float32, h) + U * h.abs(), "h")
    ref.assert_close(p.y, y, ref.half_step(torch.float16, y) + NORM * y.abs(), "y")
    _check_q(*q["y"], y, E4)
    _check_q8(p.y.t(), *q["yt"], E4, "y transposed")

    def product(got, a, b, name):
        want = val[a] @ val[b].t()
        ref.assert_close(got, want, _gemm_tol(val[a], val[b], q[a][1], q[b][1], got.dtype, want),
                         name)

    product(p.logits, "y", "w", "logits")
    want = ref.distill(p.logits, p.index, p.teacher, 2.0, p.weight, S)
    tl, te, tg = _tols(p.logits, p.index, p.teacher, 2.0, p.weight, S, *want)
    ref.assert_close(p.loss, want[0], tl, "loss")
    ref.assert_close(p.dlogits, want[2], tg, "dlogits")
    _check_q8(p.dlogits, *q["d"], E4, "dlogits")
    _check_q8(p.dlogits.t(), *q["dt"], E4, "dlogits transposed")
    product(p.dy, "d", "wt", "dy")
    product(p.dw, "dt", "yt", "dw")
    wx, ww = ref.rmsnorm_backward(p.dy, p.h, norm_w, p.rstd, p.dres)
    _assert_backward(p.dx, p.dnorm, wx, ww, p.dy, p.h, norm_w, p.rstd, p.dres)
    assert torch.equal(p.bucket[:VOCAB * WIDTH].view(VOCAB, WIDTH), p.dw)
    assert torch.equal(p.bucket[VOCAB * WIDTH:N_PARAMS], p.dnorm)


def test_two_steps_match_their_definitions_and_the_oracle():
    dev = device()
    p = Program(dev, 1024.0)
    for t in (1, 2):
        before = [x.cpu().numpy() for x in p.state]
        p.step()
        torch.cuda.synchronize()
        ctl = zs.control_read(p.ctl)
        assert ctl.overflow == 0 and ctl.step == t + 1 and ctl.scale == 1024.0
        after = [x.clone() for x in p.state]
        # the gradients came from the parameters before the step
        p.state[3].copy_(torch.from_numpy(before[3]))
        _check_gradients(p, 1024.0)
        p.state[3].copy_(after[3])
        want = ozs.shard_step([p.bucket.cpu().numpy()], before[0], before[1], before[2], before[3],
                              p.hyper.replace(step=t), 1024.0)
        for got, w in zip(after, (want.master, want.m, want.v, want.p16)):
            bits = np.uint16 if w.dtype == np.float16 else np.uint32
            assert np.array_equal(got.cpu().numpy().view(bits), w.view(bits))


def test_a_gradient_beyond_fp16_skips_the_step_and_halves_the_scale():
    """A scale that pushes the gradient past fp16's range: dlogits turn inf, their
    8-bit blocks NaN, the bucket non-finite, and the step leaves the state."""
    dev = device()
    p = Program(dev, 2.0 ** 24)
    # one entry has nearly all of the mass: the gradient there is about
    # -S w tau p = -2^24 / 203 * 2 * 0.97 = -1.6e5 (where p spreads over the 16
    # entries, at most 0.39 of it, the largest would stay below 65504)
    p.teacher[:, 0] += 14.0
    before = [x.clone() for x in p.state]
    p.step()
    torch.cuda.synchronize()
    ctl = zs.control_read(p.ctl)
    assert torch.isinf(p.dlogits).any() and not torch.isfinite(p.bucket).all()
    assert ctl.overflow == 1 and ctl.skip == 1 and ctl.step == 1 and ctl.scale == 2.0 ** 23
    assert all(torch.equal(a, b) for a, b in zip(before, p.state))
    # the next loss uses the halved scale, read on the device
    loss, finite = p.loss.clone(), torch.isfinite(p.dlogits)
    small = p.dlogits.float().abs() < 1000
    half = p.dlogits.clone()
    p.gradients()
    torch.cuda.synchronize()
    assert torch.equal(loss, p.loss)
    pick = finite & small & (half.float().abs() > 1)    # halving is exact there
    assert torch.equal(p.dlogits[pick].float(), half[pick].float() / 2)


def test_quantize_params_follows_the_committed_copy():
    """Single pass: the copy the step has made current is quantized, and after
    a skipped step the one that stayed."""
    dev = device()
    p = Program(dev, 1024.0)
    copies = (tuple(p.state), tuple(torch.empty_like(t) for t in p.state))
    table = [(0, VOCAB, WIDTH, p.q["w"], p.q["wt"]),
             (VOCAB * WIDTH, 1, WIDTH, tuple(t[:1] for t in p.q["y"]), None)]
    p.gradients()
    for k, clean in enumerate((True, False, True)):
        if not clean:
            p.bucket[7] = float("inf")
        p.stepper.single_pass([p.bucket], copies)
        p.stepper.quantize_params(copies, table)
        torch.cuda.synchronize()
        ctl = zs.control_read(p.ctl)
        assert ctl.skip == (not clean)
        p16 = copies[ctl.cur][3]
        w = p16[:VOCAB * WIDTH].view(VOCAB, WIDTH)
        _check_q8(w, *p.q["w"], E4, "w")
        _check_q8(w.t(), *p.q["wt"], E4, "w transposed")
        _check_q8(p16[VOCAB * WIDTH:N_PARAMS].view(1, WIDTH), *table[1][3], E4, "norm weight")
        p.bucket[7] = 0.0
    with pytest.raises(ValueError):
        p.stepper.quantize_params(copies, [(0, VOCAB * WIDTH, WIDTH, p.q["w"], None)])


def test_a_captured_step_replays_like_the_eager_one():
    dev = device()
    eager, graphed = Program(dev, 1024.0), Program(dev, 1024.0)
    want = []
    for _ in range(4):
        eager.step()
        want.append(eager.outputs())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.step()
    for k in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(graphed.outputs(), want[k])), k
        eager.gradients()                       # the program's own work in between
        torch.cuda.synchronize()
    assert zs.control_read(graphed.ctl).step == 5
