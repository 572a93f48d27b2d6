"""zero_model.h's operators together with the training operators and the shard step, as
one rank's program runs them: a model of one gated feed-forward layer between an
embedding and a head that share their table, from tokens to log probabilities and back
to every parameter's slot in one gradient bucket.  Each stage is checked against its
64-bit definition on what the stage before it left, the step against the oracle."""
import numpy as np
import pytest
import torch

import model_ref as ref
import oracle.zero_step as ozs
import sharded_mixed_precision_step_amd as zs
import train_ref
import workloads as wl
from gpu_util import device
from test_gpu_q8 import _check_q8, _gemm_tol

pytestmark = pytest.mark.gpu

E4, F16 = torch.float8_e4m3fn, torch.float16
U = ref.U
EPS = 1e-5
TOKENS, WIDTH, INNER, VOCAB = 203, 256, 384, 500
SHAPES = dict(table=(VOCAB, WIDTH), gate_up=(2 * INNER, WIDTH), down=(WIDTH, INNER),
              w1=(WIDTH,), b1=(WIDTH,), w2=(WIDTH,), b2=(WIDTH,))


class Program:
    def __init__(self, dev, scale):
        g = torch.Generator(device=dev)
        g.manual_seed(5)
        rnd = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
        at, self.slots = 0, {}
        for name, shape in SHAPES.items():
            n = int(np.prod(shape))
            self.slots[name] = (at, n, shape)
            at += -(-n // 256) * 256
        master = torch.zeros(at, device=dev)
        for name, (o, n, shape) in self.slots.items():
            v = rnd(n) * (0.1 if len(shape) > 1 else 0.05)
            master[o:o + n] = 1 + v if name[0] == "w" else v
        self.bucket = torch.zeros(at, dtype=F16, device=dev)
        self.state = [master, torch.zeros(at, device=dev), torch.zeros(at, device=dev),
                      master.half()]
        self.grads = {k: self.bucket[o:o + n].view(shape)
                      for k, (o, n, shape) in self.slots.items()}
        ids = torch.randint(0, VOCAB, (TOKENS + 1,), generator=g, device=dev)
        ids[40:90] = 7                                  # a frequent token
        self.ids, self.next = ids[:-1].clone(), ids[1:].clone()
        self.ids[5], self.next[9:12] = -1, -1           # padding; tokens left out
        n = int((self.next >= 0).sum())
        self.dlogp = torch.full((TOKENS,), -1.0 / n, device=dev)
        self.dent = torch.full((TOKENS,), 0.01 / n, device=dev)
        self.ctl = zs.control_new(zs.LossScaler.create(scale=scale), 1, dev)
        self.hyper = wl.AdamWHyper()
        self.stepper = zs.DeviceStepper(self.ctl, zs.adamw_params(self.hyper))
        self.q = {k: zs.q8_empty(r, c, E4, dev) for k, (r, c) in dict(
            table=(VOCAB, WIDTH), table_t=(WIDTH, VOCAB), gate_up=(2 * INNER, WIDTH),
            gate_up_t=(WIDTH, 2 * INNER), down=(WIDTH, INNER), down_t=(INNER, WIDTH),
            y1=(TOKENS, WIDTH), y1_t=(WIDTH, TOKENS), gate=(TOKENS, INNER), up=(TOKENS, INNER),
            y2=(TOKENS, INNER), y2_t=(INNER, TOKENS), y3=(TOKENS, WIDTH), y3_t=(WIDTH, TOKENS),
            dl=(TOKENS, VOCAB), dl_t=(VOCAB, TOKENS), do=(TOKENS, WIDTH), do_t=(WIDTH, TOKENS),
            dgu=(TOKENS, 2 * INNER), dgu_t=(2 * INNER, TOKENS)).items()}
        half = lambda *s: torch.empty(*s, dtype=F16, device=dev)  # noqa: E731
        row = lambda: torch.empty(TOKENS, device=dev)             # noqa: E731
        self.x0, self.y1, self.o, self.h2, self.y3 = (half(TOKENS, WIDTH) for _ in range(5))
        self.gu, self.y2, self.logits = half(TOKENS, 2 * INNER), half(TOKENS, INNER), \
            half(TOKENS, VOCAB)
        self.m1, self.r1, self.m2, self.r2, self.logp, self.ent, self.lse = (row() for _ in range(7))
        self.dlogits, self.dgu = half(TOKENS, VOCAB), half(TOKENS, 2 * INNER)
        self.dy3, self.dh2, self.dy1, self.dx0 = (half(TOKENS, WIDTH) for _ in range(4))
        self.dy2, self.y2_again = half(TOKENS, INNER), half(TOKENS, INNER)
        self.table_head = half(VOCAB, WIDTH)            # the head's share, for the check
        self.work = torch.empty(zs.zero_layernorm_backward_workspace(TOKENS, WIDTH),
                                dtype=torch.uint8, device=dev)
        self.sort = torch.empty(zs.zero_embed_backward_workspace(TOKENS, VOCAB, WIDTH),
                                dtype=torch.uint8, device=dev)

    def params(self):
        return {k: self.state[3][o:o + n].view(shape) for k, (o, n, shape) in self.slots.items()}

    def forward(self):
        p, q = self.params(), self.q
        for k in ("table", "gate_up", "down"):
            zs.zero_q8_quantize(p[k], *q[k], *q[k + "_t"])
        zs.zero_embed(p["table"], self.ids, self.x0, scale=16.0)
        zs.zero_layernorm(self.x0, p["w1"], p["b1"], EPS, y=self.y1, q=q["y1"][0], s=q["y1"][1],
                          mean=self.m1, rstd=self.r1)
        zs.zero_q8_gemm(*q["y1"], *q["gate_up"], self.gu)
        zs.zero_act(self.gu[:, :INNER], "silu", up=self.gu[:, INNER:], y=self.y2, q=q["y2"][0],
                    s=q["y2"][1], gate_q=q["gate"][0], gate_s=q["gate"][1], up_q=q["up"][0],
                    up_s=q["up"][1])
        zs.zero_q8_gemm(*q["y2"], *q["down"], self.o)
        zs.zero_layernorm(self.o, p["w2"], p["b2"], EPS, residual=self.x0, h=self.h2, y=self.y3,
                          q=q["y3"][0], s=q["y3"][1], mean=self.m2, rstd=self.r2)
        zs.zero_q8_gemm(*q["y3"], *q["table"], self.logits)
        zs.zero_logprob(self.logits, self.next, self.logp, entropy=self.ent, lse=self.lse)

    def backward(self):
        p, q, g = self.params(), self.q, self.grads
        self.stepper.logprob_backward(self.logits, self.next, self.lse, self.dlogp, self.dlogits,
                                      entropy=self.ent, dentropy=self.dent)
        zs.zero_q8_quantize(self.dlogits, *q["dl"], *q["dl_t"])
        zs.zero_q8_gemm(*q["dl"], *q["table_t"], self.dy3)
        zs.zero_q8_quantize(self.y3, qt=q["y3_t"][0], st=q["y3_t"][1])
        zs.zero_q8_gemm(*q["dl_t"], *q["y3_t"], g["table"])
        self.table_head.copy_(g["table"])
        zs.zero_layernorm_backward(self.dy3, self.h2, p["w2"], self.m2, self.r2, self.dh2, g["w2"],
                                   g["b2"], self.work)
        zs.zero_q8_quantize(self.dh2, *q["do"], *q["do_t"])
        zs.zero_q8_gemm(*q["do"], *q["down_t"], self.dy2)
        zs.zero_act_backward(self.dy2, *q["gate"], self.dgu[:, :INNER], "silu", up_q=q["up"][0],
                             up_s=q["up"][1], dup=self.dgu[:, INNER:], y=self.y2_again)
        zs.zero_q8_quantize(self.y2_again, qt=q["y2_t"][0], st=q["y2_t"][1])
        zs.zero_q8_gemm(*q["do_t"], *q["y2_t"], g["down"])
        zs.zero_q8_quantize(self.dgu, *q["dgu"], *q["dgu_t"])
        zs.zero_q8_gemm(*q["dgu"], *q["gate_up_t"], self.dy1)
        zs.zero_q8_quantize(self.y1, qt=q["y1_t"][0], st=q["y1_t"][1])
        zs.zero_q8_gemm(*q["dgu_t"], *q["y1_t"], g["gate_up"])
        zs.zero_layernorm_backward(self.dy1, self.x0, p["w1"], self.m1, self.r1, self.dx0, g["w1"],
                                   g["b1"], self.work, dres=self.dh2)
        # the embedding's share is added to the head's in their common slot
        zs.zero_embed_backward(self.dx0, self.ids, g["table"], self.sort, scale=16.0,
                               accumulate=True)

    def step(self):
        self.forward()
        self.backward()
        self.stepper.two_pass([self.bucket], *self.state)

    def outputs(self):
        return [t.clone() for t in (self.logits, self.logp, self.dlogits, self.dx0, self.bucket,
                                    *self.state)]


def _check(p, S):
    par, q, g = p.params(), p.q, p.grads
    val = {k: train_ref.from_blocks(*t) for k, t in q.items()}
    half = lambda w: ref.half_step(F16, w)  # noqa: E731

    def product(got, a, b, name):
        want = val[a] @ val[b].t()
        ref.assert_close(got, want, _gemm_tol(val[a], val[b], q[a][1], q[b][1], got.dtype, want),
                         name)

    def norm(x, res, w, b, y, kq, mean, rstd, name):
        h, wm, wr, wy = ref.layernorm(x, res, w, b, EPS)
        tm, tr, ty = ref.layernorm_bounds(x, res, w, b, EPS)
        ref.assert_close(mean, wm, tm, name + " mean")
        ref.assert_close(rstd, wr, tr, name + " rstd")
        ref.assert_close(y, wy, half(wy) + ty, name)
        ref.check_q8(*q[kq], wy, ty, E4, name + " q8")
        return h

    def norm_backward(dy, h, w, mean, rstd, dres, dx, dw, db, name):
        wx, ww, wb, tx, tw, tb = ref.layernorm_backward(dy, h, w, mean, rstd, dres)
        ref.assert_close(dx, wx, half(wx) + tx, name + " dx")
        ref.assert_close(dw, ww, half(ww) + tw, name + " dw")
        ref.assert_close(db, wb, half(wb) + tb, name + " db")

    want = ref.embed(par["table"], p.ids, 16.0)
    ref.assert_close(p.x0, want, half(want) + U * want.abs(), "x0")
    norm(p.x0, None, par["w1"], par["b1"], p.y1, "y1", p.m1, p.r1, "norm 1")
    product(p.gu, "y1", "gate_up", "gate and up")
    gate, up = p.gu[:, :INNER], p.gu[:, INNER:]
    want, tol = ref.act("silu", gate, up)
    ref.assert_close(p.y2, want, half(want) + tol, "y2")
    ref.check_q8(*q["y2"], want, tol, E4, "y2 q8")
    _check_q8(gate, *q["gate"], E4, "gate")
    _check_q8(up, *q["up"], E4, "up")
    product(p.o, "y2", "down", "o")
    h = norm(p.o, p.x0, par["w2"], par["b2"], p.y3, "y3", p.m2, p.r2, "norm 2")
    ref.assert_close(p.h2, h, half(h) + U * h.abs(), "h2")
    product(p.logits, "y3", "table", "logits")
    out, tol = ref.logprob(p.logits, p.next, 1.0, 0)
    for got, w, t, name in zip((p.logp, p.ent, p.lse), out, tol, ("logp", "entropy", "lse")):
        ref.assert_close(got, w, t + ref.half_step(torch.float32, w), name)
    want, tol = ref.logprob_backward(p.logits, p.next, 1.0, p.lse, p.dlogp, p.ent, p.dent, S)
    ref.assert_close(p.dlogits, want, half(want) + tol, "dlogits")
    product(p.dy3, "dl", "table_t", "dy3")
    product(p.table_head, "dl_t", "y3_t", "the head's gradient")
    norm_backward(p.dy3, p.h2, par["w2"], p.m2, p.r2, None, p.dh2, g["w2"], g["b2"], "norm 2")
    product(p.dy2, "do", "down_t", "dy2")
    want, tol = ref.act_backward("silu", p.dy2, val["gate"][:, :INNER], val["up"][:, :INNER])
    for got, w, t, name in zip((p.dgu[:, :INNER], p.dgu[:, INNER:], p.y2_again), want, tol,
                               ("dgate", "dup", "y2 again")):
        ref.assert_close(got, w, half(w) + t, name)
    product(g["down"], "do_t", "y2_t", "ddown")
    product(p.dy1, "dgu", "gate_up_t", "dy1")
    product(g["gate_up"], "dgu_t", "y1_t", "dgate_up")
    norm_backward(p.dy1, p.x0, par["w1"], p.m1, p.r1, p.dh2, p.dx0, g["w1"], g["b1"], "norm 1")
    want, tol = ref.embed_backward(p.dx0, p.ids, VOCAB, 16.0)
    both = want + p.table_head.double()
    has = torch.zeros(VOCAB, dtype=torch.bool, device=p.ids.device)
    has[p.ids[p.ids >= 0]] = True
    assert torch.equal(g["table"][~has], p.table_head[~has])
    ref.assert_close(g["table"][has], both[has],
                     (half(both) + tol + 2 * U * (want.abs() + both.abs()))[has], "dtable")


def test_two_steps_match_their_definitions_and_the_oracle():
    p = Program(device(), 1024.0)
    for t in (1, 2):
        before = [x.cpu().numpy() for x in p.state]
        p.step()
        torch.cuda.synchronize()
        ctl = zs.control_read(p.ctl)
        assert ctl.overflow == 0 and ctl.step == t + 1 and ctl.scale == 1024.0
        after = [x.clone() for x in p.state]
        # the gradients came from the parameters before the step
        p.state[3].copy_(torch.from_numpy(before[3]))
        _check(p, 1024.0)
        p.state[3].copy_(after[3])
        want = ozs.shard_step([p.bucket.cpu().numpy()], before[0], before[1], before[2], before[3],
                              p.hyper.replace(step=t), 1024.0)
        for got, w in zip(after, (want.master, want.m, want.v, want.p16)):
            bits = np.uint16 if w.dtype == np.float16 else np.uint32
            assert np.array_equal(got.cpu().numpy().view(bits), w.view(bits))


def test_a_token_without_a_row_skips_the_step():
    """An id beyond the table makes its row NaN; through every product and sum the
    gradients turn NaN, and the step leaves the state and halves the scale."""
    p = Program(device(), 1024.0)
    p.ids[17] = VOCAB
    before = [x.clone() for x in p.state]
    p.step()
    torch.cuda.synchronize()
    ctl = zs.control_read(p.ctl)
    assert torch.isnan(p.x0[17]).all() and torch.isnan(p.logp[17])
    assert not torch.isfinite(p.bucket).all()
    assert ctl.overflow == 1 and ctl.skip == 1 and ctl.step == 1 and ctl.scale == 512.0
    assert all(torch.equal(a, b) for a, b in zip(before, p.state))


def test_the_embedding_follows_the_committed_copy():
    """Single pass: tokens are looked up in the copy the step has made current, and
    after a skipped step in the one that stayed."""
    dev = device()
    p = Program(dev, 1024.0)
    copies = (tuple(p.state), tuple(torch.empty_like(t) for t in p.state))
    p.forward()
    p.backward()
    o, n, shape = p.slots["table"]
    y, want = torch.empty_like(p.x0), torch.empty_like(p.x0)
    for clean in (True, False, True):
        if not clean:
            p.bucket[7] = float("inf")
        p.stepper.single_pass([p.bucket], copies)
        p.stepper.embed(copies, o, *shape, p.ids, y)
        torch.cuda.synchronize()
        ctl = zs.control_read(p.ctl)
        assert ctl.skip == (not clean)
        zs.zero_embed(copies[ctl.cur][3][o:o + n].view(shape), p.ids, want)
        assert torch.equal(y, want)
        p.bucket[7] = 0.0
    with pytest.raises(ValueError):
        p.stepper.embed(copies, o, p.bucket.numel(), WIDTH, p.ids, y)


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
        eager.forward()                             # the program's own work in between
        torch.cuda.synchronize()
    assert zs.control_read(graphed.ctl).step == 5


def test_two_programs_on_two_streams():
    """Both at once, each with its own workspaces, give what each gives alone."""
    dev = device()
    alone, one, two = Program(dev, 1024.0), Program(dev, 1024.0), Program(dev, 1024.0)
    for _ in range(3):
        alone.step()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, p in zip(streams, (one, two)):
            with torch.cuda.stream(s):
                p.step()
    torch.cuda.synchronize()
    want = alone.outputs()
    for p in (one, two):
        assert all(torch.equal(a, b) for a, b in zip(p.outputs(), want))
