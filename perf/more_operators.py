"""The operators of a language model's two ends and of its feed-forward layers,
as measured cases.

Four groups of calls that a mixed-precision training step makes around its
matrix products: the embedding of tokens and its gradient by sorted tokens, the
residual add with layer norm and its backward pass, the (gated) activation that
keeps its inputs as 8-bit checkpoints and its backward pass from them, and the
log probabilities of given tokens with entropy and top alternatives, and their
loss-scaled gradient.

``run`` computes them either in plain torch operations, in fp32 and rounded
once at the end (``own`` false), or with the library's calls (``own`` true).

The 8-bit layout: a matrix [rows, cols] is held as [rows, P] 8-bit values, P =
cols rounded up to 128, zeros behind cols, and [rows, Q] scale bytes (biased
exponents of a power of two), Q = P / 128 rounded up to 4, ones behind the
last block.  A block's scale is the smallest power of two that brings its
largest magnitude to the 8-bit type's largest value or below.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FP8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
BLOCK = 128
EPS = 1e-5


def listed():
    return [
        # a few tokens looked up: the call's own latency
        dict(name="embed few tokens", op="embed", tokens=16, vocab=131072, cols=4096, t="f16",
             y="f16", scale=1.0),
        # gradient of the whole table over a micro-batch: most rows stay zero
        dict(name="embed gradient", op="embed_backward", tokens=8192, vocab=131072, cols=4096,
             dy="f16", dt="f16", scale=1.0),
        # an odd token count, width and vocabulary, scaled embeddings
        dict(name="embed gradient ragged", op="embed_backward", tokens=4099, vocab=32001,
             cols=1000, dy="bf16", dt="f32", scale=31.622776601683793),
        # a few tokens through a layer's norm: the call's own latency
        dict(name="layernorm few rows", op="layernorm", rows=16, cols=4096, x="f16", res="f16",
             fp8="e4m3"),
        # a micro-batch through a layer's norm, fp32 residual stream, the 8-bit
        # operand of the next product written at once
        dict(name="layernorm micro-batch", op="layernorm", rows=8192, cols=4096, x="f16",
             res="f32", fp8="e4m3"),
        # the backward pass of an odd number of narrow odd rows
        dict(name="layernorm backward ragged", op="layernorm_backward", rows=16387, cols=1001,
             dy="bf16", h="bf16", dres="bf16"),
        # a feed-forward layer's gated activation over a micro-batch: the 8-bit
        # operand of the next product, gate and up kept in 8 bits
        dict(name="act micro-batch", op="act", rows=8192, cols=14336, kind="silu", up=True,
             x="f16", y="none", fp8="e4m3"),
        # its backward pass from the checkpoints, the activation computed again
        dict(name="act backward", op="act_backward", rows=8192, cols=14336, kind="silu", up=True,
             dy="f16", dx="f16", fp8="e4m3", again=True),
        # an activation without a gate, odd number of rows and width
        dict(name="act backward ragged", op="act_backward", rows=1003, cols=5001, kind="gelu",
             up=False, dy="bf16", dx="bf16", fp8="e5m2", again=False),
        # a few rows over an odd vocabulary: log probabilities while answering
        dict(name="logprob few rows", op="logprob", rows=37, vocab=32001, top=20, x="bf16",
             tau=1.0),
        # the teacher's side of a micro-batch of distillation: log probabilities,
        # entropy and the top entries that the distillation loss takes
        dict(name="logprob micro-batch", op="logprob", rows=4096, vocab=131072, top=64, x="f16",
             tau=1.0),
        # gradient of log probabilities with an entropy term, odd vocabulary
        dict(name="logprob gradient", op="logprob_backward", rows=2048, vocab=50001, x="f16",
             tau=1.0, entropy=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_backward", "layernorm", "layernorm_backward", "act",
                     "act_backward", "logprob", "logprob_backward"])
    half = rng.choice(["f16", "bf16"])
    if op in ("embed", "embed_backward"):
        c = dict(op=op, tokens=_log(rng, 1, 32768 if op == "embed" else 16384),
                 vocab=_log(rng, 256, 65536), cols=_log(rng, 64, 4096),
                 scale=rng.choice([1.0, 32.0]))
        if op == "embed":
            return dict(c, t=rng.choice(["f16", "bf16", "f32"]), y=half)
        return dict(c, dy=half, dt=rng.choice([half, "f32"]))
    if op == "layernorm":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 64, 8192),
                    x=rng.choice(["f16", "bf16", "f32"]),
                    res=rng.choice(["f16", "bf16", "f32", "none"]),
                    fp8=rng.choice(["e4m3", "e5m2", "none"]))
    if op == "layernorm_backward":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 64, 8192), dy=half,
                    h=rng.choice([half, "f32"]), dres=rng.choice([half, "none"]))
    if op == "act":
        fp8 = rng.choice(["e4m3", "e5m2"])
        return dict(op=op, rows=_log(rng, 1, 4096), cols=_log(rng, 64, 14336),
                    kind=rng.choice(["silu", "gelu", "gelu_tanh"]), up=rng.random() < 0.5,
                    x=rng.choice(["f16", "bf16", "f32"]), y=rng.choice(["none", half]), fp8=fp8)
    if op == "act_backward":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 64, 14336),
                    kind=rng.choice(["silu", "gelu", "gelu_tanh"]), up=rng.random() < 0.5,
                    dy=half, dx=half, fp8=rng.choice(["e4m3", "e5m2"]),
                    again=rng.random() < 0.5)
    c = dict(op=op, rows=_log(rng, 1, 1024), vocab=_log(rng, 1000, 131072),
             x=rng.choice(["f16", "bf16", "f32"]), tau=rng.choice([1.0, 0.7]))
    if op == "logprob":
        return dict(c, top=rng.choice([0, 1, _log(rng, 1, 128)]))
    return dict(c, entropy=rng.random() < 0.5)


def _pad(n, to):
    return -(-n // to) * to


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _to_blocks(x, fp8):
    """x [rows, cols] (any float type) in the 8-bit layout, in plain torch."""
    rows, cols = x.shape
    p = _pad(max(cols, 1), BLOCK)
    nb = p // BLOCK
    xb = torch.zeros(rows, p, dtype=torch.float32, device=x.device)
    xb[:, :cols] = x
    xb = xb.view(rows, nb, BLOCK)
    amax = xb.abs().amax(-1)
    m, e = torch.frexp(amax)
    top, etop = math.frexp(FP8_MAX[fp8])
    e = torch.where(amax == 0, 0, (e - etop + (m > top)).clamp(-127, 127))
    bad = ~torch.isfinite(amax)
    e = torch.where(bad, 0, e)
    # 2^-e from its bits: a power function need not be exact
    q = xb * ((127 - e.int()) << 23).view(torch.float32)[..., None]
    q = torch.where(bad[..., None], math.nan, q).to(FP8[fp8])
    s = torch.full((rows, _pad(nb, 4)), 127, dtype=torch.uint8, device=x.device)
    s[:, :nb] = torch.where(bad, 255, e + 127).to(torch.uint8)
    return q.view(rows, p), s.view(torch.float8_e8m0fnu)


def _from_blocks(q, s, cols):
    nb = q.shape[1] // BLOCK
    v = q.to(torch.float32).view(-1, nb, BLOCK) * s[:, :nb].to(torch.float32)[..., None]
    return v.view(q.shape)[:, :cols]


def _plain_embed(c, s):
    ids = s["ids"].long()
    y = s["table"][ids.clamp_min(0)].float() * c["scale"]
    return {"y": torch.where(ids[:, None] < 0, 0.0, y).to(s["y"].dtype)}


def _plain_embed_backward(c, s):
    ids = s["ids"].long()
    dy = torch.where(ids[:, None] < 0, 0.0, s["dy"].float())
    d = torch.zeros(s["dtable"].shape, device=dy.device).index_add_(0, ids.clamp_min(0), dy)
    return {"dtable": d.mul_(c["scale"]).to(s["dtable"].dtype)}


def _plain_layernorm(c, s):
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    mean = h.mean(-1)
    xhat = h - mean[:, None]
    rstd = torch.rsqrt(xhat.square().mean(-1) + EPS)
    y = xhat * rstd[:, None] * s["w"].float() + s["b"].float()
    out = {"mean": mean, "rstd": rstd}
    if s["res"] is not None:
        out["h"] = h.to(s["h"].dtype)
    if c["fp8"] == "none":
        out["y"] = y.to(s["y"].dtype)
    else:
        out["q"], out["s"] = _to_blocks(y, c["fp8"])
    return out


def _plain_layernorm_backward(c, s):
    xhat = (s["h"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["w"].float()
    dx = s["rstd"][:, None] * (g - g.mean(-1, keepdim=True)
                               - xhat * (g * xhat).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["dx"].dtype), "dw": (dy * xhat).sum(0).to(s["dw"].dtype),
            "db": dy.sum(0).to(s["db"].dtype)}


def _activation(kind, g):
    """f(g) and f'(g)"""
    if kind == "silu":
        sig = 1 / (1 + torch.exp(-g))
        return g * sig, sig * (1 + g * (1 - sig))
    if kind == "gelu":
        phi = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * phi, phi + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    k, c3 = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(k * (g + c3 * g * g * g))
    return (0.5 * g * (1 + t),
            0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * c3 * g * g))


def _plain_act(c, s):
    y = _activation(c["kind"], s["gate"].float())[0]
    out = {}
    out["gq"], out["gs"] = _to_blocks(s["gate"], c["fp8"])
    if c["up"]:
        y = y * s["up"].float()
        out["uq"], out["us"] = _to_blocks(s["up"], c["fp8"])
    if c["y"] == "none":
        out["q"], out["s"] = _to_blocks(y, c["fp8"])
    else:
        out["y"] = y.to(s["y"].dtype)
    return out


def _plain_act_backward(c, s):
    cols = c["cols"]
    f, slope = _activation(c["kind"], _from_blocks(s["gq"], s["gs"], cols))
    dy = s["dy"].float()
    out = {}
    if c["up"]:
        up = _from_blocks(s["uq"], s["us"], cols)
        out["dgate"] = (dy * up * slope).to(s["dgate"].dtype)
        out["dup"] = (dy * f).to(s["dup"].dtype)
        f = f * up
    else:
        out["dgate"] = (dy * slope).to(s["dgate"].dtype)
    if c["again"]:
        out["y"] = f.to(s["y"].dtype)
    return out


def _ordered(x):
    """Whole numbers in the order of x's values (both zeros alike)."""
    b = (x.float() + 0.0).view(torch.int32).long()
    return torch.where(b < 0, -(b & 0x7fffffff), b)


def _plain_logprob(c, s):
    x, ids = s["logits"], s["ids"].long()
    on = ids >= 0
    z = x.float() / c["tau"]
    lse = torch.logsumexp(z, -1)
    logq = z - lse[:, None]
    logp = logq.gather(1, ids.clamp_min(0)[:, None])[:, 0]
    q = torch.exp(logq)
    entropy = -torch.where(q > 0, q * logq, 0.0).sum(-1)
    del z, q, logq
    out = {"logp": torch.where(on, logp, 0.0), "lse": torch.where(on, lse, 0.0),
           "entropy": torch.where(on, entropy, 0.0)}
    if c["top"]:
        # value and place in one number: ties go to the lowest index
        v = x.shape[1]
        key = _ordered(x) * v + (v - 1 - torch.arange(v, device=x.device))
        key = torch.topk(key, c["top"], dim=-1, sorted=True).values
        at = v - 1 - key % v
        value = x.gather(1, at)
        live = on[:, None] & (value > -math.inf)
        out["index"] = torch.where(live, at, -1).to(s["index"].dtype)
        out["value"] = torch.where(live, value, -math.inf)
    return out


def _plain_logprob_backward(c, s):
    ids = s["ids"].long()
    on = (ids >= 0)[:, None]
    logq = s["logits"].float() / c["tau"] - s["lse"][:, None]
    q = torch.exp(logq)
    g = -s["dlogp"][:, None] * q
    if c["entropy"]:
        g -= torch.where(q > 0, s["dentropy"][:, None] * q * (logq + s["entropy"][:, None]), 0.0)
    g.scatter_add_(1, ids.clamp_min(0)[:, None], s["dlogp"][:, None])
    return {"grad": torch.where(on, g * (s["scale"] / c["tau"]), 0.0).to(s["grad"].dtype)}


PLAIN = {"embed": _plain_embed, "embed_backward": _plain_embed_backward,
         "layernorm": _plain_layernorm, "layernorm_backward": _plain_layernorm_backward,
         "act": _plain_act, "act_backward": _plain_act_backward, "logprob": _plain_logprob,
         "logprob_backward": _plain_logprob_backward}


# --------------------------------------------------------------------------
# the program's side of a pass
# --------------------------------------------------------------------------

def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=dev)

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device=dev)

    def empty8(rows, cols, fp8):
        p = _pad(max(cols, 1), BLOCK)
        return (empty(rows, p, dtype=torch.uint8).view(FP8[fp8]),
                empty(rows, _pad(p // BLOCK, 4), dtype=torch.uint8).view(torch.float8_e8m0fnu))

    s = {"case": dict(c)}
    if c["op"] in ("embed", "embed_backward"):
        tokens, vocab, cols = c["tokens"], c["vocab"], c["cols"]
        # token frequencies fall as 1 / rank, ranks spread over the vocabulary;
        # some tokens are padding
        rank = torch.exp(uniform(tokens) * math.log(vocab)).long().clamp(1, vocab) - 1
        step = next(k for k in range(int(0.618 * vocab) | 1, 2 * vocab + 3)
                    if math.gcd(k, vocab) == 1)
        ids = torch.where(uniform(tokens) < 0.02, -1, rank * step % vocab)
        s["ids"] = ids.to(torch.int64)
        if c["op"] == "embed":
            s["table"] = (0.02 * normal(vocab, cols)).to(DTYPES[c["t"]])
            s["y"] = empty(tokens, cols, dtype=DTYPES[c["y"]])
        else:
            # gradients of about 1e-6, loss-scaled by 65536
            s["dy"] = (0.07 * normal(tokens, cols)).to(DTYPES[c["dy"]])
            s["dtable"] = empty(vocab, cols, dtype=DTYPES[c["dt"]])
            s["work"] = empty(tokens * cols + 64 * tokens + 8 * cols + (4 << 20),
                              dtype=torch.uint8)
    elif c["op"] == "layernorm":
        rows, cols = c["rows"], c["cols"]
        # a residual stream with some channels much larger than the rest
        gain, shift = torch.exp(0.5 * normal(cols)), 0.2 * normal(cols)
        s["x"] = (normal(rows, cols) * gain + shift).to(DTYPES[c["x"]])
        s["res"] = None if c["res"] == "none" else (2 * normal(rows, cols) * gain + shift
                                                    ).to(DTYPES[c["res"]])
        s["h"] = None if s["res"] is None else torch.empty_like(s["res"])
        s["w"] = (1 + 0.1 * normal(cols)).to(torch.float16)
        s["b"] = (0.1 * normal(cols)).to(torch.float16)
        s["mean"], s["rstd"] = empty(rows), empty(rows)
        if c["fp8"] == "none":
            s["y"] = torch.empty_like(s["x"])
        else:
            s["q"], s["s"] = empty8(rows, cols, c["fp8"])
    elif c["op"] == "layernorm_backward":
        rows, cols = c["rows"], c["cols"]
        s["h"] = (2 * normal(rows, cols) * torch.exp(0.5 * normal(cols)) + 0.2 * normal(cols)
                  ).to(DTYPES[c["h"]])
        h = s["h"].float()
        s["mean"] = h.mean(-1)
        s["rstd"] = torch.rsqrt((h - s["mean"][:, None]).square().mean(-1) + EPS)
        s["w"] = (1 + 0.1 * normal(cols)).to(torch.float16)
        s["dy"] = (0.07 * normal(rows, cols)).to(DTYPES[c["dy"]])
        s["dres"] = None if c["dres"] == "none" else (0.1 * normal(rows, cols)
                                                      ).to(DTYPES[c["dres"]])
        s["dx"] = torch.empty_like(s["dy"])
        s["dw"], s["db"] = torch.empty_like(s["w"]), torch.empty_like(s["w"])
        s["work"] = empty(8 * 1024 * cols, dtype=torch.uint8)
    elif c["op"] == "act":
        rows, cols = c["rows"], c["cols"]
        s["gate"] = (normal(rows, cols) * torch.exp(0.5 * normal(cols))).to(DTYPES[c["x"]])
        s["up"] = normal(rows, cols).to(DTYPES[c["x"]]) if c["up"] else None
        s["gq"], s["gs"] = empty8(rows, cols, c["fp8"])
        s["uq"], s["us"] = empty8(rows, cols, c["fp8"]) if c["up"] else (None, None)
        if c["y"] == "none":
            s["q"], s["s"] = empty8(rows, cols, c["fp8"])
        else:
            s["y"] = empty(rows, cols, dtype=DTYPES[c["y"]])
    elif c["op"] == "act_backward":
        rows, cols = c["rows"], c["cols"]
        s["gq"], s["gs"] = _to_blocks(normal(rows, cols) * torch.exp(0.5 * normal(cols)),
                                      c["fp8"])
        s["uq"], s["us"] = _to_blocks(normal(rows, cols), c["fp8"]) if c["up"] else (None, None)
        s["dy"] = (0.07 * normal(rows, cols)).to(DTYPES[c["dy"]])
        s["dgate"] = empty(rows, cols, dtype=DTYPES[c["dx"]])
        s["dup"] = torch.empty_like(s["dgate"]) if c["up"] else None
        s["y"] = torch.empty_like(s["dgate"]) if c["again"] else None
    else:
        rows, vocab = c["rows"], c["vocab"]
        logits = 2.5 * normal(rows, vocab)
        # each row has some likely tokens, the given one often among them
        likely = (uniform(rows, 32) * vocab * 0.99).long()
        logits.scatter_(1, likely, 1.5 * normal(rows, 32) + 9.0)
        # the places that only fill up the vocabulary cannot be chosen
        logits[:, vocab - vocab // 100:] = -math.inf
        s["logits"] = logits.to(DTYPES[c["x"]])
        pick = (uniform(rows) * 32).long()
        ids = likely.gather(1, pick[:, None])[:, 0]
        # prompt tokens are left out
        ids = torch.where(uniform(rows) < 0.1, -1, ids)
        ids[0] = likely[0, 0]
        s["ids"] = ids
        if c["op"] == "logprob":
            s["logp"], s["lse"], s["entropy"] = empty(rows), empty(rows), empty(rows)
            if c["top"]:
                s["index"] = empty(rows, c["top"], dtype=torch.int32)
                s["value"] = torch.empty(rows, c["top"], dtype=s["logits"].dtype, device=dev)
        else:
            z = s["logits"].double() / c["tau"]
            lse = torch.logsumexp(z, -1)
            z -= lse[:, None]
            entropy = -torch.special.xlogy(z.exp(), z.exp()).sum(-1)
            s["lse"] = torch.where(ids < 0, 0.0, lse).float()
            s["entropy"] = torch.where(ids < 0, 0.0, entropy).float()
            # a policy's step: the advantages' mean over the tokens that count
            s["dlogp"] = normal(rows) / rows
            s["dentropy"] = 0.01 * (0.5 + uniform(rows)) / rows if c["entropy"] else None
            s["scale"] = 65536.0
            s["grad"] = torch.empty_like(s["logits"])
    return s


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return PLAIN[op](c, s)
    import sharded_mixed_precision_step_amd as zs
    if op == "embed":
        zs.zero_embed(s["table"], s["ids"], s["y"], scale=c["scale"])
        return {"y": s["y"]}
    if op == "embed_backward":
        zs.zero_embed_backward(s["dy"], s["ids"], s["dtable"], s["work"], scale=c["scale"])
        return {"dtable": s["dtable"]}
    if op == "layernorm":
        out = {"mean": s["mean"], "rstd": s["rstd"]}
        if s["res"] is not None:
            out["h"] = s["h"]
        if c["fp8"] == "none":
            zs.zero_layernorm(s["x"], s["w"], s["b"], EPS, residual=s["res"], h=s["h"], y=s["y"],
                              mean=s["mean"], rstd=s["rstd"])
            out["y"] = s["y"]
        else:
            zs.zero_layernorm(s["x"], s["w"], s["b"], EPS, residual=s["res"], h=s["h"], q=s["q"],
                              s=s["s"], mean=s["mean"], rstd=s["rstd"])
            out["q"], out["s"] = s["q"], s["s"]
        return out
    if op == "layernorm_backward":
        zs.zero_layernorm_backward(s["dy"], s["h"], s["w"], s["mean"], s["rstd"], s["dx"], s["dw"],
                                   s["db"], s["work"], dres=s["dres"])
        return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}
    if op == "act":
        if c["y"] == "none":
            zs.zero_act(s["gate"], c["kind"], up=s["up"], q=s["q"], s=s["s"], gate_q=s["gq"],
                        gate_s=s["gs"], up_q=s["uq"], up_s=s["us"])
        else:
            zs.zero_act(s["gate"], c["kind"], up=s["up"], y=s["y"], gate_q=s["gq"],
                        gate_s=s["gs"], up_q=s["uq"], up_s=s["us"])
        return {k: s[k] for k in ("gq", "gs", "uq", "us", "q", "s", "y")
                if s.get(k) is not None}
    if op == "act_backward":
        zs.zero_act_backward(s["dy"], s["gq"], s["gs"], s["dgate"], c["kind"], up_q=s["uq"],
                             up_s=s["us"], dup=s["dup"], y=s["y"])
        return {k: s[k] for k in ("dgate", "dup", "y") if s[k] is not None}
    if op == "logprob":
        out = {"logp": s["logp"], "lse": s["lse"], "entropy": s["entropy"]}
        if c["top"]:
            zs.zero_logprob(s["logits"], s["ids"], s["logp"], entropy=s["entropy"], lse=s["lse"],
                            top_index=s["index"], top_logit=s["value"], temperature=c["tau"])
            out["index"], out["value"] = s["index"], s["value"]
        else:
            zs.zero_logprob(s["logits"], s["ids"], s["logp"], entropy=s["entropy"], lse=s["lse"],
                            temperature=c["tau"])
        return out
    if c["entropy"]:
        zs.zero_logprob_backward(s["logits"], s["ids"], s["lse"], s["dlogp"], s["grad"],
                                 entropy=s["entropy"], dentropy=s["dentropy"],
                                 temperature=c["tau"], loss_scale=s["scale"])
    else:
        zs.zero_logprob_backward(s["logits"], s["ids"], s["lse"], s["dlogp"], s["grad"],
                                 temperature=c["tau"], loss_scale=s["scale"])
    return {"grad": s["grad"]}


def _size(name):
    return {"none": 0, "f32": 4, "f16": 2, "bf16": 2}[name]


def work(case):
    c = case
    q8 = 1 + 1 / BLOCK
    if c["op"] == "embed":
        n = c["tokens"] * c["cols"]
        return {"bytes": n * (_size(c["t"]) + _size(c["y"])) + 8 * c["tokens"], "flops": n}
    if c["op"] == "embed_backward":
        n = c["tokens"] * c["cols"]
        return {"bytes": n * _size(c["dy"]) + c["vocab"] * c["cols"] * _size(c["dt"]) +
                8 * c["tokens"], "flops": n}
    if c["op"] == "layernorm":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (_size(c["x"]) + 2 * _size(c["res"]) +
                              (_size(c["x"]) if c["fp8"] == "none" else q8)) +
                4 * c["cols"] + 8 * c["rows"], "flops": 8 * n}
    if c["op"] == "layernorm_backward":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (2 * _size(c["dy"]) + _size(c["h"]) + _size(c["dres"])) +
                6 * c["cols"] + 8 * c["rows"], "flops": 14 * n}
    if c["op"] == "act":
        n, parts = c["rows"] * c["cols"], 1 + c["up"]
        return {"bytes": n * (parts * (_size(c["x"]) + q8) +
                              (q8 if c["y"] == "none" else _size(c["y"]))), "flops": 8 * n}
    if c["op"] == "act_backward":
        n, parts = c["rows"] * c["cols"], 1 + c["up"]
        return {"bytes": n * (parts * (_size(c["dx"]) + q8) + _size(c["dy"]) +
                              c["again"] * _size(c["dx"])), "flops": 14 * n}
    n = c["rows"] * c["vocab"]
    if c["op"] == "logprob":
        return {"bytes": n * _size(c["x"]) + c["rows"] * (20 + c["top"] * (4 + _size(c["x"]))),
                "flops": 6 * n}
    return {"bytes": 2 * n * _size(c["x"]) + c["rows"] * (16 + 8 * c["entropy"]), "flops": 6 * n}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_scale(amax, fp8):
    """The power of two of a block with this largest magnitude: the smallest
    with amax <= max * 2^e, found from the logarithm and put right by one."""
    big = FP8_MAX[fp8]
    e = torch.ceil(torch.log2(amax.clamp_min(2.0 ** -1000) / big))
    e = torch.where(amax <= big * _exact_pow2(e - 1), e - 1, e)
    e = torch.where(amax > big * _exact_pow2(e), e + 1, e)
    return torch.where(amax == 0, torch.zeros_like(e), e.clamp(-127, 127))


def _exact_round(v, fp8):
    """v rounded half to even to the 8-bit type's grid."""
    bits, low = (3, -6) if fp8 == "e4m3" else (2, -14)
    a = v.abs().clamp_min(2.0 ** -60)
    e = torch.floor(torch.log2(a))
    e = torch.where(_exact_pow2(e) > a, e - 1, e)
    step = _exact_pow2(e.clamp_min(low) - bits)
    return torch.round(v / step) * step


def _exact_blocks(x, fp8):
    rows, cols = x.shape
    p = _pad(max(cols, 1), BLOCK)
    x = torch.nn.functional.pad(x, (0, p - cols)).unflatten(1, (p // BLOCK, BLOCK))
    e = _exact_scale(x.abs().amax(-1), fp8)
    q = _exact_round(x * _exact_pow2(-e)[..., None], fp8).flatten(1)
    s = _exact_pow2(e)
    return q, torch.nn.functional.pad(s, (0, _pad(s.shape[1], 4) - s.shape[1]), value=1.0)


def _exact_values(q, s, cols):
    v = q.to(torch.float64).unflatten(1, (-1, BLOCK))
    e = s[:, :v.shape[1]].to(torch.float32).double()
    return (v * e[:, :, None]).flatten(1)[:, :cols]


def _exact_activation(kind, g):
    """f(g) and f'(g), by the normal distribution's function for GELU and as
    g / (1 + exp(-..)) for the other two: (1 + tanh u) / 2 = 1 / (1 + exp(-2u))."""
    if kind == "gelu":
        cdf = 0.5 * torch.special.erfc(-g / 2 ** 0.5)
        return g * cdf, cdf + g * torch.exp(-g * g / 2) * (2 * math.pi) ** -0.5
    if kind == "silu":
        u, du = g, torch.ones_like(g)
    else:
        k = (8 / math.pi) ** 0.5
        u, du = k * (g + 0.044715 * g ** 3), k * (1 + 3 * 0.044715 * g ** 2)
    sig = torch.special.expit(u)
    return g * sig, sig + g * sig * torch.special.expit(-u) * du


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "embed":
        live = (s["ids"] >= 0).double()[:, None]
        return {"y": s["table"].index_select(0, s["ids"].clamp_min(0)).double() * c["scale"] *
                live}
    if c["op"] == "embed_backward":
        order = torch.argsort(s["ids"], stable=True)
        ids = s["ids"][order]
        order, ids = order[ids >= 0], ids[ids >= 0]
        unique, counts = torch.unique_consecutive(ids, return_counts=True)
        sums = torch.segment_reduce(s["dy"][order].double(), "sum", lengths=counts, axis=0)
        out = torch.zeros(c["vocab"], c["cols"], dtype=torch.float64, device=ids.device)
        out[unique] = sums * c["scale"]
        return {"dtable": out}
    if c["op"] == "layernorm":
        h = s["x"].double() if s["res"] is None else s["x"].double() + s["res"].double()
        var, mean = torch.var_mean(h, 1, correction=0)
        rstd = (var + EPS) ** -0.5
        y = torch.addcmul(s["b"].double(), (h - mean[:, None]) * s["w"].double(), rstd[:, None])
        out = {"mean": mean, "rstd": rstd}
        if s["res"] is not None:
            out["h"] = h
        if c["fp8"] == "none":
            out["y"] = y
        else:
            out["q"], out["s"] = _exact_blocks(y, c["fp8"])
        return out
    if c["op"] == "layernorm_backward":
        # y_i = w_i (h_i - m) r + b_i: the derivative of r is
        # -r^3 (h_i - m) / cols, that of m is 1 / cols; m and r come with the state
        r, dy = s["rstd"].double()[:, None], s["dy"].double()
        centred = s["h"].double() - s["mean"].double()[:, None]
        wdy = dy * s["w"].double()
        n = c["cols"]
        dx = r * wdy - r / n * wdy.sum(1, keepdim=True) \
            - r ** 3 / n * centred * (wdy * centred).sum(1, keepdim=True)
        if s["dres"] is not None:
            dx = dx + s["dres"].double()
        return {"dx": dx, "dw": torch.einsum("tc,tc->c", dy, centred * r),
                "db": torch.einsum("tc->c", dy)}
    if c["op"] == "act":
        y = _exact_activation(c["kind"], s["gate"].double())[0]
        out = {}
        out["gq"], out["gs"] = _exact_blocks(s["gate"].double(), c["fp8"])
        if c["up"]:
            y = y * s["up"].double()
            out["uq"], out["us"] = _exact_blocks(s["up"].double(), c["fp8"])
        if c["y"] == "none":
            out["q"], out["s"] = _exact_blocks(y, c["fp8"])
        else:
            out["y"] = y
        return out
    if c["op"] == "act_backward":
        f, slope = _exact_activation(c["kind"], _exact_values(s["gq"], s["gs"], c["cols"]))
        dy = s["dy"].double()
        up = _exact_values(s["uq"], s["us"], c["cols"]) if c["up"] else torch.ones_like(dy)
        out = {"dgate": dy * slope * up}
        if c["up"]:
            out["dup"] = dy * f
        if c["again"]:
            out["y"] = f * up
        return out
    parts = []
    for r in range(0, c["rows"], 256):
        cut = slice(r, r + 256)
        x, ids = s["logits"][cut].double(), s["ids"][cut]
        on = ids >= 0
        z = x / c["tau"]
        m = z.max(1, keepdim=True).values
        e = torch.exp(z - m)
        total = e.sum(1, keepdim=True)
        p = e / total
        at = ids.clamp_min(0)[:, None]
        if c["op"] == "logprob":
            # H = log total - sum p (z - m), over what can be chosen
            shifted = torch.where(e > 0, z - m, torch.zeros_like(z))
            part = {"logp": (torch.gather(z, 1, at) - m - torch.log(total))[:, 0],
                    "lse": (m + torch.log(total))[:, 0],
                    "entropy": (torch.log(total) - (p * shifted).sum(1, keepdim=True))[:, 0]}
            part = {k: torch.where(on, v, torch.zeros_like(v)) for k, v in part.items()}
            if c["top"]:
                value, index = torch.sort(x, dim=1, descending=True, stable=True)
                value, index = value[:, :c["top"]], index[:, :c["top"]]
                dead = ~on[:, None] | torch.isinf(value)
                part["index"] = index.masked_fill(dead, -1).to(torch.int32)
                part["value"] = value.masked_fill(dead, -math.inf)
        else:
            a, lse = s["dlogp"][cut].double(), s["lse"][cut].double()[:, None]
            p = torch.exp(z - lse)
            g = torch.zeros_like(z).scatter_(1, at, 1.0) - p
            g = g * a[:, None]
            if c["entropy"]:
                # dH/dz_v = -p_v (log p_v + H)
                b, h = s["dentropy"][cut].double(), s["entropy"][cut].double()
                g = g - b[:, None] * (torch.special.xlogy(p, p) + p * h[:, None])
            part = {"grad": g * (on.double() * s["scale"] / c["tau"])[:, None]}
        parts.append(part)
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
