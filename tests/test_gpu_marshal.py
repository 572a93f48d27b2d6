"""The binding without its host library (csrc/marshal.cpp): the same results."""
import pytest
import torch

import sharded_mixed_precision_step_amd as zs
from gpu_util import device
from sharded_mixed_precision_step_amd import model, train

pytestmark = pytest.mark.gpu


def _calls(dev):
    """One call of each operator that goes through the host library; the outputs."""
    g = torch.Generator(device="cuda")
    g.manual_seed(7)

    def randn(*shape, dtype=torch.float16):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    rows, cols, vocab = 37, 300, 500
    out = {}

    def empty(name, *shape, dtype=torch.float32):
        out[name] = torch.zeros(*shape, dtype=dtype, device=dev)
        return out[name]

    ids = torch.randint(-1, vocab, (rows,), generator=g, device=dev)
    x = empty("x", rows, cols, dtype=torch.float16)
    zs.zero_embed(randn(vocab, cols), ids, x, scale=2.0)
    ws = torch.empty(zs.zero_embed_backward_workspace(rows, vocab, cols), dtype=torch.uint8,
                     device=dev)
    zs.zero_embed_backward(randn(rows, cols), ids, empty("dtable", vocab, cols), ws)
    w, b, res = randn(cols), randn(cols), randn(rows, cols, dtype=torch.float32)
    mean, rstd = empty("mean", rows), empty("rstd", rows)
    q, s = zs.q8_empty(rows, cols, device=dev)
    h = empty("h", rows, cols)
    zs.zero_layernorm(x, w, b, 1e-5, residual=res, h=h, q=q, s=s, mean=mean, rstd=rstd)
    ws = torch.empty(zs.zero_layernorm_backward_workspace(rows, cols), dtype=torch.uint8,
                     device=dev)
    dy = randn(rows, cols)
    zs.zero_layernorm_backward(dy, h, w, mean, rstd, empty("dx", rows, cols), empty("dw", cols),
                               empty("db", cols), ws, dres=res)
    gq, uq = zs.q8_empty(rows, cols, device=dev), zs.q8_empty(rows, cols, device=dev)
    zs.zero_act(x, "silu", up=dy, y=empty("y", rows, cols), gate_q=gq[0], gate_s=gq[1],
                up_q=uq[0], up_s=uq[1])
    zs.zero_act_backward(dy, *gq, empty("dgate", rows, cols), "silu", up_q=uq[0], up_s=uq[1],
                         dup=empty("dup", rows, cols))
    logits = randn(rows, vocab)
    lse = empty("lse", rows)
    zs.zero_logprob(logits, ids, empty("logp", rows), entropy=empty("entropy", rows), lse=lse,
                    top_index=empty("index", rows, 5, dtype=torch.int32),
                    top_logit=empty("value", rows, 5, dtype=torch.float16))
    zs.zero_logprob_backward(logits, ids, lse, randn(rows, dtype=torch.float32),
                             empty("grad", rows, vocab, dtype=torch.float16))
    out.update(q=q, s=s, gq=gq[0], gs=gq[1], uq=uq[0], us=uq[1])
    return out


def test_the_calls_through_ctypes_give_the_same_bits(monkeypatch):
    dev = device()
    assert zs._marshal is not None
    want = _calls(dev)
    for module in (train, model):
        for name in ("_mat", "_like", "_vec", "_q8"):
            if hasattr(module, name):
                monkeypatch.setattr(module, name, getattr(train, f"{name}_checked"))
    monkeypatch.setattr(model, "_calls", zs.lib)
    got = _calls(dev)
    assert want.keys() == got.keys()
    for name in want:
        assert torch.equal(want[name].view(torch.uint8), got[name].view(torch.uint8)), name
    with pytest.raises(TypeError):
        zs.zero_embed(want["x"].double(), torch.zeros(3, dtype=torch.int32, device=dev), want["x"])
