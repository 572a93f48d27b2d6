"""One row of a wider matrix: whatever stride torch gives a dimension of one, the
training operators take it like the same row by itself, in place too."""
import pytest
import torch

import sharded_mixed_precision_step_amd as zs
from gpu_util import device

pytestmark = pytest.mark.gpu


def _wide(row, width):
    """`row` [1, n] as the first columns of a wider matrix's only row."""
    base = torch.zeros(1, width, dtype=row.dtype, device=row.device)
    base[:, :row.shape[1]] = row
    out = base[:, :row.shape[1]]
    assert out.stride(0) == width
    return out


def test_distillation_of_one_row_with_entries_of_different_strides():
    dev = device()
    logits = torch.randn(1, 300, device=dev)
    index = torch.randint(0, 300, (1, 7), device=dev)
    teacher = torch.randn(1, 7, device=dev)
    outs = []
    for i, t in ((index, teacher), (_wide(index, 12), teacher), (index, _wide(teacher, 9))):
        loss, lse = torch.empty(1, device=dev), torch.empty(1, device=dev)
        grad = torch.empty_like(logits)
        zs.zero_distill(logits, i, t, loss, lse, grad)
        outs.append((loss, lse, grad))
    for other in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], other))


def test_distillation_of_one_row_in_place_under_another_stride():
    dev = device()
    logits = _wide(torch.randn(1, 300, device=dev), 512)
    index, teacher = torch.randint(0, 300, (1, 7), device=dev), torch.randn(1, 7, device=dev)
    want = torch.empty(1, 300, device=dev)
    zs.zero_distill(logits, index, teacher, None, None, want)
    grad = logits[0].unsqueeze(0)
    assert grad.stride(0) != logits.stride(0)
    zs.zero_distill(logits, index, teacher, None, None, grad)
    assert torch.equal(logits, want)


def test_norm_of_one_row_in_place_under_another_stride():
    dev = device()
    x = _wide(torch.randn(1, 100, device=dev), 256)
    w = torch.randn(100, device=dev)
    want = torch.empty(1, 100, device=dev)
    zs.zero_rmsnorm(x, w, 1e-5, y=want)
    zs.zero_rmsnorm(x, w, 1e-5, y=x[0].unsqueeze(0))
    assert torch.equal(x, want)


def test_conversion_of_one_row_of_two_copies_with_different_strides():
    dev = device()
    ctl = zs.control_new(zs.LossScaler.create(), 1, dev)
    copies = [torch.randn(1, 200, device=dev).half() for _ in range(2)]
    q, s = zs.q8_empty(1, 200)
    want, want_s = zs.q8_empty(1, 200)
    zs.zero_q8_quantize(copies[0], want, want_s)
    zs.zero_q8_quantize_ctl([_wide(copies[0], 512), copies[1]], ctl, q, s)
    assert torch.equal(q.view(torch.uint8), want.view(torch.uint8))
    assert torch.equal(s.view(torch.uint8), want_s.view(torch.uint8))


def test_conversion_and_product_of_one_row_of_any_stride():
    """q8 data whose only row lies in a matrix of a width that is no multiple of
    16, with scales in one whose width is no multiple of 4."""
    dev = device()
    x, w = torch.randn(1, 200, device=dev), torch.randn(50, 200, device=dev)
    q = torch.empty(1, 264 + 3, dtype=torch.uint8, device=dev)[:, :256].view(torch.float8_e4m3fn)
    s = torch.empty(1, 7, dtype=torch.uint8, device=dev)[:, :4]
    zs.zero_q8_quantize(x, q, s)
    want, want_s = zs.q8_empty(1, 200)
    zs.zero_q8_quantize(x, want, want_s)
    assert torch.equal(q.view(torch.uint8), want.view(torch.uint8))
    b = zs.q8_empty(50, 200)
    zs.zero_q8_quantize(w, *b)
    c, c2 = torch.empty(1, 50, device=dev), torch.empty(1, 50, device=dev)
    zs.zero_q8_gemm(q, s, *b, c)
    zs.zero_q8_gemm(want, want_s, *b, c2)
    assert torch.equal(c, c2)
