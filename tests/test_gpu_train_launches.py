"""Calls of the training operators with more workgroups than one HIP launch may
have (2^32 - 1 lanes): each goes out in several, and gives what calls of a part
of the rows give, bit for bit."""
import pytest
import torch

import sharded_mixed_precision_step_amd as zs
import train_ref as ref
from gpu_util import device
from test_gpu_q8 import _gemm_tol, _operand

pytestmark = [pytest.mark.gpu, pytest.mark.slow]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def test_norm_of_more_rows_than_a_launch():
    """64 lanes a row: 2^26 - 1 rows a launch."""
    dev = device()
    rows, cols = (1 << 26) + 3, 8
    print(f"case: norm {rows}x{cols}", flush=True)
    x = torch.randn(rows, cols, device=dev, dtype=torch.float16, generator=_gen(1))
    w = torch.randn(cols, device=dev, generator=_gen(2))
    y, rstd = torch.full_like(x, 7.0), torch.full((rows,), 7.0, device=dev)
    zs.zero_rmsnorm(x, w, 1e-5, y=y, rstd=rstd)
    part, part_rstd = torch.empty(1 << 24, cols, dtype=x.dtype, device=dev), \
        torch.empty(1 << 24, device=dev)
    for r in range(0, rows, 1 << 24):
        n = min(1 << 24, rows - r)
        zs.zero_rmsnorm(x[r:r + n], w, 1e-5, y=part[:n], rstd=part_rstd[:n])
        assert torch.equal(y[r:r + n], part[:n]) and torch.equal(rstd[r:r + n], part_rstd[:n])


def test_distillation_of_more_rows_than_a_launch():
    """256 lanes a row: 2^24 - 1 rows a launch."""
    dev = device()
    rows, vocab = (1 << 24) + 5, 5
    print(f"case: distill {rows}x{vocab}", flush=True)
    logits = torch.randn(rows, vocab, device=dev, generator=_gen(1)).to(torch.float16)
    index = torch.randint(0, vocab, (rows, 2), device=dev, generator=_gen(2), dtype=torch.int32)
    teacher = torch.randn(rows, 2, device=dev, generator=_gen(3)).to(torch.float16)

    def call(cut, loss, lse, both, grad):
        args = logits[cut], index[cut], teacher[cut]
        zs.zero_distill_forward(*args, loss, lse)
        zs.zero_distill_backward(*args, lse, grad, loss_scale=16.0)
        zs.zero_distill(*args, None, None, both, loss_scale=16.0)

    def outputs(n):
        return (torch.full((n,), 7.0, device=dev), torch.full((n,), 7.0, device=dev),
                torch.full((n, vocab), 7.0, dtype=torch.float16, device=dev),
                torch.full((n, vocab), 7.0, dtype=torch.float16, device=dev))

    whole = outputs(rows)
    call(slice(0, rows), *whole)
    for r in range(0, rows, 1 << 22):
        cut = slice(r, min(r + (1 << 22), rows))
        part = outputs(cut.stop - r)
        call(cut, *part)
        for a, b in zip(whole, part):
            assert torch.equal(a[cut], b)


def test_conversion_of_more_tiles_than_a_launch():
    """256 lanes a tile: 2^24 - 1 tiles a launch, here of one column each.  The
    column's blocks are the rows of the same elements as a matrix of 128."""
    dev = device()
    rows = (1 << 31) + 300
    print(f"case: convert {rows}x1", flush=True)
    x = torch.empty(rows, 1, dtype=torch.bfloat16, device=dev)
    for r in range(0, rows, 1 << 28):
        n = min(1 << 28, rows - r)
        x[r:r + n] = torch.randn(n, 1, device=dev, generator=_gen(r % 1000 + 1))
    qt, st = zs.q8_empty(1, rows)
    qt.view(torch.uint8).fill_(0x55)
    st.view(torch.uint8).fill_(0x55)
    zs.zero_q8_quantize(x, qt=qt, st=st)
    blocks = rows // 128
    q, s = zs.q8_empty(blocks, 128)
    zs.zero_q8_quantize(x[:128 * blocks].view(blocks, 128), q, s)
    got, scales = qt.view(torch.uint8)[0], st.view(torch.uint8)[0]
    assert torch.equal(got[:128 * blocks].view(blocks, 128), q.view(torch.uint8))
    assert torch.equal(scales[:blocks], s.view(torch.uint8)[:, 0])
    tail = rows - 128 * blocks
    q, s = zs.q8_empty(1, tail)
    zs.zero_q8_quantize(x[128 * blocks:].view(1, tail), q, s)
    assert torch.equal(got[128 * blocks:], q.view(torch.uint8)[0])
    assert int(scales[blocks]) == int(s.view(torch.uint8)[0, 0])
    assert (scales[blocks + 1:] == 127).all()


@pytest.mark.parametrize("m,n", [(185_500, 185_600), (371_000, 92_750)])
def test_product_of_more_tiles_than_a_launch(m, n):
    """More than 2^23 tiles of 64 x 64, cut along n and along m."""
    dev = device()
    k = 128
    print(f"case: gemm {m}x{n}x{k}", flush=True)
    a, sa = _operand(m, k, torch.float8_e4m3fn, 3, dev)
    b, sb = _operand(n, k, torch.float8_e4m3fn, 9, dev)
    c = torch.empty(m, n, dtype=torch.bfloat16, device=dev)
    zs.zero_q8_gemm(a, sa, b, sb, c)
    va, vb = ref.from_blocks(a, sa), ref.from_blocks(b, sb)
    cut = (max(m, n) // 2 + 255) // 256 * 256
    ends = [slice(0, 20), slice(-20, None)]
    rows = ends + ([slice(cut - 20, cut + 20)] if m > n else [slice(1000, 1020)])
    cols = ends + ([slice(1000, 1020)] if m > n else [slice(cut - 20, cut + 20)])
    for r in rows:
        want = va[r] @ vb.t()
        ref.assert_close(c[r], want, _gemm_tol(va[r], vb, sa[r], sb, c.dtype, want), f"rows {r}")
    for q in cols:
        want = va @ vb[q].t()
        ref.assert_close(c[:, q].contiguous(), want,
                         _gemm_tol(va, vb[q], sa, sb[q], c.dtype, want), f"columns {q}")


def test_product_of_a_long_column():
    """2^24 tiles of 64 x 64 and two more, for which the small tiles are chosen;
    no columns of k, so that c alone is large."""
    dev = device()
    m = (1 << 30) + 70
    print(f"case: gemm {m}x1x0", flush=True)
    c = torch.full((m, 1), 7.0, dtype=torch.float16, device=dev)
    stream = torch.cuda.current_stream().cuda_stream
    rc = zs.lib.zero_q8_gemm(None, 0, 128, None, 4, None, 0, 128, None, 4, m, 1, 0, c.data_ptr(),
                             zs.ZERO_F16, 1, 0, stream)
    assert rc == 0, zs.lib.zero_last_error_string()
    assert not c.any()
