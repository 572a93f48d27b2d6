"""The model operators at sizes where another way through them begins: many tokens,
large vocabularies, strided tables, last packs that share elements with another
wave's, single rows of wider matrices; and calls of more workgroups than one HIP
launch may have (2^32 - 1 lanes)."""
import math

import pytest
import torch

import model_ref as ref
import sharded_mixed_precision_step_amd as zs
from gpu_util import device

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-5


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(seed, *shape, dtype=F32):
    return torch.randn(*shape, generator=_gen(seed), device="cuda").to(dtype)


def _whole(seed, *shape):
    """Whole numbers, so that sums are exact and have to be equal."""
    return torch.randint(-3, 4, shape, device="cuda", generator=_gen(seed)).to(F16)


def _backward(dy, ids, vocab, old=None, gap=0):
    """The gradient, and what lies between its rows."""
    cols = dy.shape[1]
    base = torch.full((vocab, cols + gap), 7.0, device="cuda")
    d = base[:, :cols]
    if old is not None:
        d.copy_(old)
    n = zs.zero_embed_backward_workspace(len(ids), vocab, cols)
    work = torch.full((n,), 0xa5, dtype=torch.uint8, device="cuda")
    zs.zero_embed_backward(dy, ids, d, work, accumulate=old is not None)
    assert (base[:, cols:] == 7).all()
    return d


@pytest.mark.parametrize("gap", [0, 5])
@pytest.mark.parametrize("tokens,vocab,cols", [(511, 40, 520), (512, 40, 520), (513, 40, 520),
                                               (512, 1, 3), (512, 300001, 9), (600, 300001, 9),
                                               (2000, 1 << 18, 16), (20000, (1 << 18) - 1, 8),
                                               (20000, (1 << 18) + 1, 8), (16384, 1 << 20, 8),
                                               (530000, 3000, 8), (530000, 1 << 19, 8),
                                               (66000, 100, 4104), (9000, 30000, 80),
                                               (12345, 40000, 300), (16384, 60000, 400)])
def test_embedding_gradient_where_its_ways_change(tokens, vocab, cols, gap):
    device()
    print(f"case: embed backward {tokens} of {vocab}x{cols} gap {gap}", flush=True)
    g = _gen(tokens)
    ids = torch.exp(torch.rand(tokens, device="cuda", generator=g) * math.log(vocab + 1)).long() - 1
    ids[torch.rand(tokens, device="cuda", generator=g) < 0.05] = -1
    ids[tokens // 2] = vocab - 1
    ids[tokens // 3] = vocab
    dy = _whole(tokens, tokens, cols)
    want = torch.zeros(vocab, cols, device="cuda")  # whole numbers below 2^24: exact
    live = (ids >= 0) & (ids < vocab)
    want.index_add_(0, ids[live], dy[live].float())
    assert torch.equal(_backward(dy, ids, vocab, gap=gap), want)
    old = _whole(3, vocab, cols).float()
    assert torch.equal(_backward(dy, ids, vocab, old, gap), want + old)


@pytest.mark.parametrize("dy_dtype,dt_dtype", [(F32, F16), (F16, BF16), (BF16, F16), (F32, F32)])
@pytest.mark.parametrize("tokens,cols", [(300, 20), (3000, 20), (530000, 16)])
def test_embedding_gradient_types_where_its_ways_change(tokens, cols, dy_dtype, dt_dtype):
    """Whole numbers: the fp32 sums are exact, and rounded once."""
    device()
    vocab = 700
    ids = torch.randint(-9, vocab // 2, (tokens,), device="cuda", generator=_gen(1))
    dy = _whole(2, tokens, cols).to(dy_dtype)
    want = torch.zeros(vocab, cols, device="cuda")
    want.index_add_(0, ids[ids >= 0], dy[ids >= 0].float())
    work = torch.empty(zs.zero_embed_backward_workspace(tokens, vocab, cols), dtype=torch.uint8,
                       device="cuda")
    d = torch.full((vocab, cols), 7.0, dtype=dt_dtype, device="cuda")
    zs.zero_embed_backward(dy, ids, d, work)
    assert torch.equal(d, want.to(dt_dtype))
    d = _whole(3, vocab, cols).to(dt_dtype)
    old = d.float().clone()
    zs.zero_embed_backward(dy, ids, d, work, accumulate=True)
    assert torch.equal(d, (want + old).to(dt_dtype))


@pytest.mark.parametrize("tokens", [512, 513, 16384, 16385, 300000])
def test_embedding_gradient_of_one_token_over_and_over(tokens):
    device()
    dy = _whole(1, tokens, 24)
    ids = torch.full((tokens,), 17, device="cuda", dtype=torch.int32)
    d = _backward(dy, ids, 20, gap=1)
    assert torch.equal(d[17].double(), dy.double().sum(0)) and d[:17].eq(0).all() and \
        d[18:].eq(0).all()


@pytest.mark.parametrize("cols", [1025, 1537, 2561, 9217, 12289])
def test_layernorm_in_place_where_a_wave_begins_with_the_last_elements(cols):
    """The last pack is the row's last eight elements, which another wave's lane owns
    but for one."""
    dev = device()
    rows = 1100
    h, w = _randn(2, rows, cols, dtype=F16), _randn(3, cols, dtype=F16)
    mean, rstd = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
    x, res = _randn(5, rows, cols, dtype=F16), _randn(6, rows, cols, dtype=F16)
    hh, y = torch.empty_like(x), torch.empty_like(x)
    zs.zero_layernorm(x, w, None, EPS, residual=res, h=hh, y=y, mean=mean, rstd=rstd)
    for t in (x, res):
        x1, r1 = x.clone(), res.clone()
        zs.zero_layernorm(x1, w, None, EPS, residual=r1, h=x1 if t is x else r1,
                          y=x1 if t is res else None)
        assert torch.equal(x1 if t is x else r1, hh)
        assert t is x or torch.equal(x1, y)
    dy, dres = _randn(1, rows, cols, dtype=F16), _randn(4, rows, cols, dtype=F16)
    ws = torch.empty(zs.zero_layernorm_backward_workspace(rows, cols), dtype=torch.uint8, device=dev)
    dx, dw, db = torch.empty_like(h), torch.empty_like(w), torch.empty_like(w)
    zs.zero_layernorm_backward(dy, hh, w, mean, rstd, dx, dw, db, ws, dres=dres)
    wx, _, _, tx, _, _ = ref.layernorm_backward(dy, hh, w, mean, rstd, dres)
    ref.assert_close(dx, wx, ref.half_step(F16, wx) + tx, "dx")
    for place in range(3):
        t = [dy.clone(), hh.clone(), dres.clone()]
        zs.zero_layernorm_backward(t[0], t[1], w, mean, rstd, t[place], dw, db, ws, dres=t[2])
        assert torch.equal(t[place], dx), place


def _wide(row, width):
    """`row` [1, n] as the first columns of a wider matrix's only row."""
    base = torch.zeros(1, width, dtype=row.dtype, device=row.device)
    base[:, :row.shape[1]] = row
    out = base[:, :row.shape[1]]
    assert out.stride(0) == width
    return out


def test_single_rows_of_wider_matrices():
    dev = device()
    x, w = _randn(1, 1, 100), _randn(2, 100)
    want, y = torch.empty_like(x), _wide(x, 256)
    zs.zero_layernorm(x, w, None, EPS, y=want)
    zs.zero_layernorm(y, w, None, EPS, y=y[0].unsqueeze(0))
    assert torch.equal(y, want)
    zs.zero_act(x, "gelu", y=want)
    y = _wide(x, 130)
    zs.zero_act(y, "gelu", y=y[0].unsqueeze(0))
    assert torch.equal(y, want)
    ids = torch.tensor([3], device=dev)
    lse, logp = torch.empty(1, device=dev), torch.empty(1, device=dev)
    zs.zero_logprob(x, ids, logp, lse=lse)
    one = torch.ones(1, device=dev)
    zs.zero_logprob_backward(x, ids, lse, one, want)
    y = _wide(x, 200)
    zs.zero_logprob_backward(y, ids, lse, one, y[0].unsqueeze(0))
    assert torch.equal(y, want)
    table = _wide(_randn(3, 1, 60), 64)
    got, d = torch.empty(1, 60, device=dev), _wide(torch.ones(1, 60, device=dev), 77)
    zs.zero_embed(table, ids * 0, got)
    assert torch.equal(got, table)
    work = torch.empty(zs.zero_embed_backward_workspace(1, 1, 60), dtype=torch.uint8, device=dev)
    zs.zero_embed_backward(got, ids * 0, d, work, accumulate=True)
    assert torch.equal(d, got + 1)


# Logits that rise along the row, are all alike, or lie on few values: many reach the
# border.
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("vocab", [2000, 8192, 16001, 40000, 131072])
@pytest.mark.parametrize("rows", ["rising", "falling", "alike", "few values", "saw", "masked"])
def test_alternatives_of_rows_with_many_on_the_border(rows, vocab, dtype):
    device()
    i = torch.arange(vocab, device="cuda", dtype=torch.float64)
    x = {"rising": i / vocab, "falling": 1 - i / vocab, "alike": 0 * i + 2.5, "few values": i % 3,
         "saw": (i * 7919 % 4096) / 4096,
         "masked": torch.where(i % 1111 == 7, i / vocab, torch.finfo(dtype).min)}[rows]
    few = torch.stack([x, x.flip(0), x - 5, x * 1e4]).to(dtype).clamp_min(torch.finfo(dtype).min)
    # a stable sort of the negatives: ties by the lowest place
    order = torch.sort(-few.double(), dim=1, stable=True).indices[:, :128]
    for times in (1, 128, 512):  # as few, more and many rows
        logits = few.repeat(times, 1)
        for top in (1, 20, 128):
            index = torch.empty(4 * times, top, dtype=torch.int32, device="cuda")
            value = torch.empty(4 * times, top, dtype=dtype, device="cuda")
            zs.zero_logprob(logits, None, None, top_index=index, top_logit=value)
            want = order[:, :top].repeat(times, 1)
            assert torch.equal(index.long(), want)
            assert torch.equal(value, logits.gather(1, want))


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("vocab", [8193, 16385, 32009, 70001])
@pytest.mark.parametrize("rows", [511, 512, 2047, 2048])
def test_log_probabilities_of_many_rows(rows, vocab, dtype):
    device()
    logits = 3 * _randn(1, rows, vocab, dtype=dtype)
    logits[5, 9:] = -math.inf
    logits[6, 77] = math.nan
    ids = torch.randint(-1, vocab, (rows,), generator=_gen(2), device="cuda")
    ids[7], ids[8] = -1, vocab
    out = [torch.full((rows,), 7.0, device="cuda") for _ in range(3)]
    index = torch.empty(rows, 20, dtype=torch.int32, device="cuda")
    value = torch.empty(rows, 20, dtype=dtype, device="cuda")
    zs.zero_logprob(logits, ids, out[0], entropy=out[1], lse=out[2], top_index=index,
                    top_logit=value)
    for cut in torch.arange(rows, device="cuda").split(256):
        want, tol = ref.logprob(logits[cut], ids[cut], 1.0, 20)
        for got, w, t in zip(out, want, tol):
            ref.assert_close(got[cut], w, t + ref.half_step(F32, w.nan_to_num(0, 0, 0)), "sums")
        assert torch.equal(index[cut], want[3])
        assert torch.equal(value[cut].float().nan_to_num(9e9), want[4].float().nan_to_num(9e9))


@pytest.mark.parametrize("times,vocab", [(1, 4000003), (120, 600011), (410, 262145)])
def test_alternatives_of_long_rows(times, vocab):
    """The border moves several times on its way."""
    device()
    few = _randn(1, 5, vocab, dtype=F16)
    few[1] = few[1].sort().values
    few[2] = few[2].sort(descending=True).values
    few[3, 100:-100] = -math.inf
    few[4] = (few[4] * 2).round()
    order = torch.sort(-few.float(), dim=1, stable=True).indices[:, :128]
    logits, want = few.repeat(times, 1), order.repeat(times, 1)
    index = torch.empty(5 * times, 128, dtype=torch.int32, device="cuda")
    value = torch.empty(5 * times, 128, dtype=F16, device="cuda")
    zs.zero_logprob(logits, None, None, top_index=index, top_logit=value)
    assert torch.equal(index.long(), want) and torch.equal(value, logits.gather(1, want))


# ---- more workgroups than a launch has ------------------------------------------------


@pytest.mark.slow
def test_narrow_rows_of_more_workgroups_than_a_launch():
    """16 rows to 256 lanes: 2^28 - 16 rows a launch."""
    dev = device()
    rows, cols, step = (1 << 28) + 37, 4, 1 << 26
    print(f"case: layernorm and act {rows}x{cols}", flush=True)
    x = _randn(1, 1 << 20, cols, dtype=F16).repeat(257, 1)[:rows]
    w = _randn(2, cols)
    y, z = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    zs.zero_layernorm(x, w, None, EPS, y=y)
    zs.zero_act(x, "silu", y=z)
    part = torch.empty(step, cols, dtype=F16, device=dev)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        zs.zero_layernorm(x[r:r + n], w, None, EPS, y=part[:n])
        assert torch.equal(y[r:r + n], part[:n])
        zs.zero_act(x[r:r + n], "silu", y=part[:n])
        assert torch.equal(z[r:r + n], part[:n])


@pytest.mark.slow
def test_log_probabilities_of_more_rows_than_a_launch():
    """Four rows to 256 lanes: 2^26 - 4 rows a launch."""
    dev = device()
    rows, vocab, step = (1 << 26) + 11, 3, 1 << 24
    print(f"case: logprob {rows}x{vocab}", flush=True)
    x = _randn(1, rows, vocab, dtype=F16)
    ids = torch.randint(-1, vocab, (rows,), device=dev, generator=_gen(2), dtype=torch.int32)
    logp, top = torch.full((rows,), 7.0, device=dev), torch.full((rows, 1), 7, dtype=torch.int32,
                                                                device=dev)
    value = torch.full((rows, 1), 7.0, dtype=F16, device=dev)
    zs.zero_logprob(x, ids, logp, top_index=top, top_logit=value)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        a, b, c = torch.empty(n, device=dev), torch.empty_like(top[:n]), torch.empty_like(value[:n])
        zs.zero_logprob(x[r:r + n], ids[r:r + n], a, top_index=b, top_logit=c)
        assert torch.equal(logp[r:r + n], a) and torch.equal(top[r:r + n], b)
        assert torch.equal(value[r:r + n], c)


@pytest.mark.slow
@pytest.mark.parametrize("tokens", [3, 700])
def test_a_table_of_more_rows_than_a_launch(tokens):
    """A strided table of more workgroups of zeros than a launch has (2^24 - 1 of 256
    lanes for few tokens, 2^22 - 1 of 1,024 for more), and a gather of as many rows."""
    dev = device()
    vocab, cols = ((1 << 24) + 9, 1032) if tokens == 3 else ((1 << 22) + 9, 4104)
    print(f"case: embed {tokens} of {vocab}x{cols}", flush=True)
    base = torch.full((vocab, cols + 8), 7.0, dtype=F16, device=dev)
    d = base[:, :cols]
    dy = _whole(1, tokens, cols)
    ids = torch.randint(0, vocab, (tokens,), device=dev, generator=_gen(2))
    ids[0], ids[-1], ids[tokens // 2] = 0, vocab - 1, vocab - 1
    work = torch.empty(zs.zero_embed_backward_workspace(tokens, vocab, cols), dtype=torch.uint8,
                       device=dev)
    zs.zero_embed_backward(dy, ids, d, work)
    assert (base[:, cols:] == 7).all()
    rows, which = ids.unique(return_inverse=True)
    want = torch.zeros(len(rows), cols, device=dev).index_add_(0, which, dy.float())
    assert torch.equal(d[rows].float(), want)
    zeros = torch.zeros(1, cols, dtype=F16, device=dev)
    d[rows] = zeros
    assert all((d[r:r + (1 << 18)] == 0).all() for r in range(0, vocab, 1 << 18))
    if tokens == 3:
        table = _randn(5, 5, cols, dtype=F16)
        ids = torch.arange(vocab, device=dev, dtype=torch.int32) % 5
        zs.zero_embed(table, ids, d)
        assert (base[:, cols:] == 7).all()
        whole = vocab // 5 * 5
        for r in range(0, whole, 5 << 16):
            n = min(5 << 16, whole - r)
            assert torch.equal(d[r:r + n].reshape(-1, 5, cols), table.expand(n // 5, 5, cols))
        assert torch.equal(d[whole:], table[:vocab - whole])
