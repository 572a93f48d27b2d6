"""Embedding and its gradient by sorted tokens, against the 64-bit definitions."""
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


def _ids(seed, tokens, vocab, dtype=torch.int64, skew=True):
    """Frequencies fall as 1 / rank; some tokens have no row."""
    g = _gen(seed)
    u = torch.rand(tokens, generator=g, device="cuda")
    ids = torch.exp(u * math.log(vocab)).long().clamp(1, vocab) - 1 if skew else \
        (u * vocab).long().clamp_max(vocab - 1)
    out = torch.rand(tokens, generator=g, device="cuda")
    return torch.where(out < 0.05, -1, ids).to(dtype)


def _work(tokens, vocab, cols):
    n = zs.zero_embed_backward_workspace(tokens, vocab, cols)
    return torch.full((n,), 0xa5, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("t_dtype,y_dtype", [(F16, F16), (BF16, BF16), (F32, F16), (F32, F32),
                                             (F16, BF16), (BF16, F32)])
@pytest.mark.parametrize("tokens,vocab,cols", [(1, 1, 1), (3, 7, 5), (16, 1000, 64), (37, 101, 130),
                                               (5, 11, 1001), (129, 50, 4096), (9, 3, 9001)])
@pytest.mark.parametrize("scale", [1.0, 31.6])
def test_embed_is_the_definition(tokens, vocab, cols, t_dtype, y_dtype, scale):
    print(f"case: embed {tokens} of {vocab}x{cols} {t_dtype} {y_dtype}", flush=True)
    device()
    table = _randn(1, vocab, cols, dtype=t_dtype)
    ids = _ids(2, tokens, vocab)
    y = torch.full((tokens, cols), 7.0, dtype=y_dtype, device="cuda")
    zs.zero_embed(table, ids, y, scale=scale)
    want = ref.embed(table, ids, torch.tensor(scale, dtype=F32).double().item())
    ref.assert_close(y, want, ref.half_step(y_dtype, want) + U * want.abs(), "y")
    y2 = torch.empty_like(y)
    zs.zero_embed(table, ids.int(), y2, scale=scale)
    assert torch.equal(y, y2)


def test_embed_ids_outside_strides_and_what_lies_beside():
    device()
    base = _randn(1, 20, 77, dtype=F16)
    table = base[:, 3:3 + 61]
    ids = torch.tensor([[0, 19, -1], [20, -2 ** 40, 2 ** 33], [5, 5, 19]], device="cuda")
    out = torch.full((9, 70), 7.0, dtype=BF16, device="cuda")
    y = out[:, 5:66]
    zs.zero_embed(table, ids, y, scale=2.0)
    want = ref.embed(table, ids, 2.0)
    assert torch.isnan(y[[3, 5]]).all() and (y[[2, 4]] == 0).all()
    ref.assert_close(y, want, ref.half_step(BF16, want.nan_to_num(0)), "y")
    assert (out[:, :5] == 7).all() and (out[:, 66:] == 7).all()


def test_embed_of_the_current_copy():
    dev = device()
    two = [_randn(k, 30, 40, dtype=F16) for k in (1, 2)]
    ids = _ids(3, 25, 30)
    ctl = zs.control_new(zs.LossScaler.create(scale=8.0), 1, dev)
    y, want = torch.empty(25, 40, dtype=F16, device=dev), torch.empty(25, 40, dtype=F16, device=dev)
    zs.zero_embed_ctl(two, ctl, ids, y)
    zs.zero_embed(two[zs.control_read(ctl).cur], ids, want)
    assert torch.equal(y, want)


TYPES = [(F16, F16), (BF16, F32), (F32, F32), (F32, BF16), (BF16, BF16)]


@pytest.mark.parametrize("dy_dtype,dt_dtype", TYPES)
@pytest.mark.parametrize("tokens,vocab,cols", [(1, 1, 1), (2, 3, 7), (33, 5, 64), (100, 64, 130),
                                               (1000, 63, 129), (4099, 500, 72), (5000, 70000, 40),
                                               (8192, 1000, 264), (16384, 300, 64),
                                               (16385, 300, 64), (40000, 4097, 65), (70, 9, 9001)])
def test_backward_is_the_sum(tokens, vocab, cols, dy_dtype, dt_dtype):
    print(f"case: embed backward {tokens} of {vocab}x{cols} {dy_dtype} {dt_dtype}", flush=True)
    device()
    dy = _randn(1, tokens, cols, dtype=dy_dtype)
    ids = _ids(2, tokens, vocab)
    d = torch.full((vocab, cols), 7.0, dtype=dt_dtype, device="cuda")
    work = _work(tokens, vocab, cols)
    zs.zero_embed_backward(dy, ids, d, work, scale=0.5)
    want, tol = ref.embed_backward(dy, ids, vocab, 0.5)
    ref.assert_close(d, want, ref.half_step(dt_dtype, want) + tol, "dtable")
    # the same bits again, with 32-bit ids and whatever the workspace held
    d2 = torch.full_like(d, 3.0)
    zs.zero_embed_backward(dy, ids.int(), d2, work.random_(generator=_gen(9)), scale=0.5)
    assert torch.equal(d, d2)
    # added to what is there; rows without tokens keep their bits
    old = _randn(5, vocab, cols, dtype=dt_dtype)
    d3 = old.clone()
    zs.zero_embed_backward(dy, ids, d3, work, scale=0.5, accumulate=True)
    both = want + old.double()
    has = torch.zeros(vocab, dtype=torch.bool, device="cuda")
    has[ids[ids >= 0]] = True
    assert torch.equal(d3[~has], old[~has])
    ref.assert_close(d3, torch.where(has[:, None], both, old.double()),
                     ref.half_step(dt_dtype, both) + tol + 2 * U * (want.abs() + old.double().abs()),
                     "accumulated")


@pytest.mark.parametrize("tokens", [1, 31, 32, 33, 64, 65, 4096, 4097, 16384, 20000])
@pytest.mark.parametrize("pattern", ["one row", "each its own", "border runs", "none", "sorted",
                                     "reversed"])
def test_backward_runs_and_pieces(tokens, pattern):
    """Runs that end at, cross and cover the pieces of the sorted list; whole
    numbers, so that the sums are exact and have to be equal."""
    device()
    vocab, cols = tokens + 3, 24
    i = torch.arange(tokens, device="cuda")
    ids = {"one row": torch.full_like(i, vocab - 1), "each its own": (i * 7919) % vocab,
           "border runs": (i // 32 + (i % 32 == 31)) % vocab, "none": torch.full_like(i, -1),
           "sorted": i // 5, "reversed": (tokens - 1 - i) // 45}[pattern]
    dy = torch.randint(-3, 4, (tokens, cols), device="cuda", generator=_gen(tokens)).to(F16)
    d = torch.full((vocab, cols), 7.0, device="cuda")
    zs.zero_embed_backward(dy, ids, d, _work(tokens, vocab, cols))
    want, _ = ref.embed_backward(dy, ids, vocab, 1.0)
    assert torch.equal(d.double(), want)


def test_backward_of_a_row_ignores_the_others():
    """A row's sum has the same bits whatever other tokens there are, as long as
    its own keep their places in the pieces: the order is the tokens'."""
    device()
    tokens, cols = 3000, 96
    dy = _randn(1, tokens, cols)
    ids = torch.zeros(tokens, dtype=torch.int64, device="cuda")
    one, two = torch.empty(4, cols, device="cuda"), torch.empty(4, cols, device="cuda")
    zs.zero_embed_backward(dy, ids, one, _work(tokens, 4, cols))
    order = torch.cat([torch.arange(tokens, device="cuda"), torch.zeros(50, dtype=torch.int64,
                                                                      device="cuda")])
    more = torch.cat([ids, torch.full((50,), 2, device="cuda")])
    zs.zero_embed_backward(dy[order], more, two, _work(tokens + 50, 4, cols))
    assert torch.equal(one[0], two[0])


def test_backward_ids_outside_no_tokens_and_strides():
    device()
    ids = torch.tensor([0, 9, 10, -1, 2 ** 40, -2 ** 40, 9], device="cuda")
    base = _randn(1, 7, 50, dtype=F16)
    dy = base[:, 3:3 + 45]
    out = torch.full((10, 60), 7.0, dtype=F16, device="cuda")
    d = out[:, 1:46]
    zs.zero_embed_backward(dy, ids, d, _work(7, 10, 45))
    want, tol = ref.embed_backward(dy, ids, 10, 1.0)
    ref.assert_close(d, want, ref.half_step(F16, want) + tol, "dtable")
    assert (out[:, 0] == 7).all() and (out[:, 46:] == 7).all()
    zs.zero_embed_backward(dy[:0], ids[:0], d, None)
    assert (d == 0).all() and (out[:, 0] == 7).all() and (out[:, 46:] == 7).all()
    d.fill_(3)
    zs.zero_embed_backward(dy[:0], ids[:0], d, None, accumulate=True)
    assert (d == 3).all()


def test_backward_passes_non_finite_values_on():
    device()
    dy = torch.zeros(40, 8, device="cuda")
    dy[3, 1], dy[5, 2], dy[6, 2], dy[7, 3] = math.nan, math.inf, -math.inf, math.inf
    dy[8] = 3e38
    dy[9] = 3e38
    ids = torch.zeros(40, dtype=torch.int64, device="cuda")
    ids[8] = 1
    d = torch.empty(2, 8, dtype=F16, device="cuda")
    zs.zero_embed_backward(dy, ids, d, _work(40, 2, 8))
    assert torch.isnan(d[0, 1:3]).all() and d[0, 3] == math.inf and (d[1] == math.inf).all()


def test_backward_is_the_derivative():
    """sum(forward(table + t direction) * dy) changes by t (dtable . direction):
    the forward is linear, so one difference is exact but for rounding."""
    device()
    vocab, cols, tokens = 50, 40, 300
    table, direction = _randn(1, vocab, cols), _randn(2, vocab, cols)
    ids, dy = _ids(3, tokens, vocab), _randn(4, tokens, cols)
    d = torch.empty_like(table)
    zs.zero_embed_backward(dy, ids, d, _work(tokens, vocab, cols), scale=3.0)
    f = lambda t: (ref.embed(t, ids, 3.0) * dy.double()).sum()  # noqa: E731
    up = f(table.double() + direction.double()) - f(table.double() - direction.double())
    got = (d.double() * direction.double()).sum()
    size = (ref.embed(direction.abs(), ids, 3.0) * dy.double().abs()).sum()
    assert abs(up / 2 - got) <= (tokens + 4) * U * size


def test_an_embedding_in_a_graph_and_on_another_stream():
    device()
    tokens, vocab, cols = 700, 300, 200
    table, ids, dy = _randn(1, vocab, cols, dtype=F16), _ids(2, tokens, vocab), \
        _randn(3, tokens, cols, dtype=F16)
    y, d = torch.empty(tokens, cols, dtype=F16, device="cuda"), torch.empty_like(table)
    work = _work(tokens, vocab, cols)

    def call():
        zs.zero_embed(table, ids, y)
        zs.zero_embed_backward(dy, ids, d, work)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(3):
        ids.copy_(_ids(10 + k, tokens, vocab))
        dy.copy_(_randn(20 + k, tokens, cols))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone(), d.clone()
        call()
        torch.cuda.synchronize()
        assert torch.equal(got[0], y) and torch.equal(got[1], d)


@pytest.mark.slow
def test_offsets_past_32_bits():
    """Tables of more than 2^32 bytes: rows at both ends, in both directions."""
    device()
    vocab, cols = 1_200_000, 2048
    print(f"case: embed of {vocab}x{cols}", flush=True)
    table = torch.zeros(vocab, cols, dtype=F16, device="cuda")
    ids = torch.tensor([0, vocab - 1, 1_048_576, 1_100_001, vocab - 1], device="cuda")
    table[ids] = _randn(1, 5, cols, dtype=F16)
    y = torch.empty(5, cols, dtype=F16, device="cuda")
    zs.zero_embed(table, ids, y)
    assert torch.equal(y, table[ids])
    dy = torch.randint(-3, 4, (5, cols), device="cuda", generator=_gen(2)).to(F16)
    table.fill_(7.0)
    zs.zero_embed_backward(dy, ids, table, _work(5, vocab, cols))
    assert torch.equal(table[ids[:4]], torch.stack([dy[0], dy[1] + dy[4], dy[2], dy[3]]))
    table[ids] = 0
    assert not table.any()
