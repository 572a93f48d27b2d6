"""Residual layer norm, forward and backward, against the 64-bit definitions."""
import math

import pytest
import torch

import model_ref as ref
import sharded_mixed_precision_step_amd as zs
from gpu_util import device

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
U = ref.U
EPS = 1e-5


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(seed, *shape, dtype=F32):
    return torch.randn(*shape, generator=_gen(seed), device="cuda").to(dtype)


SHAPES = [(1, 1), (3, 7), (70, 64), (35, 127), (5, 128), (4, 129), (9, 250), (7, 500), (6, 513),
          (9, 1000), (5, 1025), (17, 2048), (16, 4096), (3, 5001), (4, 8192), (2, 12000),
          (2, 16385), (2, 33000), (1, 65536)]
TYPES = [(F16, F16), (BF16, BF16), (F16, F32), (BF16, F32), (F32, F32), (F32, F16), (F16, None),
         (F32, None)]


@pytest.mark.parametrize("x_dtype,r_dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm_is_the_definition(rows, cols, x_dtype, r_dtype):
    dev = device()
    print(f"case: layernorm {rows}x{cols} {x_dtype} {r_dtype}", flush=True)
    x = (_randn(1, rows, cols) + 0.5).to(x_dtype)
    res = None if r_dtype is None else _randn(2, rows, cols, dtype=r_dtype)
    wt = F16 if x_dtype != BF16 else BF16
    w, b = (1 + 0.1 * _randn(3, cols)).to(wt), (0.1 * _randn(4, cols)).to(wt)
    h = None if res is None else torch.empty_like(res)
    y = torch.empty(rows, cols, dtype=x_dtype, device=dev)
    mean, rstd = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
    q, s = zs.q8_empty(rows, cols, E4)
    zs.zero_layernorm(x, w, b, EPS, residual=res, h=h, y=y, q=q, s=s, mean=mean, rstd=rstd)
    wh, wm, wr, wy = ref.layernorm(x, res, w, b, EPS)
    tm, tr, ty = ref.layernorm_bounds(x, res, w, b, EPS)
    if h is not None:
        ref.assert_close(h, wh, ref.half_step(r_dtype, wh) + U * wh.abs(), "h")
    ref.assert_close(mean, wm, tm, "mean")
    ref.assert_close(rstd, wr, tr, "rstd")
    ref.assert_close(y, wy, ref.half_step(x_dtype, wy) + ty, "y")
    ref.check_q8(q, s, wy, ty, E4, "q")


@pytest.mark.parametrize("fp8", [E4, E5])
@pytest.mark.parametrize("rows,cols,w_dtype", [(33, 384, F32), (8, 4100, BF16), (3, 77, F16),
                                               (21, 100, F32)])
def test_outputs_alone_and_strided(rows, cols, w_dtype, fp8):
    """Each output by itself has the bits it has among the others; strided, oddly
    aligned rows; no bias; what lies beside an output stays."""
    dev = device()
    base = _randn(5, rows + 1, cols + 21, dtype=F16)
    rbase = _randn(6, rows + 1, cols + 5, dtype=BF16)
    x, res = base[:rows, 7:7 + cols], rbase[1:, 3:3 + cols]
    w = (1 + 0.1 * _randn(7, cols)).to(w_dtype)
    hb, yb = torch.full((rows, cols + 9), 7.0, device=dev, dtype=BF16), \
        torch.full((rows, cols + 3), 7.0, device=dev, dtype=F32)
    h, y = hb[:, 1:1 + cols], yb[:, :cols]
    mean, rstd = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
    q, s = zs.q8_empty(rows, cols, fp8)
    call = lambda **kw: zs.zero_layernorm(x, w, None, EPS, residual=res, **kw)  # noqa: E731
    call(h=h, y=y, q=q, s=s, mean=mean, rstd=rstd)
    wh, wm, wr, wy = ref.layernorm(x, res, w, None, EPS)
    tm, tr, ty = ref.layernorm_bounds(x, res, w, None, EPS)
    ref.assert_close(h, wh, ref.half_step(BF16, wh) + U * wh.abs(), "h")
    ref.assert_close(mean, wm, tm, "mean")
    ref.assert_close(rstd, wr, tr, "rstd")
    ref.assert_close(y, wy, ref.half_step(F32, wy) + ty, "y")
    ref.check_q8(q, s, wy, ty, fp8, "q")
    assert (hb[:, 0] == 7).all() and (hb[:, 1 + cols:] == 7).all() and (yb[:, cols:] == 7).all()
    h2, y2, mean2, rstd2 = torch.empty_like(h), torch.empty_like(y), torch.empty_like(mean), \
        torch.empty_like(rstd)
    q2, s2 = zs.q8_empty(rows, cols, fp8)
    call(h=h2)
    call(y=y2)
    call(q=q2, s=s2)
    call(mean=mean2)
    call(rstd=rstd2)
    assert torch.equal(h, h2) and torch.equal(y, y2)
    assert torch.equal(mean, mean2) and torch.equal(rstd, rstd2)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8))
    assert torch.equal(s.view(torch.uint8), s2.view(torch.uint8))


@pytest.mark.parametrize("cols", [100, 1500, 1501])
def test_in_place(cols):
    device()
    x, res = _randn(1, 9, cols, dtype=F16), _randn(2, 9, cols, dtype=F16)
    w, b = _randn(3, cols, dtype=F16), _randn(4, cols, dtype=F16)
    h, y = torch.empty_like(x), torch.empty_like(x)
    zs.zero_layernorm(x, w, b, EPS, residual=res, h=h, y=y)
    x1, r1 = x.clone(), res.clone()
    zs.zero_layernorm(x1, w, b, EPS, residual=r1, h=r1, y=x1)
    assert torch.equal(r1, h) and torch.equal(x1, y)
    x2, y2 = x.clone(), torch.empty_like(x)
    zs.zero_layernorm(x2, w, b, EPS, residual=res, h=x2, y=y2)
    assert torch.equal(x2, h) and torch.equal(y2, y)


@pytest.mark.parametrize("cols", [90, 200, 3000])
def test_rows_far_from_zero_constant_and_non_finite(cols):
    """A mean of 2000 beside a spread of 1 keeps its variance; a constant row gives
    the bias; a NaN or inf spoils its own row, blocks and padding scales only."""
    dev = device()
    x = _randn(1, 6, cols)
    x[0] += 2000.0
    x[1] = 3.0
    x[2, 5] = math.nan
    x[3, cols - 1] = math.inf
    w, b = torch.ones(cols, device=dev), 0.5 * torch.ones(cols, device=dev)
    y = torch.empty_like(x)
    q, s = zs.q8_empty(6, cols)
    mean, rstd = torch.empty(6, device=dev), torch.empty(6, device=dev)
    zs.zero_layernorm(x, w, b, EPS, y=y, q=q, s=s, mean=mean, rstd=rstd)
    ok = [0, 1, 4, 5]
    _, wm, wr, wy = ref.layernorm(x[ok], None, w, b, EPS)
    tm, tr, ty = ref.layernorm_bounds(x[ok], None, w, b, EPS)
    ref.assert_close(mean[ok], wm, tm, "mean")
    ref.assert_close(rstd[ok], wr, tr, "rstd")
    ref.assert_close(y[ok], wy, ty + ref.half_step(F32, wy), "y")
    assert torch.isnan(y[2:4]).all() and torch.isnan(mean[2]) and mean[3] == math.inf
    blocks = -(-cols // 128)
    byte = s.view(torch.uint8)
    assert (byte[2:4, :blocks] == 255).all() and (byte[:, blocks:] == 127).all()
    assert torch.isnan(q[2:4].float()).all() and torch.isfinite(q[ok].float()).all()
    assert (q[ok, cols:].float() == 0).all()


BACK = [(1, 1), (2, 9), (200, 64), (3, 128), (70, 250), (70, 300), (6, 513), (1500, 130),
        (33, 1025), (40, 4096), (1003, 1001), (5, 5001), (3, 9000), (3, 16385), (2, 40000)]


@pytest.mark.parametrize("dt,hdt,rdt", [(F16, F32, F16), (BF16, BF16, BF16), (F16, F16, None),
                                        (F32, F32, F32), (F32, F16, None), (BF16, F32, F32)])
@pytest.mark.parametrize("rows,cols", BACK)
def test_backward_is_the_formula(rows, cols, dt, hdt, rdt):
    dev = device()
    print(f"case: layernorm backward {rows}x{cols} {dt} {hdt} {rdt}", flush=True)
    h = (0.3 + 2 * _randn(1, rows, cols)).to(hdt)
    w = (1 + 0.1 * _randn(2, cols)).to(F16)
    _, mean, rstd, _ = ref.layernorm(h, None, w, None, EPS)
    mean, rstd = mean.float(), rstd.float()
    dy = _randn(3, rows, cols, dtype=dt)
    dres = None if rdt is None else _randn(4, rows, cols, dtype=rdt)
    dx = torch.empty_like(dy)
    dw, db = torch.empty(cols, device=dev), torch.empty(cols, device=dev)
    ws = torch.empty(zs.zero_layernorm_backward_workspace(rows, cols), dtype=torch.uint8, device=dev)
    zs.zero_layernorm_backward(dy, h, w, mean, rstd, dx, dw, db, ws, dres=dres)
    wx, ww, wb, tx, tw, tb = ref.layernorm_backward(dy, h, w, mean, rstd, dres)
    ref.assert_close(dx, wx, ref.half_step(dt, wx) + tx, "dx")
    ref.assert_close(dw, ww, ref.half_step(F32, ww) + tw, "dw")
    ref.assert_close(db, wb, ref.half_step(F32, wb) + tb, "db")
    # 16-bit sums are those rounded once; each alone has the same bits; none leaves
    # dx as it is
    dx2, dw2, db2 = torch.empty_like(dx), dw.half(), db.half()
    zs.zero_layernorm_backward(dy, h, w, mean, rstd, dx2, dw2.zero_(), db2.zero_(), ws, dres=dres)
    assert torch.equal(dw2, dw.half()) and torch.equal(db2, db.half()) and torch.equal(dx, dx2)
    one = torch.empty_like(dw)
    zs.zero_layernorm_backward(dy, h, w, mean, rstd, dx2.zero_(), one, None, ws, dres=dres)
    assert torch.equal(one, dw) and torch.equal(dx, dx2)
    zs.zero_layernorm_backward(dy, h, w, mean, rstd, dx2.zero_(), None, one, ws, dres=dres)
    assert torch.equal(one, db) and torch.equal(dx, dx2)
    zs.zero_layernorm_backward(dy, h, w, mean, rstd, dx2.zero_(), None, None, None, dres=dres)
    assert torch.equal(dx, dx2)


@pytest.mark.parametrize("cols", [60, 700, 701, 9001, 17001])
def test_backward_in_place_and_strided(cols):
    dev = device()
    rows = 37
    base = _randn(1, rows, cols + 13, dtype=F16)
    dy = base[:, 5:5 + cols]
    h, w = _randn(2, rows, cols, dtype=F16), _randn(3, cols, dtype=F16)
    _, mean, rstd, _ = ref.layernorm(h, None, w, None, EPS)
    mean, rstd = mean.float(), rstd.float()
    dres = _randn(4, rows, cols, dtype=F16)
    ws = torch.empty(zs.zero_layernorm_backward_workspace(rows, cols), dtype=torch.uint8, device=dev)
    dx, dw, db = torch.empty_like(h), torch.empty_like(w), torch.empty_like(w)
    zs.zero_layernorm_backward(dy, h, w, mean, rstd, dx, dw, db, ws, dres=dres)
    for place in range(3):
        bases = base.clone()
        t = [bases[:, 5:5 + cols], h.clone(), dres.clone()]
        dw2, db2 = torch.empty_like(w), torch.empty_like(w)
        zs.zero_layernorm_backward(t[0], t[1], w, mean, rstd, t[place], dw2, db2, ws, dres=t[2])
        assert torch.equal(t[place], dx) and torch.equal(dw2, dw) and torch.equal(db2, db), place
        assert torch.equal(bases[:, :5], base[:, :5])
        assert torch.equal(bases[:, 5 + cols:], base[:, 5 + cols:])


def test_backward_of_no_rows_and_non_finite_rows():
    dev = device()
    w = torch.ones(50, device=dev)
    dw, db = torch.full((50,), 7.0, device=dev), torch.full((50,), 7.0, device=dev)
    none = torch.empty(0, 50, device=dev)
    zs.zero_layernorm_backward(none, none, w, none[:, 0].contiguous(), none[:, 0].contiguous(),
                               none, dw, db, torch.empty(0, dtype=torch.uint8, device=dev))
    assert (dw == 0).all() and (db == 0).all()
    dy, h = _randn(1, 5, 50), _randn(2, 5, 50)
    dy[2, 3] = math.inf
    _, mean, rstd, _ = ref.layernorm(h, None, w, None, EPS)
    dx = torch.empty_like(dy)
    ws = torch.empty(zs.zero_layernorm_backward_workspace(5, 50), dtype=torch.uint8, device=dev)
    zs.zero_layernorm_backward(dy, h, w, mean.float(), rstd.float(), dx, dw, db, ws)
    # g - inf - xhat * (+-inf): -inf where the two agree in sign, else NaN
    assert not torch.isfinite(dx[2]).any() and torch.isfinite(dx[[0, 1, 3, 4]]).all()
    assert not torch.isfinite(db[3]) and torch.isfinite(db[:3]).all()


@pytest.mark.parametrize("cols", [40, 333])
def test_backward_is_the_derivative(cols):
    """Against central differences of the 64-bit forward along random directions of
    x, weight and bias: the third derivative's share is step^2 of the whole."""
    dev = device()
    rows = 20
    x, w, b, dy = _randn(1, rows, cols), 1 + 0.1 * _randn(2, cols), _randn(3, cols), \
        _randn(4, rows, cols)
    _, mean, rstd, _ = ref.layernorm(x, None, w, b, EPS)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    ws = torch.empty(zs.zero_layernorm_backward_workspace(rows, cols), dtype=torch.uint8, device=dev)
    zs.zero_layernorm_backward(dy, x, w, mean.float(), rstd.float(), dx, dw, db, ws)
    vx, vw, vb = _randn(5, rows, cols).double(), _randn(6, cols).double(), _randn(7, cols).double()

    def f(t):
        return (ref.layernorm(x.double() + t * vx, None, w.double() + t * vw, b.double() + t * vb,
                              EPS)[3] * dy.double()).sum()

    step = 1e-4
    slope = (f(step) - f(-step)) / (2 * step)
    got = (dx.double() * vx).sum() + (dw.double() * vw).sum() + (db.double() * vb).sum()
    size = (dx.double() * vx).abs().sum() + (dw.double() * vw).abs().sum() \
        + (db.double() * vb).abs().sum()
    assert abs(slope - got) <= 1e-5 * size


def test_in_a_graph_and_on_another_stream():
    dev = device()
    rows, cols = 300, 700
    x, w, b, dy = _randn(1, rows, cols, dtype=F16), _randn(2, cols), _randn(3, cols), \
        _randn(4, rows, cols, dtype=F16)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
    dw, db = torch.empty_like(w), torch.empty_like(w)
    ws = torch.empty(zs.zero_layernorm_backward_workspace(rows, cols), dtype=torch.uint8, device=dev)

    def call():
        zs.zero_layernorm(x, w, b, EPS, y=y, mean=mean, rstd=rstd)
        zs.zero_layernorm_backward(dy, x, w, mean, rstd, dx, dw, db, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(3):
        x.copy_(_randn(10 + k, rows, cols))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, dx, dw, db)]
        call()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, (y, dx, dw, db)))
