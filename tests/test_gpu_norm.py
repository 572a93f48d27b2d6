"""Residual RMS norm, forward and backward, against the 64-bit definitions."""
import math

import pytest
import torch

import sharded_mixed_precision_step_amd as zs
import train_ref as ref
from gpu_util import device

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
U = ref.U
EPS = 1e-5
# a row's sum of squares: at most 64 terms per lane, 6 wave steps, 16 waves; half
# of that on its root, and 8 for the rest of the formula
NORM = 64 * U


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(seed, *shape, dtype=F32):
    return torch.randn(*shape, generator=_gen(seed), device="cuda").to(dtype)


SHAPES = [(1, 1), (3, 7), (5, 128), (4, 129), (7, 500), (6, 513), (9, 1000), (5, 1025), (17, 2048),
          (16, 4096), (3, 5001), (4, 8192), (2, 12000), (2, 16385), (2, 33000), (1, 65536)]
TYPES = [(F16, F16), (BF16, BF16), (F16, F32), (BF16, F32), (F32, F32), (F32, F16), (F16, None),
         (F32, None)]


@pytest.mark.parametrize("x_dtype,r_dtype", TYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm_is_the_definition(rows, cols, x_dtype, r_dtype):
    dev = device()
    print(f"case: norm {rows}x{cols} {x_dtype} {r_dtype}", flush=True)
    x = _randn(1, rows, cols, dtype=x_dtype)
    res = None if r_dtype is None else _randn(2, rows, cols, dtype=r_dtype)
    w = (1 + 0.1 * _randn(3, cols)).to(F16 if x_dtype != BF16 else BF16)
    h = None if res is None else torch.empty_like(res)
    y = torch.empty(rows, cols, dtype=x_dtype, device=dev)
    rstd = torch.empty(rows, device=dev)
    q, s = zs.q8_empty(rows, cols, E4)
    zs.zero_rmsnorm(x, w, EPS, residual=res, h=h, y=y, q=q, s=s, rstd=rstd)
    wh, wr, wy = ref.rmsnorm(x, res, w, EPS)
    if h is not None:
        ref.assert_close(h, wh, ref.half_step(r_dtype, wh) + U * wh.abs(), "h")
    ref.assert_close(rstd, wr, NORM * wr, "rstd")
    ref.assert_close(y, wy, ref.half_step(x_dtype, wy) + NORM * wy.abs(), "y")
    _check_q(q, s, wy, E4)


def _check_q(q, s, wy, fp8):
    """Values: half a step of the 8-bit type at the block's scale.  Scales: the
    definition's, or its neighbour where amax is within NORM of the border."""
    rows, cols = wy.shape
    blocks = q.shape[1] // 128
    pad = torch.zeros(rows, q.shape[1], dtype=torch.float64, device=wy.device)
    pad[:, :cols] = wy
    amax = pad.view(rows, blocks, 128).abs().amax(-1)
    e = s.view(torch.uint8).to(torch.int64) - 127
    assert (e[:, blocks:] == 0).all()
    lo, hi = (ref.scale_exponent(amax * (1 + d), fp8) for d in (-NORM, NORM))
    assert ((e[:, :blocks] == lo) | (e[:, :blocks] == hi)).all()
    scale = ref.pow2(e[:, :blocks]).repeat_interleave(128, 1)
    got = q.to(F32).double() * scale
    assert (got[:, cols:] == 0).all()
    tol = ref.half_step(fp8, pad / scale) * scale + NORM * pad.abs()
    ref.assert_close(got, pad, tol, "q")


@pytest.mark.parametrize("fp8", [E4, E5])
@pytest.mark.parametrize("rows,cols,w_dtype", [(33, 384, F32), (8, 4100, BF16), (1, 77, F16)])
def test_norm_outputs_alone_and_strided(rows, cols, w_dtype, fp8):
    """Each output by itself has the bits it has among the others; strided,
    oddly aligned rows; what lies beside an output stays."""
    dev = device()
    base = _randn(5, rows + 1, cols + 21, dtype=F16)
    rbase = _randn(6, rows + 1, cols + 5, dtype=BF16)
    x, res = base[:rows, 7:7 + cols], rbase[1:, 3:3 + cols]
    w = (1 + 0.1 * _randn(7, cols)).to(w_dtype)
    hb, yb = torch.full((rows, cols + 9), 7.0, device=dev, dtype=BF16), \
        torch.full((rows, cols + 3), 7.0, device=dev, dtype=F32)
    h, y = hb[:, 1:1 + cols], yb[:, :cols]
    rstd = torch.empty(rows, device=dev)
    q, s = zs.q8_empty(rows, cols, fp8)
    zs.zero_rmsnorm(x, w, EPS, residual=res, h=h, y=y, q=q, s=s, rstd=rstd)
    wh, wr, wy = ref.rmsnorm(x, res, w, EPS)
    ref.assert_close(h, wh, ref.half_step(BF16, wh) + U * wh.abs(), "h")
    ref.assert_close(y, wy, ref.half_step(F32, wy) + NORM * wy.abs(), "y")
    _check_q(q, s, wy, fp8)
    assert (hb[:, 0] == 7).all() and (hb[:, 1 + cols:] == 7).all() and (yb[:, cols:] == 7).all()
    h2, y2, rstd2 = torch.empty_like(h), torch.empty_like(y), torch.empty_like(rstd)
    q2, s2 = zs.q8_empty(rows, cols, fp8)
    zs.zero_rmsnorm(x, w, EPS, residual=res, h=h2)
    zs.zero_rmsnorm(x, w, EPS, residual=res, y=y2)
    zs.zero_rmsnorm(x, w, EPS, residual=res, q=q2, s=s2)
    zs.zero_rmsnorm(x, w, EPS, residual=res, rstd=rstd2)
    assert torch.equal(h, h2) and torch.equal(y, y2) and torch.equal(rstd, rstd2)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8))
    assert torch.equal(s.view(torch.uint8), s2.view(torch.uint8))


def test_norm_in_place():
    x, res, w = _randn(1, 9, 1500, dtype=F16), _randn(2, 9, 1500, dtype=F16), \
        _randn(3, 1500, dtype=F16)
    h, y = torch.empty_like(x), torch.empty_like(x)
    zs.zero_rmsnorm(x, w, EPS, residual=res, h=h, y=y)
    x1, r1 = x.clone(), res.clone()
    zs.zero_rmsnorm(x1, w, EPS, residual=r1, h=r1, y=x1)   # both in place
    assert torch.equal(r1, h) and torch.equal(x1, y)
    x2 = x.clone()
    y2 = torch.empty_like(x)
    zs.zero_rmsnorm(x2, w, EPS, residual=res, h=x2, y=y2)  # h over x
    assert torch.equal(x2, h) and torch.equal(y2, y)


def test_norm_rows_of_zeros_and_non_finite_rows():
    """A row of zeros stays zero (eps > 0); a NaN or inf row is NaN where the
    formula is, and only that row; its 8-bit blocks are NaN, the zeros behind
    the row's end are not."""
    dev = device()
    x = _randn(1, 6, 200)
    x[1] = 0
    x[2, 5] = math.nan
    x[3, 150] = math.inf
    w = torch.ones(200, device=dev)
    y = torch.empty_like(x)
    q, s = zs.q8_empty(6, 200)
    zs.zero_rmsnorm(x, w, EPS, y=y, q=q, s=s)
    _, _, wy = ref.rmsnorm(x, None, w, EPS)
    ref.assert_close(y, wy, NORM * wy.abs().nan_to_num(0) + ref.half_step(F32, wy.nan_to_num(0)),
                     "y")
    assert torch.isnan(y[2]).all() and torch.isnan(y[3, 150]) and (y[3, :150] == 0).all()
    byte = s.view(torch.uint8)
    assert (byte[2, :2] == 255).all() and byte[3].tolist() == [127, 255, 127, 127]
    assert torch.isnan(q[2].float()).all() and (q[1].float() == 0).all()
    assert torch.isfinite(q[[0, 1, 4, 5]].float()).all()


BACK = [(1, 1), (2, 9), (3, 128), (70, 300), (6, 513), (1500, 130), (33, 1025), (40, 4096),
        (1003, 1001), (5, 5001), (3, 16385), (2, 40000)]


@pytest.mark.parametrize("dt,hdt,rdt", [(F16, F32, F16), (BF16, BF16, BF16), (F16, F16, None),
                                        (F32, F32, F32), (F32, F16, None), (BF16, F32, F32)])
@pytest.mark.parametrize("rows,cols", BACK)
def test_backward_is_the_formula(rows, cols, dt, hdt, rdt):
    dev = device()
    print(f"case: norm backward {rows}x{cols} {dt} {hdt} {rdt}", flush=True)
    h = (2 * _randn(1, rows, cols)).to(hdt)
    w = (1 + 0.1 * _randn(2, cols)).to(F16)
    rstd = (1 / torch.sqrt((h.double() ** 2).mean(-1) + EPS)).float()
    dy = _randn(3, rows, cols, dtype=dt)
    dres = None if rdt is None else _randn(4, rows, cols, dtype=rdt)
    dx, dw = torch.empty_like(dy), torch.empty(cols, dtype=F32, device=dev)
    ws = torch.empty(zs.zero_rmsnorm_backward_workspace(rows, cols), dtype=torch.uint8, device=dev)
    zs.zero_rmsnorm_backward(dy, h, w, rstd, dx, dw, ws, dres=dres)
    wx, ww = ref.rmsnorm_backward(dy, h, w, rstd, dres)
    _assert_backward(dx, dw, wx, ww, dy, h, w, rstd, dres)
    # 16-bit dw is that sum rounded once; no dw leaves dx as it is
    dx2, dw2 = torch.empty_like(dx), torch.empty(cols, dtype=F16, device=dev)
    zs.zero_rmsnorm_backward(dy, h, w, rstd, dx2, dw2, ws, dres=dres)
    assert torch.equal(dw2, dw.half()) and torch.equal(dx, dx2)
    zs.zero_rmsnorm_backward(dy, h, w, rstd, dx2.zero_(), None, None, dres=dres)
    assert torch.equal(dx, dx2)


def _assert_backward(dx, dw, wx, ww, dy, h, w, rstd, dres):
    rows = dy.shape[0]
    g = dy.double() * w.double()
    xhat = h.double() * rstd.double()[:, None]
    r = rstd.double()[:, None]
    mag = r * (g.abs() + xhat.abs() * (g * xhat).abs().mean(-1, keepdim=True))
    if dres is not None:
        mag = mag + dres.double().abs()
    # the dot product: 64 terms per lane, 22 joins, 4 products; 10 after it
    ref.assert_close(dx, wx, ref.half_step(dx.dtype, wx) + 100 * U * mag, "dx")
    # dw: a workgroup's rows one after another (at least 128 workgroups share
    # them where there are that many), then at most 1,024 partial rows in 16
    # groups, then the groups
    n = -(-rows // 128) + 64 + 16 + 2
    ref.assert_close(dw, ww, ref.half_step(dw.dtype, ww)
                     + n * U * (dy.double() * xhat).abs().sum(0), "dw")


def test_backward_in_place_and_strided():
    dev = device()
    rows, cols = 37, 700
    base = _randn(1, rows, cols + 13, dtype=F16)
    dy = base[:, 5:5 + cols]
    h, w = _randn(2, rows, cols, dtype=F16), _randn(3, cols, dtype=F16)
    rstd = (1 / torch.sqrt((h.double() ** 2).mean(-1) + EPS)).float()
    dres = _randn(4, rows, cols, dtype=F16)
    ws = torch.empty(zs.zero_rmsnorm_backward_workspace(rows, cols), dtype=torch.uint8, device=dev)
    dx, dw = torch.empty(rows, cols, dtype=F16, device=dev), torch.empty(cols, dtype=F16,
                                                                         device=dev)
    zs.zero_rmsnorm_backward(dy, h, w, rstd, dx, dw, ws, dres=dres)
    wx, ww = ref.rmsnorm_backward(dy, h, w, rstd, dres)
    _assert_backward(dx, dw, wx, ww, dy, h, w, rstd, dres)
    for which in ("dres", "h", "dy"):
        args = dict(dy=dy.clone() if which != "dy" else base.clone()[:, 5:5 + cols],
                    h=h.clone(), dres=dres.clone())
        out = args[which]
        zs.zero_rmsnorm_backward(args["dy"], args["h"], w, rstd, out, dw, ws, dres=args["dres"])
        assert torch.equal(out, dx), which


def test_backward_without_rows_clears_dw():
    dev = device()
    dw = torch.ones(100, device=dev)
    e = torch.empty(0, 100, device=dev)
    zs.zero_rmsnorm_backward(e, e, torch.ones(100, device=dev), torch.empty(0, device=dev), e, dw,
                             torch.empty(0, dtype=torch.uint8, device=dev))
    assert (dw == 0).all()


def test_gradients_against_differences():
    """The gradients kernels give for a random direction, against central
    differences of the 64-bit forward along it.  The difference's own error is
    O(step^2); the kernel's is fp32."""
    dev = device()
    rows, cols = 12, 333
    x, res, w = _randn(1, rows, cols), _randn(2, rows, cols), 1 + 0.1 * _randn(3, cols)
    up, dh = _randn(4, rows, cols), _randn(5, rows, cols)
    h, rstd, y = torch.empty_like(res), torch.empty(rows, device=dev), torch.empty_like(x)
    zs.zero_rmsnorm(x, w, EPS, residual=res, h=h, y=y, rstd=rstd)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(zs.zero_rmsnorm_backward_workspace(rows, cols), dtype=torch.uint8, device=dev)
    zs.zero_rmsnorm_backward(up, h, w, rstd, dx, dw, ws, dres=dh)
    vx, vw = _randn(6, rows, cols).double(), _randn(7, cols).double()

    def value(t):
        hh, _, yy = ref.rmsnorm(x.double() + t * vx, res, w.double() + t * vw, EPS)
        return (yy * up.double()).sum() + (hh * dh.double()).sum()

    step = 1e-5
    want = (value(step) - value(-step)) / (2 * step)
    got = (dx.double() * vx).sum() + (dw.double() * vw).sum()
    size = (dx.double() * vx).abs().sum() + (dw.double() * vw).abs().sum()
    assert abs(float(got - want)) <= 1e-6 * float(size)


def test_norm_calls_in_a_graph_and_on_another_stream():
    dev = device()
    rows, cols = 65, 1100
    x, res, w = _randn(1, rows, cols, dtype=F16), _randn(2, rows, cols), _randn(3, cols, dtype=F16)
    h, rstd = torch.empty_like(res), torch.empty(rows, device=dev)
    q, s = zs.q8_empty(rows, cols)
    dy = _randn(4, rows, cols, dtype=F16)
    dx, dw = torch.empty_like(dy), torch.empty_like(w)
    ws = torch.empty(zs.zero_rmsnorm_backward_workspace(rows, cols), dtype=torch.uint8, device=dev)

    def both(stream=None):
        zs.zero_rmsnorm(x, w, EPS, residual=res, h=h, q=q, s=s, rstd=rstd, stream=stream)
        zs.zero_rmsnorm_backward(dy, h, w, rstd, dx, dw, ws, stream=stream)

    outs = (h, rstd, q.view(torch.uint8), s.view(torch.uint8), dx, dw)
    both()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    both(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for k in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), k
        both()
        torch.cuda.synchronize()


@pytest.mark.parametrize("rows,cols", [(8200, 1001), (4100, 7), (4100, 15), (2100, 2047),
                                       (2100, 1024)])
def test_backward_of_many_narrow_rows(rows, cols):
    """More partial rows of dw than CUs; rows with and without a last eight."""
    dev = device()
    dy, h = _randn(1, rows, cols, dtype=BF16), _randn(2, rows, cols, dtype=F16)
    w, rstd = _randn(3, cols, dtype=F16), 1 + 0.1 * _randn(4, rows)
    dx, dw = torch.empty_like(dy), torch.empty(cols, device=dev)
    ws = torch.empty(zs.zero_rmsnorm_backward_workspace(rows, cols), dtype=torch.uint8, device=dev)
    zs.zero_rmsnorm_backward(dy, h, w, rstd, dx, dw, ws)
    wx, ww = ref.rmsnorm_backward(dy, h, w, rstd, None)
    _assert_backward(dx, dw, wx, ww, dy, h, w, rstd, None)


@pytest.mark.parametrize("rows,cols", [(600, 5), (600, 9), (300, 5001), (260, 8185), (20, 9003),
                                       (3, 17001)])
def test_backward_in_place_where_rows_end_inside_a_pack(rows, cols):
    """A row's last pack repeats elements of the one before: in place too the
    same bits, and an inf among them stays in its row and column."""
    dev = device()
    dy, h, dres = (_randn(k, rows, cols, dtype=F16) for k in (1, 2, 3))
    w, rstd = _randn(4, cols, dtype=F16), 1 + 0.1 * _randn(5, rows)
    ws = torch.empty(zs.zero_rmsnorm_backward_workspace(rows, cols), dtype=torch.uint8, device=dev)
    dx, dw, dw2 = torch.empty_like(dy), torch.empty_like(w), torch.empty_like(w)
    zs.zero_rmsnorm_backward(dy, h, w, rstd, dx, dw, ws, dres=dres)
    wx, ww = ref.rmsnorm_backward(dy, h, w, rstd, dres)
    _assert_backward(dx, dw, wx, ww, dy, h, w, rstd, dres)
    for which in ("dres", "h", "dy"):
        args = dict(dy=dy.clone(), h=h.clone(), dres=dres.clone())
        out = args[which]
        zs.zero_rmsnorm_backward(args["dy"], args["h"], w, rstd, out, dw2, ws, dres=args["dres"])
        assert torch.equal(out, dx) and torch.equal(dw, dw2), which
    bad = dy.clone()
    bad[1, cols - 4] = math.inf
    out = torch.empty_like(dx)
    zs.zero_rmsnorm_backward(bad, h, w, rstd, out, dw2, ws, dres=dres)
    others = torch.arange(rows, device=dev) != 1
    assert torch.equal(out[others], dx[others]) and not torch.isfinite(out[1]).any()
    ok = torch.arange(cols, device=dev) != cols - 4
    assert torch.equal(dw2[ok], dw[ok]) and not torch.isfinite(dw2[cols - 4])


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,cols", [(600, 9), (300, 513), (300, 1028), (200, 4101), (40, 9001),
                                       (9, 16383), (5, 16387)])
def test_norm_in_place_where_rows_end_inside_a_pack(rows, cols, dtype):
    """h in the residual's place and in x's, y in x's: the bits of a call with
    arrays of its own, which is checked against the definition."""
    dev = device()
    x, res = _randn(1, rows, cols, dtype=dtype), _randn(2, rows, cols, dtype=dtype)
    w = _randn(3, cols, dtype=F16)

    def call(x, res, h, y):
        q, s = zs.q8_empty(rows, cols)
        zs.zero_rmsnorm(x, w, EPS, residual=res, h=h, y=y, q=q, s=s)
        return q.view(torch.uint8), s.view(torch.uint8)

    h, y = torch.empty_like(x), torch.empty_like(x)
    q, s = call(x, res, h, y)
    wh, _, wy = ref.rmsnorm(x, res, w, EPS)
    ref.assert_close(h, wh, ref.half_step(dtype, wh) + U * wh.abs(), "h")
    # the mean of squares: 24 terms a lane and 22 joins; sqrt, division and two products
    ref.assert_close(y, wy, ref.half_step(dtype, wy) + 100 * U * wy.abs(), "y")
    for h_in, y_in in (("res", None), ("x", None), ("res", "x"), (None, "x")):
        a = dict(x=x.clone(), res=res.clone())
        own_h, own_y = torch.empty_like(x), torch.empty_like(x)
        got_h, got_y = a.get(h_in, own_h), a.get(y_in, own_y)
        got = call(a["x"], a["res"], got_h, got_y)
        assert torch.equal(got_h, h) and torch.equal(got_y, y), (h_in, y_in)
        assert torch.equal(got[0], q) and torch.equal(got[1], s), (h_in, y_in)


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("rows,cols", [(700, 513), (900, 1025), (600, 1543), (500, 2561), (300, 8191),
                                       (300, 9217), (280, 12289), (260, 16383)])
def test_backward_in_place_where_the_last_pack_is_another_waves(rows, cols, dtype):
    """The row's last eight elements belong to a wave whose neighbour writes some of
    them: in place the bits of a call with arrays of its own, which is checked
    against the definition.  (8191 and 16383: a lane beside, the same wave.)"""
    dev = device()
    print(f"case: norm backward in place {rows}x{cols} {dtype}", flush=True)
    dy, h, dres = (_randn(k, rows, cols, dtype=dtype) for k in (1, 2, 3))
    w, rstd = _randn(4, cols, dtype=F16), 1 + 0.1 * _randn(5, rows)
    ws = torch.empty(zs.zero_rmsnorm_backward_workspace(rows, cols), dtype=torch.uint8, device=dev)
    dx, dw, dw2 = torch.empty_like(dy), torch.empty_like(w), torch.empty_like(w)
    zs.zero_rmsnorm_backward(dy, h, w, rstd, dx, dw, ws, dres=dres)
    wx, ww = ref.rmsnorm_backward(dy, h, w, rstd, dres)
    _assert_backward(dx, dw, wx, ww, dy, h, w, rstd, dres)
    for turn in range(4):
        for which in ("dres", "h", "dy"):
            args = dict(dy=dy.clone(), h=h.clone(), dres=dres.clone())
            out = args[which]
            zs.zero_rmsnorm_backward(args["dy"], args["h"], w, rstd, out, dw2, ws,
                                     dres=args["dres"])
            assert torch.equal(out, dx) and torch.equal(dw, dw2), (which, turn)
