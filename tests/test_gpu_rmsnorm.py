"""GPU tests of the residual addition with RMS norm and its gradient
(sn_add_rmsnorm, sn_add_rmsnorm_backward) against the definition in 64 bits.

Tolerances, per element: h is one fp32 addition and one rounding.  A row's sum
of squares (or of dy w h) has at most 64 roundings on any path (32 in a
lane, 5 between lanes, 16 between warps, the rest), so with rsqrt's own (2 ulp)
the fp32 part of y is within (64 / 2 + 8) 2^-24 of it, and of dx within 80
2^-24 of the magnitudes that it sums; then comes one rounding to the output's
type.  e4m3 has 3 bits of mantissa and steps of 2^-9 below 2^-6: half a step is
2^-4 of the value or 2^-10 of the scale, plus the fp32 part."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
U = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
FP = 2.0 ** -24


@pytest.fixture(scope="module")
def sr():
    import scan_runtime_gb300 as sr
    sr.build()
    return sr


@pytest.fixture()
def ctx(sr):
    c = sr.Context(0)
    yield c
    torch.cuda.synchronize()
    assert c.last_error() == sr.SN_OK
    c.close()


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _normal(g, *shape, dtype=F32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _ref(x, r, w, eps):
    h = x.double() + (0 if r is None else r.double())
    rstd = 1.0 / (h.square().mean(-1) + eps).sqrt()
    y = h * rstd[..., None] * (1.0 if w is None else w.double())
    return h, rstd, y


def _near(got, ref, rel):
    return bool(((got.double() - ref).abs() <= rel * ref.abs() * 1.001).all())


SHAPES = [(1, 1), (1, 2048), (3, 31), (5, 128), (7, 129), (300, 511), (17, 1021), (9, 1536), (2, 4096), (3, 4104),
          (5, 9001), (2, 16384), (1500, 64), (4000, 256)]


@pytest.mark.parametrize("dt,ydt", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("R,D", SHAPES)
def test_forward(ctx, dt, ydt, R, D):
    g = _gen(R + D)
    x, r, w = _normal(g, R, D, dtype=dt), _normal(g, R, D, dtype=dt) * 3, 1 + 0.2 * _normal(g, D)
    y, scales, h, rstd = ctx.add_rmsnorm(x, r, w, eps=1e-6, dtype=ydt, rstd=True)
    rh, rr, ry = _ref(x, r, w, 1e-6)
    assert scales is None and y.dtype == ydt and h.dtype == dt
    assert _near(h, rh, U[dt] + (FP if dt == BF16 else 0))
    assert _near(rstd, rr, 40 * FP)
    assert _near(y, ry, 42 * FP + U[ydt])
    # without the residual, the weight and the optional outputs
    y, _, h, rstd = ctx.add_rmsnorm(x, eps=1e-3, dtype=ydt, h=False)
    assert h is None and rstd is None
    assert _near(y, _ref(x, None, None, 1e-3)[2], 42 * FP + U[ydt])


@pytest.mark.parametrize("dt,ydt", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("R,D", [(5, 4), (700, 332), (3, 388), (900, 1020), (7, 4100), (2, 8196), (2, 16380)])
def test_widths_of_four(ctx, dt, ydt, R, D):
    """Multiples of four columns, not of eight."""
    test_forward(ctx, dt, ydt, R, D)
    test_gradient(ctx, dt, ydt, R, D)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("R,D", SHAPES)
def test_eight_bits(ctx, dt, group, R, D):
    g = _gen(2 * R + D)
    x, r, w = _normal(g, R, D, dtype=dt), _normal(g, R, D, dtype=dt), 1 + 0.2 * _normal(g, D)
    y, scales, h, _ = ctx.add_rmsnorm(x, r, w, eps=1e-6, dtype=E4M3, group=group)
    _, _, ry = _ref(x, r, w, 1e-6)
    ng = 1 if group == 0 else -(-D // 128)
    assert y.dtype == E4M3 and scales.shape == (R, ng)
    width = D if group == 0 else 128
    pad = torch.nn.functional.pad(ry.abs(), (0, ng * width - D)).view(R, ng, width)
    want = pad.amax(-1) / 448.0
    sc = scales.view(R, ng)
    assert bool(((sc.double() - want).abs() <= 44 * FP * want).all())
    full = sc.double().repeat_interleave(width, 1)[:, :D]
    back = y.float().double() * full
    tol = torch.maximum(ry.abs() * 2.0 ** -4, full * 2.0 ** -10) * 1.001 + 50 * FP * ry.abs()
    assert bool(((back - ry).abs() <= tol).all())
    assert float(y.float().abs().max()) == 448.0


def test_eight_bits_of_zeros_tiny_rows_and_nan(ctx):
    x = torch.zeros(5, 256, device="cuda")
    x[1, 200] = 1e-30                       # a row far below eps: y about 1e-27
    x[2, :128] = 1.0                        # the second group of 128 is zero
    x[3, 7] = float("nan")
    w = torch.ones(256, device="cuda")
    y, s, _, _ = ctx.add_rmsnorm(x, None, w, eps=1e-6, dtype=E4M3, group=128)
    assert bool((y[0].float() == 0).all()) and bool((s[0] == 0).all())
    assert bool((y[2, 128:].float() == 0).all()) and float(s[2, 1]) == 0.0
    assert bool(y[3].float().isnan().all()) and bool(s[3].isnan().all())
    assert bool((y[4].float() == 0).all())
    # a weight so small that 448 / max|y| overflows
    x = torch.randn(3, 256, generator=_gen(3), device="cuda")
    w = torch.full((256,), 2.0 ** -130, device="cuda")
    y, s, _, _ = ctx.add_rmsnorm(x, None, w, eps=1e-6, dtype=E4M3)
    assert bool(y.float().isfinite().all()) and bool((y.float().abs().amax(1) > 400).all())


def test_zero_rows_need_eps(ctx):
    x = torch.zeros(2, 64, device="cuda")
    y, _, _, rstd = ctx.add_rmsnorm(x, eps=1e-6, rstd=True)
    assert bool((y == 0).all()) and bool((rstd - 1e3).abs().max() < 1e-2)
    y, _, _, _ = ctx.add_rmsnorm(x, eps=0.0)
    assert bool(y.isnan().all())


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("D", [96, 1021])
def test_in_place(ctx, dt, D):
    g = _gen(D)
    x, r, w = _normal(g, 33, D, dtype=dt), _normal(g, 33, D, dtype=dt), 1 + 0.2 * _normal(g, D)
    y0, _, h0, _ = ctx.add_rmsnorm(x, r, w, eps=1e-6)
    for name in ("x", "r"):
        a, b = x.clone(), r.clone()
        y, _, h, _ = ctx.add_rmsnorm(a, b, w, eps=1e-6, h=a if name == "x" else b)
        assert h.data_ptr() == (a if name == "x" else b).data_ptr()
        assert torch.equal(h, h0) and torch.equal(y, y0)
    a = x.clone()
    y, _, _, _ = ctx.add_rmsnorm(a, r, w, eps=1e-6, h=False, y=a)
    assert torch.equal(a, y0)


@pytest.mark.parametrize("shift", [1, 4])
def test_misaligned_views(ctx, shift):
    g = _gen(shift)
    R, D = 12, 512
    x = _normal(g, R * D + shift, dtype=BF16)[shift:].view(R, D)
    w = (1 + 0.2 * _normal(g, D + 1))[1:]
    y, _, h, rstd = ctx.add_rmsnorm(x, None, w, eps=1e-6, rstd=True)
    _, _, ry = _ref(x, None, w, 1e-6)
    assert _near(y, ry, 42 * FP + U[BF16])
    q, s, _, _ = ctx.add_rmsnorm(x, None, w, eps=1e-6, dtype=E4M3, group=128)
    q2, s2, _, _ = ctx.add_rmsnorm(x.clone(), None, w.clone(), eps=1e-6, dtype=E4M3, group=128)
    assert bool(((s - s2).abs() <= 90 * FP * s2).all())


def _bwd_ref(dy, h, w, rstd, dh):
    dyw = dy.double() * (1.0 if w is None else w.double())
    h, rs = h.double(), rstd.double()[..., None]
    c = (dyw * h).mean(-1, keepdim=True) * rs * rs
    cm = (dyw * h).abs().mean(-1, keepdim=True) * rs * rs
    d = 0 if dh is None else dh.double()
    dx = d + rs * (dyw - h * c)
    mag = (0 if dh is None else d.abs()) + rs * (dyw.abs() + h.abs() * cm)
    t = dy.double() * h * rs
    return dx, mag, t.sum(0), t.abs().sum(0)


@pytest.mark.parametrize("dt,ydt", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("R,D", SHAPES)
def test_gradient(ctx, dt, ydt, R, D):
    g = _gen(5 * R + D)
    h, w = _normal(g, R, D, dtype=dt) * 2, 1 + 0.2 * _normal(g, D)
    dy, dh = _normal(g, R, D, dtype=ydt), _normal(g, R, D, dtype=dt)
    _, _, _, rstd = ctx.add_rmsnorm(h, None, w, eps=1e-6, rstd=True)
    for ww, dd in ((w, dh), (None, None)):
        dx, dw = ctx.add_rmsnorm_backward(dy, h, ww, rstd, dd)
        rx, mag, rw, wmag = _bwd_ref(dy, h, ww, rstd, dd)
        assert dx.dtype == dt and dw.dtype == F32
        assert bool(((dx.double() - rx).abs() <= 80 * FP * mag + U[dt] * rx.abs() * 1.001).all())
        assert bool(((dw.double() - rw).abs() <= (R + 16) * FP * wmag).all())
    # in place over dh, without the weight's gradient; a second run: the same bits
    again, dw2 = ctx.add_rmsnorm_backward(dy, h, None, rstd)
    assert torch.equal(dx, again) and torch.equal(dw, dw2)
    d2 = dh.clone()
    full, _ = ctx.add_rmsnorm_backward(dy, h, w, rstd, dh)
    got, none = ctx.add_rmsnorm_backward(dy, h, w, rstd, d2, dx=d2, dw=False)
    assert none is None and torch.equal(got, full)


def test_gradient_against_differences(ctx):
    """Directional derivatives of sum(c y) + sum(e h) by central differences of
    the definition in 64 bits."""
    g = _gen(77)
    R, D, eps = 6, 80, 1e-5
    x, r, w = _normal(g, R, D), _normal(g, R, D), 1 + 0.2 * _normal(g, D)
    c, e = _normal(g, R, D), _normal(g, R, D)
    _, _, h, rstd = ctx.add_rmsnorm(x, r, w, eps=eps, rstd=True)
    dx, dw = ctx.add_rmsnorm_backward(c, h, w, rstd, e)

    def f(xx, ww):
        hh, _, yy = _ref(xx, r, ww, eps)
        return (c.double() * yy).sum() + (e.double() * hh).sum()

    step = 1e-4
    for grad, arg in ((dx, 0), (dw, 1)):
        d = _normal(g, *grad.shape).double()
        hi = f(x.double() + (step * d if arg == 0 else 0), w.double() + (step * d if arg == 1 else 0))
        lo = f(x.double() - (step * d if arg == 0 else 0), w.double() - (step * d if arg == 1 else 0))
        got = (grad.double() * d).sum()
        # the gradient's 80 roundings; the difference's own error is of order step^2
        assert abs(float(got - (hi - lo) / (2 * step))) <= 6e-6 * float((grad.double() * d).abs().sum())


def test_on_another_stream(ctx):
    g = _gen(9)
    x, dy = _normal(g, 2000, 512), _normal(g, 2000, 512)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y, _, h, rstd = ctx.add_rmsnorm(x, eps=1e-6, rstd=True, stream=s)
    dx, dw = ctx.add_rmsnorm_backward(dy, h, None, rstd, stream=s)
    s.synchronize()
    rx, mag, rw, wmag = _bwd_ref(dy, h, None, rstd, None)
    assert bool(((dx.double() - rx).abs() <= 80 * FP * mag + FP * rx.abs()).all())
    assert bool(((dw.double() - rw).abs() <= 2016 * FP * wmag).all())


def test_refusals(ctx, sr):
    abi, E = sr._abi, sr.SN_E_INVAL
    x, y, s = torch.zeros(2, 64, device="cuda"), torch.full((2, 64), 3.0, device="cuda"), torch.zeros(2, device="cuda")
    call = lambda R=2, D=64, dt=0, yt=0, gr=0, xx=x, r=None, w=None, eps=1e-6, h=None, yy=y, sc=None, rs=None: (  # noqa: E731
        abi.sn_add_rmsnorm(ctx.handle, R, D, dt, yt, gr, xx, r, w, eps, h, yy, sc, rs))
    for bad in (dict(R=0), dict(D=0), dict(dt=2), dict(yt=5), dict(gr=128), dict(yt=2), dict(yt=2, sc=s, gr=64),
                dict(sc=s), dict(eps=-1.0), dict(eps=float("nan")), dict(xx=None), dict(yy=None), dict(h=y),
                dict(rs=y), dict(xx=x.data_ptr() + 2), dict(r=y, h=y)):
        assert call(**bad) == E, bad
    assert call(D=16385) == sr.SN_E_UNSUPPORTED
    assert bool((y == 3.0).all())
    rstd = torch.ones(2, device="cuda")
    dw = torch.zeros(64, device="cuda")
    back = lambda dt=0, yt=0, dy=x, h=x, dx=y, w=None: abi.sn_add_rmsnorm_backward(     # noqa: E731
        ctx.handle, 2, 64, dt, yt, dy, h, None, rstd, None, dx, w)
    assert back(w=dw) == sr.SN_E_NOMEM
    for bad in (dict(dt=2), dict(yt=2), dict(dy=None), dict(h=None), dict(dx=None)):
        assert back(**bad) == E, bad
    h2 = torch.zeros(2, 64, device="cuda")
    assert back(h=h2, dx=h2) == E                       # dx over h
    with pytest.raises(ValueError):
        ctx.add_rmsnorm(x, x[:1], eps=1e-6)
    with pytest.raises(ValueError):
        ctx.add_rmsnorm(x, x.bfloat16(), eps=1e-6)
    with pytest.raises(ValueError):
        ctx.add_rmsnorm(x.half(), eps=1e-6)
    with pytest.raises(ValueError):
        ctx.add_rmsnorm(x, None, torch.zeros(63, device="cuda"), eps=1e-6)
    with pytest.raises(ValueError):
        ctx.add_rmsnorm(x.cpu(), eps=1e-6)
    with pytest.raises(sr.SnError):
        ctx.add_rmsnorm(x[:0], eps=1e-6)


def test_the_grid_follows_the_width_alone(ctx):
    """Calls of several widths run the same kernel in CTAs of different sizes;
    each width's grid fills the GPU whatever width came first.  CTAs of half
    the threads: at least twice as many of them."""
    from tests._graph_nodes import nodes
    grids = {}
    for D in (4096, 2048, 1024, 4096, 2048):
        x = torch.zeros(20000, D, dtype=BF16, device="cuda")
        call = lambda: ctx.add_rmsnorm(x, x, None, eps=1e-6)    # noqa: E731
        call()
        (k,), _ = nodes(call)
        threads = k.block[0] * k.block[1]
        assert grids.setdefault(D, (k.grid[0], threads)) == (k.grid[0], threads)
    (g1, t1), (g2, t2) = grids[4096], grids[2048]
    assert t1 == 2 * t2 and g2 >= 2 * g1
    assert grids[1024] == grids[2048]       # two rows a CTA
