"""GPU tests of the embedding lookup and its gradient (sn_embed,
sn_embed_backward) against the definition in 64 bits.

Tolerances, per element: the lookup is one fp32 product and one rounding to
the output's type (unit roundoff U: 2^-24 for fp32, 2^-8 for bf16 with its 8 significant bits); a
gradient element is a sum of m fp32 terms in some order, within (m + 1) 2^-24
of the sum of their magnitudes, then one rounding."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


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


def _lookup_ref(ids, table, scale):
    ok = (ids >= 0) & (ids < table.shape[0])
    rows = table.double()[torch.where(ok, ids, 0).long()] * scale
    return torch.where(ok[..., None], rows, torch.zeros_like(rows))


def _grad_ref(ids, g, V, scale):
    """The gradient, the sum of magnitudes and the number of terms of each row."""
    ids, g = ids.reshape(-1).long(), g.reshape(-1, g.shape[-1]).double()
    ok = (ids >= 0) & (ids < V)
    ids, g = ids[ok], g[ok]
    ref = torch.zeros(V, g.shape[1], dtype=torch.float64, device="cuda").index_add_(0, ids, g) * scale
    mag = torch.zeros_like(ref).index_add_(0, ids, g.abs()) * abs(scale)
    return ref, mag, torch.bincount(ids, minlength=V)


def _check_grad(got, ref, mag, m, base=None):
    base = torch.zeros_like(ref) if base is None else base.double()
    tol = (m[:, None] + 2) * 2.0 ** -24 * (mag + base.abs()) + U[got.dtype] * (ref + base).abs() * 1.001
    assert bool(((got.double() - ref - base).abs() <= tol).all())


@pytest.mark.parametrize("tdt,odt", [(F32, F32), (BF16, F32), (BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
@pytest.mark.parametrize("n,V,D", [(1, 1, 1), (3, 7, 8), (257, 1000, 511), (64, 33, 256), (1000, 5000, 768)])
def test_lookup(ctx, tdt, odt, idt, n, V, D):
    g = _gen(n + V + D)
    table = _normal(g, V, D, dtype=tdt)
    ids = torch.randint(0, V, (n,), generator=g, device="cuda").to(idt)
    scale = math.sqrt(D)
    out = ctx.embed(ids, table, scale=scale, dtype=odt)
    ref = _lookup_ref(ids, table, float(torch.tensor(scale, dtype=F32)))
    assert out.dtype == odt and out.shape == (n, D)
    assert bool(((out.double() - ref).abs() <= (U[odt] + 2.0 ** -24) * ref.abs() * 1.001).all())


def test_lookup_of_padding_reads_no_row(ctx):
    """Ids outside [0, V) give zeros, also where table rows hold NaN, and with
    ids far beyond what 32 bits index."""
    table = torch.full((4, 64), float("nan"), device="cuda")
    table[2] = 1.0
    ids = torch.tensor([[-1, 2, 4], [-(2 ** 40), 2 ** 40, 2]], device="cuda")
    out = ctx.embed(ids, table, scale=3.0)
    want = torch.zeros(2, 3, 64, device="cuda")
    want[0, 1] = want[1, 2] = 3.0
    assert torch.equal(out, want)


def test_lookup_beyond_32_bit_offsets(ctx):
    V, D = (1 << 20) + 77, 2064          # 2.16e9 elements
    table = torch.zeros(V, D, dtype=BF16, device="cuda")
    ids = torch.tensor([V - 1, 0, V - 2, (1 << 31) // D + 1], device="cuda")
    rows = _normal(_gen(5), 4, D, dtype=BF16)
    table[ids] = rows
    assert torch.equal(ctx.embed(ids, table), rows)
    grad = ctx.embed_backward(ids, rows, V)
    assert torch.equal(grad[ids], rows)
    assert int(torch.count_nonzero(grad.sum(1))) <= 4
    del table, grad
    torch.cuda.empty_cache()


def test_views_and_misaligned_rows(ctx):
    """A view that starts inside a buffer: aligned to its element only."""
    g = _gen(11)
    buf = _normal(g, 40 * 96 + 3, dtype=BF16)
    table = buf[3:].view(40, 96)
    ids = torch.randint(0, 40, (50,), generator=g, device="cuda")
    assert torch.equal(ctx.embed(ids, table), table[ids])
    gbuf = _normal(g, 50 * 96 + 1)
    go = gbuf[1:].view(50, 96)
    obuf = torch.full((40 * 96 + 5,), 7.0, device="cuda")
    gt = obuf[5:].view(40, 96)
    ctx.embed_backward(ids, go, 40, grad_table=gt)
    _check_grad(gt, *_grad_ref(ids, go, 40, 1.0))
    assert bool((obuf[:5] == 7.0).all())


SIZES = [(1, 1, 1), (1, 300, 8), (2, 259, 511), (31, 5, 32), (2047, 1, 40), (2048, 3, 64), (2049, 70000, 16),
         (5000, 259, 511), (40000, 65537, 24), (9000, 100, 1032)]


@pytest.mark.parametrize("gdt,tdt", [(F32, F32), (BF16, F32), (BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("n,V,D", SIZES)
def test_gradient(ctx, gdt, tdt, n, V, D):
    g = _gen(3 * n + V)
    # skewed: id 0 takes a tenth of the tokens, some are padding
    ids = torch.randint(-max(1, V // 20), V + max(1, V // 20), (n,), generator=g, device="cuda")
    ids = torch.where(torch.rand(n, generator=g, device="cuda") < 0.1, 0, ids)
    go = _normal(g, n, D, dtype=gdt)
    got = ctx.embed_backward(ids, go, V, scale=0.5, dtype=tdt)
    assert got.dtype == tdt
    _check_grad(got, *_grad_ref(ids, go, V, 0.5))
    # 32-bit ids and a second run: the same bits
    assert torch.equal(got, ctx.embed_backward(ids.to(torch.int32), go, V, scale=0.5, dtype=tdt))


@pytest.mark.parametrize("gdt,tdt", [(F32, F32), (BF16, BF16)])
@pytest.mark.parametrize("n,V,D", [(32767, 1200, 8), (32768, 70000, 16), (250001, 3, 264), (300000, 65536, 21)])
def test_gradient_of_many_tokens(ctx, gdt, tdt, n, V, D):
    g = _gen(n)
    # skewed: a third of the tokens are id V - 1, some are padding
    ids = torch.randint(-max(1, V // 20), V + max(1, V // 20), (n,), generator=g, device="cuda")
    ids = torch.where(torch.rand(n, generator=g, device="cuda") < 0.3, V - 1, ids)
    go = _normal(g, n, D, dtype=gdt)
    got = ctx.embed_backward(ids, go, V, scale=0.5, dtype=tdt)
    _check_grad(got, *_grad_ref(ids, go, V, 0.5))
    assert torch.equal(got, ctx.embed_backward(ids, go, V, scale=0.5, dtype=tdt))


@pytest.mark.parametrize("tdt", [F32, BF16])
@pytest.mark.parametrize("D", [8, 64, 256, 264, 520, 768, 1032, 1280, 1536, 1800, 2048, 2056, 4104])
def test_rows_without_tokens(ctx, tdt, D):
    """Every row that no token names is zero, whatever the buffer held, at
    every number of threads that the width may give."""
    n, V = 60, 900
    g = _gen(D)
    ids = torch.randint(0, V, (n,), generator=g, device="cuda")
    go = _normal(g, n, D)
    for _ in range(3):
        out = torch.full((V, D), float("nan"), dtype=tdt, device="cuda")
        ctx.embed_backward(ids, go, V, grad_table=out)
        ref, mag, m = _grad_ref(ids, go, V, 1.0)
        assert bool((out[m == 0] == 0).all())
        _check_grad(out, ref, mag, m)
        # other contents for the next call's shared memory
        ctx.add_rmsnorm(_normal(g, 4000, 2048), eps=1e-6)


@pytest.mark.parametrize("case", ["one id", "no id", "sorted", "reversed", "last"])
def test_gradient_of_lopsided_ids(ctx, case):
    n, V, D = 6000, 1000, 72
    ids = {"one id": torch.full((n,), 37), "no id": torch.full((n,), -1), "sorted": torch.arange(n) % V,
           "reversed": V - 1 - torch.arange(n) % V, "last": torch.full((n,), V - 1)}[case].cuda()
    if case == "sorted":
        ids = ids.sort().values
    go = _normal(_gen(1), n, D)
    got = ctx.embed_backward(ids, go, V)
    _check_grad(got, *_grad_ref(ids, go, V, 1.0))


@pytest.mark.parametrize("tdt", [F32, BF16])
def test_gradient_added_to_what_is_there(ctx, tdt):
    """accumulate: the rows that tokens name get their sums added, the others
    keep their bits, NaN among them; NaN in padding tokens' gradients is not read."""
    g = _gen(21)
    n, V, D = 700, 50, 96
    ids = torch.randint(0, V - 10, (n,), generator=g, device="cuda")
    ids[::7] = -100
    go = _normal(g, n, D)
    go[::7] = float("nan")
    base = _normal(g, V, D, dtype=tdt)
    base[V - 1] = float("nan")
    got = base.clone()
    out = ctx.embed_backward(ids, go, V, grad_table=got, accumulate=True)
    assert out.data_ptr() == got.data_ptr()
    ref, mag, m = _grad_ref(ids, torch.where((ids >= 0)[:, None], go, torch.zeros_like(go)), V, 1.0)
    named = m > 0
    _check_grad(got[named], ref[named], mag[named], m[named], base[named])
    assert torch.equal(got[~named].view(torch.uint8), base[~named].view(torch.uint8))


def test_gradient_against_differences(ctx):
    """The directional derivative of sum(c * embed(table)) by differences of
    the definition in 64 bits."""
    g = _gen(31)
    n, V, D = 500, 60, 48
    ids = torch.randint(0, V, (n,), generator=g, device="cuda")
    table, c, d = _normal(g, V, D), _normal(g, n, D), _normal(g, V, D)
    grad = ctx.embed_backward(ids, c, V, scale=2.0)
    f = lambda t: (c.double() * t[ids] * 2.0).sum()          # noqa: E731
    eps = 1e-3
    diff = (f(table.double() + eps * d.double()) - f(table.double() - eps * d.double())) / (2 * eps)
    got = (grad.double() * d.double()).sum()
    scale = (grad.double() * d.double()).abs().sum()
    assert abs(float(got - diff)) <= 1e-6 * float(scale)


def test_on_another_stream(ctx):
    g = _gen(41)
    n, V, D = 3000, 500, 128
    ids = torch.randint(0, V, (n,), generator=g, device="cuda")
    table, go = _normal(g, V, D), _normal(g, n, D)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = ctx.embed(ids, table, stream=s)
    gt = ctx.embed_backward(ids, go, V, stream=s)
    s.synchronize()
    assert torch.equal(out, table[ids])
    _check_grad(gt, *_grad_ref(ids, go, V, 1.0))


def test_refusals(ctx, sr):
    abi, E = sr._abi, sr.SN_E_INVAL
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    table, out = torch.zeros(8, 16, device="cuda"), torch.full((4, 16), 5.0, device="cuda")
    call = lambda n=4, V=8, D=16, dt=0, ot=0, it=1, i=ids, t=table, o=out: abi.sn_embed(    # noqa: E731
        ctx.handle, n, V, D, dt, ot, it, i, t, 1.0, o)
    for bad in (dict(n=0), dict(V=0), dict(D=-1), dict(dt=2), dict(ot=3), dict(it=2), dict(i=None), dict(t=None),
                dict(o=None), dict(o=table), dict(i=ids.data_ptr() + 4), dict(t=table.data_ptr() + 2),
                dict(n=(1 << 30) + 1)):
        assert call(**bad) == E, bad
    assert bool((out == 5.0).all())
    go = torch.zeros(4, 16, device="cuda")
    assert abi.sn_embed_backward(ctx.handle, 4, 8, 16, 0, 0, 1, ids, go, 1.0, 0, table) == sr.SN_E_NOMEM
    ctx.ensure_workspace_bytes(abi.sn_embed_backward_workspace_bytes(4, 8, 16))
    assert abi.sn_embed_backward(ctx.handle, 4, 8, 16, 0, 0, 1, ids, go, 1.0, 2, table) == E
    assert abi.sn_embed_backward(ctx.handle, 4, 8, 16, 0, 0, 1, ids, go, 1.0, 0, go) == E
    assert abi.sn_embed_backward(ctx.handle, 4, 8, 16, 0, 0, 1, ids, go, 1.0, 0, ctx._ws) == E
    with pytest.raises(ValueError):
        ctx.embed(ids, table.half())
    with pytest.raises(ValueError):
        ctx.embed(ids.float(), table)
    with pytest.raises(ValueError):
        ctx.embed(ids, table.t())
    with pytest.raises(ValueError):
        ctx.embed(ids.cpu(), table)
    with pytest.raises(ValueError):
        ctx.embed_backward(ids, go[:3], 8)
    with pytest.raises(ValueError):
        ctx.embed_backward(ids, go, 8, accumulate=True)
    with pytest.raises(sr.SnError):
        ctx.embed(ids[:0], table)


@pytest.mark.parametrize("as_handle", [False, True])
def test_memory_used_on_another_stream_is_not_handed_out(ctx, as_handle):
    """The call's tensors are dropped while it still waits behind a busy
    stream: their memory is not given to the next tensors."""
    g = _gen(61)
    n, V, D = 3000, 50, 96
    ids = torch.randint(0, V, (n,), generator=g, device="cuda")
    rows = _normal(g, n, D)
    want = ctx.embed_backward(ids, rows, V)
    used = rows.clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)       # about 10 ms
    got = ctx.embed_backward(ids, used, V, stream=s.cuda_stream if as_handle else s)
    at = used.data_ptr()
    del used
    others = [torch.full((n, D), 9.0, device="cuda") for _ in range(8)]
    assert s.query() or all(x.data_ptr() != at for x in others)
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("odt", [F32, BF16])
@pytest.mark.parametrize("D", [64, 33])
@pytest.mark.parametrize("scale", [float("inf"), float("-inf"), float("nan"), -2.0])
def test_padding_is_zeros_whatever_the_scale(ctx, odt, D, scale):
    g = _gen(67)
    table = _normal(g, 20, D)
    ids = torch.tensor([3, -1, 20, 7, 2 ** 40, 19], device="cuda")
    out = ctx.embed(ids, table, scale=scale, dtype=odt)
    pad = torch.tensor([1, 2, 4], device="cuda")
    assert bool((out[pad] == 0).all())
    rows = (table[ids[[0, 3, 5]]] * scale).to(odt)
    assert torch.equal(out[[0, 3, 5]].nan_to_num(nan=5.0), rows.nan_to_num(nan=5.0))


def test_many_tokens_take_a_cluster_of_sixteen(ctx):
    """Where the device grants it, as a whole GB300 does."""
    from tests._graph_nodes import nodes
    for n, ctas in ((2048, 1), (32767, 8), (32768, 16)):
        ids = torch.zeros(n, dtype=torch.int64, device="cuda")
        rows = torch.ones(n, 8, device="cuda")
        ctx.embed_backward(ids, rows, 4)
        kernels, _ = nodes(lambda: ctx.embed_backward(ids, rows, 4))
        assert [k.grid[0] for k in kernels if "sort_kernel" in k.name] == [ctas]


@pytest.mark.parametrize("handle", [0, 1])
def test_the_default_stream_by_its_handles(ctx, handle):
    """0 and 1 (cudaStreamLegacy) while another stream is the current one."""
    g = _gen(71)
    ids = torch.randint(-1, 50, (300,), generator=g, device="cuda")
    rows = _normal(g, 300, 40)
    want = ctx.embed_backward(ids, rows, 50)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        used = rows.clone()
        s.synchronize()
        got = ctx.embed_backward(ids, used, 50, stream=handle)
        del used
    torch.cuda.synchronize()
    assert torch.equal(got, want)
