"""GPU tests of calls that share a context's workspace, some of them captured
in CUDA graphs and replayed between others: every call and every replay gives
the bits of the same call alone."""
import pytest
import torch

from tests._graph_nodes import nodes

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
B, T, N = 1, 16384, 64


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


def _scan_inputs(seed, t=T):
    g = torch.Generator("cuda").manual_seed(seed)
    a = torch.rand(B, t, N, generator=g, device="cuda") * 0.2 + 0.8
    return a, torch.randn(B, t, N, generator=g, device="cuda")


def _operators(ctx):
    """Calls that leave integers, bf16 and fp32 data all over the workspace."""
    g = torch.Generator("cuda").manual_seed(5)
    n, V, D = 8192, 300, 64
    ids = torch.randint(0, V, (n,), generator=g, device="cuda")
    rows = torch.randn(n, D, generator=g, device="cuda")
    h, w = rows[:500].to(BF16), torch.zeros(V, D, dtype=BF16, device="cuda")
    w[::2] = 0.1
    t = ids[:500]

    def embed():
        return ctx.embed_backward(ids, rows, V)

    def head():
        loss, lse = ctx.linear_ce(h, w, t)
        return ctx.linear_ce_backward(h, w, t, lse)

    return embed, head


def _kernels(sr):
    return [("look-back", sr.SN_SCAN_KERNEL_LOOKBACK), ("fused", sr.SN_SCAN_KERNEL_FUSED)]


def _room(sr, ctx):
    ctx.ensure_workspace_bytes(1 << 26)
    assert sr.sn_workspace_bytes(sr.SN_OP_SCAN_FMA, B, T, N) < 1 << 26


@pytest.mark.parametrize("which", [0, 1], ids=["look-back", "fused"])
def test_a_captured_scan_clears_its_words(sr, ctx, which):
    """A replay cannot know what came before it: the clearing is part of the
    graph although the capture found the workspace clean.  Outside of a graph
    only the first call clears."""
    _room(sr, ctx)
    ctx.set_option(sr.SN_OPT_SCAN_KERNEL, _kernels(sr)[which][1])
    a, b = _scan_inputs(1)
    ctx.scan_fma(a, b)
    ctx.scan_fma(a, b)
    kernels, memsets = nodes(lambda: ctx.scan_fma(a, b))
    assert len(kernels) == 1 and memsets >= 2       # the tagged words, the abort tag


@pytest.mark.parametrize("which", [0, 1], ids=["look-back", "fused"])
def test_scan_replayed_among_other_calls(sr, ctx, which):
    """A scan captured after the usual warm-up and replayed after calls that
    write the same workspace."""
    _room(sr, ctx)
    ctx.set_option(sr.SN_OPT_SCAN_KERNEL, _kernels(sr)[which][1])
    embed, head = _operators(ctx)
    a, b = _scan_inputs(2)
    a2, b2 = _scan_inputs(3, T // 2)
    want, last = ctx.scan_fma(a, b)
    want2, _ = ctx.scan_fma(a2, b2)
    ctx.scan_fma(a, b)
    dtable = embed()
    dh, dw = head()
    ctx.scan_fma(a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, fin = ctx.scan_fma(a, b)
    for between in (lambda: None, embed, head, lambda: ctx.scan_fma(a2, b2), embed, embed):
        between()
        out.zero_()
        fin.zero_()
        graph.replay()
        assert torch.equal(out, want) and torch.equal(fin, last)
        # and calls outside of the graph behind it
        assert torch.equal(ctx.scan_fma(a2, b2)[0], want2)
        assert torch.equal(ctx.scan_fma(a, b)[0], want)
        assert torch.equal(embed(), dtable)
        assert all(torch.equal(x, y) for x, y in zip(head(), (dh, dw)))


@pytest.mark.parametrize("which", [0, 1], ids=["look-back", "fused"])
def test_scan_after_replays_of_other_calls(sr, ctx, which):
    """The host sees no replay: a scan behind one finds the workspace
    overwritten although the last call it knows of was a scan."""
    _room(sr, ctx)
    ctx.set_option(sr.SN_OPT_SCAN_KERNEL, _kernels(sr)[which][1])
    embed, head = _operators(ctx)
    a, b = _scan_inputs(4)
    want, _ = ctx.scan_fma(a, b)
    dtable = embed()
    head()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        head()
        got = embed()
    for _ in range(3):
        assert torch.equal(ctx.scan_fma(a, b)[0], want)
        graph.replay()
        assert torch.equal(ctx.scan_fma(a, b)[0], want)
        graph.replay()
        assert torch.equal(got, dtable)


def test_a_capture_alone_clears_nothing(sr, ctx):
    """A captured clearing has not run: the next call clears for itself.  Said
    by the bits: the workspace holds embed_backward's integers."""
    _room(sr, ctx)
    ctx.set_option(sr.SN_OPT_SCAN_KERNEL, sr.SN_SCAN_KERNEL_FUSED)
    embed, _ = _operators(ctx)
    a, b = _scan_inputs(6)
    want, _ = ctx.scan_fma(a, b)
    embed()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = ctx.scan_fma(a, b)
    assert torch.equal(ctx.scan_fma(a, b)[0], want)
    graph.replay()
    assert torch.equal(out, want)


def _beyond(x, y):
    return x.data_ptr() + x.numel() <= y[0] or y[0] + y[1] <= x.data_ptr()


def test_a_grown_workspace_leaves_graphs_theirs(sr, ctx):
    """A step captured with a small workspace, then a call that needs a larger
    one: the memory that the graph writes belongs to nobody else, and it still
    gives the step's bits."""
    g = torch.Generator("cuda").manual_seed(8)
    h, w = (torch.randn(s, 128, generator=g, device="cuda").to(BF16) for s in (3, 700))
    t = torch.tensor([0, 5, 699], device="cuda")
    assert ctx.get_option(sr.SN_OPT_WORKSPACE_CAPTURED) == 0
    want, _ = ctx.linear_ce(h, w, t)
    torch.cuda.synchronize()
    assert ctx.get_option(sr.SN_OPT_WORKSPACE_CAPTURED) == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, _ = ctx.linear_ce(h, w, t)
    assert ctx.get_option(sr.SN_OPT_WORKSPACE_CAPTURED) == 1
    old = ctx._ws.data_ptr(), ctx._ws.numel()
    embed, _ = _operators(ctx)
    dtable = embed()
    assert ctx._ws.numel() > old[1] and ctx.get_option(sr.SN_OPT_WORKSPACE_CAPTURED) == 0
    others = [torch.full((old[1],), 7, dtype=torch.uint8, device="cuda") for _ in range(64)]
    assert all(_beyond(x, old) for x in others)
    graph.replay()
    assert torch.equal(loss, want) and all(bool((x == 7).all()) for x in others)
    assert torch.equal(embed(), dtable)
    with pytest.raises(sr.SnError):
        ctx.set_option(sr.SN_OPT_WORKSPACE_CAPTURED, 0)


def test_a_workspace_of_no_graph_is_not_kept(sr, ctx):
    for n in (1 << 12, 1 << 14, 1 << 16):
        ctx.ensure_workspace_bytes(n)
    assert ctx._kept == []


@pytest.mark.parametrize("which", [0, 1], ids=["look-back", "fused"])
def test_scan_replayed_across_a_growth(sr, ctx, which):
    """The scan's graph stays with the workspace that it was captured with, the
    calls behind it with the new one."""
    _room(sr, ctx)
    ctx.set_option(sr.SN_OPT_SCAN_KERNEL, _kernels(sr)[which][1])
    embed, head = _operators(ctx)
    a, b = _scan_inputs(9)
    want, _ = ctx.scan_fma(a, b)
    dtable = embed()
    ctx.scan_fma(a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = ctx.scan_fma(a, b)
    ctx.ensure_workspace_bytes(1 << 27)
    assert len(ctx._kept) == 1
    for _ in range(3):
        assert torch.equal(embed(), dtable)
        graph.replay()
        assert torch.equal(out, want)
        assert torch.equal(ctx.scan_fma(a, b)[0], want)
        head()


def _captured(call):
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    return graph, out


@pytest.mark.parametrize("n,V,D,dt", [(1, 300, 768, BF16), (1024, 300, 33, torch.float32), (40000, 64, 16, BF16)])
def test_lookup_and_its_gradient_replayed(ctx, n, V, D, dt):
    """On new ids and rows each time, one and eight and sixteen CTAs sorting."""
    g = torch.Generator("cuda").manual_seed(n)
    table, rows = torch.randn(V, D, generator=g, device="cuda").to(dt), torch.empty(n, D, dtype=dt, device="cuda")
    ids = torch.zeros(n, dtype=torch.int64, device="cuda")
    graph, got = _captured(lambda: (ctx.embed(ids, table, scale=3.0), ctx.embed_backward(ids, rows, V, scale=3.0)))
    for _ in range(3):
        ids.copy_(torch.randint(-2, V, (n,), generator=g, device="cuda"))
        rows.normal_(generator=g)
        graph.replay()
        want = ctx.embed(ids, table, scale=3.0), ctx.embed_backward(ids, rows, V, scale=3.0)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("R,D,dt", [(1, 2048, BF16), (300, 511, BF16), (2000, 1536, torch.float32)])
def test_norm_and_its_gradient_replayed(ctx, R, D, dt):
    g = torch.Generator("cuda").manual_seed(R)
    x, r, c = (torch.empty(R, D, dtype=dt, device="cuda") for _ in range(3))
    w = torch.rand(D, generator=g, device="cuda")

    def step():
        q, scales, _, _ = ctx.add_rmsnorm(x, r, w, eps=1e-6, dtype=torch.float8_e4m3fn, group=128)
        y, _, h, rstd = ctx.add_rmsnorm(x, r, w, eps=1e-6, rstd=True)
        return (q.view(torch.uint8), scales, y, h, rstd, *ctx.add_rmsnorm_backward(y, h, w, rstd, c))

    for t in (x, r, c):
        t.normal_(generator=g)
    graph, got = _captured(step)
    for _ in range(3):
        for t in (x, r, c):
            t.normal_(generator=g)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
