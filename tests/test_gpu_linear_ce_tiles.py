"""GPU tests of the linear head's cross entropy by the tiles that its products
run in: each shape says which it is there for, the test reads from a captured
call that it runs them, and holds the results against the definition.

The logits' tiles go by the bounds of test_gpu_linear_ce.py, with few enough
columns that a probability in a wrong place shows.  The gradients' tiles go by
exact values: with h (or w) zero all logits are 0 and p is 1 / V, V a power of
two; grad_loss is 1 or 2 of either sign and w (or h) small integers, so that dz
(1 / V, and -1 at the target, which bf16 makes of 1 / V - 1) and every partial
sum are exact in any order, and the result is the definition's, rounded once."""
import re

import pytest
import torch

from tests._graph_nodes import nodes
from tests.test_gpu_linear_ce import Ref, _inputs

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


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


def _tiles(call):
    """What the products of a call run in: {"z" | "dh" | "dw": text}.  Wide tiles (256 x 512) whole, as halves, or
    both; else the columns of a tile; the sum in splits; results of several pieces of the vocabulary added."""
    call()
    found = {}
    for k in nodes(call, ("ce_gemm", 3, 10))[0]:
        kind = re.search(r"ce_gemmILi(\d)ELb([01])ELb[01]EL.*?4ModeE(\d)E", k.name)
        if kind is None:
            continue
        M, N, kblocks, seg, bw, mt, nt, splits, items, whole = k.ints
        what = "z" if kind[1] != "2" else "dw" if kind[2] == "1" else "dh"
        text = str(bw)
        if kind[3] == "1":
            text = "wide" + " whole" * (whole > 0) + " halves" * (items > whole)
        text += " splits" * (splits > 1)
        if what in found:
            assert found[what].split(" pieces")[0] == text or what == "z"
            text = found[what].split(" pieces")[0] + " pieces"
        found[what] = text
    return found


LOGITS = [(5000, 1100, 64 * nk, "wide whole") for nk in range(1, 9)] + [
    (5000, 1100, 520, "wide whole"), (5000, 1100, 1021, "wide whole"), (3000, 1400, 2048, "wide halves"),
    (3000, 4096, 2048, "wide whole halves"), (4000, 8000, 2112, "256"), (3000, 1400, 2112, "256"),
    (300, 700, 320, "64"), (700, 3000, 4096, "128")]


@pytest.mark.parametrize("N,V,D,tiles", LOGITS)
def test_logits(ctx, N, V, D, tiles):
    h, w, t, gl = _inputs(N, V, D, BF16, N + V + D, masked=0.05)
    loss, lse = ctx.linear_ce(h, w, t)
    assert _tiles(lambda: ctx.linear_ce(h, w, t)) == {"z": tiles}
    back = lambda: ctx.linear_ce_backward(h, w, t, lse, gl)     # noqa: E731
    assert _tiles(back)["z"] == tiles
    dh, dw = back()
    r = Ref(h, w, t, 1.0, gl)
    r.check(loss, lse)
    r.check_grad(dh, dw)


GRADIENTS = [
    (1000, 32768, 512, "wide halves splits", "wide whole"),
    (4096, 32768, 1024, "wide whole splits", "wide whole halves"),
    (16384, 32768, 512, "wide whole pieces", "wide whole pieces"),
    (2000, 8192, 1021, "128", "wide whole"),                        # rows of odd widths
    (5000, 1024, 1021, "wide whole", "64"),
    (33000, 1024, 1021, "wide whole halves", "wide whole splits"),
    (33000, 1024, 1000, "wide whole halves", "wide whole splits"),
    (20000, 2048, 2000, "wide whole halves", "wide whole splits"),
    (40000, 16384, 256, "256 pieces", "256 splits pieces"),
    (300, 32768, 520, "256 splits", "wide whole halves"),
    (700, 32768, 72, "128 splits", "128"),
    (700, 4096, 100, "64 splits", "64"),
    # few rows of h
    (1, 65536, 768, None, None), (16, 32768, 768, None, None), (64, 32768, 1100, None, None)]


@pytest.mark.parametrize("N,V,D,dh_tiles,dw_tiles", GRADIENTS)
def test_gradients(ctx, N, V, D, dh_tiles, dw_tiles):
    g = torch.Generator("cuda").manual_seed(N + V + D)

    def integers(least, most, *shape):
        return torch.randint(least, most + 1, shape, generator=g, device="cuda")

    t = integers(0, V - 1, N)
    gl = (integers(1, 2, N) * (2 * integers(0, 1, N) - 1)).float()
    h, w = integers(-1, 1, N, D).to(BF16), integers(-2, 2, V, D).to(BF16)
    none_h, none_w = torch.zeros_like(h), torch.zeros_like(w)
    _, lse = ctx.linear_ce(none_h, w, t)

    def grad_h():
        return ctx.linear_ce_backward(none_h, w, t, lse, gl, dw=False)[0]

    def grad_w():
        return ctx.linear_ce_backward(h, none_w, t, lse, gl, dh=False)[1]

    assert _tiles(grad_h).get("dh") == dh_tiles
    if dw_tiles is not None:
        assert _tiles(grad_w)["dw"] == dw_tiles
    wt = w.double()[t]
    dh = gl.double()[:, None] * ((w.double().sum(0) - wt) / V - wt)
    assert torch.equal(grad_h(), dh.to(BF16))
    gh = gl.double()[:, None] * h.double()
    own = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, t, gh)
    dw = (gh.sum(0) - own) / V - own
    assert torch.equal(grad_w(), dw.to(BF16))
