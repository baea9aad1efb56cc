"""Every form of the tiled products over several steps of k, on the GPU: the timing
hook's name says which form a call took.  Inputs are small whole numbers, so that
every sum is exact in fp32 (below 2^24) and equality is asked for: a step that is
left out, taken twice or read from the other buffer, and a short first step, change
the result.  The choices are those of a GPU of 256 CUs."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import farthest_vector_search_amd as vs  # noqa: E402
from test_table_ops import dev, i32, rng  # noqa: E402

HALF = [torch.float16, torch.bfloat16]


def whole(r, shape, top):
    """Whole numbers -top .. top as fp32 on the CPU."""
    return torch.from_numpy(r.integers(-top, top + 1, shape).astype(np.float32))


def places(r, G, lo, hi, empty):
    """Places of G units of lo .. hi rows, `empty` of them without, and 9 rows of no unit
    before and 70 behind."""
    count = r.integers(lo, hi + 1, G)
    count[r.choice(G, empty, replace=False)] = 0
    off = 9 + np.concatenate([[0], np.cumsum(count)])
    return off, int(off[-1]) + 70


def named(call):
    with vs.KernelTimer(8) as kt:
        out = call()
    assert kt.launches == 1
    return out, kt.name


def same(got, want, t):
    got = got.cpu()
    want = want.to(t)
    assert torch.equal(got, want), int((got != want).sum())


ROWS = [
    # form, across's form, units, rows a unit (least, most, empty units), d, cols
    ("256x256,16", "256x256,16", 64, 200, 300, 2, 1032, 1024),
    ("256x256,16", "256x256,16", 64, 130, 170, 0, 1032, 1048),
    ("256x256,16", "256x256,16", 300, 190, 260, 5, 520, 512),      # found by slots
    ("128x128,16", "128x128,16", 64, 100, 140, 3, 1032, 1048),
    ("128x128,16", "128x128,16", 300, 90, 130, 5, 264, 272),       # found by slots
    ("128x128,4", "128x128,4", 64, 100, 180, 3, 1030, 1042),
    ("128x128,0", "128x128,0", 64, 100, 180, 3, 1027, 1033),
    ("64x128,16", "64x128,16", 64, 20, 64, 3, 1032, 1048),
    ("64x128,16", "64x128,16", 400, 20, 64, 9, 520, 264),          # found by slots
    ("64x64,16", "64x64,16", 5, 20, 300, 1, 1032, 264),
    ("64x64,4", "64x64,4", 20, 20, 90, 1, 1030, 262),
    ("64x64,0", "64x64,0", 20, 20, 90, 1, 1027, 261),
    ("64x64,4", "64x64,4", 300, 20, 60, 5, 262, 70),               # found by slots
    ("64x64,0", "64x64,0", 300, 20, 60, 5, 263, 71),               # found by slots
]


@pytest.mark.parametrize("form,across,G,lo,hi,empty,d,cols", ROWS)
def test_rows(form, across, G, lo, hi, empty, d, cols):
    r = rng(80, G, d, cols)
    off, m = places(r, G, lo, hi, empty)
    X, W, dY = whole(r, (m, d), 3), whole(r, (G, cols, d), 3), whole(r, (m, cols), 3)
    Y, dX = torch.zeros(m, cols), torch.zeros(m, d)
    for g in range(G):
        s = slice(off[g], off[g + 1])
        Y[s], dX[s] = X[s] @ W[g].T, dY[s] @ W[g]
    for t in HALF:
        x, w, dy, o = X.to(t).to(dev()), W.to(t).to(dev()), dY.to(t).to(dev()), i32(off)
        got, name = named(lambda: vs.vs_unit_products(x, w, o))
        assert name == f"k_unit_rows<{form}>"
        same(got, Y, t)
        (got, _), name = named(lambda: vs.vs_unit_products_backward(dy, x, w, o, want_dW=False))
        assert name == f"k_unit_rows<{across},across>"
        same(got, dX, t)


@pytest.mark.parametrize("G,lo,hi,empty,d,cols,piece", [
    (64, 20, 200, 3, 264, 328, 16), (64, 20, 200, 3, 257, 333, 4), (300, 20, 70, 3, 136, 132, 16),
    (300, 20, 70, 3, 133, 135, 4)])
def test_rows_in_full_precision(G, lo, hi, empty, d, cols, piece):
    r = rng(81, G, d, cols)
    off, m = places(r, G, lo, hi, empty)
    X, W, dY = whole(r, (m, d), 9), whole(r, (G, cols, d), 9), whole(r, (m, cols), 9)
    Y, dX = torch.zeros(m, cols), torch.zeros(m, d)
    for g in range(G):
        s = slice(off[g], off[g + 1])
        Y[s], dX[s] = X[s] @ W[g].T, dY[s] @ W[g]
    x, w, dy, o = X.to(dev()), W.to(dev()), dY.to(dev()), i32(off)
    got, name = named(lambda: vs.vs_unit_products(x, w, o))
    assert name == f"k_unit_rows<64x64,{piece}>"
    same(got, Y, torch.float32)
    (got, _), name = named(lambda: vs.vs_unit_products_backward(dy, x, w, o, want_dW=False))
    assert name == f"k_unit_rows<64x64,{piece},across>"
    same(got, dX, torch.float32)


MATS = [
    # form, units, rows a unit (least, most, empty units), d, cols, in runs
    ("256x256,16", 64, 130, 300, 3, 1024, 1024, False),
    ("128x128,16", 20, 130, 250, 2, 512, 520, False),
    ("128x128,4", 20, 130, 250, 2, 510, 506, False),
    ("128x128,0", 20, 130, 250, 2, 509, 507, False),
    ("128x128,16", 4, 4200, 5300, 0, 512, 504, True),
    ("128x128,4", 4, 4200, 5300, 0, 506, 510, True),
    ("128x128,0", 4, 4200, 5300, 0, 507, 509, True),
    ("64x64,16", 20, 130, 250, 2, 264, 72, False),
    ("64x64,4", 20, 130, 250, 2, 262, 70, False),
    ("64x64,0", 20, 130, 250, 2, 261, 71, False),
    ("64x64,16", 4, 1100, 1500, 0, 512, 504, False),   # rows too few for runs
    ("64x64,16", 4, 2200, 2500, 0, 512, 504, False),
    ("128x128,0", 4, 2200, 2500, 0, 511, 503, True),
    ("64x64,16", 3, 2200, 2500, 0, 128, 72, True),
    ("64x64,16", 3, 800, 1000, 0, 128, 72, False),
]


@pytest.mark.parametrize("form,G,lo,hi,empty,d,cols,runs", MATS)
def test_matrices(form, G, lo, hi, empty, d, cols, runs):
    r = rng(82, G, d, cols)
    off, m = places(r, G, lo, hi, empty)
    need = vs.lib().vs_unit_products_backward_workspace(m, d, G, cols)
    ws = torch.empty(need + 256, dtype=torch.uint8, device=dev())
    X, dY = whole(r, (m, d), 3), whole(r, (m, cols), 3)
    dW = torch.stack([dY[a:b].T @ X[a:b] for a, b in zip(off, off[1:])])
    X[:9], X[off[-1]:], dY[:9], dY[off[-1]:] = (float("nan"),) * 4  # rows of no unit
    for t in HALF:
        x, dy, o = X.to(t).to(dev()), dY.to(t).to(dev()), i32(off)
        w = torch.zeros(G, cols, d, dtype=t, device=dev())
        for gt in (t, torch.float32):
            ws.fill_(0xA5)
            (_, got), name = named(lambda: vs.vs_unit_products_backward(
                dy, x, w, o, grad_dtype=gt, want_dXs=False, workspace=ws))
            assert name == f"k_unit_mats<{form}>"
            assert bool((ws[:need] != 0xA5).any()) == runs  # runs leave their sums there
            same(got, dW, gt)


@pytest.mark.parametrize("G,r,d,cols,runs", [(4, 600, 64, 64, True), (4, 400, 64, 64, False),
                                             (16, 1100, 256, 256, False), (16, 2100, 256, 257, True)])
def test_matrices_in_full_precision(G, r, d, cols, runs):
    m = G * r
    gen = rng(84, G, r)
    X, dY = whole(gen, (m, d), 9), whole(gen, (m, cols), 9)
    off = np.arange(G + 1) * r
    dW = torch.stack([dY[a:b].T @ X[a:b] for a, b in zip(off, off[1:])])
    need = vs.lib().vs_unit_products_backward_workspace(m, d, G, cols)
    ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device=dev())
    w = torch.zeros(G, cols, d, device=dev())
    _, got = vs.vs_unit_products_backward(dY.to(dev()), X.to(dev()), w, i32(off), want_dXs=False,
                                          workspace=ws)
    assert bool((ws[:need] != 0xA5).any()) == runs
    same(got, dW, torch.float32)


SCORES = [
    # form, queries, table rows, d
    ("256x256,16", 300, 65500, 400), ("128x128,16", 130, 40000, 400), ("128x128,4", 130, 40000, 404),
    ("128x128,0", 130, 40000, 403), ("64x64,16", 40, 5000, 912), ("64x64,4", 40, 5000, 908),
    ("64x64,0", 40, 5000, 911),
]


@pytest.mark.parametrize("form,nq,nc,d", SCORES)
def test_scores(form, nq, nc, d):
    r = rng(83, nq, nc, d)
    x, t = (torch.from_numpy(r.integers(-128, 128, s).astype(np.int8)) for s in ((nq, d), (nc, d)))
    one = torch.ones(nc, device=dev())
    got, name = named(lambda: vs.vs_q8_scores(x.to(dev()), one[:nq], t.to(dev()), one))
    assert name == f"k_q8_scores<{form}>"
    same(got, x.float() @ t.float().T, torch.float32)  # below 2^24


FEW = [
    # type, rows, units, d, cols, the form the call takes
    (torch.bfloat16, 1, 64, 1024, 2048, "<64x64,16>"),     # empty workgroups would be the most
    (torch.bfloat16, 1, 64, 4096, 1024, "_few"),
    (torch.bfloat16, 31, 64, 1024, 2048, "<64x128,16>"),   # as for 32
    (torch.bfloat16, 32, 64, 1024, 2048, "<64x128,16>"),
    (torch.bfloat16, 16, 8, 2048, 2048, "_few"),
    (torch.bfloat16, 512, 32, 2048, 2048, "<64x128,16>"),
    (torch.float16, 64, 16, 1027, 1025, "_few"),
    (torch.float16, 4096, 256, 515, 131, "<64x64,0>"),     # 16 rows a unit at odd addresses
    (torch.float32, 1, 64, 1024, 8192, "<64x64,16>"),
    (torch.float32, 1, 64, 1024, 1024, "_few"),
    (torch.float32, 31, 64, 1024, 2048, "_few"),
    (torch.float32, 32, 64, 1024, 2048, "_few"),
    (torch.float32, 256, 64, 1024, 1024, "_few"),
    (torch.float32, 1024, 64, 1024, 1024, "<64x64,16>"),
]


@pytest.mark.parametrize("t,m,G,d,cols,form", FEW)
def test_few_rows(t, m, G, d, cols, form):
    """The form for units of few rows, on both sides of each border."""
    gen = torch.Generator(device=dev()).manual_seed(m + cols)
    X, W = (torch.randint(-3, 4, s, generator=gen, device=dev()).to(t) for s in ((m, d), (G, cols, d)))
    unit = torch.sort(torch.randint(0, G, (m,), generator=gen, device=dev()))[0]
    off = torch.searchsorted(unit, torch.arange(G + 1, device=dev())).int()
    got, name = named(lambda: vs.vs_unit_products(X, W, off))
    assert name == "k_unit_rows" + form
    want = torch.empty(m, cols)
    for g in unit.unique().tolist():
        a, b = int(off[g]), int(off[g + 1])
        want[a:b] = X[a:b].float().cpu() @ W[g].float().cpu().T
    same(got, want, t)


@pytest.mark.parametrize("nq,nc,d,form", [
    (4, 4096, 256, "_few"), (4, 4096, 255, "<64x64,0>"), (4, 4096, 767, "_few"),
    (4, 32768, 767, "<64x64,0>"), (5, 4096, 256, "<64x64,16>"), (16, 9000, 1024, "_few"),
    (17, 9000, 1024, "<64x64,16>"), (16, 4096, 1027, "_few"), (16, 9000, 1027, "<64x64,0>"),
    (256, 300, 1024, "_few"), (1024, 300, 1024, "<64x64,16>"), (16, 9000, 1020, "<64x64,4>"),
    (16, 9000, 1028, "_few")])
def test_few_queries(nq, nc, d, form):
    """The form for few queries, on both sides of each border."""
    r = rng(85, nq, nc, d)
    x, t = (torch.from_numpy(r.integers(-120, 121, s).astype(np.int8)) for s in ((nq, d), (nc, d)))
    one = torch.ones(max(nq, nc), device=dev())
    got, name = named(lambda: vs.vs_q8_scores(x.to(dev()), one[:nq], t.to(dev()), one[:nc]))
    assert name == "k_q8_scores" + form
    same(got, x.float() @ t.float().T, torch.float32)  # below 2^24


def test_few_queries_over_very_many_rows():
    """More workgroups than a launch takes at a time, in the form for few queries."""
    nc, d = 150000000, 4
    gen = torch.Generator(device=dev()).manual_seed(9)
    t = torch.empty(nc, d, dtype=torch.int8, device=dev()).random_(-100, 101, generator=gen)
    one = torch.ones(nc, device=dev())
    q = t[nc // 2:nc // 2 + 1].contiguous()
    got, name = named(lambda: vs.vs_q8_scores(q, one[:1], t, one))
    assert name == "k_q8_scores_few"
    for lo in range(0, nc, 1 << 25):
        assert torch.equal(got[0, lo:lo + (1 << 25)], (t[lo:lo + (1 << 25)].float() * q.float()).sum(1))


def test_timed_names():
    """The timing hook names each call's own kernel; both gradients are timed."""
    x = torch.ones(6, 64, device=dev())
    w, rs = torch.ones(64, device=dev()), torch.ones(6, device=dev())
    for call, name in ((lambda: vs.vs_norm_rows(x, w), "k_norm_rows"),
                       (lambda: vs.vs_norm_rows_q8(x, w), "k_norm_rows_q8"),
                       (lambda: vs.vs_q8_quantize(x), "k_q8_quantize"),
                       (lambda: vs.vs_norm_rows_backward(x, x, w, rs), "k_norm_rows_bwd")):
        assert named(call)[1] == name
    W, off = torch.ones(2, 8, 64, device=dev()), i32(np.array([0, 2, 6]))
    with vs.KernelTimer(8) as kt:
        vs.vs_unit_products_backward(torch.ones(6, 8, device=dev()), x, W, off)
    assert kt.launches == 2 and kt.ms > 0 and kt.name.startswith("k_unit_mats")
