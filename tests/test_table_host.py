"""Host-side checks of the table operators (rows grouped by unit, row lookup,
routing, 4-bit tables): every refusal comes before anything is enqueued, so
fake, never-dereferenced addresses are enough (no GPU needed)."""
import ctypes

import pytest

import farthest_vector_search_amd as vs

torch = pytest.importorskip("torch")

FAKE = 0x10000  # 256-byte aligned
NULL, SHAPE, WORKSPACE, ALIGN, DTYPE = 1, 2, 4, 5, 9
BIG = 1 << 40


def _P(x):
    return ctypes.c_void_p(x)


@pytest.fixture(scope="module")
def L():
    return vs.lib()


def test_status_text(L):
    assert L.vs_status_str(DTYPE).decode() == "unknown or unsuitable element type"
    assert vs.STATUS[DTYPE] == "VS_ERR_DTYPE"


def test_group_rows(L):
    def call(ids=FAKE, n=10, g=4, order=FAKE, offsets=FAKE, slot=FAKE, ws=FAKE, size=BIG):
        return L.vs_group_rows(_P(ids), n, g, _P(order), _P(offsets), _P(slot), _P(ws), size,
                               None)
    assert call(n=-1) == SHAPE
    assert call(n=2 ** 31) == SHAPE
    assert call(g=0) == SHAPE
    assert call(g=2 ** 31 - 1) == SHAPE
    for name in ("ids", "order", "offsets"):
        assert call(**{name: 0}) == NULL
    assert call(n=5000, ws=0) == NULL and call(n=50, g=5000, ws=0) == NULL
    for name in ("ids", "order", "offsets", "slot"):
        assert call(**{name: FAKE + 2}) == ALIGN
    assert call(ws=FAKE + 64) == ALIGN
    need = L.vs_group_rows_workspace(1 << 20, 1000)
    assert need >= 16 << 20
    assert call(n=1 << 20, g=1000, size=need - 1) == WORKSPACE
    assert L.vs_group_rows_workspace(-1, 4) == 0
    assert L.vs_group_rows_workspace(4, 0) == 0
    assert L.vs_group_rows_workspace(10, 4) == 0  # counted in one launch
    assert L.vs_group_rows_workspace(10, 100000) == 256


def test_row_lookup(L):
    def call(T=FAKE, g=4, d=8, dtype=0, ids=FAKE, n=3, Y=FAKE):
        return L.vs_row_lookup(_P(T), g, d, dtype, _P(ids), n, 1.0, _P(Y), None)
    assert call(dtype=3) == DTYPE
    assert call(dtype=-1) == DTYPE
    for bad in (dict(g=0), dict(d=0), dict(n=-1), dict(d=(1 << 20) + 1), dict(n=2 ** 31)):
        assert call(**bad) == SHAPE
    assert call(n=0, T=0, ids=0, Y=0) == 0
    for name in ("T", "ids", "Y"):
        assert call(**{name: 0}) == NULL
        assert call(**{name: FAKE + 2}) == ALIGN
        assert call(**{name: FAKE + 1}, dtype=1) == ALIGN


def test_row_lookup_backward(L):
    def call(dY=FAKE, n=3, d=8, dtype=1, ids=FAKE, order=FAKE, offsets=FAKE, g=4, gd=1, dT=FAKE,
             ws=FAKE, size=BIG):
        return L.vs_row_lookup_backward(_P(dY), n, d, dtype, _P(ids), _P(order), _P(offsets), g,
                                        1.0, gd, _P(dT), _P(ws), size, None)
    assert call(dtype=5) == DTYPE
    assert call(gd=2) == DTYPE          # neither the rows' type nor float32
    assert call(dtype=0, gd=1) == DTYPE
    for bad in (dict(g=0), dict(d=0), dict(n=-1)):
        assert call(**bad) == SHAPE
    for name in ("dY", "ids", "order", "offsets", "dT"):
        assert call(**{name: 0}) == NULL
    # two float32 rows per 16 rows (64 beyond 4,096 rows), none up to 16
    assert call(n=17, ws=0) == NULL
    assert L.vs_row_lookup_backward_workspace(16, 8) == 0
    assert L.vs_row_lookup_backward_workspace(17, 8) == 2 * 2 * 8 * 4
    assert L.vs_row_lookup_backward_workspace(4097, 8) == 65 * 2 * 8 * 4
    assert call(n=0, dY=0, ids=0, order=0, dT=0) == NULL  # the gradient is still written
    for name in ("ids", "order", "offsets"):
        assert call(**{name: FAKE + 2}) == ALIGN
    assert call(dY=FAKE + 1) == ALIGN
    assert call(gd=0, dT=FAKE + 2) == ALIGN
    assert call(ws=FAKE + 4) == ALIGN
    need = L.vs_row_lookup_backward_workspace(1000, 64)
    assert call(n=1000, d=64, size=need - 1) == WORKSPACE
    assert L.vs_row_lookup_backward_workspace(-1, 64) == 0
    assert L.vs_row_lookup_backward_workspace(1, 0) == 0


def test_route_and_combine(L):
    def route(X=FAKE, n=3, d=8, dtype=0, slot=FAKE, off=FAKE, g=4, k=2, Xs=FAKE):
        return L.vs_route_rows(_P(X), n, d, dtype, _P(slot), _P(off), g, k, _P(Xs), None)

    def route_b(dXs=FAKE, n=3, d=8, dtype=0, slot=FAKE, k=2, dX=FAKE):
        return L.vs_route_rows_backward(_P(dXs), n, d, dtype, _P(slot), k, _P(dX), None)

    def comb(Ys=FAKE, n=3, d=8, dtype=0, slot=FAKE, w=FAKE, k=2, Y=FAKE):
        return L.vs_combine_rows(_P(Ys), n, d, dtype, _P(slot), _P(w), k, _P(Y), None)

    def comb_b(dY=FAKE, Ys=FAKE, n=3, d=8, dtype=0, slot=FAKE, w=FAKE, off=FAKE, g=4, k=2,
               dYs=FAKE, dw=FAKE):
        return L.vs_combine_rows_backward(_P(dY), _P(Ys), n, d, dtype, _P(slot), _P(w), _P(off),
                                          g, k, _P(dYs), _P(dw), None)
    for call, ptrs in ((route, ("X", "slot", "off", "Xs")), (route_b, ("dXs", "slot", "dX")),
                       (comb, ("Ys", "slot", "w", "Y")),
                       (comb_b, ("dY", "Ys", "slot", "w", "off", "dYs", "dw"))):
        assert call(dtype=3) == DTYPE
        for bad in (dict(n=-1), dict(d=0), dict(k=0), dict(k=1025), dict(n=2 ** 30, k=2)):
            assert call(**bad) == SHAPE
        for name in ptrs:
            assert call(**{name: 0}) == NULL
            assert call(**{name: FAKE + 2}) == ALIGN
        assert call(n=0, **{name: 0 for name in ptrs}) == 0
    assert route(g=0) == SHAPE
    assert comb_b(g=0) == SHAPE


def test_q4(L):
    # 16 x 128 blocks of 1 KiB of codes and 128 / group x 16 scales of 2 bytes
    assert L.vs_q4_bytes(1, 1, 32) == 1024 + 128
    assert L.vs_q4_bytes(17, 129, 64) == 4 * (1024 + 64)
    assert L.vs_q4_bytes(16, 256, 128) == 2 * (1024 + 32)
    for bad in ((0, 8, 32), (8, 0, 32), (8, 8, 16), (8, 8, 256), (2 ** 31, 8, 32)):
        assert L.vs_q4_bytes(*bad) == 0

    def quant(T=FAKE, nc=4, d=8, dtype=0, group=32, sd=1, codes=FAKE, scales=FAKE):
        return L.vs_q4_quantize(_P(T), nc, d, dtype, group, sd, _P(codes), _P(scales), None)

    def layout(codes=FAKE, scales=FAKE, nc=4, d=8, group=32, out=FAKE):
        return L.vs_q4_layout(_P(codes), _P(scales), nc, d, group, _P(out), None)

    def scores(x=FAKE, nq=2, d=8, dtype=2, table=FAKE, nc=4, group=32, sd=1, y=FAKE):
        return L.vs_q4_scores(_P(x), nq, d, dtype, _P(table), nc, group, sd, _P(y), None)
    assert quant(dtype=3) == DTYPE and scores(dtype=-1) == DTYPE
    assert quant(sd=0) == DTYPE and scores(sd=0) == DTYPE  # scales are 16 bits
    for call in (quant, layout, scores):
        for bad in (dict(nc=0), dict(d=0), dict(group=48), dict(nc=2 ** 31)):
            assert call(**bad) == SHAPE
    assert scores(nq=-1) == SHAPE
    assert scores(nq=0, x=0, y=0) == 0
    for call, ptrs in ((quant, ("T", "codes", "scales")), (layout, ("codes", "scales", "out")),
                       (scores, ("x", "table", "y"))):
        for name in ptrs:
            assert call(**{name: 0}) == NULL
    assert quant(T=FAKE + 2) == ALIGN and quant(scales=FAKE + 1) == ALIGN
    assert layout(scales=FAKE + 1) == ALIGN and layout(out=FAKE + 8) == ALIGN
    assert scores(x=FAKE + 1) == ALIGN and scores(table=FAKE + 8) == ALIGN
    assert scores(y=FAKE + 2) == ALIGN


def test_host_tensors_are_refused():
    X = torch.ones(4, 8)
    i = torch.zeros(4, dtype=torch.int32)
    o = torch.zeros(3, dtype=torch.int32)
    w = torch.ones(4, 1)
    c = torch.zeros(4, 4, dtype=torch.uint8)
    for call in (lambda: vs.vs_group_rows(i, 2), lambda: vs.vs_row_lookup(X, i),
                 lambda: vs.vs_row_lookup_backward(X, i, i, o),
                 lambda: vs.vs_route_rows(X, i, o, 1), lambda: vs.vs_route_rows_backward(X, i, 1),
                 lambda: vs.vs_combine_rows(X, i, w),
                 lambda: vs.vs_combine_rows_backward(X, X, i, w, o),
                 lambda: vs.vs_q4_quantize(X), lambda: vs.vs_q4_layout(c, X.half(), 8),
                 lambda: vs.vs_q4_scores(X, c, 4)):
        with pytest.raises(TypeError, match="CUDA"):
            call()
