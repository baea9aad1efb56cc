"""Host-side checks of the units' products, the row norm and the 8-bit tables:
every refusal comes before anything is enqueued, so fake, never-dereferenced
addresses are enough (no GPU needed)."""
import ctypes

import pytest

import farthest_vector_search_amd as vs

torch = pytest.importorskip("torch")

FAKE = 0x10000  # 256-byte aligned
NULL, SHAPE, WORKSPACE, ALIGN, DTYPE = 1, 2, 4, 5, 9
BIG = 1 << 40
WIDE = (1 << 20) + 1


def _P(x):
    return ctypes.c_void_p(x)


@pytest.fixture(scope="module")
def L():
    return vs.lib()


def test_unit_products(L):
    def call(Xs=FAKE, m=5, d=8, dtype=0, W=FAKE, off=FAKE, g=3, cols=4, Ys=FAKE):
        return L.vs_unit_products(_P(Xs), m, d, dtype, _P(W), _P(off), g, cols, _P(Ys), None)
    assert call(dtype=3) == DTYPE and call(dtype=-1) == DTYPE
    for bad in (dict(m=-1), dict(m=2 ** 31), dict(d=0), dict(d=WIDE), dict(cols=0),
                dict(cols=WIDE), dict(g=0), dict(g=2 ** 31 - 1)):
        assert call(**bad) == SHAPE
    assert call(m=0, Xs=0, W=0, off=0, Ys=0) == 0
    for name in ("Xs", "W", "off", "Ys"):
        assert call(**{name: 0}) == NULL
        assert call(**{name: FAKE + 2}) == ALIGN
        assert call(**{name: FAKE + 1}, dtype=2) == ALIGN


def test_unit_products_backward(L):
    def call(dYs=FAKE, Xs=FAKE, m=5, d=8, dtype=0, W=FAKE, off=FAKE, g=3, cols=4, dXs=FAKE, gd=0,
             dW=FAKE, ws=FAKE, size=BIG):
        return L.vs_unit_products_backward(_P(dYs), _P(Xs), m, d, dtype, _P(W), _P(off), g, cols,
                                           _P(dXs), gd, _P(dW), _P(ws), size, None)
    assert call(dtype=3) == DTYPE
    assert call(gd=1) == DTYPE and call(dtype=1, gd=2) == DTYPE and call(gd=-1) == DTYPE
    for bad in (dict(m=-1), dict(m=2 ** 31), dict(d=0), dict(d=WIDE), dict(cols=0),
                dict(cols=WIDE), dict(g=0), dict(g=2 ** 31 - 1)):
        assert call(**bad) == SHAPE
    for name in ("dYs", "Xs", "W", "off"):
        assert call(**{name: 0}) == NULL
    assert call(dXs=0, dW=0) == NULL          # nothing to compute
    assert call(dXs=0, Xs=0) == NULL          # dW needs Xs
    assert call(dW=0, W=0) == NULL            # dXs needs W
    assert call(m=0, dYs=0, Xs=0, W=0, dXs=0, off=0) == NULL  # dW is still written
    for name in ("dYs", "Xs", "W", "off", "dXs", "dW"):
        assert call(**{name: FAKE + 2}) == ALIGN
    assert call(dtype=1, gd=0, dW=FAKE + 2) == ALIGN
    # units of many rows and few, small matrices are summed in runs of rows
    need = L.vs_unit_products_backward_workspace(4096, 64, 4, 32)
    assert need >= 2 * 4 * 64 * 32 * 4 and need % (4 * 64 * 32 * 4) == 0
    many = dict(m=4096, d=64, g=4, cols=32)
    assert call(**many, size=need - 1) == WORKSPACE
    assert call(**many, ws=0) == NULL and call(**many, ws=FAKE + 64) == ALIGN
    assert L.vs_unit_products_backward_workspace(100, 64, 4, 32) == 0
    assert L.vs_unit_products_backward_workspace(1 << 20, 2048, 64, 2048) == 0
    for bad in ((-1, 64, 4, 32), (100, 0, 4, 32), (100, 64, 0, 32), (100, 64, 4, 0)):
        assert L.vs_unit_products_backward_workspace(*bad) == 0


def test_norm_rows(L):
    def rows(X=FAKE, R=FAKE, w=FAKE, n=5, d=8, dtype=0, eps=1e-6, H=FAKE, Y=FAKE, rstd=FAKE):
        return L.vs_norm_rows(_P(X), _P(R), _P(w), n, d, dtype, eps, _P(H), _P(Y), _P(rstd), None)

    def q8(X=FAKE, R=FAKE, w=FAKE, n=5, d=8, dtype=0, eps=1e-6, H=FAKE, codes=FAKE, scales=FAKE):
        return L.vs_norm_rows_q8(_P(X), _P(R), _P(w), n, d, dtype, eps, _P(H), _P(codes),
                                 _P(scales), None)
    for call, need, aligned in ((rows, ("X", "H", "Y"), ("X", "R", "w", "H", "Y", "rstd")),
                                (q8, ("X", "H", "codes", "scales"),
                                 ("X", "R", "w", "H", "scales"))):
        assert call(dtype=3) == DTYPE and call(dtype=-1) == DTYPE
        for bad in (dict(n=-1), dict(n=2 ** 31), dict(d=0), dict(d=WIDE), dict(eps=-1e-6),
                    dict(eps=float("nan")), dict(eps=float("inf"))):
            assert call(**bad) == SHAPE
        assert call(n=0, X=0, H=0) == 0
        for name in need:
            assert call(**{name: 0}) == NULL
        for name in aligned:
            assert call(**{name: FAKE + 2}) == ALIGN


def test_norm_rows_backward(L):
    def call(dY=FAKE, H=FAKE, w=FAKE, dH=FAKE, rstd=FAKE, n=5, d=8, dtype=1, dX=FAKE, gd=1,
             dw=FAKE, ws=FAKE, size=BIG):
        return L.vs_norm_rows_backward(_P(dY), _P(H), _P(w), _P(dH), _P(rstd), n, d, dtype, _P(dX),
                                       gd, _P(dw), _P(ws), size, None)
    assert call(dtype=3, gd=3) == DTYPE and call(gd=2) == DTYPE and call(gd=5) == DTYPE
    for bad in (dict(n=-1), dict(n=2 ** 31), dict(d=0), dict(d=WIDE)):
        assert call(**bad) == SHAPE
    assert call(n=0, dw=0, dY=0, H=0, rstd=0, dX=0) == 0
    for name in ("dY", "H", "rstd", "dX", "ws"):
        assert call(**{name: 0}) == NULL
    for name in ("dY", "H", "w", "dH", "dX", "dw"):
        assert call(**{name: FAKE + 1}) == ALIGN
    assert call(rstd=FAKE + 2) == ALIGN and call(ws=FAKE + 64) == ALIGN
    assert call(gd=0, dw=FAKE + 2) == ALIGN
    need = L.vs_norm_rows_backward_workspace(1000, 64)
    assert 64 * 4 <= need <= 1000 * 64 * 4
    assert call(n=1000, d=64, size=need - 1) == WORKSPACE
    assert L.vs_norm_rows_backward_workspace(-1, 64) == 0
    assert L.vs_norm_rows_backward_workspace(1, 0) == 0
    assert L.vs_norm_rows_backward_workspace(0, 64) == 0


def test_q8(L):
    def quant(T=FAKE, n=5, d=8, dtype=0, codes=FAKE, scales=FAKE):
        return L.vs_q8_quantize(_P(T), n, d, dtype, _P(codes), _P(scales), None)

    def scores(x=FAKE, xs=FAKE, nq=2, d=8, t=FAKE, ts=FAKE, nc=4, od=0, y=FAKE):
        return L.vs_q8_scores(_P(x), _P(xs), nq, d, _P(t), _P(ts), nc, od, _P(y), None)
    assert quant(dtype=3) == DTYPE and scores(od=3) == DTYPE and scores(od=-1) == DTYPE
    for bad in (dict(n=-1), dict(n=2 ** 31), dict(d=0), dict(d=WIDE)):
        assert quant(**bad) == SHAPE
    for bad in (dict(nq=-1), dict(nq=2 ** 31), dict(nc=0), dict(nc=2 ** 31), dict(d=0),
                dict(d=131072)):
        assert scores(**bad) == SHAPE
    assert quant(n=0, T=0, codes=0, scales=0) == 0
    assert scores(nq=0, x=0, xs=0, t=0, ts=0, y=0) == 0
    for name in ("T", "codes", "scales"):
        assert quant(**{name: 0}) == NULL
    for name in ("x", "xs", "t", "ts", "y"):
        assert scores(**{name: 0}) == NULL
    assert quant(T=FAKE + 2) == ALIGN and quant(scales=FAKE + 2) == ALIGN
    assert scores(xs=FAKE + 2) == ALIGN and scores(ts=FAKE + 1) == ALIGN
    assert scores(y=FAKE + 2) == ALIGN and scores(od=2, y=FAKE + 1) == ALIGN


def test_host_tensors_are_refused():
    X, W, v = torch.ones(4, 8), torch.ones(2, 3, 8), torch.ones(4)
    o = torch.zeros(3, dtype=torch.int32)
    c = torch.zeros(4, 8, dtype=torch.int8)
    for call in (lambda: vs.vs_unit_products(X, W, o),
                 lambda: vs.vs_unit_products_backward(X, X, W, o),
                 lambda: vs.vs_norm_rows(X), lambda: vs.vs_norm_rows_q8(X),
                 lambda: vs.vs_norm_rows_backward(X, X, None, v),
                 lambda: vs.vs_q8_quantize(X), lambda: vs.vs_q8_scores(c, v, c, v)):
        with pytest.raises(TypeError, match="CUDA"):
            call()
