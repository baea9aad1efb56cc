"""Products of rows in unit order with their unit's matrix and their gradients, on
the GPU against plain implementations in 64 bits.

Tolerances.  u(t) = eps(t) / 2 is the rounding of a stored result, v = 2^-24 that
of one fp32 operation.  A sum of K products: products of 16-bit values are exact
in fp32, fp32 ones round once, and the K additions inside the matrix instructions
are taken at a whole unit 2 v each, because their rounding is not documented to be
to nearest: 2 v (K + 1) sum |a b| + u(t) |exact|, plus half the smallest subnormal
of t, and 2^-149 per product that falls below the normal numbers.  Where inputs
are small whole numbers every sum is exact in fp32, and equality is asked for."""
import warnings

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import farthest_vector_search_amd as vs  # noqa: E402
from test_table_ops import SUB, TYPES, U, V, close, dev, host, i32, rng, rows  # noqa: E402


def make_offsets(r, m, G, kind):
    """Places of G units' rows among m: even, skewed, all on one, none, some units
    empty; but for `even` some rows belong to none."""
    if kind == "none":
        count = np.zeros(G, np.int64)
    elif kind == "one":
        count = np.zeros(G, np.int64)
        count[G // 2] = m
    else:
        p = np.ones(G) if kind == "even" else np.exp(2 * r.random(G)) * (r.random(G) < 0.7)
        p[r.integers(0, G)] += 1e-3
        kept = m if kind == "even" else m - m // 9
        count = r.multinomial(kept, p / p.sum())
    return np.concatenate([[0], np.cumsum(count)]).astype(np.int32)


def reference(X, W, off, dY=None):
    """Y, dX, dW in 64 bits, and the sums of magnitudes behind each."""
    m, (G, cols, d) = X.shape[0], W.shape
    out = [np.zeros((m, cols)), np.zeros((m, d)), np.zeros(W.shape)]
    mag = [np.zeros((m, cols)), np.zeros((m, d)), np.zeros(W.shape)]
    for g in range(G):
        s = slice(off[g], off[g + 1])
        out[0][s] = X[s] @ W[g].T
        mag[0][s] = np.abs(X[s]) @ np.abs(W[g]).T
        if dY is not None:
            out[1][s], mag[1][s] = dY[s] @ W[g], np.abs(dY[s]) @ np.abs(W[g])
            out[2][g], mag[2][g] = dY[s].T @ X[s], np.abs(dY[s]).T @ np.abs(X[s])
    return out, mag


def bound(K, mag, exact, t):
    return 2 * V * (K + 1) * mag + U(t) * np.abs(exact) + SUB[t] + K * 2.0 ** -149


def check_all(r, m, G, d, cols, kind, t, grad=None):
    off = make_offsets(r, m, G, kind)
    X, X64 = rows(r, (m, d), t)
    W, W64 = rows(r, (G, cols, d), t, 1 / np.sqrt(d))
    dY, dY64 = rows(r, (m, cols), t)
    X[off[-1]:], dY[off[-1]:] = float("nan"), float("inf")  # never used
    (Y, dX, dW), (mY, mX, mW) = reference(X64, W64, off, dY64)
    o = i32(off)
    close(vs.vs_unit_products(X, W, o), Y, bound(d, mY, Y, t))
    gX, gW = vs.vs_unit_products_backward(dY, X, W, o, grad_dtype=grad)
    assert gW.dtype == (grad or t)
    close(gX, dX, bound(cols, mX, dX, t))
    close(gW, dW, bound(np.diff(off)[:, None, None], mW, dW, grad or t))


CASES = [
    # m, G, d, cols, kind
    (1, 1, 1, 1, "even"), (1, 3, 8, 8, "one"), (5, 7, 3, 2, "even"), (16, 64, 64, 40, "even"),
    (33, 4, 17, 65, "skew"), (200, 3, 64, 64, "skew"), (64, 1, 32, 16, "even"),
    (130, 5, 250, 33, "skew"), (257, 2, 129, 257, "even"), (300, 9, 264, 136, "skew"),
    (40, 5, 96, 72, "none"), (700, 3, 72, 520, "one"), (1, 300, 40, 24, "even"),
    (90, 4200, 8, 8, "skew"), (1000, 6, 128, 256, "skew"), (515, 2, 1000, 24, "even"),
    (2049, 17, 56, 120, "skew"), (600, 1, 513, 300, "even"),
]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("m,G,d,cols,kind", CASES)
def test_unit_products(m, G, d, cols, kind, t):
    check_all(rng(40, m, G, d, cols), m, G, d, cols, kind, t)


@pytest.mark.parametrize("t", [torch.float16, torch.bfloat16])
def test_matrices_gradient_in_32_bits(t):
    check_all(rng(41), 210, 4, 48, 80, "skew", t, grad=torch.float32)
    check_all(rng(41), 3000, 3, 48, 80, "skew", t, grad=torch.float32)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("m,G,d,cols,kind", [(3000, 2, 24, 40, "skew"), (6000, 3, 65, 33, "one"),
                                             (2600, 2, 8, 8, "none"), (5001, 1, 130, 70, "even"),
                                             (40000, 4, 16, 16, "skew")])
def test_matrices_gradient_in_runs(m, G, d, cols, kind, t):
    """Units of many rows with few, small matrices: their rows are summed in runs.
    One addition more per run (32 at most), which the bound's K covers."""
    assert vs.lib().vs_unit_products_backward_workspace(m, d, G, cols) > 0
    check_all(rng(53, m, d), m, G, d, cols, kind, t)


def whole(r, shape, t, top=3):
    x = r.integers(-top, top + 1, shape).astype(np.float64)
    return torch.from_numpy(x).to(t).to(dev()), x


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("m,G,d,cols", [(70, 3, 40, 24), (513, 4, 128, 136), (1100, 2, 328, 512),
                                        (300, 5, 131, 77), (900, 3, 256, 264), (24, 6, 2048, 512),
                                        (20, 9, 1000, 96)])
def test_whole_numbers_are_exact(m, G, d, cols, t):
    """Sums of small whole numbers: every product lands in its place, once.
    Results below 256 in magnitude or rounded once from an exact sum."""
    r = rng(42, m, d)
    off = make_offsets(r, m, G, "skew")
    (X, X64), (W, W64), (dY, dY64) = (whole(r, s, t) for s in ((m, d), (G, cols, d), (m, cols)))
    (Y, dX, dW), _ = reference(X64, W64, off, dY64)
    gX, gW = vs.vs_unit_products_backward(dY, X, W, i32(off))
    for got, want in ((vs.vs_unit_products(X, W, i32(off)), Y), (gX, dX), (gW, dW)):
        assert np.array_equal(host(got), host(torch.from_numpy(want).to(t)))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("m,G,d,cols", [(300, 5, 66, 130), (700, 2, 258, 514), (900, 4, 30, 6),
                                        (2000, 3, 10, 700), (70, 9, 1030, 36), (5000, 20, 390, 262)])
def test_rows_on_four_bytes(m, G, d, cols, t):
    """Even widths that no multiple of 8 divides: rows of 16 bits on 4-byte addresses,
    and the same a half-word off them."""
    check_all(rng(54, m, d), m, G, d, cols, "skew", t)
    r = rng(55, m, d)
    off = i32(make_offsets(r, m, G, "skew"))
    X, W = rows(r, (m, d), t)[0], rows(r, (G, cols, d), t)[0]
    want = vs.vs_unit_products(X, W, off)
    for s in (1, 2):
        at = torch.empty(X.numel() + 8, dtype=t, device=dev())[s:s + X.numel()].view(X.shape)
        close(vs.vs_unit_products(at.copy_(X), W, off), host(want),
              2 * bound(d, host(X.float().abs()) @ np.ones((d, cols)) * float(W.abs().max()),
                        host(want), t))


@pytest.mark.parametrize("t", [torch.float16, torch.bfloat16])
def test_last_tiles_of_every_height(t):
    """Units of some hundred rows, whose last tiles have few rows, many, or all."""
    r = rng(56)
    G, d, cols = 120, 512, 1024
    count = 256 * r.integers(0, 3, G) + np.resize(
        [0, 1, 15, 63, 64, 65, 100, 127, 128, 129, 192, 255], G)
    off = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    m = int(off[-1])
    assert m // G >= 200
    (X, X64), (W, W64), (dY, dY64) = (whole(r, s, t, 1) for s in ((m, d), (G, cols, d), (m, cols)))
    Y = vs.vs_unit_products(X, W, i32(off))
    dX, _ = vs.vs_unit_products_backward(dY, X, W, i32(off), want_dW=False)
    for g in range(G):
        a, b = off[g], off[g + 1]
        w = W64[g].astype(np.float32)  # sums below 2^24: exact
        for got, want in ((Y, X64[a:b].astype(np.float32) @ w.T),
                          (dX, dY64[a:b].astype(np.float32) @ w)):
            assert torch.equal(got[a:b].cpu(), torch.from_numpy(want).to(t))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("G", [1, 2, 63, 64, 65, 129, 200, 255, 256, 257, 400])
def test_every_row_is_taken_once(G, t):
    """Few and many units, some empty, with rows before the first and behind the last:
    each row is its unit's alone."""
    r = rng(57, G)
    d, cols = 24, 200
    count = r.integers(0, 150, G) * (r.random(G) < 0.8)
    count[r.integers(0, G)] += 70
    off = (37 + np.concatenate([[0], np.cumsum(count)])).astype(np.int32)
    m = int(off[-1]) + 333
    (X, X64), (W, W64), (dY, dY64) = (whole(r, s, t, 1) for s in ((m, d), (G, cols, d), (m, cols)))
    (Y, dX, _), _ = reference(X64, W64, off, dY64)
    X[:37], X[off[-1]:], dY[:37], dY[off[-1]:] = (float("nan"),) * 4
    assert np.array_equal(host(vs.vs_unit_products(X, W, i32(off))), Y)
    gX, _ = vs.vs_unit_products_backward(dY, X, W, i32(off), want_dW=False)
    assert np.array_equal(host(gX), host(torch.from_numpy(dX).to(t)))


@pytest.mark.parametrize("t", TYPES)
def test_differences(t):
    """The loss sum(R * Y) is linear in X and in W, and exact for small whole
    numbers: moving one element by 1 moves it by that element's gradient."""
    r = rng(43)
    m, G, d, cols = 23, 4, 24, 16
    off = make_offsets(r, m, G, "skew")
    (X, _), (W, _), (R, R64) = (whole(r, s, t, 2) for s in ((m, d), (G, cols, d), (m, cols)))
    gX, gW = (host(a) for a in vs.vs_unit_products_backward(R, X, W, i32(off)))
    loss = lambda: (host(vs.vs_unit_products(X, W, i32(off))) * R64).sum()  # noqa: E731
    base = loss()
    for T, grad in ((X, gX), (W, gW)):
        flat = T.view(-1)
        for at in r.integers(0, flat.numel(), 12):
            keep = flat[at].clone()
            flat[at] += 1
            assert loss() - base == grad.reshape(-1)[at]
            flat[at] = keep


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d,cols", [(64, 64), (65, 63), (200, 136)])
def test_values_stay_with_their_unit(d, cols, t):
    """A NaN or an infinity in a row, a matrix or an upstream row reaches the results
    that it is a factor of, and no others: neighbouring units' results are
    the same bits with and without it."""
    r = rng(44, d)
    m, G = 150, 5
    off = np.array([0, 31, 31, 70, 149, 150], np.int32)
    X, _ = rows(r, (m, d), t)
    W, _ = rows(r, (G, cols, d), t)
    dY, _ = rows(r, (m, cols), t)
    o = i32(off)
    Y0 = vs.vs_unit_products(X, W, o)
    dX0, dW0 = vs.vs_unit_products_backward(dY, X, W, o)
    X[70, 0], X[69, d - 1], X[148, d // 2] = float("nan"), float("inf"), float("-inf")
    W[3, cols - 1, d - 1], dY[30, cols - 1] = float("nan"), float("inf")
    Y = vs.vs_unit_products(X, W, o)
    dX, dW = vs.vs_unit_products_backward(dY, X, W, o)
    bad = torch.zeros(m, cols, dtype=torch.bool)
    bad[[69, 70, 148]] = True
    bad[70:149, cols - 1] = True
    assert torch.equal(Y[~bad], Y0[~bad]) and not torch.isfinite(Y.cpu()[bad]).any()
    bad = torch.zeros(m, d, dtype=torch.bool)
    bad[70:149, d - 1] = True
    bad[30] = True
    assert torch.equal(dX[~bad], dX0[~bad]) and not torch.isfinite(dX.cpu()[bad]).any()
    bad = torch.zeros(G, cols, d, dtype=torch.bool)
    bad[0, cols - 1] = True
    bad[2, :, d - 1] = True
    bad[3, :, 0] = True
    bad[3, :, d // 2] = True
    assert torch.equal(dW[~bad], dW0[~bad]) and not torch.isfinite(dW.cpu()[bad]).any()


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("shift", [1, 3, 4])
def test_addresses_and_outputs(t, shift):
    """Matrices at every alignment of their element; outputs are written whole and
    nothing beside them."""
    r = rng(45, shift)
    m, G, d, cols = 77, 3, 64, 48
    off = i32(make_offsets(r, m, G, "skew"))

    def at(x):
        buf = torch.empty(x.numel() + 16, dtype=x.dtype, device=dev())
        v = buf[shift:shift + x.numel()].view(x.shape)
        v.copy_(x)
        return v

    def guarded(*shape):
        n = int(np.prod(shape))
        buf = torch.full((n + 64,), 7.0, dtype=t, device=dev())
        return buf, buf[32 + shift:32 + shift + n].view(shape)
    X, W, dY = (rows(r, s, t)[0] for s in ((m, d), (G, cols, d), (m, cols)))
    want = (vs.vs_unit_products(X, W, off),) + vs.vs_unit_products_backward(dY, X, W, off)
    bufs = [guarded(m, cols), guarded(m, d), guarded(G, cols, d)]
    vs.vs_unit_products(at(X), at(W), off, out=bufs[0][1])
    vs.vs_unit_products_backward(at(dY), at(X), at(W), off, out=bufs[1][1], dW=bufs[2][1])
    for (buf, v), w in zip(bufs, want):
        # the sums' order may follow the alignment
        assert torch.allclose(v.float(), w.float(), rtol=8 * U(t), atol=1e-3)
        v.fill_(7.0)
        assert bool((buf == 7.0).all())


def test_places_outside_the_rows():
    """Offsets that do not rise or lie outside [0, m] are held inside: nothing
    beside the outputs is written, and units with sound places keep their results."""
    r = rng(46)
    m, G, d, cols = 100, 4, 64, 32
    X, X64 = rows(r, (m, d), torch.bfloat16)
    W, W64 = rows(r, (G, cols, d), torch.bfloat16)
    for off in ([-5, 30, 60, 90, 1000], [0, 2 ** 31 - 1, -2 ** 31, 50, 100], [100, 80, 40, 20, 0]):
        buf = torch.full(((m + 40) * cols,), 7.0, dtype=torch.bfloat16, device=dev())
        out = buf[20 * cols:(20 + m) * cols].view(m, cols)
        vs.vs_unit_products(X, W, i32(off), out=out)
        dW = torch.empty(G, cols, d, dtype=torch.bfloat16, device=dev())
        vs.vs_unit_products_backward(X[:, :cols].contiguous(), X, W, i32(off), dW=dW)
        assert bool((buf[:20 * cols] == 7.0).all()) and bool((buf[(20 + m) * cols:] == 7.0).all())
        if off[0] == -5:
            (Y, _, _), (mag, _, _) = reference(X64, W64, np.clip(off, 0, m))
            close(out, Y, bound(d, mag, Y, torch.bfloat16))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("m,first,d,cols", [(20, 3, 24, 16), (400, 150, 64, 72), (3000, 1000, 33, 40)])
def test_rows_before_the_first_unit(m, first, d, cols, t):
    """Places that begin behind row 0: the rows before belong to no unit."""
    r = rng(54, m)
    G = 3
    off = first + make_offsets(r, m - first, G, "skew")
    X, X64 = rows(r, (m, d), t)
    W, W64 = rows(r, (G, cols, d), t)
    dY, dY64 = rows(r, (m, cols), t)
    X[:first], dY[:first] = float("nan"), float("inf")
    (Y, dX, dW), (mY, mX, mW) = reference(X64, W64, off, dY64)
    close(vs.vs_unit_products(X, W, i32(off)), Y, bound(d, mY, Y, t))
    gX, gW = vs.vs_unit_products_backward(dY, X, W, i32(off))
    close(gX, dX, bound(cols, mX, dX, t))
    close(gW, dW, bound(np.diff(off)[:, None, None], mW, dW, t))


def test_very_many_units():
    """More tiles than a launch takes at a time."""
    m, G, d, cols = 500, 2500000, 2, 3
    r = rng(55)
    units = np.sort(r.choice(G, m // 2, replace=False))
    units = np.sort(np.concatenate([units, units[:m - m // 2]]))
    off = np.searchsorted(units, np.arange(G + 1)).astype(np.int32)
    (X, X64), (W, W64), (dY, dY64) = (whole(r, s, torch.float32)
                                      for s in ((m, d), (G, cols, d), (m, cols)))
    Y = vs.vs_unit_products(X, W, i32(off))
    dX, dW = vs.vs_unit_products_backward(dY, X, W, i32(off))
    assert np.array_equal(host(Y), np.einsum("mk,mjk->mj", X64, W64[units]))
    assert np.array_equal(host(dX), np.einsum("mj,mjk->mk", dY64, W64[units]))
    want = np.zeros((G, cols, d))
    np.add.at(want, units, dY64[:, :, None] * X64[:, None, :])
    assert np.array_equal(host(dW), want)


@pytest.mark.parametrize("t,step", [(torch.float32, 2.0 ** -149), (torch.float16, 2.0 ** -24),
                                    (torch.bfloat16, 2.0 ** -133)])
@pytest.mark.parametrize("m", [6, 100, 700])
def test_subnormal_factors(m, t, step):
    """Subnormal values are multiplied, not flushed: small multiples of the smallest
    one times small whole numbers."""
    r = rng(56, m)
    d, cols = 24, 32
    off = np.array([0, m // 2, m], np.int32)
    X64 = r.integers(-3, 4, (m, d)) * step
    X = torch.from_numpy(X64).to(t).to(dev())
    (W, W64), (dY, dY64) = whole(r, (2, cols, d), t, 2), whole(r, (m, cols), t, 2)
    (Y, _, dW), _ = reference(X64, W64, off, dY64)
    assert np.array_equal(host(vs.vs_unit_products(X, W, i32(off))), host(torch.from_numpy(Y).to(t)))
    _, gW = vs.vs_unit_products_backward(dY, X, W, i32(off))
    assert np.array_equal(host(gW), host(torch.from_numpy(dW).to(t)))


def test_no_rows():
    W = torch.ones(3, 5, 8, device=dev())
    off = i32([0, 0, 0, 0])
    X, dY = torch.empty(0, 8, device=dev()), torch.empty(0, 5, device=dev())
    assert vs.vs_unit_products(X, W, off).shape == (0, 5)
    dX, dW = vs.vs_unit_products_backward(dY, X, W, off, dW=torch.full_like(W, 3.0))
    assert dX.shape == (0, 8) and bool((dW == 0).all())


def test_one_gradient_alone():
    r = rng(47)
    off = i32([0, 3, 9])
    X, W, dY = (rows(r, s, torch.float16)[0] for s in ((9, 16), (2, 24, 16), (9, 24)))
    dX, dW = vs.vs_unit_products_backward(dY, X, W, off)
    a, none = vs.vs_unit_products_backward(dY, X, W, off, want_dW=False)
    assert none is None and torch.equal(a, dX)
    none, b = vs.vs_unit_products_backward(dY, X, W, off, want_dXs=False)
    assert none is None and torch.equal(b, dW)


def test_refusals():
    f = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device=dev())  # noqa: E731
    X, W, dY, off = f(6, 8), f(2, 4, 8), f(6, 4), i32([0, 3, 6])
    for call, error in (
            (lambda: vs.vs_unit_products(X.double(), W, off), TypeError),
            (lambda: vs.vs_unit_products(X, W.half(), off), TypeError),
            (lambda: vs.vs_unit_products(X, W, off.long()), TypeError),
            (lambda: vs.vs_unit_products(X, W.cpu(), off), TypeError),
            (lambda: vs.vs_unit_products(X, f(2, 4, 9), off), ValueError),
            (lambda: vs.vs_unit_products(X, W, off[:2]), ValueError),
            (lambda: vs.vs_unit_products(X, W[:, ::2], off), ValueError),
            (lambda: vs.vs_unit_products(X.t(), W, off), ValueError),
            (lambda: vs.vs_unit_products(X[None], W, off), ValueError),
            (lambda: vs.vs_unit_products(X, W, off, out=f(5, 4)), ValueError),
            (lambda: vs.vs_unit_products(X, f(0, 4, 8), off[:1]), vs.VsError),
            (lambda: vs.vs_unit_products_backward(f(6, 5), X, W, off), ValueError),
            (lambda: vs.vs_unit_products_backward(dY, X.float(), W, off), TypeError),
            (lambda: vs.vs_unit_products_backward(dY, X, W, off, grad_dtype=torch.float16),
             vs.VsError),
            (lambda: vs.vs_unit_products_backward(dY, X, W, off, want_dXs=False, want_dW=False),
             ValueError),
            (lambda: vs.vs_unit_products_backward(f(4096, 4), f(4096, 8), W, off,
                                                  workspace=f(8)), ValueError)):
        with pytest.raises(error):
            call()
    for call in (lambda: vs.vs_unit_products(X, W.clone().requires_grad_(), off),
                 lambda: vs.vs_unit_products_backward(dY, X.clone().requires_grad_(), W, off)):
        with pytest.warns(UserWarning, match="gradient"):
            call()


def test_streams_and_graphs():
    """Another stream; two graphs captured and replayed with new inputs, eager
    calls between the replays."""
    r = rng(48)
    m, G, d, cols = 160, 6, 96, 64
    off = i32(make_offsets(r, m, G, "skew"))
    t = torch.bfloat16
    X, W, dY = (rows(r, s, t)[0] for s in ((m, d), (G, cols, d), (m, cols)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = vs.vs_unit_products(X, W, off)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, vs.vs_unit_products(X, W, off))

    def step():
        return (vs.vs_unit_products(X, W, off),) + vs.vs_unit_products_backward(dY, X, W, off)
    step()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step()
        graphs.append((g, outs))
    for k in range(3):
        X.copy_(rows(rng(49, k), (m, d), t)[0])
        off.copy_(i32(make_offsets(rng(50, k), m, G, "skew")))
        for g, outs in graphs:
            g.replay()
            torch.cuda.synchronize()
            for got, want in zip(outs, step()):
                assert torch.equal(got, want)


def test_inside_an_autograd_function():
    class Units(torch.autograd.Function):
        @staticmethod
        def forward(ctx, X, W, off):
            ctx.save_for_backward(X, W, off)
            return vs.vs_unit_products(X, W, off)

        @staticmethod
        def backward(ctx, dY):
            X, W, off = ctx.saved_tensors
            return (*vs.vs_unit_products_backward(dY.contiguous(), X, W, off), None)
    r = rng(51)
    off = np.array([0, 4, 9], np.int32)
    (X, X64), (W, W64), (R, R64) = (whole(r, s, torch.float32) for s in ((9, 8), (2, 6, 8), (9, 6)))
    X.requires_grad_(), W.requires_grad_()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        (Units.apply(X, W, i32(off)) * R).sum().backward()
    (_, dX, dW), _ = reference(X64, W64, off, R64)
    assert np.array_equal(host(X.grad), dX) and np.array_equal(host(W.grad), dW)


def test_routed_and_combined():
    """The run of calls that a layer of units makes: picks grouped, rows routed,
    multiplied by their unit's matrix, brought back with weights; and its backward
    pass.  Small whole numbers and weights that are powers of two: exact."""
    r = rng(52)
    n, k, G, d, cols = 50, 2, 7, 32, 24
    picks = r.integers(-1, G, (n, k)).astype(np.int32)
    w64 = 2.0 ** r.integers(-2, 1, (n, k))
    (X, X64), (W, W64), (dO, dO64) = (whole(r, s, torch.float32, 2)
                                      for s in ((n, d), (G, cols, d), (n, cols)))
    w = torch.from_numpy(w64).float().to(dev())
    order, off, slot = vs.vs_group_rows(i32(picks), G)
    Xs = vs.vs_route_rows(X, slot, off, k)
    Ys = vs.vs_unit_products(Xs, W, off)
    out = vs.vs_combine_rows(Ys, slot, w)
    dYs, dw = vs.vs_combine_rows_backward(dO, Ys, slot, w, off)
    dXs, dW = vs.vs_unit_products_backward(dYs, Xs, W, off)
    dX = vs.vs_route_rows_backward(dXs, slot, k)
    want, wX, ww, wW = np.zeros((n, cols)), np.zeros((n, d)), np.zeros((n, k)), np.zeros(W64.shape)
    for i in range(n):
        for j in range(k):
            g = picks[i, j]
            if g >= 0:
                y = W64[g] @ X64[i]
                want[i] += w64[i, j] * y
                ww[i, j] = dO64[i] @ y
                wX[i] += w64[i, j] * (dO64[i] @ W64[g])
                wW[g] += w64[i, j] * np.outer(dO64[i], X64[i])
    for got, ref in ((out, want), (dX, wX), (dw, ww), (dW, wW)):
        assert np.array_equal(host(got), ref)


def test_matrices_past_32_bit_offsets():
    """More than 2^31 elements of W and of its gradient."""
    G, cols, d, m = 600, 2048, 2048, 30
    gen = torch.Generator(device=dev()).manual_seed(5)
    W = torch.empty(G, cols, d, dtype=torch.bfloat16, device=dev()).random_(-2, 3, generator=gen)
    X = torch.empty(m, d, dtype=torch.bfloat16, device=dev()).random_(-2, 3, generator=gen)
    dY = torch.empty(m, cols, dtype=torch.bfloat16, device=dev()).random_(-2, 3, generator=gen)
    count = np.zeros(G, np.int64)
    for g in (0, 511, 512, G - 1):
        count[g] = 7
    off = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    Y = vs.vs_unit_products(X, W, i32(off))
    dX, dW = vs.vs_unit_products_backward(dY, X, W, i32(off))
    for g in (0, 511, 512, G - 1):
        s = slice(off[g], off[g + 1])
        x, w, dy = host(X[s]), host(W[g]), host(dY[s])
        for got, want in ((Y[s], x @ w.T), (dX[s], dy @ w), (dW[g], dy.T @ x)):
            assert np.array_equal(host(got), host(torch.from_numpy(want).bfloat16()))
    assert bool((Y[28:] == 0).all()) and bool((dX[28:] == 0).all())
    for g in (1, 300, 513, G - 2):
        assert bool((dW[g] == 0).all())


def test_largest_number_of_rows():
    """2^31 - 1 rows of one element: every row its unit's factor times itself."""
    m = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[1] < 64 << 30:
        pytest.skip("needs 64 GiB")
    X = torch.ones((m, 1), dtype=torch.bfloat16, device=dev())
    W = torch.tensor([2.0, 3.0, 5.0], dtype=torch.bfloat16, device=dev()).view(3, 1, 1)
    for cuts in ((0, 0, 0, m), (0, 1, m - 1, m), (7, 2 ** 30 + 5, 2 ** 30 + 5, m - 9)):
        off = i32(np.array(cuts))
        for Y in (vs.vs_unit_products(X, W, off),
                  vs.vs_unit_products_backward(X, X, W, off, want_dW=False)[0]):
            ends = (0, *cuts, m)
            for f, a, b in zip((0.0, 2.0, 3.0, 5.0, 0.0), ends, ends[1:]):
                assert bool((Y[a:b] == f).all()), (cuts, f)
            del Y


@pytest.mark.parametrize("G", [2, 64, 130, 300])
def test_places_that_fall(G):
    """Offsets that go up and down: results are nobody's, but nothing beside the
    output is written, and the call ends."""
    m, d, cols = 700, 40, 72
    r = rng(58, G)
    X, W = rows(r, (m, d), torch.bfloat16)[0], rows(r, (G, cols, d), torch.bfloat16)[0]
    buf = torch.full((m + 2, cols), 7.0, dtype=torch.bfloat16, device=dev())
    for off in (np.arange(G + 1) % 2 * m, (np.arange(G + 1) + 1) % 2 * m, r.integers(-9, m + 9, G + 1)):
        vs.vs_unit_products(X, W, i32(off.astype(np.int32)), out=buf[1:-1])
        assert bool((buf[0] == 7).all()) and bool((buf[-1] == 7).all())
