"""The row norm with its 8-bit output and gradients, and scores over 8-bit tables,
on the GPU against plain implementations in 64 bits.

Tolerances.  u(t) = eps(t) / 2 is the rounding of a stored result, v = 2^-24 that
of one fp32 operation.  Sums of d terms in any order: d v relative to the sum of
magnitudes.  The mean square is a sum of d positive terms (d v), divided, added to
eps; its root halves that, and root and reciprocal round once each: rstd is within
r = (d / 2 + 4) v of its value.  Then
  Y        two products more: (r + 2 v) |Y| + u(t) |Y|
  scale    max |v| exact but for v's rounding: (r + 3 v) scale
  dX       c = mean of w dy x^ : its terms are off by r + 2 v, their sum by d v and
           the division v: e_c = (r + (d + 3) v) mean |w dy x^|; then
           rstd (w dy - x^ c): (2 r + 6 v) rstd (|w dy| + |x^ c|) + rstd |x^| e_c,
           + v |result| for dH's addition, + u(t) |result|
  dweight  n terms off by r + 2 v each: (r + (n + 2) v) sum |dy x^| + u(t) |exact|
plus half the smallest subnormal of t; everything times 1.01 for products of the
small quantities.  H is one rounding of an fp32 sum of two values, which is
the rounding of their exact sum in all cases tested (exponents less than 13 apart
for 16-bit types; fp32 addition itself for fp32).  Codes are whole numbers that
follow from H and the weight: they have to be equal.  Scores: the sum is exact,
rounded to fp32, two products: 3 v + u(t)."""
import warnings

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import farthest_vector_search_amd as vs  # noqa: E402
from test_table_ops import SUB, TYPES, U, V, close, dev, host, rng, rows  # noqa: E402

EPS = 1e-6
WIDTHS = [1, 2, 3, 7, 8, 9, 64, 100, 257, 511, 512, 513, 1030, 2048, 2055, 4096, 4099, 8192, 9000,
          20001]


def norm_ref(x, r, w, eps, t):
    """h, rms, y of rows in 64 bits; h rounded to t."""
    h = x if r is None else host(torch.from_numpy(x + r).to(t))
    ms = (h * h).mean(1, keepdims=True) + eps
    with np.errstate(divide="ignore"):
        rstd = np.where(ms > 0, 1 / np.sqrt(ms), 0.0)
    return h, rstd, h * rstd * w


def codes_ref(h, w):
    """Codes and largest magnitudes: v = h w held in fp32."""
    v = (h.astype(np.float32) * w.astype(np.float32)).astype(np.float64)
    top = np.abs(v).max(1, keepdims=True)
    return np.rint(v * 127.0 / np.where(top > 0, top, 1)), top


def r_of(d):
    return (d / 2 + 4) * V


def inputs(r, n, d, t, residual):
    x, x64 = rows(r, (n, d), t)
    res, r64 = rows(r, (n, d), t, 2.0) if residual else (None, None)
    w, w64 = rows(r, (1, d), t)
    return x, x64, res, r64, w[0] + 1, host(w[0] + 1)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("d", WIDTHS)
def test_norm_rows(d, residual, t):
    n = 5 if d > 600 else 9
    x, x64, res, r64, w, w64 = inputs(rng(60, d, residual), n, d, t, residual)
    h, rstd, y = norm_ref(x64, r64, w64, EPS, t)
    Y, H, rs = vs.vs_norm_rows(x, w, EPS, residual=res)
    assert np.array_equal(host(H), h)
    assert (H is x) == (not residual)
    close(rs, rstd[:, 0], 1.01 * r_of(d) * rstd[:, 0])
    close(Y, y, 1.01 * (r_of(d) + 2 * V + U(t)) * np.abs(y) + SUB[t])
    codes, scales, H = vs.vs_norm_rows_q8(x, w, EPS, residual=res)
    assert np.array_equal(host(H), h)
    c, top = codes_ref(h, w64)
    assert np.array_equal(host(codes), c)
    scale = (top * rstd / 127)[:, 0]
    close(scales, scale, 1.01 * (r_of(d) + 3 * V) * scale)
    codes, scales = vs.vs_q8_quantize(x)
    c, top = codes_ref(x64, np.ones(d))
    assert np.array_equal(host(codes), c)
    close(scales, top[:, 0] / 127, V * top[:, 0] / 127)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n,d", [(1, 64), (1500, 64), (1500, 768), (1501, 1000), (1200, 2048),
                                 (1030, 2041), (5000, 12), (2000, 4096), (20000, 5)])
def test_norm_rows_many(n, d, t):
    """Row counts on both sides of each change of form."""
    x, x64, res, r64, w, w64 = inputs(rng(61, n, d), n, d, t, True)
    h, rstd, y = norm_ref(x64, r64, w64, EPS, t)
    Y, H, rs = vs.vs_norm_rows(x, w, EPS, residual=res)
    assert np.array_equal(host(H), h)
    close(Y, y, 1.01 * (r_of(d) + 2 * V + U(t)) * np.abs(y) + SUB[t])
    codes, scales, H = vs.vs_norm_rows_q8(x, w, EPS, residual=res)
    c, top = codes_ref(h, w64)
    assert np.array_equal(host(codes), c)


def backward_ref(dY, h, rstd, w, dH):
    xh = h * rstd
    g = dY * w
    c = (g * xh).mean(1, keepdims=True)
    dX = rstd * (g - xh * c) + (0 if dH is None else dH)
    return dX, (dY * xh).sum(0)


def backward_tol(dY, h, rstd, w, dX, dw, t, gt):
    n, d = h.shape
    xh, r = np.abs(h * rstd), r_of(d)
    g = np.abs(dY * w)
    m = (g * xh).mean(1, keepdims=True)
    tx = ((2 * r + 6 * V) * rstd * (g + xh * m) + rstd * xh * (r + (d + 3) * V) * m
          + (V + U(t)) * np.abs(dX))
    tw = (r + (n + 2) * V) * (np.abs(dY) * xh).sum(0) + U(gt) * np.abs(dw)
    return 1.01 * tx + SUB[t], 1.01 * tw + SUB[gt]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("more", [False, True])
@pytest.mark.parametrize("n,d", [(1, 1), (3, 7), (9, 64), (700, 100), (5, 513), (1100, 768), (1023, 257),
                                 (6, 4099), (1300, 2048), (40, 8192), (7, 20001), (600, 9000),
                                 (2, 1 << 20)])
def test_norm_rows_backward(n, d, more, t):
    r = rng(62, n, d, more)
    x, x64, res, r64, w, w64 = inputs(r, n, d, t, more)
    dY, dY64 = rows(r, (n, d), t)
    dH, dH64 = rows(r, (n, d), t) if more else (None, None)
    h, rstd, _ = norm_ref(x64, r64, w64, EPS, t)
    _, H, rs = vs.vs_norm_rows(x, w, EPS, residual=res)
    dX, dw = backward_ref(dY64, h, rstd, w64, dH64)
    for gt in {t, torch.float32}:
        gX, gw = vs.vs_norm_rows_backward(dY, H, w, rs, dH=dH, grad_dtype=gt)
        assert gw.dtype == gt
        tx, tw = backward_tol(dY64, h, rstd, w64, dX, dw, t, gt)
        close(gX, dX, tx)
        close(gw, dw, tw)
    # without a weight, and the weight's gradient not wanted
    alone, none = vs.vs_norm_rows_backward(dY, H, w, rs, dH=dH, want_dweight=False)
    assert none is None and torch.equal(alone, gX)
    one = np.ones((1, d))
    dX, _ = backward_ref(dY64, h, rstd, one, dH64)
    gX, none = vs.vs_norm_rows_backward(dY, H, None, rs, dH=dH)
    assert none is None
    close(gX, dX, backward_tol(dY64, h, rstd, one, dX, dw, t, t)[0])


def test_backward_against_differences():
    """Central differences of the loss sum(R Y) in 64 bits (the forward pass's formula)
    at step e: their error is below e^2 max |L'''| + 2^-50 |L| / e, far below 1e-6
    here; the gradient's own is the bound of the formula."""
    r = rng(63)
    n, d, e = 4, 24, 1e-4
    x, x64, _, _, w, w64 = inputs(r, n, d, torch.float32, False)
    R, R64 = rows(r, (n, d), torch.float32)
    _, H, rs = vs.vs_norm_rows(x, w, EPS)
    gX, gw = (host(a) for a in vs.vs_norm_rows_backward(R, H, w, rs))

    def loss(x, w):
        return (norm_ref(x, None, w, EPS, torch.float32)[2] * R64).sum()
    for at in [(0, 0), (1, 5), (3, 23), (2, 11)]:
        step = np.zeros_like(x64)
        step[at] = e
        assert abs((loss(x64 + step, w64) - loss(x64 - step, w64)) / (2 * e) - gX[at]) < 2e-5
        step = np.zeros_like(w64)
        step[at[1]] = e
        assert abs((loss(x64, w64 + step) - loss(x64, w64 - step)) / (2 * e) - gw[at[1]]) < 2e-5


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d", [6, 40, 1001, 20000])
def test_unit_rows(d, t):
    """Weight d^-1/2 and eps 0: the unit rows the cosine metrics take; a row of
    zeros stays one."""
    x, x64 = rows(rng(64, d), (5, d), t)
    x[3] = 0
    x64[3] = 0
    w = torch.full((d,), d ** -0.5, dtype=torch.float32, device=dev()).to(t)
    Y, _, rs = vs.vs_norm_rows(x, w, 0.0)
    h, rstd, y = norm_ref(x64, None, host(w), 0.0, t)
    close(Y, y, 1.01 * (r_of(d) + 2 * V + U(t)) * np.abs(y) + SUB[t])
    assert float(rs[3]) == 0 and bool((Y[3] == 0).all())
    codes, scales, _ = vs.vs_norm_rows_q8(x, w, 0.0)
    assert float(scales[3]) == 0 and bool((codes[3] == 0).all())
    dX, dw = vs.vs_norm_rows_backward(torch.ones_like(x), x, w, rs)
    assert bool((dX[3] == 0).all()) and bool(torch.isfinite(dw).all())


@pytest.mark.parametrize("t,e", [(torch.float32, 100), (torch.float32, 64), (torch.float32, -50),
                                 (torch.float32, -100), (torch.bfloat16, 120),
                                 (torch.bfloat16, -90), (torch.float16, -12)])
@pytest.mark.parametrize("d", [64, 777, 10000])
def test_squares_beyond_the_range(d, t, e):
    """Rows whose squares over- or underflow in fp32 (in the ranges rstd has)."""
    x64 = rng(65, d).standard_normal((4, d)).clip(-4, 4) * 2.0 ** e
    x = torch.from_numpy(x64).to(t).to(dev())
    x64 = host(x)
    for eps in (0.0, 1e-6):
        h, rstd, y = norm_ref(x64, None, np.ones(d), eps, t)
        # two roundings more than the plain way: scaling and its way back
        Y, _, rs = vs.vs_norm_rows(x, None, eps)
        close(rs, rstd[:, 0], 1.01 * (r_of(d) + 8 * V) * rstd[:, 0] + 2.0 ** -149)
        # results below the normal numbers round to their spacing
        close(Y, y, 1.01 * (r_of(d) + 10 * V + U(t)) * np.abs(y) + 2 * SUB[t] + 2.0 ** -126 * (rstd < 2.0 ** -126))
        codes, scales, _ = vs.vs_norm_rows_q8(x, None, eps)
        assert np.array_equal(host(codes), codes_ref(x64, np.ones(d))[0])


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d", [20, 600, 9001])
def test_rows_that_are_not_finite(d, t):
    """A NaN or an infinity costs its own row, and no other."""
    x, x64 = rows(rng(66, d), (6, d), t)
    w = torch.ones(d, dtype=t, device=dev())
    Y0, _, _ = vs.vs_norm_rows(x, w)
    c0, s0, _ = vs.vs_norm_rows_q8(x, w)
    q0, z0 = vs.vs_q8_quantize(x)
    x[1, d - 1], x[4, 0] = float("nan"), float("inf")
    good = [0, 2, 3, 5]
    Y, _, rs = vs.vs_norm_rows(x, w)
    assert torch.equal(Y[good], Y0[good]) and bool(torch.isnan(Y[[1, 4]]).all())
    for (c, s), (cc, ss) in (((c0, s0), vs.vs_norm_rows_q8(x, w)[:2]),
                             ((q0, z0), vs.vs_q8_quantize(x))):
        assert torch.equal(cc[good], c[good]) and torch.equal(ss[good], s[good])
        assert bool((cc[[1, 4]] == 0).all()) and bool(torch.isnan(ss[[1, 4]]).all())


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n,d", [(1030, 1024), (700, 1600), (1030, 2800), (40, 6000), (1030, 6000),
                                 (1030, 6008), (9, 12001), (1030, 12000), (5, 24000), (1025, 17000),
                                 (3, 40003)])
def test_norm_rows_wide(n, d, t):
    """Wide rows, few and many: one row a workgroup of each size, held or read twice."""
    r = rng(71, n, d)
    x, x64, res, r64, w, w64 = inputs(r, n, d, t, True)
    h, rstd, y = norm_ref(x64, r64, w64, EPS, t)
    Y, H, rs = vs.vs_norm_rows(x, w, EPS, residual=res)
    assert np.array_equal(host(H), h)
    close(Y, y, 1.01 * (r_of(d) + 2 * V + U(t)) * np.abs(y) + SUB[t])
    codes, scales, _ = vs.vs_norm_rows_q8(H, w, EPS)
    c, top = codes_ref(h, w64)
    assert np.array_equal(host(codes), c)
    scale = (top * rstd / 127)[:, 0]
    close(scales, scale, 1.01 * (r_of(d) + 3 * V) * scale)
    assert np.array_equal(host(vs.vs_q8_quantize(H)[0]), codes_ref(h, np.ones(d))[0])
    dY, dY64 = rows(r, (n, d), t)
    dX, dw = backward_ref(dY64, h, rstd, w64, None)
    gX, gw = vs.vs_norm_rows_backward(dY, H, w, rs)
    tx, tw = backward_tol(dY64, h, rstd, w64, dX, dw, t, t)
    close(gX, dX, tx)
    close(gw, dw, tw)


def test_codes_beside_borders():
    """Values next to the borders of rows with any largest magnitude: the float
    nearest to each border, and the two beside it on both sides."""
    r = rng(72)
    top = np.concatenate([r.uniform(1, 2, 300), 2.0 ** -130 * r.uniform(1, 2, 20),
                          2.0 ** 126 * r.uniform(1, 2, 20)]).astype(np.float32)[:, None]
    border = np.concatenate([np.arange(0.5, 127), -np.arange(0.5, 127)])
    v = (border * top.astype(np.float64) / 127).astype(np.float32)
    bits = v.view(np.int32)
    x = np.concatenate([top] + [(bits + k).view(np.float32) for k in (-2, -1, 0, 1, 2)], 1)
    got = host(vs.vs_q8_quantize(torch.from_numpy(x).to(dev()))[0])
    assert np.array_equal(got, codes_ref(x, np.ones(x.shape[1]))[0])


@pytest.mark.parametrize("t", TYPES)
def test_codes_at_borders(t):
    """Quotients exactly halfway between whole numbers go to the even one, and
    those one step of the type beside them to their side."""
    half = np.arange(0.5, 127.5, 1.0)
    x = np.concatenate([[127.0], half, -half, np.zeros(1)])[None]
    T = torch.from_numpy(np.concatenate([x * 2.0 ** k for k in (0, -3, 5)])).to(t).to(dev())
    for a in (T, T * 3):
        got = host(vs.vs_q8_quantize(a)[0])
        assert np.array_equal(got, codes_ref(host(a), np.ones(T.shape[1]))[0])
    bits = T.view(torch.int32 if t == torch.float32 else torch.int16)
    for step in (1, -1):
        moved = (T != 0) & (T.abs() < 127 * 2.0 ** 5)
        near = (bits + step * moved.to(bits.dtype)).view(t)
        near[:, 0] = T[:, 0]
        got = host(vs.vs_q8_quantize(near.contiguous())[0])
        assert np.array_equal(got, codes_ref(host(near), np.ones(T.shape[1]))[0])


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d", [64, 1003, 9000])
def test_in_place(d, t):
    """H over X or over the residual, Y over X, dX over each of its inputs."""
    r = rng(67, d)
    x, _, res, _, w, _ = inputs(r, 7, d, t, True)
    Y, H, rs = vs.vs_norm_rows(x, w, residual=res)
    for which in (0, 1):
        a, b = x.clone(), res.clone()
        y, h, _ = vs.vs_norm_rows(a, w, residual=b, H=(a, b)[which])
        assert torch.equal(y, Y) and torch.equal((a, b)[which], H)
        a, b = x.clone(), res.clone()
        c, s, h = vs.vs_norm_rows_q8(a, w, residual=b, H=(a, b)[which])
        assert torch.equal((a, b)[which], H)
        assert torch.equal(c, vs.vs_norm_rows_q8(x, w, residual=res)[0])
    y0, _, _ = vs.vs_norm_rows(x, w)
    a = x.clone()
    assert vs.vs_norm_rows(a, w, out=a)[0] is a and torch.equal(a, y0)
    dY, _ = rows(r, (7, d), t)
    dX, dw = vs.vs_norm_rows_backward(dY, H, w, rs, dH=x)
    for which in range(3):
        a = [dY.clone(), H.clone(), x.clone()]
        gX, gw = vs.vs_norm_rows_backward(a[0], a[1], w, rs, dH=a[2], out=a[which])
        assert torch.equal(a[which], dX) and torch.equal(gw, dw)


@pytest.mark.parametrize("n,d", [(3, 40003), (1030, 9001), (1030, 17000)])
def test_wide_in_place(n, d):
    """The same for rows that are read twice."""
    r = rng(73, n)
    x, _, res, _, w, _ = inputs(r, n, d, torch.bfloat16, True)
    dY = rows(r, (n, d), torch.bfloat16)[0]
    Y, H, rs = vs.vs_norm_rows(x, w, residual=res)
    codes, scales, _ = vs.vs_norm_rows_q8(x, w, residual=res)
    dX, dw = vs.vs_norm_rows_backward(dY, H, w, rs, dH=x)
    for which in (0, 1):
        a, b = x.clone(), res.clone()
        assert torch.equal(vs.vs_norm_rows(a, w, residual=b, H=(a, b)[which])[0], Y)
        assert torch.equal((a, b)[which], H)
        a, b = x.clone(), res.clone()
        c, s, _ = vs.vs_norm_rows_q8(a, w, residual=b, H=(a, b)[which])
        assert torch.equal(c, codes) and torch.equal(s, scales) and torch.equal((a, b)[which], H)
    a = H.clone()
    assert torch.equal(vs.vs_norm_rows(a, w, out=a)[0], Y)
    for which in (0, 1, 2):
        a = [dY.clone(), H.clone(), x.clone()]
        g, gw = vs.vs_norm_rows_backward(a[0], a[1], w, rs, dH=a[2], out=a[which])
        assert torch.equal(g, dX) and torch.equal(gw, dw)


@pytest.mark.parametrize("d", [64, 8000])
def test_largest_magnitudes(d):
    """fp32 rows up to the largest number: rstd and the scale as in 64 bits, one
    rounding to a subnormal rstd more."""
    x = torch.from_numpy(rng(74, d).uniform(-1, 1, (3, d)) * 3.4e38).float().to(dev())
    x64 = host(x)
    h, rstd, y = norm_ref(x64, None, np.ones(d), 0.0, torch.float32)
    Y, _, rs = vs.vs_norm_rows(x, None, 0.0)
    sub = 2.0 ** -150 / rstd  # of a subnormal rstd, relative
    close(rs, rstd[:, 0], 1.01 * ((r_of(d) + 8 * V + sub) * rstd)[:, 0])
    close(Y, y, 1.01 * (r_of(d) + 10 * V + sub) * np.abs(y))
    codes, scales, _ = vs.vs_norm_rows_q8(x, None, 0.0)
    c, top = codes_ref(h, np.ones(d))
    assert np.array_equal(host(codes), c)
    scale = top * rstd / 127
    close(scales, scale[:, 0], 1.01 * ((r_of(d) + 10 * V + sub) * scale)[:, 0])


@pytest.mark.parametrize("t", TYPES)
def test_outputs_and_addresses(t):
    """Odd addresses; nothing beside the outputs is written."""
    r = rng(68)
    for n, d in ((11, 64), (11, 131), (3, 2), (2, 9001)):
        x, _, res, _, w, _ = inputs(r, n, d, t, True)
        Y, H, rs = vs.vs_norm_rows(x, w, residual=res)

        def at(a, s=1):
            buf = torch.empty(a.numel() + 16, dtype=a.dtype, device=dev())
            v = buf[s:s + a.numel()].view(a.shape)
            return v.copy_(a)

        def guarded(shape, dt):
            k = int(np.prod(shape))
            buf = torch.full((k + 40,), 7, dtype=dt, device=dev())
            return buf, buf[17:17 + k].view(shape)
        bufs = [guarded((n, d), t), guarded((n, d), t), guarded((n,), torch.float32),
                guarded((n, d), torch.int8), guarded((n,), torch.float32), guarded((n, d), t),
                guarded((d,), t)]
        o = [b[1] for b in bufs]
        vs.vs_norm_rows(at(x), at(w), residual=at(res), out=o[0], H=o[1], rstd=o[2])
        assert torch.equal(o[0], Y) and torch.equal(o[1], H) and torch.equal(o[2], rs)
        vs.vs_norm_rows_q8(at(x), at(w), residual=at(res), codes=o[3], scales=o[4], H=o[1])
        want = vs.vs_norm_rows_q8(x, w, residual=res)
        assert torch.equal(o[3], want[0]) and torch.equal(o[4], want[1])
        vs.vs_norm_rows_backward(at(x), at(H), at(w), rs, out=o[5], dweight=o[6])
        want = vs.vs_norm_rows_backward(x, H, w, rs)
        assert torch.equal(o[5], want[0]) and torch.equal(o[6], want[1])
        for buf, v in bufs:
            v.fill_(7)
            assert bool((buf == 7).all())


def test_norm_no_rows():
    x, w = torch.empty(0, 8, device=dev()), torch.ones(8, device=dev())
    Y, H, rs = vs.vs_norm_rows(x, w, residual=x)
    assert Y.shape == (0, 8) and rs.shape == (0,)
    codes, scales, _ = vs.vs_norm_rows_q8(x, w)
    assert codes.shape == (0, 8) and scales.shape == (0,)
    dX, dw = vs.vs_norm_rows_backward(x, x, w, rs, dweight=torch.full((8,), 3.0, device=dev()))
    assert dX.shape == (0, 8) and bool((dw == 0).all())


def test_norm_refusals():
    x, w = torch.ones(4, 8, device=dev()), torch.ones(8, device=dev())
    rs = torch.ones(4, device=dev())
    for call, error in (
            (lambda: vs.vs_norm_rows(x.double(), w), TypeError),
            (lambda: vs.vs_norm_rows(x, w.half()), TypeError),
            (lambda: vs.vs_norm_rows(x, w[:7]), ValueError),
            (lambda: vs.vs_norm_rows(x, w, residual=x[:3]), ValueError),
            (lambda: vs.vs_norm_rows(x, w, residual=x.half()), TypeError),
            (lambda: vs.vs_norm_rows(x, w, H=x.clone()), ValueError),
            (lambda: vs.vs_norm_rows(x.t(), w[:4]), ValueError),
            (lambda: vs.vs_norm_rows(x, w, -1.0), vs.VsError),
            (lambda: vs.vs_norm_rows_q8(x, w, float("nan")), vs.VsError),
            (lambda: vs.vs_norm_rows_backward(x, x[:3], w, rs), ValueError),
            (lambda: vs.vs_norm_rows_backward(x, x, w, rs[:3]), ValueError),
            (lambda: vs.vs_norm_rows_backward(x, x, w, rs.half()), TypeError),
            (lambda: vs.vs_norm_rows_backward(x, x, None, rs, dweight=w), ValueError),
            (lambda: vs.vs_norm_rows_backward(x, x, w, rs, grad_dtype=torch.float16), vs.VsError),
            (lambda: vs.vs_norm_rows_backward(x, x, w, rs, workspace=torch.empty(
                16, dtype=torch.uint8, device=dev())), ValueError),
            (lambda: vs.vs_q8_quantize(x, codes=torch.empty(31, dtype=torch.int8, device=dev())),
             ValueError)):
        with pytest.raises(error):
            call()
    for call in (lambda g: vs.vs_norm_rows(g, w), lambda g: vs.vs_norm_rows_q8(g, w),
                 lambda g: vs.vs_norm_rows_backward(g, x, w, rs), lambda g: vs.vs_q8_quantize(g)):
        with pytest.warns(UserWarning, match="gradient"):
            call(x.clone().requires_grad_())
        with warnings.catch_warnings(), torch.no_grad():
            warnings.simplefilter("error")
            call(x.clone().requires_grad_())


# -------------------------------------------------------------------- scores --

SCORES = [
    # nq, nc, d
    (1, 1, 1), (1, 5, 16), (2, 3, 15), (1, 300, 256), (1, 1000, 4096), (3, 17, 100), (16, 64, 128),
    (17, 65, 129), (37, 209, 767), (64, 40, 1024), (65, 130, 64), (128, 128, 2048), (130, 515, 96),
    (300, 700, 272), (257, 1, 40), (1, 2, 131071), (5, 4100, 33), (600, 260, 513), (33, 48, 16),
]


def codes8(r, shape):
    c = r.integers(-128, 128, shape)
    return torch.from_numpy(c.astype(np.int8)).to(dev()), c


def scales8(r, n):
    s = torch.from_numpy((0.5 + r.random(n)).astype(np.float32)).to(dev())
    return s, host(s)


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("nq,nc,d", SCORES)
def test_q8_scores(nq, nc, d, out):
    r = rng(70, nq, nc, d)
    (x, xc), (t, tc) = codes8(r, (nq, d)), codes8(r, (nc, d))
    (xs, xs64), (ts, ts64) = scales8(r, nq), scales8(r, nc)
    if out == torch.float16:  # hold the scores inside its range
        xs, xs64 = xs * 2.0 ** -20, xs64 * 2.0 ** -20
    want = (xc @ tc.T).astype(np.float64) * xs64[:, None] * ts64
    tol = 1.01 * (3 * V + U(out)) * np.abs(want) + SUB[out]
    close(vs.vs_q8_scores(x, xs, t, ts, out_dtype=out), want, tol)


@pytest.mark.parametrize("shift", [0, 4, 2])
@pytest.mark.parametrize("nq,nc,d", [(37, 209, 764), (130, 515, 100), (300, 700, 268), (6, 33, 4),
                                     (300, 17000, 132)])
def test_q8_scores_on_four_bytes(nq, nc, d, shift):
    """Widths that 4 divides and 16 does not, on addresses of 4 bytes and of 2."""
    r = rng(75, nq, d)
    (x, xc), (t, tc) = codes8(r, (nq, d)), codes8(r, (nc, d))
    (xs, xs64), (ts, ts64) = scales8(r, nq), scales8(r, nc)

    def at(a):
        return torch.empty(a.numel() + 8, dtype=a.dtype, device=dev())[shift:shift + a.numel()].view(
            a.shape).copy_(a)

    want = (xc @ tc.T).astype(np.float64) * xs64[:, None] * ts64
    close(vs.vs_q8_scores(at(x), xs, at(t), ts), want,
          1.01 * (3 * V + U(torch.float32)) * np.abs(want) + SUB[torch.float32])


@pytest.mark.parametrize("nq,d", [(1, 131071), (40, 131071), (200, 131056), (3, 100000)])
def test_q8_scores_largest_sums(nq, d):
    """Every code -128, the sums next to 2^31, and of either sign."""
    x = torch.full((nq, d), -128, dtype=torch.int8, device=dev())
    t = torch.full((20, d), -128, dtype=torch.int8, device=dev())
    t[1::2] = 127
    one = torch.ones(max(nq, 20), device=dev())
    want = np.tile(np.where(np.arange(20) % 2, -128.0 * 127 * d, 128.0 * 128 * d), (nq, 1))
    got = host(vs.vs_q8_scores(x, one[:nq], t, one[:20]))
    assert np.array_equal(got, want.astype(np.float32))


@pytest.mark.parametrize("nq,nc,d", [(1, 70, 64), (40, 70, 100), (300, 140, 256), (9, 50, 31)])
def test_q8_scores_addresses(nq, nc, d):
    """Codes at any address; the same scores; nothing beside the output written."""
    r = rng(71, nq, d)
    (x, xc), (t, tc) = codes8(r, (nq, d)), codes8(r, (nc, d))
    (xs, _), (ts, _) = scales8(r, nq), scales8(r, nc)
    want = vs.vs_q8_scores(x, xs, t, ts)
    for s in (1, 2, 4, 8):
        a = torch.empty(x.numel() + 16, dtype=torch.int8, device=dev())[s:s + x.numel()].view(nq, d)
        b = torch.empty(t.numel() + 16, dtype=torch.int8, device=dev())[16 - s:16 - s + t.numel()].view(nc, d)
        buf = torch.full((nq * nc + 40,), 7.0, device=dev())
        out = buf[19:19 + nq * nc].view(nq, nc)
        vs.vs_q8_scores(a.copy_(x), xs, b.copy_(t), ts, out=out)
        assert torch.equal(out, want)
        out.fill_(7.0)
        assert bool((buf == 7.0).all())


@pytest.mark.parametrize("nq", [1, 20, 200])
def test_q8_scores_scales_that_are_not_finite(nq):
    """A NaN scale costs its query's or its row's scores, and no others."""
    r = rng(72, nq)
    (x, _), (t, _) = codes8(r, (nq, 80)), codes8(r, (30, 80))
    (xs, _), (ts, _) = scales8(r, nq), scales8(r, 30)
    want = vs.vs_q8_scores(x, xs, t, ts)
    ts[7] = float("nan")
    xs[nq - 1] = float("inf")
    got = vs.vs_q8_scores(x, xs, t, ts)
    bad = torch.zeros(nq, 30, dtype=torch.bool)
    bad[:, 7] = True
    bad[nq - 1] = True
    assert torch.equal(got[~bad], want[~bad]) and not torch.isfinite(got.cpu()[bad & (want.cpu() != 0)]).any()


def test_q8_refusals():
    c, s = torch.ones(4, 8, dtype=torch.int8, device=dev()), torch.ones(4, device=dev())
    for call, error in (
            (lambda: vs.vs_q8_scores(c.float(), s, c, s), TypeError),
            (lambda: vs.vs_q8_scores(c, s.half(), c, s), TypeError),
            (lambda: vs.vs_q8_scores(c, s[:3], c, s), ValueError),
            (lambda: vs.vs_q8_scores(c, s, c[:, :7].contiguous(), s), ValueError),
            (lambda: vs.vs_q8_scores(c, s, c[:, ::2], s), ValueError),
            (lambda: vs.vs_q8_scores(c, s, c[:0], s[:0]), vs.VsError),
            (lambda: vs.vs_q8_scores(c, s, c, s, out_dtype=torch.float64), TypeError),
            (lambda: vs.vs_q8_scores(c, s, c, s, out=torch.empty(15, device=dev())), ValueError)):
        with pytest.raises(error):
            call()
    assert vs.vs_q8_scores(c[:0], s[:0], c, s).shape == (0, 4)


def test_streams_and_graphs():
    """Another stream; two captured graphs replayed with new inputs, eager calls
    between the replays."""
    r = rng(73)
    n, d, nc = 40, 200, 90
    t = torch.bfloat16
    x, _, res, _, w, _ = inputs(r, n, d, t, True)
    dY, _ = rows(r, (n, d), t)
    table, ts = vs.vs_q8_quantize(rows(r, (nc, d), t)[0])

    def step():
        Y, H, rs = vs.vs_norm_rows(x, w, residual=res)
        codes, scales, _ = vs.vs_norm_rows_q8(x, w, residual=res)
        return (Y, H, rs, *vs.vs_norm_rows_backward(dY, H, w, rs, dH=x),
                vs.vs_q8_scores(codes, scales, table, ts))
    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step()
        graphs.append((g, outs))
    for k in range(3):
        x.copy_(rows(rng(74, k), (n, d), t)[0])
        for g, outs in graphs:
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(outs, step()):
                assert torch.equal(a, b)


def test_rows_scored_and_sent_to_units():
    """The run of calls between two layers: rows added and normalised in 8 bits,
    scored against the units' centroids, sent to the best of them, multiplied by
    their matrix, brought back, and added and normalised again."""
    r = rng(75)
    n, d, G, k = 60, 48, 9, 2
    t = torch.float32
    x, x64, res, r64, w, w64 = inputs(r, n, d, t, True)
    cent, _ = rows(r, (G, d), t)
    W, W64 = rows(r, (G, d, d), t, d ** -0.5)
    table, ts = vs.vs_q8_quantize(cent)
    codes, scales, H = vs.vs_norm_rows_q8(x, w, EPS, residual=res)
    scores = vs.vs_q8_scores(codes, scales, table, ts)
    val, picks = torch.topk(scores, k, dim=1)
    weights = torch.softmax(val, 1)
    order, off, slot = vs.vs_group_rows(picks.int(), G)
    Y, _, _ = vs.vs_norm_rows(H, w, EPS)
    Ys = vs.vs_unit_products(vs.vs_route_rows(Y, slot, off, k), W, off)
    out, H2, _ = vs.vs_norm_rows(vs.vs_combine_rows(Ys, slot, weights), w, EPS, residual=H)
    # the same in 64 bits from the formulas; picks as found (the scores are checked)
    h, rstd, y = norm_ref(x64, r64, w64, EPS, t)
    c, top = codes_ref(h, w64)
    want = (c * (top * rstd / 127)) @ (host(table) * host(ts)[:, None]).T
    close(scores, want, 1e-5 * np.abs(want) + 1e-5 * np.abs(want).max())
    p, ww = host(picks).astype(int), host(weights)
    add = np.stack([sum(ww[i, j] * (W64[p[i, j]] @ y[i]) for j in range(k)) for i in range(n)])
    h2 = add + h
    y2 = h2 / np.sqrt((h2 * h2).mean(1, keepdims=True) + EPS) * w64
    # every value is a few hundred fp32 roundings from its inputs, which are of size 1 to 10
    close(H2, h2, 400 * V * 10)
    close(out, y2, 800 * V * 10)


def test_more_tiles_than_a_launch_takes():
    """A table of very many short rows, for one query and for some."""
    nc, d = 150000000, 2
    gen = torch.Generator(device=dev()).manual_seed(8)
    t = torch.empty(nc, d, dtype=torch.int8, device=dev()).random_(-100, 101, generator=gen)
    one = torch.ones(nc, device=dev())
    at = torch.tensor([0, 1, 2 ** 27 - 1, 2 ** 27, 2 ** 27 + 129, nc - 1], device=dev())
    for nq in (1, 9):
        q = t[nc // 2:nc // 2 + nq].contiguous()
        got = vs.vs_q8_scores(q, one[:nq], t, one)
        assert np.array_equal(host(got[:, at]), host(q) @ host(t[at]).T)
        assert int(torch.count_nonzero(got)) > nq * nc // 2  # every part was written
        del got


def test_past_32_bit_offsets():
    """More than 2^31 codes, and more than 2^31 scores."""
    d, n = 4096, 530000
    gen = torch.Generator(device=dev()).manual_seed(6)
    x = torch.empty(n, d, dtype=torch.bfloat16, device=dev()).random_(-100, 101, generator=gen)
    codes, scales, _ = vs.vs_norm_rows_q8(x, None, 0.0)
    Y, _, rs = vs.vs_norm_rows(x, None, 0.0)
    at = [0, 1, 262143, 524287, 524288, 524289, n - 1]
    x64 = host(x[at])
    h, rstd, y = norm_ref(x64, None, np.ones(d), 0.0, torch.bfloat16)
    assert np.array_equal(host(codes[at]), codes_ref(x64, np.ones(d))[0])
    close(Y[at], y, 1.01 * (r_of(d) + 2 * V + U(torch.bfloat16)) * np.abs(y))
    gX, gw = vs.vs_norm_rows_backward(Y, x, torch.ones(d, dtype=torch.bfloat16, device=dev()), rs)
    dX, _ = backward_ref(host(Y[at]), h, rstd, np.ones((1, d)), None)
    close(gX[at], dX, backward_tol(host(Y[at]), h, rstd, np.ones((1, d)), dX, np.zeros(d),
                                   torch.bfloat16, torch.bfloat16)[0])
    del Y, gX, x
    one = torch.ones(n, device=dev())
    for nq in (3, 200):
        q = codes[n - nq:].contiguous()
        got = vs.vs_q8_scores(q, one[:nq], codes, one)
        want = host(q) @ host(codes[at]).T
        assert np.array_equal(host(got[:, at]), want)
    del got
    nq = 4200
    q, t = codes[:nq, :64].contiguous(), codes[:, :64].contiguous()
    got = vs.vs_q8_scores(q, one[:nq], t, one, out_dtype=torch.bfloat16)
    rows_at = [0, 4095, 4096, nq - 1]
    want = host(q[rows_at]) @ host(t[at]).T
    assert np.array_equal(host(got[rows_at][:, at]), host(torch.from_numpy(want).bfloat16()))
