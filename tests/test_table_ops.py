"""Table operators on the GPU against plain implementations in 64 bits (numpy).

Tolerances.  u(t) = eps(t) / 2 is the rounding of a stored result, v = 2^-24
that of one fp32 operation; e counts fp32 operations on a term's path:
  lookup            |y - scale T| <= (u(t) + 2 v) |scale T|            (1 product)
  lookup backward   c terms summed, 1 product:
                    2 (c + 1) v scale sum |dY| + u(t) |exact|
  combine           k fused multiply-adds: 2 (k + 1) v sum |w y| + u(t) |exact|
  dweights          d fused multiply-adds in any order: 2 d v sum |dY Ys|
plus half the smallest subnormal of t.  Scores: every product (16 + c) x and
24 x is exact; the 2 group of them in a group are added inside the matrix
instruction, taken at a whole unit 2 v per addition because its rounding is
not documented to be to nearest, then groups + 4 fp32 operations join groups,
waves and pieces:  2 v (2 group + groups + 4) sum s (16 + c + 24) |x|.
Where inputs are small whole numbers and scales powers of two every sum is
exact in fp32, and equality is asked for.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import farthest_vector_search_amd as vs  # noqa: E402

V = 2.0 ** -24
TYPES = [torch.float32, torch.float16, torch.bfloat16]
SUB = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


def U(t):
    return torch.finfo(t).eps / 2


def dev():
    return torch.device("cuda:0")


def rng(*key):
    return np.random.default_rng(list(key))


def rows(r, shape, t, scale=1.0):
    """Random rows of type t: the tensor on the GPU and its values in 64 bits."""
    x = torch.from_numpy((r.standard_normal(shape) * scale).astype(np.float32)).to(t)
    return x.to(dev()), x.to(torch.float64).numpy()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev())


def host(t):
    return t.detach().to("cpu").to(torch.float64).numpy()


def close(got, want, tol):
    got = host(got)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4],
                           np.broadcast_to(tol, want.shape)[bad][:4])


def make_ids(r, n, G, kind):
    if kind == "even":
        ids = r.integers(0, G, n)
    elif kind == "hot":   # half of the entries on one unit, the rest anywhere
        ids = np.where(r.random(n) < 0.5, G // 2, r.integers(0, G, n))
    elif kind == "one":
        ids = np.full(n, G - 1)
    elif kind == "none":
        ids = np.full(n, -1)
    else:                 # wild: every sort of id that drops an entry among them
        ids = r.integers(0, G, n)
        out = np.array([-1, G, -2 ** 31, 2 ** 31 - 1, G + 7 if G < 2 ** 31 - 8 else G])
        gone = r.random(n) < 0.3
        ids = np.where(gone, out[r.integers(0, 5, n)], ids)
    return ids.astype(np.int64).astype(np.int32)


def group_ref(ids, G):
    n = len(ids)
    keep = np.nonzero((ids >= 0) & (ids < G))[0]
    kept = keep[np.argsort(ids[keep], kind="stable")]
    order = np.full(n, -1, np.int32)
    order[:len(kept)] = kept
    slot = np.full(n, -1, np.int32)
    slot[kept] = np.arange(len(kept))
    offsets = np.zeros(G + 1, np.int32)
    offsets[1:] = np.cumsum(np.bincount(ids[keep], minlength=G))
    return order, offsets, slot


# ------------------------------------------------------------------ grouping --

GROUP_CASES = [
    # n, G, kind
    (0, 5, "even"), (1, 1, "even"), (1, 300000, "one"), (3, 2, "none"), (16, 64, "wild"),
    (63, 7, "even"), (64, 1, "even"), (65, 64, "wild"), (1000, 63, "hot"), (1023, 1000, "wild"),
    (4097, 100, "wild"), (5000, 8359, "even"), (3000, 262144, "wild"),
    (32768, 128, "hot"),
    # beyond the counting path: one digit, two and three of them, tile edges
    (32769, 255, "wild"), (65536, 256, "even"), (40960, 1023, "hot"), (70001, 1024, "wild"),
    (131072, 65536, "hot"), (50000, 262144, "wild"), (33000, 1 << 21, "wild"),
    (100003, 1, "even"), (90000, 5, "none"), (2000000, 300, "hot"), (600000, 1 << 20, "even"),
]


@pytest.mark.parametrize("n,G,kind", GROUP_CASES)
def test_group_rows(n, G, kind):
    ids = make_ids(rng(1, n, G), n, G, kind)
    order, offsets, slot = vs.vs_group_rows(i32(ids), G)
    o, f, s = group_ref(ids, G)
    assert np.array_equal(offsets.cpu().numpy(), f)
    assert np.array_equal(order.cpu().numpy(), o)
    assert np.array_equal(slot.cpu().numpy(), s)


@pytest.mark.parametrize("n,G", [(70, 9), (50000, 3000)])
def test_group_rows_writes_its_outputs_only(n, G):
    ids = make_ids(rng(2, n), n, G, "wild")
    big = [torch.full((c + 64,), 77, dtype=torch.int32, device=dev()) for c in (n, G + 1, n)]
    vs.vs_group_rows(i32(ids), G, order=big[0][:n], offsets=big[1][:G + 1], slot=big[2][:n])
    for t, want in zip(big, group_ref(ids, G)):
        assert np.array_equal(t[:len(want)].cpu().numpy(), want)
        assert bool((t[len(want):] == 77).all())
    # without slots, a caller's workspace, a 2-d index matrix
    ws = torch.empty(vs.lib().vs_group_rows_workspace(n, G), dtype=torch.uint8, device=dev())
    order, offsets, slot = vs.vs_group_rows(i32(ids).view(-1, 10), G, workspace=ws,
                                            want_slot=False)
    assert slot is None and torch.equal(order, big[0][:n]) and torch.equal(offsets, big[1][:G + 1])


# -------------------------------------------------------------------- lookup --

LOOKUP_CASES = [
    # n, G, d
    (1, 1, 1), (16, 8359, 768), (5, 3, 7), (333, 50, 8), (1000, 300, 64), (77, 10, 250),
    (64, 9, 1030), (4099, 257, 96), (2, 4, 5000),
]


def away(x):
    """The same values at an address one element off 16-byte alignment."""
    buf = torch.empty(x.numel() + 1, dtype=x.dtype, device=x.device)[1:]
    return buf.copy_(x.reshape(-1)).view(x.shape)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n,G,d", LOOKUP_CASES)
def test_row_lookup(n, G, d, t):
    r = rng(3, n, G, d)
    T, T64 = rows(r, (G, d), t)
    ids = make_ids(r, n, G, "wild")
    scale = 1.7320508
    ok = (ids >= 0) & (ids < G)
    want = np.where(ok[:, None], T64[np.where(ok, ids, 0)] * np.float64(np.float32(scale)), 0.0)
    for table in (T, away(T)):
        got = vs.vs_row_lookup(table, i32(ids), scale=scale)
        assert got.dtype == t
        close(got, want, (U(t) + 2 * V) * np.abs(want) + SUB[t])
        assert not host(got)[~ok].any()
    # an output off alignment; scale 1 copies the rows
    out = away(torch.zeros(n, d, dtype=t, device=dev()))
    vs.vs_row_lookup(T, i32(ids), out=out)
    assert np.array_equal(host(out), np.where(ok[:, None], T64[np.where(ok, ids, 0)], 0.0))


def test_row_lookup_passes_infinities_and_hides_dropped_rows():
    T = torch.full((3, 16), float("nan"), device=dev())
    T[1] = float("inf")
    got = vs.vs_row_lookup(T, i32([-1, 1, 5, 0]), scale=2.0).cpu()
    assert torch.equal(got[0], torch.zeros(16)) and torch.equal(got[2], torch.zeros(16))
    assert bool(torch.isinf(got[1]).all()) and bool(torch.isnan(got[3]).all())


def test_row_lookup_past_32_bit_offsets():
    G, d = (1 << 31) // 512 + 100, 512
    T = torch.zeros(G, d, dtype=torch.bfloat16, device=dev())
    ids = np.array([0, G - 1, (1 << 31) // 512, (1 << 30) // 512, G], np.int32)
    r = rng(4)
    x, x64 = rows(r, (4, d), torch.bfloat16)
    T[torch.from_numpy(ids[:4].astype(np.int64)).to(dev())] = x
    got = vs.vs_row_lookup(T, i32(ids))
    assert np.array_equal(host(got)[:4], x64) and not host(got)[4].any()
    order, offsets, _ = vs.vs_group_rows(i32(ids), G)
    out = T.fill_(1.0)
    vs.vs_row_lookup_backward(got, i32(ids), order, offsets, out=out)
    assert np.array_equal(host(out[torch.from_numpy(ids[:4].astype(np.int64)).to(dev())]), x64)
    assert int(torch.count_nonzero(out).item()) == int(np.count_nonzero(x64))


BACK_CASES = [
    # n, G, d, kind
    (0, 5, 9, "even"), (1, 1, 1, "one"), (1, 7, 16, "none"), (63, 40, 7, "wild"),
    (257, 3, 250, "even"), (1023, 1000, 257, "wild"), (5000, 64, 8, "hot"),
    (4096, 4096, 768, "even"), (20000, 11, 100, "hot"), (300, 2, 2056, "one"),
    (65, 1, 64, "one"), (64, 1, 64, "one"), (129, 2, 1030, "hot"), (40000, 300, 33, "hot"),
]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n,G,d,kind", BACK_CASES)
def test_row_lookup_backward(n, G, d, kind, t):
    r = rng(5, n, G, d)
    dY, dY64 = rows(r, (n, d), t, 0.25)
    ids = make_ids(r, n, G, kind)
    ok = (ids >= 0) & (ids < G)
    scale = np.float64(np.float32(1.5811388))
    want, mass = np.zeros((G, d)), np.zeros((G, d))
    np.add.at(want, ids[ok], dY64[ok])
    np.add.at(mass, ids[ok], np.abs(dY64[ok]))
    c = np.bincount(ids[ok], minlength=G)[:, None]
    order, offsets, _ = vs.vs_group_rows(i32(ids), G)
    for src, gt in ((dY, t), (dY, torch.float32), (away(dY) if n else dY, t)):
        out = torch.full((G, d), 9.0, dtype=gt, device=dev())
        got = vs.vs_row_lookup_backward(src, i32(ids), order, offsets, scale=float(scale),
                                        grad_dtype=gt, out=out)
        close(got, want * scale,
              2 * (c + 1) * V * mass * scale + U(gt) * np.abs(want) * scale + SUB[gt])
        again = vs.vs_row_lookup_backward(src, i32(ids), order, offsets, scale=float(scale),
                                          grad_dtype=gt)
        assert torch.equal(got, again)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("lens", [
    [64, 65, 63, 128, 129, 1, 0, 200, 64, 0, 64], [65], [0, 0, 64, 0], [640, 640], [1, 191, 1],
    [63, 66, 62, 67, 126, 130], [2, 3, 4, 5, 6, 7, 8, 9, 15, 16, 17], [17], [16, 17, 15, 32, 33],
    [64, 65, 63, 128, 129, 1, 0, 200, 64, 0, 64] * 6, [4097], [1, 5000, 1]])
def test_row_lookup_backward_unit_lengths(lens, t):
    """Units about the length at which they are cut, at every alignment."""
    r = rng(15, len(lens), sum(lens))
    ids = r.permutation(np.repeat(np.arange(len(lens)), lens)).astype(np.int32)
    n, G = len(ids), len(lens)
    for d in (4, 320):
        # whole numbers below 2^8 in all: sums are exact in fp32 (not always in f16, bf16)
        dY64 = r.integers(-4, 5, (n, d)).astype(np.float64)
        dY = torch.from_numpy(dY64).to(t).to(dev())
        want = np.zeros((G, d))
        np.add.at(want, ids, dY64)
        order, offsets, _ = vs.vs_group_rows(i32(ids), G)
        got = vs.vs_row_lookup_backward(dY, i32(ids), order, offsets, scale=0.5,
                                        grad_dtype=torch.float32)
        assert np.array_equal(host(got), 0.5 * want)


def test_empty_calls():
    e = torch.zeros(0, dtype=torch.int32, device=dev())
    for G in (1, 70, 5000, 300000):
        order, offsets, slot = vs.vs_group_rows(e, G)
        assert order.numel() == 0 and slot.numel() == 0 and not offsets.any()
        assert offsets.numel() == G + 1
    T = torch.ones(3, 8, device=dev())
    assert vs.vs_row_lookup(T, e).shape == (0, 8)
    order, offsets, slot = vs.vs_group_rows(e, 3)
    X, w = torch.zeros(0, 8, device=dev()), torch.zeros(0, 2, device=dev())
    assert not vs.vs_row_lookup_backward(X, e, order, offsets, out=T.clone()).any()
    assert vs.vs_route_rows(X, slot, offsets, 2).shape == (0, 8)
    assert vs.vs_route_rows_backward(X, slot, 2).shape == (0, 8)
    assert vs.vs_combine_rows(X, slot, w).shape == (0, 8)
    dYs, dw = vs.vs_combine_rows_backward(X, X, slot, w, offsets)
    assert dYs.shape == (0, 8) and dw.shape == (0, 2)
    c, s = vs.vs_q4_quantize(T, 32)
    assert vs.vs_q4_scores(X, vs.vs_q4_layout(c, s, 8, 32), 3, 32).shape == (0, 3)


def test_route_and_combine_past_32_bit_offsets():
    d = 2048
    n = (1 << 31) // d + 65
    g = torch.Generator(device=dev()).manual_seed(5)
    X = torch.empty(n, d, dtype=torch.bfloat16, device=dev()).random_(-50, 51, generator=g)
    ids = torch.zeros(n, dtype=torch.int32, device=dev())
    ids[5] = 1  # the last place
    ids[9] = -1
    order, offsets, slot = vs.vs_group_rows(ids, 2)
    Xs = vs.vs_route_rows(X, slot, offsets, 1)
    p = slot.long()
    assert int(p[5]) == n - 2 and int(p[9]) == -1
    live = torch.tensor([0, 5, 10, n // 2, n - 2, n - 1], device=dev())
    assert torch.equal(Xs[p[live]], X[live]) and not Xs[n - 1].any()
    w = torch.full((n, 1), 2.0, device=dev())
    Y = vs.vs_combine_rows(Xs, slot, w, out=torch.empty_like(X))
    assert torch.equal(Y[live], 2 * X[live]) and not Y[9].any()
    dYs, dw = vs.vs_combine_rows_backward(X, Xs, slot, w, offsets, out=Y)
    assert torch.equal(dYs[p[live]], 2 * X[live]) and not dYs[n - 1].any()
    # squares below 2500, 2,048 of them: sums below 2^23, exact
    assert torch.equal(dw[live, 0], X[live].float().square().sum(1)) and float(dw[9]) == 0


def test_row_lookup_backward_hides_dropped_rows():
    dY = torch.ones(6, 40, device=dev())
    dY[1] = float("nan")
    dY[4] = float("inf")
    ids = i32([0, -1, 2, 2, 9, 0])
    order, offsets, _ = vs.vs_group_rows(ids, 3)
    got = vs.vs_row_lookup_backward(dY, ids, order, offsets)
    assert torch.equal(got.cpu(), torch.tensor([2.0, 0.0, 2.0])[:, None].expand(3, 40))


# ------------------------------------------------------------ route, combine --

ROUTE_CASES = [
    # n, k, G, d, kind
    (1, 1, 1, 1, "even"), (16, 2, 64, 1024, "even"), (7, 3, 5, 250, "wild"),
    (33, 8, 4, 64, "hot"), (100, 1, 10, 7, "wild"), (257, 9, 30, 520, "wild"),
    (64, 4, 8, 2056, "none"), (1500, 5, 100, 96, "wild"), (3, 70, 6, 33, "wild"),
]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n,k,G,d,kind", ROUTE_CASES)
def test_route_and_combine(n, k, G, d, kind, t):
    r = rng(6, n, k, d)
    m = n * k
    ids = make_ids(r, m, G, kind)
    _, off_ref, slot_ref = group_ref(ids, G)
    order, offsets, slot = vs.vs_group_rows(i32(ids).view(n, k), G)
    kept = int(off_ref[-1])
    X, X64 = rows(r, (n, d), t)
    Ys, Ys64 = rows(r, (m, d), t)
    dY, dY64 = rows(r, (n, d), t)
    Ys[kept:] = float("nan")  # rows of no unit are never read
    w = torch.from_numpy(r.random((n, k)).astype(np.float32)).to(dev())
    w64 = host(w).reshape(-1)
    live = slot_ref >= 0
    w.view(-1)[torch.from_numpy(~live).to(dev())] = float("nan")  # nor dropped entries' weights
    at, tok = slot_ref[live], np.arange(m)[live] // k

    for src in (X, away(X)):
        Xs = vs.vs_route_rows(src, slot, offsets, k,
                              out=torch.full((m, d), 5.0, dtype=t, device=dev()))
        want = np.zeros((m, d))
        want[at] = X64[tok]
        assert np.array_equal(host(Xs), want)

    want, mass = np.zeros((n, d)), np.zeros((n, d))
    np.add.at(want, tok, w64[live, None] * Ys64[at])
    np.add.at(mass, tok, w64[live, None] * np.abs(Ys64[at]))
    for src in (Ys, away(Ys)):
        Y = vs.vs_combine_rows(src, slot, w)
        close(Y, want, 2 * (k + 1) * V * mass + U(t) * np.abs(want) + SUB[t])

    want, mass = np.zeros((n, d)), np.zeros((n, d))
    np.add.at(want, tok, Ys64[at])
    np.add.at(mass, tok, np.abs(Ys64[at]))
    dX = vs.vs_route_rows_backward(Ys, slot, k)
    close(dX, want, 2 * (k + 1) * V * mass + U(t) * np.abs(want) + SUB[t])

    want_s = np.zeros((m, d))
    want_s[at] = w64[live, None] * dY64[tok]
    want_w, mass_w = np.zeros(m), np.zeros(m)
    want_w[live] = (dY64[tok] * Ys64[at]).sum(1)
    mass_w[live] = np.abs(dY64[tok] * Ys64[at]).sum(1)
    for a, b in ((dY, Ys), (away(dY), Ys)):
        dYs, dw = vs.vs_combine_rows_backward(
            a, b, slot, w, offsets, out=torch.full((m, d), 5.0, dtype=t, device=dev()))
        close(dYs, want_s, (U(t) + 2 * V) * np.abs(want_s) + SUB[t])
        close(dw.view(-1), want_w, 2 * d * V * mass_w + SUB[torch.float32])


def test_gradients_against_differences():
    """Central differences of L = sum(out * R) in float32 at values where every
    product and sum is exact (small whole numbers), so the difference quotient
    of these (bi)linear maps equals the gradient bit for bit."""
    r = rng(7)
    whole = lambda *s: torch.from_numpy(r.integers(-3, 4, s).astype(np.float32)).to(dev())  # noqa: E731
    n, k, G, d = 9, 3, 4, 12
    ids = i32(make_ids(r, n * k, G, "wild"))
    order, offsets, slot = vs.vs_group_rows(ids, G)
    # combine: by weights and by Ys
    Ys, w, R = whole(n * k, d), whole(n, k), whole(n, d)
    kept = int(offsets[-1])
    Ys[kept:] = 0
    dYs, dw = vs.vs_combine_rows_backward(R, Ys, slot, w, offsets)

    def loss(y, ww):
        return float((vs.vs_combine_rows(y, slot, ww) * R).sum())
    for e in range(n * k):
        step = torch.zeros(n * k, device=dev())
        step[e] = 1
        diff = (loss(Ys, w + step.view(n, k)) - loss(Ys, w - step.view(n, k))) / 2
        assert diff == float(dw.view(-1)[e])
    for p, c in zip(r.integers(0, n * k, 20), r.integers(0, d, 20)):
        step = torch.zeros(n * k, d, device=dev())
        step[p, c] = 1
        assert (loss(Ys + step, w) - loss(Ys - step, w)) / 2 == float(dYs[p, c])
    # route by X, lookup by T
    X, Rs = whole(n, d), whole(n * k, d)
    dX = vs.vs_route_rows_backward(Rs, slot, k)
    T, Rl = whole(G, d), whole(n * k, d)
    dT = vs.vs_row_lookup_backward(Rl, ids, order, offsets, scale=2.0)
    for i, c in zip(r.integers(0, n, 20), r.integers(0, d, 20)):
        step = torch.zeros(n, d, device=dev())
        step[i, c] = 1
        f = lambda x: float((vs.vs_route_rows(x, slot, offsets, k) * Rs).sum())  # noqa: E731
        assert (f(X + step) - f(X - step)) / 2 == float(dX[i, c])
        step = torch.zeros(G, d, device=dev())
        step[i % G, c] = 1
        f = lambda x: float((vs.vs_row_lookup(x, ids, scale=2.0) * Rl).sum())  # noqa: E731
        assert (f(T + step) - f(T - step)) / 2 == float(dT[i % G, c])


# ------------------------------------------------------------- 4-bit tables --

def unpack(codes, d):
    c = codes.cpu().numpy()
    return np.stack((c & 15, c >> 4), axis=2).reshape(c.shape[0], -1)[:, :d].astype(np.float64)


def pack(c):
    nc, d = c.shape
    p = np.full((nc, d + d % 2), 8, np.uint8)
    p[:, :d] = c
    return torch.from_numpy(p[:, 0::2] | (p[:, 1::2] << 4)).to(dev())


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("st", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("nc,d,group", [(1, 1, 32), (5, 31, 32), (16, 128, 64), (33, 257, 128),
                                        (100, 770, 64), (7, 96, 32)])
def test_q4_quantize(nc, d, group, st, t):
    T, T64 = rows(rng(8, nc, d), (nc, d), t, 3.0)
    T[0, : min(d, group)] = 0  # a group of zeros
    T64 = host(T)
    codes, scales = vs.vs_q4_quantize(T, group, st)
    groups = -(-d // group)
    v = np.zeros((nc, groups * group), np.float32)
    v[:, :d] = T64
    v = v.reshape(nc, groups, group)
    s = torch.from_numpy(np.abs(v).max(2) / np.float32(7)).to(st)
    assert torch.equal(scales.cpu(), s)
    s32 = s.float().numpy()[:, :, None]
    with np.errstate(invalid="ignore", divide="ignore"):
        c = np.where(s32 > 0, np.clip(np.rint(v / s32), -8, 7), 0) + 8
    c = c.reshape(nc, -1)[:, :d]
    assert np.array_equal(unpack(codes, d), c)
    if d % 2:
        assert bool((codes[:, -1] >> 4 == 8).all())
    # half a step of the scale, or the rounded scale's distance from max / 7
    got = (c.reshape(nc, d) - 8) * np.repeat(s.double().numpy(), group, 1)[:, :d]
    step = np.repeat(s.double().numpy(), group, 1)[:, :d]
    assert (np.abs(got - T64) <= step * (0.5 + 8 * U(st)) + 1e-7).all()


def test_q4_quantize_extremes():
    T = torch.zeros(4, 64, device=dev())
    T[0] = 3e38                       # the f16 scale stops at its largest value
    T[1] = 1e-12                      # rounds to a scale of zero: codes of zero
    T[2, 3] = float("inf")
    T[3, :2] = torch.tensor([-7.0, 6.5])
    codes, scales = vs.vs_q4_quantize(T, 32)
    assert scales[0].tolist() == [65504.0] * 2 and scales[1].tolist() == [0.0] * 2
    c = unpack(codes, 64)
    assert (c[0] == 15).all() and (c[1] == 8).all() and c[2, 3] == 15
    assert c[3, :2].tolist() == [1.0, 14.0]  # 6.5 lies between two codes: to even


SCORE_CASES = [
    # nq, nc, d, group
    (1, 1, 1, 32), (1, 17, 33, 32), (3, 100, 128, 64), (5, 333, 767, 64), (16, 64, 256, 128),
    (6, 31, 300, 32), (17, 50, 130, 128), (33, 1000, 96, 32), (2, 40, 4096, 128),
    (1, 5000, 256, 32), (16, 48, 1111, 32), (1, 20, 9000, 64), (48, 16, 20000, 128),
    (11, 129, 4100, 64), (1, 3, 70000, 32), (7, 20011, 200, 32), (16, 30000, 640, 64),
    (40, 9000, 250, 128), (2, 70000, 96, 64), (1, 300, 4096, 32),
]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("st", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("nq,nc,d,group", SCORE_CASES)
def test_q4_scores(nq, nc, d, group, st, t):
    r = rng(9, nq, nc, d)
    groups = -(-d // group)
    c = r.integers(0, 16, (nc, d))
    # whole numbers and powers of two: every sum is exact, so are the scores
    s = torch.from_numpy(2.0 ** r.integers(-2, 1, (nc, groups))).to(st).to(dev())
    x64 = r.integers(-4, 5, (nq, d)).astype(np.float64)
    x = torch.from_numpy(x64).to(t).to(dev())
    table = vs.vs_q4_layout(pack(c), s, d, group)
    y = vs.vs_q4_scores(x, table, nc, group, st)
    full = (c - 8.0) * np.repeat(host(s), group, 1)[:, :d]
    assert np.array_equal(host(y), x64 @ full.T)
    # real values, off alignment
    s = torch.from_numpy(0.02 + 0.01 * r.random((nc, groups))).to(st).to(dev())
    x, x64 = rows(r, (nq, d), t)
    table = vs.vs_q4_layout(pack(c), s, d, group)
    rep = np.repeat(host(s), group, 1)[:, :d]
    want = x64 @ ((c - 8.0) * rep).T
    mass = np.abs(x64) @ ((c + 40.0) * rep).T
    tol = 2 * V * (2 * group + groups + 4) * mass
    out = away(torch.zeros(nq, nc, device=dev()))
    for q in (x, away(x)):
        close(vs.vs_q4_scores(q, table, nc, group, st, out=out), want, tol)
    assert torch.equal(vs.vs_q4_scores(x, table, nc, group, st), out)


@pytest.mark.parametrize("t", TYPES)
def test_q4_scores_query_values(t):
    """A query that is not finite affects its own scores only; small and
    subnormal queries are not flushed; f32 queries keep all their bits."""
    r = rng(10)
    nc, d, group = 50, 160, 32
    c = r.integers(0, 16, (nc, d))
    s = torch.ones(nc, 5, dtype=torch.float16, device=dev())
    table = vs.vs_q4_layout(pack(c), s, d, group)
    x, x64 = rows(r, (4, d), t)
    x[1, 5] = float("nan")
    x[3, 159] = float("inf")
    small = 2.0 ** -20 if t == torch.float16 else 2.0 ** -100
    x[2] = torch.from_numpy(x64[2] * small).to(t).to(dev())
    x64[2] = host(x[2])
    y = host(vs.vs_q4_scores(x, table, nc, group))
    for q in (0, 2):
        want = (c - 8.0) @ x64[q]
        tol = 2 * V * (2 * group + 9) * ((c + 40.0) @ np.abs(x64[q]))
        assert (np.abs(y[q] - want) <= tol).all()
    assert np.isnan(y[1]).all() and not np.isfinite(y[3]).any()
    # one column at a time: the score is the query's value, every bit of it
    one = np.full((1, d), 8)
    one[0, 7] = 9
    table = vs.vs_q4_layout(pack(one), s[:1], d, group)
    x = torch.zeros(1, d, dtype=t, device=dev())
    x[0, 7] = 1.2345678
    assert float(vs.vs_q4_scores(x, table, 1, group)) == float(x[0, 7])


def test_q4_scores_past_32_bit_offsets():
    nc, d = (1 << 20) + 50, 4200
    g = torch.Generator(device=dev()).manual_seed(6)
    codes = torch.empty(nc, d // 2, dtype=torch.uint8, device=dev()).random_(0, 256, generator=g)
    scales = torch.ones(nc, 33, dtype=torch.float16, device=dev())
    table = vs.vs_q4_layout(codes, scales, d, 128)
    assert table.numel() > 1 << 31
    x64 = rng(16).integers(-3, 4, (2, d)).astype(np.float64)
    y = vs.vs_q4_scores(torch.from_numpy(x64).to(torch.bfloat16).to(dev()), table, nc, 128)
    for rows_ in (slice(0, 40), slice(nc - 70, nc), slice(nc // 2, nc // 2 + 30)):
        want = x64 @ (unpack(codes[rows_], d) - 8).T
        assert np.array_equal(host(y[:, rows_]), want)


# ------------------------------------------------- the operators in use --

def pipeline(ids, X, T, R, k):
    """One training pass around the units that ids (n x k) name: rows to their
    units, each unit's row of T taken from them, back with weights, and the
    gradients of weights, rows and table."""
    n, d = X.shape
    G = T.shape[0]
    order, offsets, slot = vs.vs_group_rows(ids, G)
    E = vs.vs_row_lookup(T, ids, scale=-1.0)            # by entry
    Xs = vs.vs_route_rows(X, slot, offsets, k)          # by place
    w = torch.softmax(-(E.view(n, k, d) + X.view(n, 1, d)).square().sum(2).float() / d, dim=1)
    Y = vs.vs_combine_rows(Xs, slot, w)
    dYs, dw = vs.vs_combine_rows_backward(R, Xs, slot, w, offsets)
    dX = vs.vs_route_rows_backward(dYs, slot, k)
    dE = (R.view(n, 1, d) * dw.view(n, k, 1)).reshape(n * k, d).to(X.dtype)
    dT = vs.vs_row_lookup_backward(dE, ids, order, offsets, scale=-1.0,
                                   grad_dtype=torch.float32)
    return w, Y, dX, dw, dT


def test_search_route_lookup_and_serve():
    """The operators as a user joins them to a search: best units of each row,
    a pass and its gradients through them (against autograd on the same
    formulas in 64 bits), then the trained table served in 4 bits."""
    r = rng(11)
    n, k, G, d = 700, 2, 60, 96
    X, X64 = rows(r, (n, d), torch.float32)
    T, T64 = rows(r, (G, d), torch.float32)
    R, R64 = rows(r, (n, d), torch.float32)
    best, _ = vs.vs_bmu_search(X, T, vs.VS_L2SQ_MIN)
    far, _ = vs.vs_bmu_search(X, T, vs.VS_L2SQ_MAX)
    ids = torch.stack((best, far), dim=1).contiguous()
    ids[::7, 1] = -1
    w, Y, dX, dw, dT = pipeline(ids, X, T, R, k)
    i = ids.cpu().long()
    live = (i >= 0).double()
    x = torch.from_numpy(X64)
    w64 = w.cpu().double().requires_grad_()
    xv = x.clone().requires_grad_()
    y = (w64 * live).sum(1, keepdim=True) * xv
    (y * torch.from_numpy(R64)).sum().backward()
    # per element 3 fp32 operations a term; dw adds d products
    tol = 8 * V * np.abs(host(Y)) + 1e-6 * 1e-3
    close(Y, y.detach().numpy(), tol)
    close(dX, xv.grad.numpy(), 8 * V * np.abs(R64) + 1e-9)
    close(dw, w64.grad.numpy(), 2 * d * V * np.abs(X64 * R64).sum(1)[:, None] + 1e-9)
    want = np.zeros((G, d))
    mass = np.zeros((G, d))
    flat, ok = i.reshape(-1).numpy(), i.reshape(-1).numpy() >= 0
    dE = np.repeat(R64, k, 0) * host(dw).reshape(-1, 1)
    np.add.at(want, flat[ok], -dE[ok])
    np.add.at(mass, flat[ok], np.abs(dE[ok]))
    close(dT, want, 2 * (n * k + 2) * V * mass + 1e-30)
    T = T - 0.01 * dT
    codes, scales = vs.vs_q4_quantize(T, 32)
    table = vs.vs_q4_layout(codes, scales, d, 32)
    y = vs.vs_q4_scores(X[:3], table, G, 32)
    full = (unpack(codes, d) - 8) * np.repeat(host(scales), 32, 1)
    mass = np.abs(X64[:3]) @ ((unpack(codes, d) + 40) * np.repeat(host(scales), 32, 1)).T
    close(y, X64[:3] @ full.T, 2 * V * (64 + 3 + 4) * mass)


@pytest.mark.parametrize("n,G", [(500, 40), (40000, 3000)])
def test_captured_and_replayed(n, G):
    """Captured once, replayed on new inputs with eager work in between: each
    replay equals the eager calls bit for bit."""
    r = rng(12, n)
    k, d = 2, 64
    ids = i32(make_ids(r, n * k, G, "wild")).view(n, k)
    X, _ = rows(r, (n, d), torch.bfloat16)
    T, _ = rows(r, (G, d), torch.bfloat16)
    R, _ = rows(r, (n, d), torch.bfloat16)
    codes, scales = vs.vs_q4_quantize(T, 32)
    table = vs.vs_q4_layout(codes, scales, d, 32)

    def calls():
        order, offsets, slot = vs.vs_group_rows(ids, G)
        Xs = vs.vs_route_rows(X, slot, offsets, k)
        w = torch.ones(n, k, device=dev()) * 0.5
        Y = vs.vs_combine_rows(Xs, slot, w)
        dYs, dw = vs.vs_combine_rows_backward(R, Xs, slot, w, offsets)
        dX = vs.vs_route_rows_backward(dYs, slot, k)
        E = vs.vs_row_lookup(T, ids, scale=3.0)
        dT = vs.vs_row_lookup_backward(E, ids, order, offsets)
        y = vs.vs_q4_scores(X[:3], table, G, 32)
        return [order, offsets, slot, Xs, Y, dYs, dw, dX, E, dT, y]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    for turn in range(3):
        ids.copy_(i32(make_ids(r, n * k, G, ["hot", "wild", "none"][turn])).view(n, k))
        X.copy_(rows(r, (n, d), torch.bfloat16)[0])
        R.copy_(rows(r, (n, d), torch.bfloat16)[0])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        for a, b in zip(got, calls()):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    """Two passes in flight on two streams, each with its own workspaces."""
    r = rng(13)
    n, G, d = 50000, 5000, 64
    streams = [torch.cuda.Stream() for _ in range(2)]
    ids = [i32(make_ids(r, n, G, kind)) for kind in ("hot", "even")]
    dY = [rows(r, (n, d), torch.float32)[0] for _ in range(2)]
    want = []
    for a, b in zip(ids, dY):
        order, offsets, _ = vs.vs_group_rows(a, G)
        want.append(vs.vs_row_lookup_backward(b, a, order, offsets))
    torch.cuda.synchronize()
    got = [None, None]
    for turn in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                order, offsets, _ = vs.vs_group_rows(ids[i], G)
                got[i] = vs.vs_row_lookup_backward(dY[i], ids[i], order, offsets)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_indices_that_do_not_fit_are_skipped():
    """slot, order and offsets that vs_group_rows did not make: nothing outside
    the arrays is touched, and what fits is used."""
    n, k, G, d = 6, 2, 3, 32
    X, X64 = rows(rng(14), (n, d), torch.float32)
    slot = i32([0, -5, 99, 12, 3, 1 << 30, -(1 << 31), 4, 5, 6, 7, 11])
    off = i32([0, 4, 8, 12])
    buf = torch.full((n * k + 8, d), 3.0, device=dev())
    vs.vs_route_rows(X, slot, off, k, out=buf[4:-4])
    assert bool((buf[:4] == 3).all()) and bool((buf[-4:] == 3).all())
    assert np.array_equal(host(buf[4]), X64[0]) and np.array_equal(host(buf[4 + 11]), X64[5])
    for total in (-7, 1 << 30):
        vs.vs_route_rows(X, slot, i32([0, 4, 8, total]), k, out=buf[4:-4])
        assert bool((buf[:4] == 3).all()) and bool((buf[-4:] == 3).all())
    w = torch.ones(n, k, device=dev())
    Y = vs.vs_combine_rows(buf[4:-4].contiguous(), slot, w)
    assert bool(torch.isfinite(Y).all())
    ids = i32([0, 1, 2, 0, 1, 2])
    got = vs.vs_row_lookup_backward(X, ids, i32([5, -1, 77, 3, -(1 << 31), 0]),
                                    i32([-3, 2, 99, 6]))
    assert np.array_equal(host(got)[0], X64[5])
    assert np.array_equal(host(got)[1], host(X[3] + X[0])) and not host(got)[2].any()


def test_refusals_on_the_gpu():
    X = torch.zeros(6, 8, device=dev())
    i = torch.zeros(6, dtype=torch.int32, device=dev())
    o = torch.zeros(4, dtype=torch.int32, device=dev())
    w = torch.zeros(3, 2, device=dev())
    with pytest.raises(TypeError):
        vs.vs_group_rows(i.long(), 3)
    with pytest.raises(vs.VsError):
        vs.vs_group_rows(i, 0)
    with pytest.raises(ValueError):
        vs.vs_group_rows(i, 3, order=i[:5])
    with pytest.raises(TypeError):
        vs.vs_row_lookup(X.double(), i)
    with pytest.raises(ValueError):
        vs.vs_row_lookup(X[:, ::2], i)
    with pytest.raises(ValueError):
        vs.vs_row_lookup(X.t(), i)
    with pytest.raises(ValueError):
        vs.vs_row_lookup_backward(X, i[:5], i, o)
    with pytest.raises(vs.VsError):
        vs.vs_row_lookup_backward(X, i, i, o, grad_dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        vs.vs_route_rows(X, i, o, 2)
    with pytest.raises(vs.VsError):
        vs.vs_route_rows(X, torch.zeros(0, dtype=torch.int32, device=dev()), o, 0)
    with pytest.raises(ValueError):
        vs.vs_route_rows_backward(X, i, 4)
    with pytest.raises(TypeError):
        vs.vs_combine_rows(X, i, w.half())
    with pytest.raises(ValueError):
        vs.vs_combine_rows(X[:5], i, w)
    with pytest.raises(TypeError):
        vs.vs_combine_rows_backward(X[:3].half(), X, i, w, o)
    with pytest.raises(ValueError):
        vs.vs_q4_quantize(X, 16)
    with pytest.raises(vs.VsError):
        vs.vs_q4_quantize(X, 32, torch.float32)
    c, s = vs.vs_q4_quantize(X, 32)
    with pytest.raises(ValueError):
        vs.vs_q4_layout(c, s, 9, 32)
    with pytest.raises(TypeError):
        vs.vs_q4_layout(c, s.float(), 8, 32)
    table = vs.vs_q4_layout(c, s, 8, 32)
    with pytest.raises(ValueError):
        vs.vs_q4_scores(X, table, 6, 64)  # laid out for another group
    with pytest.raises(ValueError):
        vs.vs_q4_scores(X, table, 17, 32)
