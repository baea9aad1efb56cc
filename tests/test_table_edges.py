"""Table operators on the GPU at the values, sizes and addresses where they could
go wrong, against plain implementations in 64 bits (tolerances as derived in
test_table_ops)."""
import warnings

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import farthest_vector_search_amd as vs  # noqa: E402
from test_table_ops import (TYPES, V, close, dev, host, i32, pack, rng, rows,  # noqa: E402
                            unpack)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("st", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_q4_quantize_keeps_a_nan(group, st, t):
    """A group that holds a NaN (alone, filled with them, in the cut last group,
    next to an infinity) gets a NaN scale, its row NaN scores; no other group
    changes."""
    r = rng(20, group)
    d = 2 * group + 5
    T, _ = rows(r, (8, d), t)
    nan = float("nan")
    T[0, 0] = nan
    T[1, group - 1] = nan
    T[2, group + group // 2 + 1] = nan
    T[3, :group] = nan
    T[4, 2 * group:] = nan
    T[5, d - 1] = nan
    T[6, 3], T[6, 4] = float("inf"), nan
    held = [(0, 0), (1, 0), (2, 1), (3, 0), (4, 2), (5, 2), (6, 0)]
    codes, scales = vs.vs_q4_quantize(T, group, st)
    bad = torch.zeros(8, 3, dtype=torch.bool)
    for at in held:
        bad[at] = True
    assert torch.equal(torch.isnan(scales).cpu(), bad)
    got = unpack(codes, d)
    over = np.repeat(bad.numpy(), group, 1)[:, :d]
    assert (got[over] == 8).all()
    plain_codes, plain_scales = vs.vs_q4_quantize(torch.nan_to_num(T, 0.0, 1.0, -1.0), group, st)
    assert torch.equal(scales.cpu()[~bad], plain_scales.cpu()[~bad])
    assert np.array_equal(got[~over], unpack(plain_codes, d)[~over])
    x, _ = rows(r, (2, d), t)
    table = vs.vs_q4_layout(codes, scales, d, group)
    y = vs.vs_q4_scores(x, table, 8, group, st)
    assert torch.isnan(y[:, :7]).all() and torch.isfinite(y[:, 7]).all()


@pytest.mark.parametrize("t", TYPES)
def test_q4_scores_scale_type(t):
    """The laid-out table carries its scales' type, also through copies and views;
    another one asked for is refused.  Plain bytes are taken as the caller says."""
    r = rng(21)
    nc, d = 50, 160
    T, _ = rows(r, (nc, d), torch.float32)
    x, _ = rows(r, (3, d), t)
    for st in (torch.float16, torch.bfloat16):
        codes, scales = vs.vs_q4_quantize(T, 32, st)
        table = vs.vs_q4_layout(codes, scales, d, 32)
        want = vs.vs_q4_scores(x, table, nc, 32, st)
        for same in (table, table.clone(), table[:]):
            assert torch.equal(vs.vs_q4_scores(x, same, nc, 32), want)
    with pytest.raises(ValueError, match="scale"):
        vs.vs_q4_scores(x, table, nc, 32, torch.float16)
    buf = torch.empty(table.numel(), dtype=torch.uint8, device=dev())
    again = vs.vs_q4_layout(codes, scales, d, 32, out=buf)
    assert again.data_ptr() == buf.data_ptr()
    assert torch.equal(vs.vs_q4_scores(x, again, nc, 32), want)
    assert torch.equal(vs.vs_q4_scores(x, buf, nc, 32, torch.bfloat16), want)


def test_inputs_that_require_a_gradient_warn():
    """Results are outside autograd: a warning says so where one is expected."""
    n, k, G, d = 6, 2, 4, 8
    r = rng(22)
    X, _ = rows(r, (n, d), torch.float32)
    T, _ = rows(r, (G, d), torch.float32)
    Ys, _ = rows(r, (n * k, d), torch.float32)
    w = torch.ones(n, k, device=dev())
    ids = i32(r.integers(0, G, n * k))
    order, offsets, slot = vs.vs_group_rows(ids, G)
    table = vs.vs_q4_layout(*vs.vs_q4_quantize(T, 32), d, 32)
    g = lambda a: a.clone().requires_grad_()  # noqa: E731
    calls = [lambda q: vs.vs_row_lookup(q(T), ids), lambda q: vs.vs_route_rows(q(X), slot, offsets, k),
             lambda q: vs.vs_combine_rows(q(Ys), slot, w), lambda q: vs.vs_combine_rows(Ys, slot, q(w)),
             lambda q: vs.vs_q4_scores(q(X), table, G, 32)]
    for call in calls:
        with pytest.warns(UserWarning, match="gradient"):
            a = call(g)
        assert not a.requires_grad
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            call(lambda z: z)
            with torch.no_grad():
                assert torch.equal(call(g), a)


def test_calls_inside_an_autograd_function():
    """The way the gradient is meant to be had: quiet, and equal to the formula."""
    class Lookup(torch.autograd.Function):
        @staticmethod
        def forward(ctx, T, ids):
            order, offsets, _ = vs.vs_group_rows(ids, T.shape[0])
            ctx.save_for_backward(ids, order, offsets)
            return vs.vs_row_lookup(T, ids, scale=2.0)

        @staticmethod
        def backward(ctx, dY):
            return vs.vs_row_lookup_backward(dY.contiguous(), *ctx.saved_tensors, scale=2.0), None
    r = rng(27)
    T = torch.from_numpy(r.integers(-3, 4, (5, 8)).astype(np.float32)).to(dev()).requires_grad_()
    R64 = r.integers(-3, 4, (9, 8)).astype(np.float64)
    ids = r.integers(0, 5, 9).astype(np.int32)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        (Lookup.apply(T, i32(ids)) * torch.from_numpy(R64).float().to(dev())).sum().backward()
    want = np.zeros((5, 8))
    np.add.at(want, ids, 2 * R64)
    assert np.array_equal(host(T.grad), want)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_q4_scores_table_at_16_bytes(group):
    """A table on a 16-byte boundary that is no 32-byte one."""
    r = rng(23)
    nc, d = 70, 300
    c = r.integers(0, 16, (nc, d))
    s = torch.from_numpy(2.0 ** r.integers(-2, 1, (nc, -(-d // group)))).half().to(dev())
    x64 = r.integers(-4, 5, (2, d)).astype(np.float64)
    x = torch.from_numpy(x64).half().to(dev())
    need = vs.lib().vs_q4_bytes(nc, d, group)
    buf = torch.empty(need + 64, dtype=torch.uint8, device=dev())
    at = (16 - buf.data_ptr()) % 32
    table = vs.vs_q4_layout(pack(c), s, d, group, out=buf[at:at + need])
    assert table.data_ptr() % 32 == 16
    full = (c - 8.0) * np.repeat(host(s), group, 1)[:, :d]
    assert np.array_equal(host(vs.vs_q4_scores(x, table, nc, group)), x64 @ full.T)


def test_wide_sizes_are_refused():
    """Sizes that do not fit the C interface's 32 bits are refused, not cut off."""
    big = 2 ** 32 + 8
    e = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device=dev())  # noqa: E731
    ids = e(0, t=torch.int32)
    off = i32([0, 0])
    calls = [lambda: vs.vs_row_lookup(e(1, big), ids),
             lambda: vs.vs_route_rows(e(0, big), ids, off, 2),
             lambda: vs.vs_route_rows(e(0, 8), ids, off, 2 ** 32 + 2),
             lambda: vs.vs_route_rows_backward(e(0, big), ids, 2),
             lambda: vs.vs_route_rows_backward(e(0, 8), ids, 2 ** 32 + 2),
             lambda: vs.vs_combine_rows(e(0, big), ids, e(0, 2, t=torch.float32)),
             lambda: vs.vs_combine_rows(e(0, 8), ids, e(0, 2 ** 32 + 2, t=torch.float32)),
             lambda: vs.vs_combine_rows_backward(e(0, big), e(0, big), ids,
                                                 e(0, 2, t=torch.float32), off),
             lambda: vs.vs_q4_quantize(e(1, big)),
             lambda: vs.vs_q4_layout(e(0, 4, t=torch.uint8), e(0, 1, t=torch.float16), big),
             lambda: vs.vs_q4_scores(e(0, big), e(1152, t=torch.uint8), 3)]
    for i, call in enumerate(calls):
        with pytest.raises(vs.VsError) as err:
            call()
        assert err.value.status == 2, i


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("nq,d", [(33, 768), (33, 769), (64, 700), (17, 2048), (17, 2049), (3, 4608),
                                  (16, 4608), (3, 4609), (17, 4616), (5, 768), (11, 768), (6, 2048),
                                  (6, 2049)])
def test_q4_scores_where_the_form_changes(nq, d, t):
    """Widths and query counts on both sides of each change of kernel form: the
    last ones whose operands just fit in LDS (160 KiB), and one column more.
    Small whole numbers, scales powers of two: exact."""
    nc, group = 37, 64
    r = rng(24, nq, d)
    c = r.integers(0, 16, (nc, d))
    s = torch.from_numpy(2.0 ** r.integers(-2, 1, (nc, -(-d // group)))).half().to(dev())
    x64 = r.integers(-4, 5, (nq, d)).astype(np.float64)
    x = torch.from_numpy(x64).to(t).to(dev())
    table = vs.vs_q4_layout(pack(c), s, d, group)
    full = (c - 8.0) * np.repeat(host(s), group, 1)[:, :d]
    assert np.array_equal(host(vs.vs_q4_scores(x, table, nc, group)), x64 @ full.T)


@pytest.mark.parametrize("t", TYPES)
def test_q4_scores_codes_near_zero(t):
    """Rows of one large value a group, nearly all other codes at 7 .. 9."""
    r = rng(25)
    nc, d, group, nq = 60, 512, 128, 4
    T = torch.from_numpy((r.standard_normal((nc, d)) * 0.01).astype(np.float32))
    T[:, ::group] = 1.0
    T = T.to(dev())
    codes, scales = vs.vs_q4_quantize(T, group)
    table = vs.vs_q4_layout(codes, scales, d, group)
    x, x64 = rows(r, (nq, d), t)
    c = unpack(codes, d)
    assert (np.abs(c - 8) <= 1).mean() > 0.9
    rep = np.repeat(host(scales), group, 1)[:, :d]
    want = x64 @ ((c - 8.0) * rep).T
    tol = 2 * V * (2 * group + d // group + 4) * (np.abs(x64) @ ((c + 40.0) * rep).T)
    close(vs.vs_q4_scores(x, table, nc, group), want, tol)


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("e", [-105, -112, -120, -126, -130])
def test_q4_scores_tiny_queries(e, t):
    """Queries about the smallest normal number.  Beside the usual bound: what an
    f32 query loses below 2^-133, less than that per column, times |code - 8|,
    and half the smallest subnormal, 2^-150, per fp32 operation."""
    r = rng(28, -e)
    nc, d, group, nq = 40, 160, 32, 3
    c = r.integers(0, 16, (nc, d))
    s = torch.ones(nc, 5, dtype=torch.float16, device=dev())
    table = vs.vs_q4_layout(pack(c), s, d, group)
    x = torch.from_numpy(r.standard_normal((nq, d)) * 2.0 ** e).to(t).to(dev())
    x64 = host(x)
    ops = 2 * group + d // group + 4
    tol = 2 * V * ops * (np.abs(x64) @ (c + 40.0).T) + ops * d // group * 2.0 ** -150
    if t == torch.float32:
        tol = tol + 2.0 ** -133 * np.abs(c - 8.0).sum(1)
    close(vs.vs_q4_scores(x, table, nc, group), x64 @ (c - 8.0).T, tol)


def test_subnormal_rows_pass_unchanged():
    """Subnormal values are moved and summed, not flushed."""
    for t, step in ((torch.float32, 2.0 ** -149), (torch.float16, 2.0 ** -24), (torch.bfloat16, 2.0 ** -133)):
        v = np.arange(-40, 40).reshape(2, 40) * step
        T = torch.from_numpy(v).to(t).to(dev())
        assert np.array_equal(host(T), v)
        ids = i32([1, 0])
        assert np.array_equal(host(vs.vs_row_lookup(T, ids)), v[::-1]), t
        order, offsets, slot = vs.vs_group_rows(ids, 2)
        assert np.array_equal(host(vs.vs_row_lookup_backward(T, ids, order, offsets)), v[::-1]), t
        assert np.array_equal(host(vs.vs_route_rows_backward(T, slot, 1)), v[::-1]), t


@pytest.mark.parametrize("n,G", [(131072, 2), (1 << 20, 1), (300000, 8)])
def test_row_lookup_backward_hot_units(n, G):
    """Units of a great many rows.  Whole numbers, partial sums below 2^24: exact."""
    r = rng(26, n)
    d = 64
    ids = r.integers(0, G, n).astype(np.int32)
    g = torch.Generator(device=dev()).manual_seed(3)
    # whole numbers, |sum| < 2^24: exact
    dY = torch.empty(n, d, device=dev()).random_(-4, 5, generator=g)
    order, offsets, _ = vs.vs_group_rows(i32(ids), G)
    got = vs.vs_row_lookup_backward(dY, i32(ids), order, offsets)
    want = np.stack([host(dY[torch.from_numpy(ids == u).to(dev())]).sum(0) for u in range(G)])
    assert np.array_equal(host(got), want)
