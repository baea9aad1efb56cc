"""The row norm at the ends of fp32's range, on the GPU against 64 bits.

Tolerances, in v = 2^-24, the rounding of one fp32 operation: rstd is within
(d / 2 + 4) v by the sum of d positive terms (test_norm_q8.py), and 4 v more where the
row is scaled to keep its squares in range and back.  A scale is top * rstd / 127: two
roundings more, and half a unit of the subnormal numbers where it is one of them."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import farthest_vector_search_amd as vs  # noqa: E402
from test_norm_q8 import codes_ref, norm_ref, r_of  # noqa: E402
from test_table_ops import SUB, V, close, dev, host, rng  # noqa: E402


@pytest.mark.parametrize("e", [-90, -99, -100, -101, -118, -125])
@pytest.mark.parametrize("d", [3, 8, 64, 777])
def test_scales_of_tiny_rows(d, e):
    """Rows whose largest magnitude over 127 is below the normal numbers, while the
    scale itself, over the row's root mean square, is about 1 / 127."""
    x64 = rng(90, d).uniform(0.5, 1, (200, d)) * 2.0 ** e
    x = torch.from_numpy(x64).float().to(dev())
    x64 = host(x)
    for weight in (None, torch.full((d,), 0.75, device=dev())):
        w64 = np.ones(d) if weight is None else host(weight)
        h, rstd, _ = norm_ref(x64, None, w64, 0.0, torch.float32)
        codes, scales, _ = vs.vs_norm_rows_q8(x, weight, 0.0)
        c, top = codes_ref(h, w64)
        assert np.array_equal(host(codes), c)
        scale = (top * rstd / 127)[:, 0]
        close(scales, scale, 1.01 * (r_of(d) + 10 * V) * scale + SUB[torch.float32])


@pytest.mark.parametrize("eps", [1e38, 2.9e38, 3.4e38])
@pytest.mark.parametrize("d", [1, 3, 64])
def test_largest_eps(d, eps):
    """Every finite eps is taken, also where its sum with the mean square is none."""
    x64 = rng(91, d).uniform(0.5, 1, (50, d)) * np.sqrt(2.0 ** 126 / d)
    x64[1::3] *= 2.0 ** -70
    x64[2::3] *= 1.5  # squares beyond 2^126
    x = torch.from_numpy(x64).float().to(dev())
    x64, eps = host(x), float(np.float32(eps))
    _, rstd, y = norm_ref(x64, None, np.ones(d), eps, torch.float32)
    Y, _, rs = vs.vs_norm_rows(x, None, eps)
    close(rs, rstd[:, 0], 1.01 * (r_of(d) + 8 * V) * rstd[:, 0])
    close(Y, y, 1.01 * (r_of(d) + 10 * V) * np.abs(y))


@pytest.mark.parametrize("t", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,d", [(511, 64), (513, 257), (1023, 128), (1025, 512), (4100, 7), (4101, 64),
                                 (9000, 2047), (1500, 2048), (600, 2056)])
def test_weights_gradient_of_many_rows(n, d, t):
    """The weight's gradient on both sides of each number of partial sums: whole numbers
    over rows of rms 1 (+-1), so that every sum is exact.  The workspace holds just what
    the size query says, and nothing behind it is written."""
    r = rng(92, n, d)
    h = torch.from_numpy(r.choice([-1.0, 1.0], (n, d)).astype(np.float32))
    dY = torch.from_numpy(r.integers(-3, 4, (n, d)).astype(np.float32))
    want = (h * dY).sum(0)
    w, rs = torch.ones(d, device=dev()).to(t), torch.ones(n, device=dev())
    need = vs.lib().vs_norm_rows_backward_workspace(n, d)
    buf = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device=dev())
    _, dw = vs.vs_norm_rows_backward(dY.to(t).to(dev()), h.to(t).to(dev()), w, rs,
                                     grad_dtype=torch.float32, workspace=buf[:need])
    assert torch.equal(dw.cpu(), want)
    assert bool((buf[need:] == 0x5A).all())
