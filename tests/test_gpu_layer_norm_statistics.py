"""GPU: the statistics of layer norm rows that a sum's rounding shows in (constant rows, means far larger than the
spread), and of rows with infinities, against the fp64 oracle."""
import numpy as np
import pytest

from layer_ops_util import HALF, U, check, norm_terms
from oracle import layer_ops as ops

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
WIDTHS = [1, 5, 64, 77, 200, 300, 768, 1001, 1024, 1536, 4096, 4097, 5001, 8192, 10001, 16384]


@pytest.fixture(scope="module")
def la():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kernelized_linear_attention_gb300 as m
    m.load_library()
    return m


def _np(t):
    return t.detach().cpu().double().numpy()


def _off(t, by):
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    out = buf[by:].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", WIDTHS)
def test_mean_of_rows_with_infinities(la, d, dtype, off):
    inf = float("inf")
    x = torch.randn(7, d, generator=torch.Generator().manual_seed(d)).to(TYPES[dtype])
    x[1, d // 2] = inf
    x[2, d - 1] = -inf
    x[3, 0] = inf
    x[4, 0], x[4, d - 1] = inf, -inf                 # (one value: the last one)
    x[5, d // 3] = float("nan")
    xd = _off(x.cuda(), off)
    y, mean, rstd = la.la_layer_norm(xd, return_stats=True)
    with np.errstate(invalid="ignore"):
        ref = _np(x).mean(-1)
    got = _np(mean)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[np.isinf(ref)], ref[np.isinf(ref)])
    assert torch.isnan(rstd[1:6]).all() and torch.isnan(y[1:6]).all()
    assert torch.isfinite(rstd[[0, 6]]).all() and torch.isfinite(y[[0, 6]]).all()


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", WIDTHS)
def test_constant_rows_have_their_value_as_mean(la, d, dtype, off):
    g = torch.Generator().manual_seed(d)
    c = torch.cat([torch.tensor([540.5734, 1836.8123, -0.1, 3.3e5, 1e-20, -1.7e18, 1e36, 0.0]), 1e4 * torch.randn(200, generator=g)])
    c = c.to(TYPES[dtype])
    x = _off(c[:, None].expand(-1, d).contiguous().cuda(), off)
    w, b = torch.randn(d, generator=g).cuda(), torch.randn(d, generator=g).cuda()
    y, mean, rstd = la.la_layer_norm(x, w, b, return_stats=True)
    sums_fit = c.abs().float() * d < 3e38                 # the fp32 sum of the others is an infinity
    assert torch.equal(mean[sums_fit.cuda()], c.float().cuda()[sums_fit.cuda()])
    keep = sums_fit.cuda()
    assert torch.equal(y[keep], b.to(x.dtype).expand(len(c), d)[keep])        # no deviation: the bias alone
    # 1 / sqrt(0 + eps): the root and its step of Newton's method within two steps
    exact = 1 / np.sqrt(np.float64(np.float32(1e-5)))
    assert np.abs(_np(rstd[keep]) - exact).max() <= 4 * U * exact
    y0 = la.la_layer_norm(x, w, b, eps=0.0)
    assert torch.isnan(y0[keep]).all()                    # 0 / 0, as the formula has it


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("ratio", [100.0, 3e4, 1e6])
@pytest.mark.parametrize("d", WIDTHS[1:])
def test_means_far_larger_than_the_spread(la, d, ratio, off):
    """The mean within its own rounding, the variance without the square of an error of a whole sum.

    A first mean m is within (K + 2) u mean|x| (K = norm_terms(d), and a product with a rounded 1 / d).  Deviations
    x - m are exact or off by u of themselves, their mean within (K + 3) u mean|x - m|, and adding it to m rounds
    once, by u |mean|.  So |dmu| <= u |mean| + (K + 4) u (mean|c| + (K + 2) u mean|x|), c the exact deviations.
    Where a row takes several warps, theirs are such means too, and their mean is found the same way: twice that.
    Squares are summed within (K + 3) u of mean(c^2) + dmu'^2, dmu' the error of the mean they are taken about,
    and what remains of dmu'^2 is no larger than (2 u |mean|)^2."""
    g = torch.Generator().manual_seed(int(d + ratio))
    x = ((1.0 + torch.rand(64, 1, generator=g)) * ratio + torch.randn(64, d, generator=g)).cuda()
    y, mean, rstd = la.la_layer_norm(_off(x, off), return_stats=True)
    ref, rm, rr = ops.layer_norm(_np(x), None, None, 1e-5)
    K = norm_terms(d)
    c = _np(x) - rm[:, None]
    dmu = 2 * (U * np.abs(rm) + (K + 4) * U * (np.abs(c).mean(-1) + (K + 2) * U * np.abs(_np(x)).mean(-1)))
    check(_np(mean), rm, dmu, "f32", "mean")
    var = (c * c).mean(-1)
    rel = 0.5 * (2 * (K + 6) * U * var + 2 * dmu ** 2) / (var + 1e-5) + 4 * U
    check(_np(rstd), rr, 1.01 * rel * rr, "f32", "rstd")
    xh = np.abs(c) * rr[:, None]
    by = rr[:, None] * (dmu[:, None] + U * np.abs(c)) + xh * (rel[:, None] + 3 * U)
    check(_np(y), ref, 1.01 * by, "f32", "y")


def test_one_value_differs_by_a_step(la):
    """Rows of one value but for an element one step larger: the variance is that element's, not a sum's rounding."""
    for d in (64, 77, 1001, 4096):
        x = torch.full((8, d), 1836.8123, device="cuda")
        step = 2.0 ** -13
        for i in range(8):
            x[i, i * (d - 1) // 7] += step
        _, mean, rstd = la.la_layer_norm(x, eps=0.0, return_stats=True)
        # about the rounded mean, which is the common value: step^2 / d, where exactly it is step^2 / d (1 - 1 / d)
        assert bool((mean == x.median()).all())
        ref = np.sqrt(d) / step
        assert np.abs(_np(rstd) - ref).max() <= ref * (1.0 / d + 16 * U + HALF["f32"])
