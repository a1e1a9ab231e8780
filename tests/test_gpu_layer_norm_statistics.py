"""GPU: the statistics of layer norm rows with infinities."""
import numpy as np
import pytest

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
