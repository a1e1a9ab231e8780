"""GPU: layer norms with hundreds and thousands of weight rows, more than the blocks that run at once have, against the
fp64 oracle."""
import numpy as np
import pytest

from layer_ops_util import check, layer_norm_backward_bounds, layer_norm_bounds
from oracle import layer_ops as ops

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def la():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kernelized_linear_attention_gb300 as m
    m.load_library()
    return m


def _np(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("times", [1, 3, 8])
@pytest.mark.parametrize("groups,d", [(153, 40), (304, 64), (1000, 16), (5000, 64), (5003, 7), (5000, 33), (16384, 64), (1213, 200),
                                      (700, 1030), (20011, 1), (611, 131)])
def test_many_weight_rows(la, groups, d, times, dtype):
    if groups * d * times > 1 << 21:
        times = 2
    g = torch.Generator().manual_seed(groups + d)
    x = ((torch.randn(times, groups, d, generator=g) + 0.5) * torch.exp(torch.randn(times, groups, 1, generator=g)))
    x = x.to(TYPES[dtype]).cuda()
    dy = torch.randn(times, groups, d, generator=g).to(TYPES[dtype]).cuda()
    w, b = 1 + 0.3 * torch.randn(groups, d, generator=g).cuda(), torch.randn(groups, d, generator=g).cuda()
    y, mean, rstd = la.la_layer_norm(x, w, b, return_stats=True)
    ref, rm, rr = ops.layer_norm(_np(x), _np(w), _np(b), 1e-5)
    by, bm, br = layer_norm_bounds(_np(x), _np(w), _np(b), rm, rr, 1e-5)
    check(_np(y), ref, by, dtype, "y")
    check(_np(mean), rm, bm, "f32", "mean")
    check(_np(rstd), rr, br, "f32", "rstd")
    refs = ops.layer_norm_backward(_np(x), _np(dy), _np(mean), _np(rstd), _np(w))
    bounds = layer_norm_backward_bounds(_np(x), _np(dy), _np(mean), _np(rstd), _np(w), times)
    def gradients(off):
        # whole, or from arrays that do not start on 16 bytes (taken element by element)
        def at(t):
            buf = torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")
            out = buf[off:].view(t.shape)
            out.copy_(t)
            return out
        return la.la_layer_norm_backward(at(x), at(dy), at(mean), at(rstd), at(w))
    for off in (0, 1):
        grads = gradients(off)
        for got, r, bd, t in zip(grads, refs, bounds, (dtype, "f32", "f32")):
            check(_np(got), r, bd, t, "gradient")
        assert all(torch.equal(p, q) for p, q in zip(grads, gradients(off)))
