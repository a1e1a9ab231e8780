"""The norm of queries and keys with their rotation where a row times its weights leaves fp32 although its normed values do
not: rows whose squares overflow (rstd 0, outputs 0), and rows and weights that are both small."""
import pytest

from oracle import layer_ops as ops
from test_gpu_qk_norm_rotary import TYPES, _bounds, _case, _forward, _np, check, la  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,pairs", [(64, (32,)), (83, (20, 19)), (256, (64,))])
def test_rows_whose_squares_overflow_are_zero(la, d, pairs, dtype, il):   # noqa: F811
    c = _case(20, 3, 2, d, pairs, dtype, seed=d)
    c["qw"] = c["qw"].abs() + 1.0
    c["q"][6, 1] = 3e38
    c["q"][7, 2] = -2e38
    c["k"][0, 0] = 3e38
    c["kw"] *= 1e30
    qo, ko, qr, kr = _forward(la, c, interleaved=il)
    assert not qr[6, 1].any() and not qo[6, 1].any() and not qo[7, 2].any() and not ko[0, 0].any() and not kr[0, 0].any()
    assert torch.isfinite(qo).all() and torch.isfinite(ko).all()


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,pairs", [(64, (32,)), (83, (20, 19)), (256, (64,))])
def test_small_rows_with_small_weights_keep_their_digits(la, d, pairs, dtype, il):   # noqa: F811
    c = _case(20, 3, 2, d, pairs, dtype, seed=d + 1)
    c["q"] = (c["q"].float() * 1e-15).to(TYPES[dtype])
    c["qw"] = c["qw"] * 1e-27
    qo, _, qr, _ = _forward(la, c, interleaved=il, eps=0.0)
    x, w = _np(c["q"]), _np(c["qw"])
    ref, ref_r = ops.qk_norm_rotary(x, w, _np(c["freq"]), c["pos"].cpu().numpy(), c["pairs"], il, 0.0)
    by, br = _bounds(x, w, ref_r, 0.0, c["pairs"], il)
    check(_np(qr), ref_r, br, "f32", "rstd")
    check(_np(qo), ref, by, dtype, "q_out")
