"""Operands with fewer elements than a call reads or writes are refused before anything is enqueued."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def la():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kernelized_linear_attention_gb300 as m
    m.load_library()
    return m


def test_short_operands_are_refused(la):
    x, short = torch.zeros(40, 2, 64, device="cuda"), torch.zeros(39, 2, 64, device="cuda")
    om, few = torch.zeros(128, 64, device="cuda"), torch.zeros(128, 32, device="cuda")
    state = torch.zeros(40, 2, 64, 65, device="cuda")
    g, g2 = torch.zeros(2, 64, 64, dtype=torch.float64, device="cuda"), torch.zeros(64, 2, dtype=torch.float64, device="cuda")
    calls = [lambda: la.la_forward_causal(x, short, x, "elu1"), lambda: la.la_forward_causal(x, x, short, "elu1", out=x.clone()),
             lambda: la.la_forward_causal(x, x, x, "elu1", out=short), lambda: la.la_forward_bidir(x, short, x, "elu1"),
             lambda: la.la_forward_causal(x, x, x, "favor", omega=few), lambda: la.la_forward(x, short, x, "elu1"),
             lambda: la.la_forward_causal_noalloc(x, short, x, "elu1"), lambda: la.attention(x, x, short, "elu1", out=x.clone()),
             lambda: la.la_decode_step(x, short, x, state, "elu1"), lambda: la.la_decode_step(x, x, x, state, "elu1", out=short),
             lambda: la.la_backward(x, short, x, x, "elu1"), lambda: la.la_backward(x, x, x, short, "elu1"),
             lambda: la.la_backward(x, x, x, x, "elu1", dq=short), lambda: la.la_backward(x, x, x, x, "elu1", dv=short),
             lambda: la.la_feature_map(x, "favor", few), lambda: la.la_feature_map(x, "elu1", phi=short),
             lambda: la.la_orthogonal_features(g, g2, 128), lambda: la.la_orthogonal_features(g[:1], g, 128),
             lambda: la.la_orthogonal_features(g, g, 128, omega=few)]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"call {i} was not refused")
    assert la.la_orthogonal_features(g + torch.eye(64, device="cuda"), g, 128).shape == (128, 64)
    torch.cuda.synchronize()
