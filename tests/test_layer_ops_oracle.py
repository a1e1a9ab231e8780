"""Pins of the fp64 oracle of the operators around the attention call: worked values, and
gradients against central differences."""
import numpy as np
import pytest

from oracle import layer_ops as ops


def _num_grad(f, x, eps=1e-6):
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        keep = x[i]
        x[i] = keep + eps
        up = f()
        x[i] = keep - eps
        down = f()
        x[i] = keep
        g[i] = (up - down) / (2 * eps)
    return g


def test_gated_scan_worked_values():
    a = np.array([9.0, 0.5, 0.5, 9.0, 2.0]).reshape(5, 1, 1)
    b = np.array([1.0, 1.0, 1.0, 4.0, 1.0]).reshape(5, 1, 1)
    h, out = ops.gated_scan(a, b, cu_seqlens=[0, 3, 3, 5])
    assert np.array_equal(h.ravel(), [1.0, 1.5, 1.75, 4.0, 9.0])   # a first gate has nothing to scale
    assert np.array_equal(out.ravel(), [1.75, 0.0, 9.0])
    h, out = ops.gated_scan(a, b, cu_seqlens=[0, 3, 3, 5], state_in=np.array([1.0, 7.0, -1.0]).reshape(3, 1, 1))
    assert np.array_equal(h.ravel(), [10.0, 6.0, 4.0, -5.0, -9.0])
    assert np.array_equal(out.ravel(), [4.0, 7.0, -9.0])           # the empty sequence keeps its state


@pytest.mark.parametrize("state", [False, True])
def test_gated_scan_gradients_match_differences(state):
    rng = np.random.default_rng(1)
    T, H, d, cu = 9, 2, 3, [0, 4, 4, 9]
    a, b, w = (rng.standard_normal((T, H, d)) for _ in range(3))
    s0, ws = rng.standard_normal((3, H, d)), rng.standard_normal((3, H, d))

    def loss():
        h, out = ops.gated_scan(a, b, cu, state_in=s0 if state else None)
        return (w * h).sum() + (ws * out).sum()

    h, _ = ops.gated_scan(a, b, cu, state_in=s0 if state else None)
    da, db, ds = ops.gated_scan_backward(a, h, w, cu, state_in=s0 if state else None, dstate_out=ws)
    # central differences of a function of third degree and more: eps^2 truncation and 1e-16 / eps rounding
    np.testing.assert_allclose(da, _num_grad(loss, a), atol=1e-7)
    np.testing.assert_allclose(db, _num_grad(loss, b), atol=1e-7)
    if state:
        np.testing.assert_allclose(ds, _num_grad(loss, s0), atol=1e-7)


def test_layer_norm_worked_values():
    y, mean, rstd = ops.layer_norm(np.array([[1.0, 3.0], [5.0, 5.0]]), eps=0.0)
    assert np.array_equal(y[0], [-1.0, 1.0]) and mean[1] == 5.0 and rstd[0] == 1.0
    assert np.isnan(y[1]).all()                                    # no variance and no eps
    y, _, _ = ops.layer_norm(np.array([[1.0, 3.0]]), np.array([2.0, 4.0]), np.array([1.0, 1.0]), eps=0.0)
    assert np.array_equal(y[0], [-1.0, 5.0])


@pytest.mark.parametrize("per_head", [False, True])
def test_layer_norm_gradients_match_differences(per_head):
    rng = np.random.default_rng(2)
    x, w = rng.standard_normal((4, 3, 5)), rng.standard_normal((4, 3, 5))
    weight, bias = rng.standard_normal((2, 3, 5) if per_head else (2, 5))

    def loss():
        return (w * ops.layer_norm(x, weight, bias)[0]).sum()

    _, mean, rstd = ops.layer_norm(x, weight, bias)
    dx, dw, db = ops.layer_norm_backward(x, w, mean, rstd, weight)
    np.testing.assert_allclose(dx, _num_grad(loss, x), atol=1e-6)
    np.testing.assert_allclose(dw, _num_grad(loss, weight), atol=1e-6)
    np.testing.assert_allclose(db, _num_grad(loss, bias), atol=1e-6)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_worked_values_inverse_and_gradient(interleaved):
    x = np.arange(1.0, 6.0).reshape(1, 1, 5)
    quarter = np.array([np.pi / 2, np.pi])
    y = ops.rotary(x, quarter, [[1, 1]], [1, 1], interleaved)
    want = [-2.0, 1.0, -3.0, -4.0, 5.0] if interleaved else [-3.0, -2.0, 1.0, -4.0, 5.0]
    np.testing.assert_allclose(y.ravel(), want, atol=1e-14)
    rng = np.random.default_rng(3)
    x, w = rng.standard_normal((3, 2, 7)), rng.standard_normal((3, 2, 7))
    freq, pos, pairs = rng.standard_normal(3), rng.integers(-50, 50, (3, 2)), [2, 1]
    y = ops.rotary(x, freq, pos, pairs, interleaved)
    np.testing.assert_allclose(ops.rotary(y, freq, pos, pairs, interleaved, inverse=True), x, atol=1e-12)
    num = _num_grad(lambda: (w * ops.rotary(x, freq, pos, pairs, interleaved)).sum(), x)
    np.testing.assert_allclose(ops.rotary(w, freq, pos, pairs, interleaved, inverse=True), num, atol=1e-7)


def test_rotary_scores_depend_on_position_differences():
    rng = np.random.default_rng(4)
    q, k, freq = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8)), rng.standard_normal(4)
    dot = lambda p, r: (ops.rotary(q, freq, [[p, 2 * p]], [2, 2]) * ops.rotary(k, freq, [[r, 2 * r]], [2, 2])).sum()  # noqa: E731
    assert abs(dot(5, 2) - dot(105, 102)) < 1e-10


def test_decay_attention_worked_values():
    # one channel each: S = 1*2, then 2/2 + 3*1 = 4, then a new sequence from its state 8: 8/2 + 1*1
    q, k, v = (np.array(x, float).reshape(3, 1, 1) for x in ([1, 2, 1], [1, 3, 1], [2, 1, 1]))
    half = np.log([0.5])
    out, st = ops.decay_attention(q, k, v, half, scale=0.5, cu_seqlens=[0, 2, 2, 3],
                                  state_in=np.array([0.0, 5.0, 8.0]).reshape(3, 1, 1, 1))
    assert np.allclose(out.ravel(), [1.0, 4.0, 2.5])
    assert np.allclose(st.ravel(), [4.0, 5.0, 5.0])


def test_decay_attention_is_the_sum_over_earlier_tokens():
    g = np.random.default_rng(3)
    q, k, v = g.normal(size=(9, 2, 4)), g.normal(size=(9, 2, 4)), g.normal(size=(9, 2, 3))
    ld = np.array([-0.3, -np.inf])
    out, _ = ops.decay_attention(q, k, v, ld, scale=0.7)
    for h in range(2):
        for i in range(9):
            want = sum((np.exp(ld[h] * (i - j)) if i > j else 1.0) * (q[i, h] @ k[j, h]) * v[j, h] for j in range(i + 1))
            assert np.allclose(out[i, h], 0.7 * want)


def test_decay_attention_without_decay_is_the_unnormalised_output():
    import oracle
    g = np.random.default_rng(4)
    q, k, v = g.normal(size=(12, 2, 4)), g.normal(size=(12, 2, 4)), g.normal(size=(12, 2, 4))
    out, _ = ops.decay_attention(q, k, v, np.zeros(2), cu_seqlens=[0, 5, 12])
    ref = oracle.forward(q, k, v, "identity", True, cu_seqlens=np.array([0, 5, 12]), norm="none")
    assert np.allclose(out, ref)


def test_decay_attention_gradients():
    g = np.random.default_rng(5)
    q, k, v, do = g.normal(size=(7, 2, 3)), g.normal(size=(7, 2, 3)), g.normal(size=(7, 2, 2)), g.normal(size=(7, 2, 2))
    s, ds = g.normal(size=(3, 2, 3, 2)), g.normal(size=(3, 2, 3, 2))
    ld, cu = np.array([-0.2, -1.5]), [0, 4, 4, 7]

    def loss():
        out, st = ops.decay_attention(q, k, v, ld, 0.6, cu, state_in=s)
        return (out * do).sum() + (st * ds).sum()

    got = ops.decay_attention_backward(q, k, v, do, ld, 0.6, cu, state_in=s, dstate_out=ds)
    for x, y in zip((q, k, v, s), got):
        assert np.allclose(_num_grad(loss, x), y, atol=1e-7)


def test_qk_norm_rotary_worked_values():
    x = np.array([3.0, 4.0, 0.0]).reshape(1, 1, 3)
    y, r = ops.qk_norm_rotary(x, np.array([1.0, 2.0, 5.0]), [np.pi / 2], [[1]], [1], eps=0.0)
    assert np.allclose(r, np.sqrt(3.0) / 5)
    assert np.allclose(y.ravel(), np.array([-8.0, 3.0, 0.0]) * np.sqrt(3.0) / 5)   # a quarter of a turn of (3, 8)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("per_head", [False, True])
def test_qk_norm_rotary_gradients(per_head, interleaved):
    g = np.random.default_rng(6)
    x, dy = g.normal(size=(4, 2, 7)), g.normal(size=(4, 2, 7))
    w = g.normal(size=(2, 7) if per_head else 7)
    args = ([0.3, 1.0, 0.01], [[0, 5], [1, -3], [2, 9], [70, 0]], [1, 2], interleaved)

    def loss():
        return (ops.qk_norm_rotary(x, w, *args, eps=0.1)[0] * dy).sum()

    _, r = ops.qk_norm_rotary(x, w, *args, eps=0.1)
    dx, dw = ops.qk_norm_rotary_backward(x, r, dy, w, *args)
    assert np.allclose(_num_grad(loss, x), dx, atol=1e-7)
    assert np.allclose(_num_grad(loss, w), dw, atol=1e-7)
