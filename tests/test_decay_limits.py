"""The limits of decay_limits.py on a numpy model of the tensor cores' arithmetic: it keeps them, and exceeds them where the
state loses its second part or a little in every chunk."""
import numpy as np

from decay_limits import chunked, limits, relative, rows_that_differ_little
from oracle import layer_ops as ops


def _bf16(a):
    b = np.asarray(a, np.float32).view(np.uint32)
    return ((b + 0x7fff + (b >> 16 & 1)) & 0xffff0000).astype(np.uint32).view(np.float32).astype(np.float64)


def _case(T, H, d, seed):
    g = np.random.default_rng(seed)
    q, k = (_bf16(g.standard_normal((T, H, d)) * d ** -0.25) for _ in range(2))
    return q, k, _bf16(g.standard_normal((T, H, d)))


def test_the_model_keeps_the_limits():
    for T, H, d, ld in ((1500, 4, 64, [-0.5, -0.03, -0.002, 0.0]), (700, 6, 8, [0.0, -1e-6, -1e-4, -1e-2, -1.0, -np.inf])):
        q, k, v = _case(T, H, d, T)
        ref, _ = ops.decay_attention(q, k, v, ld, 0.37)
        lim = limits(q, k, v, ref, ld, 0.37, [(0, T)], -(-T // 128))
        assert (lim < 0.005).all()
        assert (relative(chunked(q, k, v, ld, 0.37), ref) <= lim).all()


def test_a_state_that_loses_a_little_exceeds_them():
    q, k, v = _case(4000, 4, 8, 1)
    ld = [0.0, -1e-6, -1e-4, -1e-3]
    ref, _ = ops.decay_attention(q, k, v, ld, 0.37)
    lim = limits(q, k, v, ref, ld, 0.37, [(0, 4000)], 32)
    assert (relative(chunked(q, k, v, ld, 0.37), ref) <= lim).all()
    assert (relative(chunked(q, k, v, ld, 0.37, lost=2.0 ** -10), ref) > lim).all()


def test_a_state_read_as_one_bf16_exceeds_the_bound():
    q, s, ref, bound = rows_that_differ_little(3, 64, 64, 2)
    none = np.zeros_like(q)
    assert (np.abs(chunked(q, none, np.zeros((1, 3, 64)), np.zeros(3), 1.0, s) - ref) <= bound).all()
    assert (np.abs(chunked(q, none, np.zeros((1, 3, 64)), np.zeros(3), 1.0, s, low=False) - ref) > bound).mean() > 0.3
