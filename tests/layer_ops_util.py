"""Tolerances of the operators around the attention call, derived here.

u = 2^-24 is half a step of fp32; a value stored in type t is off by at most
half a step of t: HALF[t] times its magnitude.  With every bound below, an
element passes when |got - ref| <= computed bound + HALF[t] (|ref| + bound).
"""
import numpy as np

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def check(got, ref, bound, dtype, what=""):
    """Every element within `bound` (before storage) and half a step of dtype; non-finite
    reference values must come out as the same kind."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, f"{what}: shape {got.shape}, expected {ref.shape}"
    if got.size == 0:
        return
    fin = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN in other places"
    assert np.array_equal(got[~fin & ~np.isnan(ref)], ref[~fin & ~np.isnan(ref)]), f"{what}: infinities differ"
    bound = np.broadcast_to(bound, ref.shape)
    tol = bound + HALF[dtype] * (np.abs(ref) + bound)
    bad = fin & ~(np.abs(got - ref) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} beyond tolerance, first at {i}: got {got[i]!r}, "
                             f"expected {ref[i]!r} within {tol[i]:.3e}")


def scan_bound(a, b, spans, state=None, reverse=False):
    """Error of a recurrence h_t = a_t h_{t-1} + b_t in fp32 in any grouping of the tokens.

    Let M_t = |a_t| M_{t-1} + |b_t| majorise |h_t|.  Each token adds at most four roundings of a
    value no larger than M_t: the fused multiply-add of the recurrence, the same step in a tile's
    state from zero, one more factor in a tile's product of gates (whose error scales a state that
    M majorises), and the multiply-add that applies it.  So E_t = |a_t| E_{t-1} + 4 u M_t; 5 u
    covers the products of these errors with one another.
    For the adjoint (reverse) the gate into token t is a_{t+1}.  Returns (E, E behind the last
    token of each span)."""
    a, b = np.abs(np.asarray(a, np.float64)), np.abs(np.asarray(b, np.float64))
    E = np.zeros_like(b)
    edge = np.zeros((len(spans),) + b.shape[1:])
    for s, (lo, hi) in enumerate(spans):
        M = np.zeros(b.shape[1:]) if state is None else np.abs(np.asarray(state[s], np.float64))
        e = np.zeros(b.shape[1:])
        for t in (range(hi - 1, lo - 1, -1) if reverse else range(lo, hi)):
            g = 1.0 if reverse and t == hi - 1 else a[t + 1] if reverse else a[t]
            M = g * M + b[t]
            e = g * e + 5 * U * M
            E[t] = e
        # the adjoint's edge value is a_first g_first: one more product
        edge[s] = (a[lo] * (e + U * M) if reverse else e) if hi > lo else 0.0
    return E, edge


def norm_terms(d):
    """Roundings on the longest path of a sum over d values: a lane adds at most 64 of them one
    after the other, and at most 16 partial sums join above it."""
    return min(d, 64 + 16)


def layer_norm_bounds(x, weight, bias, mean, rstd, eps):
    """Bounds of y, mean and rstd.  K = norm_terms(d) roundings and one division in a mean:
    |dmu| <= (K + 1) u mean|x|.  Deviations c = x - mu are off by |dmu| + u |c|; as they sum to
    zero, the variance is off by relative 2 u + (K + 3) u and by dmu^2.  rstd = 1/sqrt(var + eps)
    takes half of that relative error and three roundings (addition, square root, division)."""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    K = norm_terms(d)
    c = x - mean[..., None]
    dmu = (K + 1) * U * np.abs(x).mean(-1)
    var = (c * c).mean(-1)
    rel = 0.5 * ((K + 5) * U * var + dmu ** 2) / (var + eps) + 3 * U
    w = 1.0 if weight is None else np.abs(weight)
    xh = np.abs(c) * rstd[..., None]
    by = w * (rstd[..., None] * (dmu[..., None] + U * np.abs(c)) + xh * (rel[..., None] + 2 * U))
    by = by + U * (w * xh + (0.0 if bias is None else np.abs(bias)))
    return 1.01 * by, 1.01 * dmu, 1.01 * rel * rstd


def layer_norm_backward_bounds(x, dy, mean, rstd, weight, chain):
    """Bounds of dx, dweight, dbias for given statistics.  xh = (x - mean) rstd: two roundings;
    w dy: one; the two row means: K = norm_terms(d) more and a division; the rest five of the
    terms' magnitudes.  A weight gradient sums `chain` values one after the other in fp32 (two
    roundings before each) and joins the sums with compensation (two roundings)."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    d = x.shape[-1]
    K = norm_terms(d)
    w = np.ones(d) if weight is None else np.abs(np.asarray(weight, np.float64))
    r = np.asarray(rstd, np.float64)[..., None]
    xh = np.abs(x - np.asarray(mean, np.float64)[..., None]) * r
    u = np.abs(dy) * w
    m1 = u.mean(-1, keepdims=True)
    m2 = (u * xh).mean(-1, keepdims=True)
    dx = r * U * (2 * u + (K + 3) * m1 + (K + 7) * xh * m2 + 5 * (u + m1 + xh * m2))
    lead = tuple(range(x.ndim - w.ndim))
    return 1.01 * dx, (chain + 4) * U * (np.abs(dy) * xh).sum(lead), (chain + 2) * U * np.abs(dy).sum(lead)


def rotary_bound(x, pairs, interleaved):
    """cos and sin: the angle in half turns is rounded once to fp32 (at most pi u radians), each
    value is within one step (2 u); the products and their sum add two roundings: 8 u (|x0| + |x1|)
    covers pi + 2 + 2.  The fixed-point angle adds at most |position| 2^-53 turns, below u for
    every position up to 2^28 and counted by the caller beyond.  Unrotated channels are exact."""
    x = np.abs(np.asarray(x, np.float64))
    P = sum(pairs)
    i0, i1 = (np.s_[..., 0:2 * P:2], np.s_[..., 1:2 * P:2]) if interleaved else (np.s_[..., :P], np.s_[..., P:2 * P])
    b = np.zeros_like(x)
    b[i0] = b[i1] = 8 * U * (x[i0] + x[i1])
    return b
