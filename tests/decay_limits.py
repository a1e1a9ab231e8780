"""What linear attention with a decay for each head may be off by on the tensor cores, as norms over a head's outputs
instead of element by element.

The bounds of decay_util.py add up the magnitudes of all terms: with slow decays and many tokens that is as much as the
outputs themselves.  The roundings are independent of one another, though, so their squares add up.  A bf16 rounding
is off by at most 2^-8 of the power of two below the value, evenly, so by 2^-8 / sqrt(3) of it in the mean square, and by
    E0 = 2^-8 / sqrt(3) sqrt(mean of 1 / m^2),   m in [1, 2) with density 1 / (m ln 2):   mean 3 / (8 ln 2)
of a value.  With terms scale g^(i-j) (x_i . y_j) z_j as in a product pass, each is rounded once, in its score or in
its weighted y, and the output once more:
    |error|^2 ~ E0^2 sum_i (|out_i|^2 + |terms of i|^2),
the terms' squares as a recurrence, V_i = g^2 V_(i-1) + (y_i z_i^T)^2, |terms of i|^2 = scale^2 (x_i^2)^T V_i.  A quarter
more is for mantissas that are not spread like that and for sums that are not their expectation.  Besides these the tensor
cores cut off what they add to the state that stays in them, 5 2^-23 of it for 16 tokens at most, 40 2^-23 a chunk of 128, for
`chunks` of a segment (64 at most): of the outputs' norm, whose queries the losses meet as the state itself.
"""
import numpy as np

E0 = 2.0 ** -8 / np.sqrt(3.0) * np.sqrt(3.0 / (8.0 * np.log(2.0)))


def relative(got, ref):
    """|got - ref| / |ref| of each head [T, H, d]."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    return np.sqrt(((got - ref) ** 2).sum((0, 2)) / (ref ** 2).sum((0, 2)))


def limits(x, y, z, out, log_decay, scale, spans, chunks, reverse=False):
    """Limit of `relative` of each head, for a product pass with these operands and output."""
    g2 = np.exp(2.0 * np.asarray(log_decay, np.float64))[:, None, None]
    x2, y2, z2 = (np.asarray(a, np.float64) ** 2 for a in (x, y, z))
    terms = np.zeros(x2.shape[1])
    for lo, hi in spans:
        V = np.zeros((x2.shape[1], x2.shape[2], z2.shape[2]))
        for t in (range(hi - 1, lo - 1, -1) if reverse else range(lo, hi)):
            V = g2 * V + y2[t][:, :, None] * z2[t][:, None, :]
            terms += (x2[t] * V.sum(2)).sum(1)
    size = (np.asarray(out, np.float64) ** 2).sum((0, 2))
    return 1.25 * E0 * np.sqrt(1.0 + scale * scale * terms / size) + 40 * 2.0 ** -23 * chunks


def chunked(q, k, v, log_decay, scale, state=None, low=True, lost=0.0, chunk=128):
    """The tensor cores' forward of one sequence in numpy: bf16 scores and weighted keys, a state read as a bf16 and, with
    `low`, what that leaves; every chunk loses `lost` of the state."""
    def bf16(a):
        b = np.asarray(a, np.float32).view(np.uint32)
        return ((b + 0x7fff + (b >> 16 & 1)) & 0xffff0000).astype(np.uint32).view(np.float32).astype(np.float64)
    T, H, dk = q.shape
    g = np.maximum(np.asarray(log_decay, np.float64), -1e30)      # (-inf times no token is none)
    out = np.zeros((T, H, v.shape[2]))
    S = np.zeros((H, dk, v.shape[2])) if state is None else np.array(state, np.float64)
    for lo in range(0, T, chunk):
        n = min(chunk, T - lo)
        i = np.arange(n)
        a = np.einsum("ihd,jhd->hij", q[lo:lo + n], k[lo:lo + n])
        apart = i[:, None] - i[None, :]
        w = np.where(apart >= 0, np.exp(g[:, None, None] * np.maximum(apart, 0)), 0.0)
        hi = bf16(S)
        S_in = hi + (bf16(S - hi) if low else 0.0)
        into = np.exp(g[:, None] * (i + 1)).T[..., None]
        out[lo:lo + n] = (np.einsum("hij,jhd->ihd", bf16(scale * w * a), v[lo:lo + n]) +
                          scale * into * np.einsum("ihd,hde->ihe", q[lo:lo + n], S_in))
        kw = bf16(k[lo:lo + n] * np.exp(g[:, None] * (n - 1 - i)).T[..., None])
        S = (1.0 - lost) * (np.exp(g * n)[:, None, None] * S + np.einsum("jhd,jhe->hde", kw, v[lo:lo + n]))
    return bf16(out)


def rows_that_differ_little(H, dk, dv, seed):
    """(q, state, reference, bound) of one token for each head whose queries take pairs of the state's rows from one
    another that differ by less than a bf16 of them holds: only a state read to more bits gives the difference.  Bound of
    an output: the state to 2^-16 and fp32's roundings of the sum, 2^-24 each, of the terms; the output's half step."""
    rng = np.random.default_rng(seed)
    s = rng.uniform(1.0, 2.0, (H, dk, dv)).astype(np.float32)
    s[:, 1::2] = (s[:, 0::2] * (1.0 + 2.0 ** -9 * rng.uniform(0.5, 1.0, (H, dk // 2, dv)))).astype(np.float32)
    q = np.ones((1, H, dk))
    q[:, :, 0::2] = -1.0
    s64 = s.astype(np.float64)
    ref = np.einsum("thd,hde->the", q, s64)
    bound = (2.0 ** -16 + (dk + 12) * 2.0 ** -24) * np.abs(s64).sum(1)[None]
    return q, s, ref, bound + 2.0 ** -8 * (np.abs(ref) + bound)
