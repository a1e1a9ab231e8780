"""fp64 oracle of the operators around the attention call, from their formulas:
the gated linear recurrence, layer norm and rotary positions, with gradients."""
import numpy as np


def _spans(T, cu_seqlens, nseq):
    if cu_seqlens is None:
        n = T // nseq
        return [(s * n, (s + 1) * n) for s in range(nseq)]
    return [(int(lo), int(hi)) for lo, hi in zip(cu_seqlens, cu_seqlens[1:])]


def gated_scan(a, b, cu_seqlens=None, nseq=1, state_in=None):
    """(h, state_out) of h_t = a_t h_{t-1} + b_t on rows [T, ...]."""
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    h = np.empty_like(b)
    spans = _spans(b.shape[0], cu_seqlens, nseq)
    out = np.zeros((len(spans),) + b.shape[1:])
    if state_in is not None:
        out[:] = state_in
    for s, (lo, hi) in enumerate(spans):
        for t in range(lo, hi):
            # the first token of a sequence without a state has nothing to scale
            out[s] = b[t] if t == lo and state_in is None else a[t] * out[s] + b[t]
            h[t] = out[s]
    return h, out


def gated_scan_backward(a, h, dh, cu_seqlens=None, nseq=1, state_in=None, dstate_out=None):
    """(da, db, dstate_in) of sum(dh * h) + sum(dstate_out * state_out), h the forward output."""
    a, h, dh = (np.asarray(x, np.float64) for x in (a, h, dh))
    da, db = np.empty_like(a), np.empty_like(dh)
    spans = _spans(dh.shape[0], cu_seqlens, nseq)
    ds = np.zeros((len(spans),) + dh.shape[1:])
    if dstate_out is not None:
        ds[:] = dstate_out
    for s, (lo, hi) in enumerate(spans):
        for t in range(hi - 1, lo - 1, -1):
            db[t] = dh[t] + ds[s]
            before = h[t - 1] if t > lo else (0.0 if state_in is None else state_in[s])
            da[t] = db[t] * before
            ds[s] = a[t] * db[t]
    return da, db, ds


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd) over the last dimension; weight and bias broadcast over the leading ones."""
    x = np.asarray(x, np.float64)
    mean = x.mean(-1)
    c = x - mean[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        rstd = 1.0 / np.sqrt((c * c).mean(-1) + eps)
        y = c * rstd[..., None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd


def layer_norm_backward(x, dy, mean, rstd, weight=None):
    """(dx, dweight, dbias) for given statistics; the last two have weight's shape ([d] without one)."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    w = np.ones(x.shape[-1]) if weight is None else np.asarray(weight, np.float64)
    r = np.asarray(rstd, np.float64)[..., None]
    xh = (x - np.asarray(mean, np.float64)[..., None]) * r
    u = dy * w
    dx = r * (u - u.mean(-1, keepdims=True) - xh * (u * xh).mean(-1, keepdims=True))
    lead = tuple(range(x.ndim - w.ndim))
    return dx, (dy * xh).sum(lead), dy.sum(lead)


def rotary(x, freq, positions, pairs, interleaved=False, inverse=False):
    """x [T, H, d] with pair p turned by positions[t, axis(p)] * freq[p]."""
    x = np.asarray(x, np.float64)
    axis = np.repeat(np.arange(len(pairs)), pairs)
    angle = np.asarray(positions, np.float64).reshape(x.shape[0], -1)[:, axis] * np.asarray(freq, np.float64)
    turn = np.exp((-1j if inverse else 1j) * angle)[:, None, :]
    P = len(axis)
    i0, i1 = (np.s_[..., 0:2 * P:2], np.s_[..., 1:2 * P:2]) if interleaved else (np.s_[..., :P], np.s_[..., P:2 * P])
    z = (x[i0] + 1j * x[i1]) * turn
    y = x.copy()
    y[i0], y[i1] = z.real, z.imag
    return y
