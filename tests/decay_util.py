"""Tolerances of linear attention with a decay for each head, derived here.

u = 2^-24 is half a step of fp32.  Let M_t = g M_{t-1} + |k_t| |v_t|^T majorise the state.  In fp32, in
any grouping of the tokens into chunks and segments, a token's term takes: its weight, a power of the
decay (off by at most 6 u: exp2f within two steps, its correction's two roundings) and the product with
it; the product k v and the addition; and, once for every chunk of at least 32 tokens that it crosses, a
factor g^n (6 u and a rounding) and an addition.  Each addition rounds a value no larger than M_t.  With
the tensor cores an addition to an accumulator may truncate, 2 u.  So
    E_t = g E_{t-1} + 3 u M_t + 10 u |k_t| |v_t|^T
bounds the state's error: 2 u a token for the addition, 16 u / 32 for a chunk's factor and addition.
An output sums d_k products of q with the state (d_k + 4 roundings of scale |q|^T M):
    |scale| |q|^T (E_t + (d_k + 12) u M_t).
The scores' form q.k first (d_k roundings), then weights (8 u) and sums over a chunk's tokens (at most 2 u
a token: counted in E), is covered by the same.

bf16 operands on the tensor cores: decayed scores, and weighted keys (queries) on their way into a state that
stays in one call, are rounded to bf16, off by 2^-8; a state goes in as a bf16 and the bf16 of what it leaves,
off by 2^-16: 2^-8 + 2^-16 + 2^-24 of M at most.  States that a call returns are sums of three such parts, 2^-24:
counted above.
"""
import numpy as np

from layer_ops_util import HALF, U, check  # noqa: F401

PARTS = {"f32": 0.0, "bf16": 2.0 ** -8 + 2.0 ** -15}


def forward_bounds(q, k, v, log_decay, scale, spans, state, dtype):
    """(bound of out, bound of state_out)."""
    q, k, v = (np.abs(np.asarray(x, np.float64)) for x in (q, k, v))
    g = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    out = np.zeros_like(v)
    edge = np.zeros((len(spans), q.shape[1], q.shape[2], v.shape[2]))
    dk = q.shape[2]
    for s, (lo, hi) in enumerate(spans):
        M = np.abs(np.asarray(state[s], np.float64)) if state is not None else np.zeros_like(edge[0])
        E = np.zeros_like(M)
        for t in range(lo, hi):
            kv = k[t][:, :, None] * v[t][:, None, :]
            M = g * M + kv
            E = g * E + U * (3 * M + 10 * kv)
            out[t] = abs(scale) * np.matmul(q[t][:, None, :], E + ((dk + 12) * U + PARTS[dtype]) * M)[:, 0]
        edge[s] = E + 8 * U * M if hi > lo else 0.0
    return 1.01 * out, 1.01 * edge


def backward_bounds(q, k, v, dout, log_decay, scale, spans, state, dstate, dtype):
    """Bounds of dq, dk, dv, dstate_in: the forward's for the same recurrences with other operands."""
    q, k, v, do = (np.abs(np.asarray(x, np.float64)) for x in (q, k, v, dout))
    g = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    d_k, d_v, sc = q.shape[2], v.shape[2], abs(scale)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    edge = np.zeros((len(spans), q.shape[1], d_k, d_v))
    more = (max(d_k, d_v) + 12) * U + PARTS[dtype]
    for s, (lo, hi) in enumerate(spans):
        M = np.abs(np.asarray(state[s], np.float64)) if state is not None else np.zeros_like(edge[0])
        E = np.zeros_like(M)
        for t in range(lo, hi):
            kv = k[t][:, :, None] * v[t][:, None, :]
            M = g * M + kv
            E = g * E + U * (3 * M + 10 * kv)
            dq[t] = sc * np.matmul(E + more * M, do[t][:, :, None])[:, :, 0]
        R = np.abs(np.asarray(dstate[s], np.float64)) if dstate is not None else np.zeros_like(edge[0])
        E = np.zeros_like(R)
        for t in range(hi - 1, lo - 1, -1):
            qd = sc * q[t][:, :, None] * do[t][:, None, :]
            R = R + qd
            E = E + U * (3 * R + 11 * qd)
            dk[t] = np.matmul(E + more * R, v[t][:, :, None])[:, :, 0]
            dv[t] = np.matmul(k[t][:, None, :], E + more * R)[:, 0]
            R, E = g * R, g * E
        edge[s] = E + 8 * U * R if hi > lo else 0.0
    return tuple(1.01 * x for x in (dq, dk, dv, edge))
