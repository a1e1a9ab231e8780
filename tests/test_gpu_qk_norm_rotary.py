"""GPU parity of the norm of queries and keys with their rotation, and of its gradients, against the
fp64 oracle.

Tolerances (u = 2^-24).  A lane adds up to 32 squares and at most 5 partial sums join above it, so the
sum of d squares is off by K u, K = min(d, 32 + 5) + 1, the mean by one more; the reciprocal root takes half of that
and two steps of its own (4 u).  u = x rstd w: two roundings.  Turning: rotary_bound's 8 u of both
channels of a pair.  A gradient's mean over d likewise takes K + 2 roundings."""
import numpy as np
import pytest

from layer_ops_util import U, check
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
    return None if t is None else t.detach().cpu().double().numpy()


def _pair_sum(x, pairs, interleaved):
    """|x0| + |x1| in both channels of a pair, |x| elsewhere."""
    x = np.abs(x)
    P = sum(pairs)
    i0, i1 = (np.s_[..., 0:2 * P:2], np.s_[..., 1:2 * P:2]) if interleaved else (np.s_[..., :P], np.s_[..., P:2 * P])
    s = x.copy()
    s[i0] = s[i1] = x[i0] + x[i1]
    return s


def _terms(d):
    return min(d, 37) + 1


def _bounds(x, w, rstd, eps, pairs, interleaved):
    """Bounds of y and rstd."""
    K = _terms(x.shape[-1])
    rel = ((K + 2) / 2 + 4) * U
    u = np.abs(x) * rstd[..., None] * (1.0 if w is None else np.abs(w))
    return 1.01 * (rel + 2 * U + 8 * U) * _pair_sum(u, pairs, interleaved), 1.01 * rel * rstd


def _backward_bounds(x, rstd, dy, w, pairs, interleaved):
    d = x.shape[-1]
    K = _terms(d)
    w = np.ones(d) if w is None else np.abs(w)
    r = rstd[..., None]
    xh, du = np.abs(x) * r, _pair_sum(dy, pairs, interleaved)
    off = 8 * U * du                          # of what is turned back; a magnitude above du's too
    g = du * w
    mean = (g * xh).mean(-1, keepdims=True)
    dx = r * (off * w + 4 * U * g + xh * ((off * w * xh).mean(-1, keepdims=True) + (K + 8) * U * mean))
    lead = tuple(range(x.ndim - w.ndim))
    chain = min(x.shape[0] * x.shape[1], 300)     # rows that a lane and a block's places add one after the other
    return 1.01 * dx, 1.01 * ((off * xh).sum(lead) + (chain + 6) * U * (du * xh).sum(lead))


def _case(T, Hq, Hk, d, pairs, dtype, per_head=False, fused=False, seed=1):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g)

    rows = (normal(T, Hq + 2 * Hk, d) * torch.exp(normal(T, Hq + 2 * Hk, 1))).to(TYPES[dtype]).cuda()
    q, k = rows[:, :Hq], rows[:, Hq:Hq + Hk]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    w = [1.0 + 0.3 * (normal(H, d) if per_head else normal(d)) for H in (Hq, Hk)]
    freq = torch.cat([10000.0 ** (-torch.arange(p).double() / max(p, 1)) for p in pairs]).float()
    pos = torch.randint(-50, 1 << 20, (T, len(pairs)), generator=g).to(torch.int32)
    return dict(q=q, k=k, qw=w[0].cuda(), kw=w[1].cuda(), freq=freq.cuda(), pos=pos.cuda(), pairs=pairs,
                dq=normal(T, Hq, d).to(TYPES[dtype]).cuda(), dk=normal(T, Hk, d).to(TYPES[dtype]).cuda(), dtype=dtype)


def _forward(la, c, **kw):
    return la.la_qk_norm_rotary(c["q"], c["k"], c["qw"], c["kw"], c["freq"], c["pos"], c["pairs"],
                                **{**dict(return_rstd=True), **kw})


def _backward(la, c, qr, kr, **kw):
    return la.la_qk_norm_rotary_backward(c["q"], c["k"], qr, kr, c["dq"], c["dk"], c["qw"], c["kw"], c["freq"], c["pos"],
                                         c["pairs"], **kw)


def _check_all(la, c, il, eps=1e-6):
    qo, ko, qr, kr = _forward(la, c, interleaved=il, eps=eps)
    grads = _backward(la, c, qr, kr, interleaved=il)
    for x, w, y, r, dy, dx, dw in (("q", "qw", qo, qr, "dq", grads[0], grads[2]), ("k", "kw", ko, kr, "dk", grads[1], grads[3])):
        if c[x] is None:
            assert y is None and dx is None and dw is None
            continue
        xn, wn, dyn = _np(c[x]), _np(c[w]), _np(c[dy])
        ref, ref_r = ops.qk_norm_rotary(xn, wn, _np(c["freq"]), c["pos"].cpu().numpy(), c["pairs"], il, eps)
        by, br = _bounds(xn, wn, ref_r, eps, c["pairs"], il)
        check(_np(y), ref, by, c["dtype"], f"{x}_out")
        check(_np(r), ref_r, br, "f32", f"{x}_rstd")
        rdx, rdw = ops.qk_norm_rotary_backward(xn, _np(r), dyn, wn, _np(c["freq"]), c["pos"].cpu().numpy(), c["pairs"], il)
        bx, bw = _backward_bounds(xn, _np(r), dyn, wn, c["pairs"], il)
        check(_np(dx), rdx, bx, c["dtype"], f"d{x}")
        if wn is None:
            assert dw is None
        else:
            check(_np(dw), rdw, bw, "f32", f"d{x}_weight")
    return qo, ko, qr, kr, grads


SHAPES = [(1, 1, 1, 2, (1,)), (5, 3, 2, 64, (32,)), (33, 16, 4, 128, (64,)), (70, 8, 8, 64, (8, 12, 12)), (7, 2, 1, 83, (20, 19)),
          (300, 5, 5, 37, (18,)), (9, 7, 3, 255, (60, 0, 67)), (6, 2, 2, 256, (128,)), (4, 1, 1, 1024, (512,)),
          (3, 2, 1, 1024, (8,)), (3, 1, 2, 1023, (511,)), (3, 1, 1, 1021, (1,)), (4, 3, 1, 512, (100, 100)), (2000, 4, 4, 16, (8,)),
          (2500, 2, 1, 64, (16,)), (40, 40, 40, 64, (32,)), (11, 300, 20, 32, (16,))]


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,Hq,Hk,d,pairs", SHAPES, ids=lambda v: str(v).replace(" ", ""))
def test_shapes(la, T, Hq, Hk, d, pairs, dtype, il):
    for per_head, fused in ((False, False), (True, True)):
        _check_all(la, _case(T, Hq, Hk, d, pairs, dtype, per_head, fused), il)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_keys_or_weights(la, dtype):
    c = _case(50, 3, 2, 64, (32,), dtype)
    both = _check_all(la, c, False)
    alone = _check_all(la, dict(c, k=None, kw=None, dk=None), False)
    assert torch.equal(both[0], alone[0]) and torch.equal(both[4][0], alone[4][0])
    _check_all(la, dict(c, qw=None), False)
    _check_all(la, dict(c, kw=None), True)
    bare = dict(c, qw=None, kw=None)
    _check_all(la, bare, False)
    ones = dict(c, qw=torch.ones(64).cuda(), kw=torch.ones(64).cuda())
    assert torch.equal(_forward(la, bare)[0], _forward(la, ones)[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,pairs", [(64, (32,)), (83, (20, 19))])
def test_operands_anywhere_and_far_apart(la, d, pairs, dtype):
    """Rows that start on no vector's boundary, tokens some way apart."""
    c = _case(60, 3, 2, d, pairs, dtype, seed=2)
    want = _forward(la, c)
    grads = _backward(la, c, want[2], want[3])
    for gap, by in ((0, 1), (1, 0), (8, 0), (17, 3), (64, 2)):
        def apart(x):
            T, H, _ = x.shape
            buf = torch.full((T * (H * d + gap) + by,), 9.0, dtype=x.dtype, device="cuda")
            y = buf[by:].as_strided((T, H, d), (H * d + gap, d, 1))
            y.copy_(x)
            return y
        m = dict(c, q=apart(c["q"]), k=apart(c["k"]))
        _check_all(la, m, False)
        if (gap, by) == (8, 0):                # still whole vectors where they were: the same arithmetic
            assert all(torch.equal(x, y) for x, y in zip(_forward(la, m), want))
            assert all(torch.equal(x, y) for x, y in zip(_backward(la, m, want[2], want[3]), grads))


def test_refused_strides(la):
    c = _case(20, 4, 4, 64, (32,), "bf16")
    for q in (c["q"].transpose(0, 1).contiguous().transpose(0, 1), c["q"][:, ::2], c["q"][..., ::2].expand(20, 4, 32),
              c["q"][:1].expand(20, 4, 64)):
        with pytest.raises(ValueError):
            la.la_qk_norm_rotary(q, None, None, None, c["freq"][:q.shape[2] // 2], c["pos"], (q.shape[2] // 2,))
    for bad in (dict(k=c["k"][:10]), dict(kw=torch.ones(4, 64).cuda()), dict(qw=torch.ones(32).cuda()),
                dict(k=c["k"].float()), dict(freq=c["freq"][:-1].contiguous()), dict(pos=c["pos"][:-1])):
        with pytest.raises(ValueError):
            _forward(la, dict(c, **bad))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place(la, dtype):
    for d, pairs in ((64, (32,)), (83, (20, 19))):
        c = _case(70, 3, 2, d, pairs, dtype, seed=3)
        qo, ko, _, _ = _forward(la, c)
        q, k = c["q"].clone(), c["k"].clone()
        la.la_qk_norm_rotary(q, k, c["qw"], c["kw"], c["freq"], c["pos"], pairs, q_out=q, k_out=k)
        assert torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_rows_values_stay_in_it(la, dtype):
    c = _case(40, 3, 2, 64, (32,), dtype, seed=4)
    clean = _forward(la, c)
    grads = _backward(la, c, clean[2], clean[3])
    for bad in (float("nan"), float("inf"), 3e38):
        d = dict(c, q=c["q"].clone(), dq=c["dq"].clone())
        d["q"][7, 1, 3] = bad
        d["dq"][9, 2, 60] = bad
        out = _forward(la, d)
        keep = torch.ones(40, 3, dtype=torch.bool, device="cuda")
        keep[7, 1] = False
        assert torch.equal(out[0][keep], clean[0][keep]) and torch.equal(out[1], clean[1])
        got = _backward(la, d, clean[2], clean[3])
        keep[9, 2] = False
        assert torch.equal(got[0][keep], grads[0][keep]) and torch.equal(got[1], grads[1])
        assert torch.equal(got[3], grads[3])


def test_rows_of_zeros_and_tiny_and_large_rows(la):
    c = _case(40, 2, 2, 64, (32,), "f32", seed=5)
    c["q"][3] = 0.0
    c["q"][4] *= 1e-18
    c["q"][5] *= 1e15
    _check_all(la, c, False)
    c["q"][6] = 1e30                       # squares beyond fp32: rstd 0
    qo, _, qr, _ = _forward(la, c)
    assert not qr[6].any() and not qo[6].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_same_bits_every_time_captured_too(la, dtype):
    c = _case(3000, 8, 4, 64, (32,), dtype, fused=True, seed=6)
    want = _forward(la, c)
    grads = _backward(la, c, want[2], want[3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _forward(la, c)
        more = _backward(la, c, got[2], got[3])
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got + more, want + grads))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = _backward(la, c, want[2], want[3], stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(other, grads))


def test_no_tokens(la):
    c = _case(1, 3, 2, 64, (32,), "bf16")
    e = dict(c, **{x: c[x][:0] for x in ("q", "k", "pos", "dq", "dk")})
    qo, ko, qr, kr = _forward(la, e)
    assert qo.shape == (0, 3, 64) and kr.shape == (0, 2)
    dq, dk, dqw, dkw = _backward(la, e, qr, kr)
    assert dq.shape == (0, 3, 64) and not dqw.any() and not dkw.any()


def test_rows_beyond_32_bits(la):
    """Tokens of a projection whose last rows lie beyond 2^32 bytes."""
    T, wide, d = 40000, 60000, 64
    buf = torch.empty(T * wide, dtype=torch.bfloat16, device="cuda")
    assert buf.numel() * 2 > 2 ** 32
    c = _case(T, 2, 1, d, (32,), "bf16", seed=7)
    q, k = (buf[at:].as_strided((T, H, d), (wide, d, 1)) for at, H in ((0, 2), (2 * d, 1)))
    q.copy_(c["q"]), k.copy_(c["k"])
    want = _forward(la, c)
    got = _forward(la, dict(c, q=q, k=k))
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert all(torch.equal(x, y) for x, y in zip(_backward(la, dict(c, q=q, k=k), want[2], want[3]),
                                                 _backward(la, c, want[2], want[3])))


def test_gradients_against_differences(la):
    c = _case(30, 3, 2, 24, (5, 4), "f32", seed=8)
    c["q"], c["k"] = c["q"] / 2, c["k"] / 2
    freq, pos = _np(c["freq"]), c["pos"].cpu().numpy()
    got = _backward(la, c, *_forward(la, c)[2:])
    rng = np.random.default_rng(1)
    for x, w, dy, dx, dw in (("q", "qw", "dq", got[0], got[2]), ("k", "kw", "dk", got[1], got[3])):
        xn, wn, dyn = _np(c[x]), _np(c[w]), _np(c[dy])
        loss = lambda a, b: (ops.qk_norm_rotary(a, b, freq, pos, c["pairs"])[0] * dyn).sum()   # noqa: E731
        r = ops.qk_norm_rotary(xn, wn, freq, pos, c["pairs"])[1]
        bx, bw = _backward_bounds(xn, r, dyn, wn, c["pairs"], False)
        # rstd itself is off by its own bound: three powers of it in dx, one in dw
        rel = 3 * ((_terms(24) + 2) / 2 + 4) * U
        way = rng.normal(size=xn.shape)
        slope = (loss(xn + 1e-6 * way, wn) - loss(xn - 1e-6 * way, wn)) / 2e-6
        size = r[..., None] * np.abs(dyn).max() * 12
        # the 64-bit rounding of two losses of about 2^12 over that step, and third derivatives of x / |x|
        assert abs((_np(dx) * way).sum() - slope) <= ((bx + rel * size + U * np.abs(_np(dx))) * np.abs(way)).sum() + 1e-5
        way = rng.normal(size=wn.shape)
        slope = (loss(xn, wn + 1e-3 * way) - loss(xn, wn - 1e-3 * way)) / 2e-3
        assert abs((_np(dw) * way).sum() - slope) <= ((bw + (rel + U) * np.abs(dyn).sum((0, 1)) * 12) * np.abs(way)).sum()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_layer_of_these_operators(la, dtype):
    """Projection -> norm and rotation of q and k -> decayed attention -> layer norm, and back, each call
    held to its own definition on what the one before it gave."""
    from decay_util import backward_bounds, forward_bounds
    T, H, d, pairs = 200, 2, 64, (32,)
    c = _case(T, H, H, d, pairs, dtype, fused=True, seed=9)
    g = torch.Generator().manual_seed(10)
    v = torch.randn(T, H, d, generator=g).to(TYPES[dtype]).cuda()
    ld = torch.tensor([-0.01, -0.3]).cuda()
    cu = torch.tensor([0, 70, T], dtype=torch.int32).cuda()
    spans = [(0, 70), (70, T)]
    qo, ko, qr, kr = _forward(la, c)
    out = la.la_decay_attention(qo, ko, v, ld, scale=0.125, cu_seqlens=cu)
    y, mean, rstd = la.la_layer_norm(out, return_stats=True)
    dout, _, _ = la.la_layer_norm_backward(out, c["dq"], mean, rstd)
    dq, dk, dv = la.la_decay_attention_backward(qo, ko, v, dout, ld, scale=0.125, cu_seqlens=cu)
    grads = la.la_qk_norm_rotary_backward(c["q"], c["k"], qr, kr, dq, dk, c["qw"], c["kw"], c["freq"], c["pos"], pairs)
    a = [_np(x) for x in (qo, ko, v)]
    ref, _ = ops.decay_attention(*a, _np(ld), 0.125, cu.cpu().numpy())
    check(_np(out), ref, forward_bounds(*a, _np(ld), 0.125, spans, None, dtype)[0], dtype, "out")
    refs = ops.decay_attention_backward(*a, _np(dout), _np(ld), 0.125, cu.cpu().numpy())
    for x, r, b in zip((dq, dk, dv), refs, backward_bounds(*a, _np(dout), _np(ld), 0.125, spans, None, None, dtype)):
        check(_np(x), r, b, dtype, "gradient")
    for x, w, r, dy, dx, dw in (("q", "qw", qr, dq, grads[0], grads[2]), ("k", "kw", kr, dk, grads[1], grads[3])):
        args = (_np(c[x]), _np(r), _np(dy), _np(c[w]))
        rdx, rdw = ops.qk_norm_rotary_backward(*args, _np(c["freq"]), c["pos"].cpu().numpy(), pairs)
        bx, bw = _backward_bounds(*args, pairs, False)
        check(_np(dx), rdx, bx, dtype, f"d{x}")
        check(_np(dw), rdw, bw, "f32", f"d{x}_weight")
