"""GPU parity of the operators around the attention call (gated linear recurrence, layer norm,
rotary positions) against the fp64 oracle; tolerances in layer_ops_util.py."""
import numpy as np
import pytest

import oracle
from layer_ops_util import (HALF, U, check, layer_norm_backward_bounds, layer_norm_bounds, rotary_bound, scan_bound)
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


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g).to(TYPES[dtype]).cuda()


def _off(t, by):
    """The same values in memory whose address is `by` elements off a 256-byte boundary."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    out = buf[by:].view(t.shape)
    out.copy_(t)
    return out


def _cu(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)


# --------------------------------------------------------------------------- gated linear recurrence

LENGTHS = [[1], [2, 1], [0, 0, 3, 0], [15, 16, 17, 0, 33], [127], [128], [129], [0, 128, 0, 128, 0], [1] * 300,
           [255, 257, 1, 640], [2500], [0, 0, 0]]


def _gates(g, shape, dtype):
    a = torch.sigmoid(2.0 + 1.5 * torch.randn(shape, generator=g))
    a[torch.rand(shape, generator=g) < 0.01] = 0.0      # forgets everything
    a[torch.rand(shape, generator=g) < 0.02] = 1.0      # forgets nothing
    a[torch.rand(shape, generator=g) < 0.02] *= -1.0
    return a.to(TYPES[dtype]).cuda()


def _scan_case(lengths, H, d, ta, tb, seed):
    g = torch.Generator().manual_seed(seed)
    T, n = sum(lengths), len(lengths)
    cu = _cu(lengths)
    return dict(a=_gates(g, (T, H, d), ta), b=_randn(g, (T, H, d), tb), dh=_randn(g, (T, H, d), tb),
                s=torch.randn(n, H, d, generator=g).cuda(), ds=torch.randn(n, H, d, generator=g).cuda(), cu=cu,
                cu_t=torch.from_numpy(cu).cuda(), spans=list(zip(cu[:-1].tolist(), cu[1:].tolist())))


def _check_scan(la, c, ta, tb, state, what="", **seqs):
    seqs = seqs or dict(cu_seqlens=c["cu_t"])
    s = c["s"] if state else None
    h, out = la.la_gated_scan(c["a"], c["b"], state_in=s, return_state=True, **seqs)
    sn = _np(c["s"]) if state else None
    ref, ref_out = ops.gated_scan(_np(c["a"]), _np(c["b"]), c["cu"], state_in=sn)
    E, edge = scan_bound(_np(c["a"]), _np(c["b"]), c["spans"], sn)
    check(_np(h), ref, E, tb, f"{what} h")
    check(_np(out), ref_out, edge, "f32", f"{what} state_out")
    return h, out


def _check_scan_backward(la, c, h, ta, tb, state, what="", **seqs):
    seqs = seqs or dict(cu_seqlens=c["cu_t"])
    s, ds = (c["s"], c["ds"]) if state else (None, None)
    da, db, dsi = la.la_gated_scan_backward(c["a"], h, c["dh"], state_in=s, dstate_out=ds, return_dstate=True, **seqs)
    sn, dsn = (_np(s), _np(ds)) if state else (None, None)
    ra, rb, rs = ops.gated_scan_backward(_np(c["a"]), _np(h), _np(c["dh"]), c["cu"], state_in=sn, dstate_out=dsn)
    E, edge = scan_bound(_np(c["a"]), _np(c["dh"]), c["spans"], dsn, reverse=True)
    before = np.zeros_like(rb)
    for i, (lo, hi) in enumerate(c["spans"]):
        if hi > lo:
            before[lo + 1:hi] = _np(h)[lo:hi - 1]
            before[lo] = sn[i] if state else 0.0
    check(_np(db), rb, E, tb, f"{what} db")
    check(_np(da), ra, np.abs(before) * (E + U * np.abs(rb)), ta, f"{what} da")
    check(_np(dsi), rs, edge, "f32", f"{what} dstate_in")
    return da, db, dsi


@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("ta,tb", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda l: "x".join(map(str, l[:5])))
def test_gated_scan_packed(la, lengths, ta, tb, state):
    c = _scan_case(lengths, 2, 40, ta, tb, 7)
    h, _ = _check_scan(la, c, ta, tb, state)
    _check_scan_backward(la, c, h, ta, tb, state)


@pytest.mark.parametrize("H,d", [(1, 1), (1, 2), (3, 21), (1, 63), (1, 64), (1, 65), (2, 64), (5, 37), (4, 80), (1, 1000)])
@pytest.mark.parametrize("ta,tb", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
def test_gated_scan_widths_and_alignment(la, H, d, ta, tb):
    c = _scan_case([200, 0, 301], H, d, ta, tb, 8)
    h, _ = _check_scan(la, c, ta, tb, True)
    _check_scan_backward(la, c, h, ta, tb, True)
    for by in (1, 2, 3):
        c2 = dict(c, a=_off(c["a"], by), b=_off(c["b"], by), dh=_off(c["dh"], by), s=_off(c["s"], by))
        out = _off(torch.zeros_like(c["b"]), by)
        assert torch.equal(la.la_gated_scan(c2["a"], c2["b"], cu_seqlens=c["cu_t"], state_in=c2["s"], h=out), h)
        da, db = la.la_gated_scan_backward(c["a"], h, c["dh"], cu_seqlens=c["cu_t"], state_in=c["s"])
        da2, db2 = la.la_gated_scan_backward(c2["a"], _off(h, by), c2["dh"], cu_seqlens=c["cu_t"], state_in=c2["s"],
                                             da=_off(torch.zeros_like(c["a"]), by),
                                             db=_off(torch.zeros_like(c["b"]), by))
        assert torch.equal(da, da2) and torch.equal(db, db2)


@pytest.mark.parametrize("nseq,length", [(1, 1), (1, 700), (3, 129), (5, 64), (40, 1), (4, 1000)])
def test_gated_scan_equal_lengths(la, nseq, length):
    c = _scan_case([length] * nseq, 2, 33, "f32", "bf16", 9)
    h, out = _check_scan(la, c, "f32", "bf16", True, nseq=nseq)
    packed = la.la_gated_scan(c["a"], c["b"], cu_seqlens=c["cu_t"], state_in=c["s"], return_state=True)
    assert torch.equal(h, packed[0]) and torch.equal(out, packed[1])
    _check_scan_backward(la, c, h, "f32", "bf16", True, nseq=nseq)


def test_gated_scan_long_sequence_with_gates_near_one(la):
    c = _scan_case([9000, 3, 7001], 1, 64, "f32", "f32", 10)
    c["a"] = 1.0 - 1e-4 * torch.rand(c["a"].shape, device="cuda")
    h, _ = _check_scan(la, c, "f32", "f32", True)
    _check_scan_backward(la, c, h, "f32", "f32", True)


@pytest.mark.parametrize("d", [64, 62, 63, 72])
@pytest.mark.parametrize("ta,tb", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
def test_gated_scan_states_that_cross_many_tiles(la, d, ta, tb):
    """Gates of 1 - 2^-7 and 1 - 2^-8 (exact in bf16) let a state reach over hundreds of tokens; the
    long sequences span several blocks of 64 tiles in every type and every kind of copy."""
    c = _scan_case([19000, 0, 5, 17003], 1, d, ta, tb, 20)
    g = torch.Generator().manual_seed(20)
    c["a"] = (1.0 - 2.0 ** -torch.randint(7, 9, c["a"].shape, generator=g).float()).to(TYPES[ta]).cuda()
    h, _ = _check_scan(la, c, ta, tb, True)
    _check_scan_backward(la, c, h, ta, tb, True)


def test_gated_scan_thousands_of_short_sequences(la):
    lengths = np.random.default_rng(21).integers(0, 4, 20000).tolist()
    for d, ta, tb in ((48, "f32", "bf16"), (33, "f32", "f32")):
        c = _scan_case(lengths, 1, d, ta, tb, 22)
        h, _ = _check_scan(la, c, ta, tb, True)
        _check_scan_backward(la, c, h, ta, tb, True)


def test_gated_scan_split_over_calls_and_steps(la):
    c = _scan_case([700], 2, 24, "f32", "f32", 11)
    whole, end = la.la_gated_scan(c["a"], c["b"], state_in=c["s"], return_state=True)
    parts, state = [], c["s"].clone()
    for lo, hi in ((0, 1), (1, 300), (300, 690)):
        parts.append(la.la_gated_scan(c["a"][lo:hi], c["b"][lo:hi], state_in=state, state_out=state))   # in place
    for t in range(690, 700):
        parts.append(la.la_gated_step(c["a"][t:t + 1], c["b"][t:t + 1], state))
    E, edge = scan_bound(_np(c["a"]), _np(c["b"]), c["spans"], _np(c["s"]))
    ref, ref_out = ops.gated_scan(_np(c["a"]), _np(c["b"]), c["cu"], state_in=_np(c["s"]))
    check(_np(torch.cat(parts)), ref, E, "f32", "h in parts")
    check(_np(state), ref_out, edge, "f32", "state in parts")
    check(_np(whole), ref, E, "f32", "h")


@pytest.mark.parametrize("lengths", [[60, 0, 2, 200, 1, 1, 300], [0] * 5 + [4] * 100])
def test_gated_scan_states_in_place(la, lengths):
    c = _scan_case(lengths, 2, 48, "f32", "bf16", 12)
    h, out = la.la_gated_scan(c["a"], c["b"], cu_seqlens=c["cu_t"], state_in=c["s"], return_state=True)
    st = c["s"].clone()
    h2 = la.la_gated_scan(c["a"], c["b"], cu_seqlens=c["cu_t"], state_in=st, state_out=st)
    assert torch.equal(h, h2) and torch.equal(out, st)
    _, _, dsi = la.la_gated_scan_backward(c["a"], h, c["dh"], cu_seqlens=c["cu_t"], state_in=c["s"],
                                          dstate_out=c["ds"], return_dstate=True)
    ds = c["ds"].clone()
    la.la_gated_scan_backward(c["a"], h, c["dh"], cu_seqlens=c["cu_t"], state_in=c["s"], dstate_out=ds, dstate_in=ds)
    assert torch.equal(dsi, ds)


def test_gated_scan_values_stay_in_their_sequence(la):
    lengths = [130, 1, 64, 400, 0, 90]
    c = _scan_case(lengths, 2, 32, "f32", "f32", 13)
    h = la.la_gated_scan(c["a"], c["b"], cu_seqlens=c["cu_t"], state_in=c["s"])
    da, db = la.la_gated_scan_backward(c["a"], h, c["dh"], cu_seqlens=c["cu_t"], state_in=c["s"], dstate_out=c["ds"])
    for poison in (float("nan"), float("inf")):
        for s in (0, 3):
            lo, hi = c["spans"][s]
            a, b, dh, st, ds, hp = (c[k].clone() for k in ("a", "b", "dh", "s", "ds")) and [
                c["a"].clone(), c["b"].clone(), c["dh"].clone(), c["s"].clone(), c["ds"].clone(), h.clone()]
            for x in (a, b, dh, hp):
                x[lo:hi] = poison
            st[s] = poison
            ds[s] = poison
            h2 = la.la_gated_scan(a, b, cu_seqlens=c["cu_t"], state_in=st)
            da2, db2 = la.la_gated_scan_backward(a, hp, dh, cu_seqlens=c["cu_t"], state_in=st, dstate_out=ds)
            for x, y in ((h, h2), (da, da2), (db, db2)):
                assert torch.equal(x[:lo], y[:lo]) and torch.equal(x[hi:], y[hi:])
                assert not torch.isfinite(y[lo:hi]).any()


def test_gated_scan_non_finite_values_follow_the_recurrence(la):
    c = _scan_case([300], 1, 8, "f32", "f32", 14)
    c["a"].abs_().clamp_(0.5, 1.0)
    c["b"][5, 0, 1] = float("inf")
    c["b"][150, 0, 2] = float("nan")
    c["b"][299, 0, 3] = -float("inf")
    with np.errstate(invalid="ignore"):
        h, _ = _check_scan(la, c, "f32", "f32", False)


def test_gated_scan_is_deterministic(la):
    c = _scan_case([5000, 3000], 3, 50, "f32", "bf16", 15)
    first = la.la_gated_scan(c["a"], c["b"], cu_seqlens=c["cu_t"], return_state=True)
    grads = la.la_gated_scan_backward(c["a"], first[0], c["dh"], cu_seqlens=c["cu_t"], return_dstate=True)
    for _ in range(5):
        again = la.la_gated_scan(c["a"], c["b"], cu_seqlens=c["cu_t"], return_state=True)
        grads2 = la.la_gated_scan_backward(c["a"], first[0], c["dh"], cu_seqlens=c["cu_t"], return_dstate=True)
        assert all(torch.equal(x, y) for x, y in zip(first + grads, again + grads2))


def test_gated_scan_writes_nothing_else_and_reports_malformed_boundaries(la):
    c = _scan_case([100, 200], 1, 16, "f32", "f32", 16)
    for cu in ([0, 200, 100, 300], [0, 100, 299], [1, 100, 300], [0, -5, 300], [0, 400, 300], [5, 5, 5]):
        ws = torch.full((la.la_gated_scan_workspace_bytes(True, len(cu) - 1, 300, 1, 16),), 255, dtype=torch.uint8,
                        device="cuda")
        h = torch.full_like(c["b"], 7.0)
        st = torch.full((len(cu) - 1, 1, 16), 3.0, device="cuda")
        la.la_gated_scan(c["a"], c["b"], cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), state_out=st, h=h,
                         workspace=ws)
        assert la.la_workspace_error(ws) == 1 and bool((h == 7.0).all()) and bool((st == 3.0).all())
        la.la_gated_scan(c["a"], c["b"], h=h, workspace=ws)     # the next call clears it
        assert la.la_workspace_error(ws) == 0
    # rows and states beside the outputs keep their values
    buf = torch.full((500, 1, 16), 9.0, device="cuda")
    la.la_gated_scan(c["a"], c["b"], cu_seqlens=c["cu_t"], h=buf[100:400])
    assert bool((buf[:100] == 9.0).all()) and bool((buf[400:] == 9.0).all())


def test_gated_scan_refuses(la):
    c = _scan_case([10], 1, 8, "f32", "f32", 17)
    a, b = c["a"], c["b"]
    for bad in (dict(h=a), dict(h=b), dict(state_out=torch.zeros(1, 1, 9, device="cuda")),
                dict(state_in=torch.zeros(1, 1, 8, dtype=torch.float64, device="cuda")),
                dict(cu_seqlens=torch.tensor([0, 10]).cuda()), dict(nseq=3),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((ValueError, la.LinAttnError)):
            la.la_gated_scan(a, b, **bad)
    for x, y in ((a.half(), b), (a, b.half()), (a[:, :, ::2], b[:, :, ::2]), (a[:5], b), (a.cpu(), b)):
        with pytest.raises(ValueError):
            la.la_gated_scan(x, y)


def test_gated_scan_offsets_beyond_32_bits(la):
    T, H, d = 70000, 16, 2048 + 64                        # 2.4 G elements per tensor
    a = torch.full((T, H, d), 0.5, dtype=torch.bfloat16, device="cuda")
    b = torch.ones((T, H, d), dtype=torch.bfloat16, device="cuda")
    b[T - 3:] = 3.0
    h, out = la.la_gated_scan(a, b, return_state=True)
    # 1, 1.5, 1.75, .. reaches 2 (the 30th term differs by 2^-29, less than half a step of bf16 and of fp32)
    assert bool((h[100:T - 3] == 2.0).all()) and bool((h[T - 3:, 5, 7] == torch.tensor([4.0, 5.0, 5.5]).cuda()).all())
    assert bool((out == 5.5).all())
    da, db = la.la_gated_scan_backward(a, h, b)
    assert bool((db[T - 3:, 3, 9] == torch.tensor([5.25, 4.5, 3.0]).cuda()).all())
    assert bool((db[:T - 100] == 2.0).all()) and bool((da[200:T - 100] == 4.0).all())
    del a, b, h, da, db
    torch.cuda.empty_cache()


@pytest.mark.parametrize("ta,tb", [("f32", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("B,H,d", [(1, 1, 1), (3, 16, 64), (7, 5, 37), (256, 2, 130)])
def test_gated_step(la, B, H, d, ta, tb):
    c = _scan_case([1] * B, H, d, ta, tb, 18)
    ref, _ = ops.gated_scan(_np(c["a"]), _np(c["b"]), None, B, _np(c["s"]))
    bound = 2 * U * (np.abs(_np(c["a"]) * _np(c["s"])) + np.abs(_np(c["b"])))
    out = torch.empty_like(c["s"])
    keep = c["s"].clone()
    h = la.la_gated_step(c["a"], c["b"], c["s"], state_out=out)
    assert torch.equal(c["s"], keep)
    check(_np(h), ref, bound, tb, "h")
    check(_np(out), ref, bound, "f32", "state")
    # the scan over one token each is the same arithmetic
    h2, out2 = la.la_gated_scan(c["a"], c["b"], nseq=B, state_in=c["s"], return_state=True)
    assert torch.equal(h, h2) and torch.equal(out, out2)
    o = _off(torch.zeros_like(c["b"]), 1)
    h3 = la.la_gated_step(_off(c["a"], 1), _off(c["b"], 1), c["s"], h=o)        # in place, unaligned
    assert torch.equal(h, h3) and torch.equal(c["s"], out)


# --------------------------------------------------------------------------- layer norm

NORM_SHAPES = [((1, 1), 1), ((3, 2), 1), ((5,), 2), ((7, 3), 37), ((2, 5, 3), 64), ((33, 4), 64), ((9, 2), 65),
               ((130, 3), 128), ((4, 3), 200), ((17, 2), 256), ((40,), 768), ((9,), 1023), ((6, 1), 1024), ((5,), 2048),
               ((3,), 4100), ((2,), 8192), ((3,), 10001), ((2, 2), 16384)]


def _norm_inputs(lead, d, dtype, seed, per_head, scale=1.0, shift=0.5):
    g = torch.Generator().manual_seed(seed)
    x = ((torch.randn(*lead, d, generator=g) + shift) * torch.exp(torch.randn(*lead, 1, generator=g)) * scale)
    shape = (lead[-1], d) if per_head else (d,)
    w, b = 1.0 + 0.3 * torch.randn(shape, generator=g), torch.randn(shape, generator=g)
    dy = torch.randn(*lead, d, generator=g)
    return x.to(TYPES[dtype]).cuda(), w.cuda(), b.cuda(), dy.to(TYPES[dtype]).cuda()


def _check_norm(la, x, w, b, dy, dtype, eps=1e-5, what=""):
    y, mean, rstd = la.la_layer_norm(x, w, b, eps=eps, return_stats=True)
    wn, bn = (None if t is None else _np(t) for t in (w, b))
    ref, rm, rr = ops.layer_norm(_np(x), wn, bn, eps)
    by, bm, br = layer_norm_bounds(_np(x), wn, bn, rm, rr, eps)
    check(_np(y), ref, by, dtype, f"{what} y")
    check(_np(mean), rm, bm, "f32", f"{what} mean")
    check(_np(rstd), rr, br, "f32", f"{what} rstd")
    assert torch.equal(y, la.la_layer_norm(x, w, b, eps=eps))
    if w is None:
        return
    dx, dw, db = la.la_layer_norm_backward(x, dy, mean, rstd, w)
    ra, rw, rb = ops.layer_norm_backward(_np(x), _np(dy), _np(mean), _np(rstd), wn)
    rows = x.numel() // w.numel()
    ba, bw, bb = layer_norm_backward_bounds(_np(x), _np(dy), _np(mean), _np(rstd), wn, min(rows, 256))
    check(_np(dx), ra, ba, dtype, f"{what} dx")
    check(_np(dw), rw, bw, "f32", f"{what} dweight")
    check(_np(db), rb, bb, "f32", f"{what} dbias")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lead,d", NORM_SHAPES, ids=str)
def test_layer_norm_shapes(la, lead, d, dtype):
    _check_norm(la, *_norm_inputs(lead, d, dtype, 21, False), dtype)
    if len(lead) > 1:
        _check_norm(la, *_norm_inputs(lead, d, dtype, 22, True), dtype, what="per head")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,H,d", [(3000, 5, 64), (6001, 1, 128), (1500, 3, 48), (700, 16, 96), (1, 16, 64), (5003, 2, 7),
                                      (900, 1, 2000), (40, 3, 5000)])
def test_layer_norm_many_rows(la, rows, H, d, dtype):
    _check_norm(la, *_norm_inputs((rows, H), d, dtype, 23, True), dtype, what="per head")
    _check_norm(la, *_norm_inputs((rows, H), d, dtype, 24, False), dtype, what="shared")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 300, 4096])
def test_layer_norm_without_weights_large_means_and_scales(la, d, dtype):
    x, w, b, dy = _norm_inputs((20, 2), d, dtype, 25, False)
    _check_norm(la, x, None, None, dy, dtype)
    _check_norm(la, x, None, b, dy, dtype)
    _check_norm(la, x, w, None, dy, dtype)
    _check_norm(la, *_norm_inputs((20, 2), d, dtype, 26, True, shift=300.0), dtype, what="large mean")
    _check_norm(la, *_norm_inputs((20, 2), d, dtype, 27, True, scale=1e12), dtype, what="large")
    _check_norm(la, *_norm_inputs((20, 2), d, dtype, 28, True, scale=1e-12), dtype, what="small")


@pytest.mark.parametrize("d", [1, 64, 1000])
def test_layer_norm_constant_and_non_finite_rows(la, d):
    x, w, b, dy = _norm_inputs((6, 2), d, "f32", 29, True)
    x[1] = 4.0                     # no variance: rstd = 1 / sqrt(eps)
    x[2] = 0.0
    _check_norm(la, x, w, b, dy, "f32")
    base, mean, rstd = la.la_layer_norm(x, w, b, return_stats=True)
    dx = la.la_layer_norm_backward(x, dy, mean, rstd, w)[0]
    for bad in (float("nan"), float("inf")):
        xb = x.clone()
        xb[3, 0, d // 2] = bad
        y, mean, rstd = la.la_layer_norm(xb, w, b, return_stats=True)
        assert not torch.isfinite(y[3, 0]).any()
        dxb = la.la_layer_norm_backward(xb, dy, mean, rstd, w)[0]
        assert not torch.isfinite(dxb[3, 0]).any()
        keep = torch.ones(6, 2, dtype=torch.bool)
        keep[3, 0] = False          # every other row as before
        assert torch.equal(y[keep], base[keep]) and torch.equal(dxb[keep], dx[keep])
    y = la.la_layer_norm(x, w, b, eps=0.0)
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()    # 0 / 0, as the formula has it


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 80, 1024])
def test_layer_norm_alignment_and_neighbours(la, d, dtype):
    x, w, b, dy = _norm_inputs((50, 2), d, dtype, 30, True)
    y, mean, rstd = la.la_layer_norm(x, w, b, return_stats=True)
    grads = la.la_layer_norm_backward(x, dy, mean, rstd, w)
    for by in (1, 2, 3):
        buf = torch.full((x.numel() + 64,), 5.0, dtype=x.dtype, device="cuda")
        out = buf[by:by + x.numel()].view(x.shape)
        y2 = la.la_layer_norm(_off(x, by), _off(w, by), _off(b, by), y=out)
        assert bool((buf[:by] == 5.0).all()) and bool((buf[by + x.numel():] == 5.0).all())
        g2 = la.la_layer_norm_backward(_off(x, by), _off(dy, by), _off(mean, by), _off(rstd, by), _off(w, by),
                                       dx=_off(torch.zeros_like(x), by))
        # sums may be grouped in another order: both within their bounds of the exact values
        ref, rm, rr = ops.layer_norm(_np(x), _np(w), _np(b), 1e-5)
        check(_np(y2), ref, layer_norm_bounds(_np(x), _np(w), _np(b), rm, rr, 1e-5)[0], dtype, "y")
        refs = ops.layer_norm_backward(_np(x), _np(dy), _np(mean), _np(rstd), _np(w))
        bounds = layer_norm_backward_bounds(_np(x), _np(dy), _np(mean), _np(rstd), _np(w), 50)
        for g, r, bd, t in zip(g2, refs, bounds, (dtype, "f32", "f32")):
            check(_np(g), r, bd, t, "gradient")
    again = la.la_layer_norm_backward(x, dy, mean, rstd, w)
    assert all(torch.equal(p, q) for p, q in zip(grads, again))


def test_layer_norm_no_rows_and_missing_gradients(la):
    x = torch.empty(0, 2, 64, device="cuda")
    w = torch.ones(2, 64, device="cuda")
    st = torch.empty(0, 2, device="cuda")
    assert la.la_layer_norm(x, w, w).shape == (0, 2, 64)
    dx, dw, db = la.la_layer_norm_backward(x, x, st, st, w)
    assert bool((dw == 0).all()) and bool((db == 0).all())
    # through the C entry point: either gradient may be left out
    x, w, b, dy = _norm_inputs((30, 2), 64, "f32", 31, True)
    y, mean, rstd = la.la_layer_norm(x, w, b, return_stats=True)
    full = la.la_layer_norm_backward(x, dy, mean, rstd, w)
    lib = la.load_library()
    ws = torch.empty(la.la_layer_norm_backward_workspace_bytes(torch.float32, 60, 2, 64), dtype=torch.uint8, device="cuda")
    for keep in ((True, False), (False, True), (False, False)):
        dx, dw, db = (torch.full_like(t, 3.0) for t in (x, w, w))
        assert lib.la_layer_norm_backward(x.data_ptr(), dy.data_ptr(), w.data_ptr(), mean.data_ptr(), rstd.data_ptr(), 0,
                                          60, 2, 64, dx.data_ptr(), dw.data_ptr() if keep[0] else None,
                                          db.data_ptr() if keep[1] else None, ws.data_ptr(), ws.numel(),
                                          torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(dx, full[0])
        assert torch.equal(dw, full[1]) if keep[0] else bool((dw == 3.0).all())
        assert torch.equal(db, full[2]) if keep[1] else bool((db == 3.0).all())


@pytest.mark.parametrize("kinds", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")], ids=str)
@pytest.mark.parametrize("T,C", [(129, 1), (257, 63), (1000, 65), (2049, 191), (777, 1001)])
def test_gated_scan_odd_rows_among_neighbours(la, T, C, kinds):
    # rows that start inside four bytes, read by whole words, against the same rows read one by one
    # (arrays that start inside four bytes): the same results, whatever lies before and after
    g = torch.Generator().manual_seed(T + C)
    ta, tb = (torch.float32 if k == "f32" else torch.bfloat16 for k in kinds)
    vals = dict(a=torch.rand(T, 1, C, generator=g).to(ta), b=torch.randn(T, 1, C, generator=g).to(tb),
                dh=torch.randn(T, 1, C, generator=g).to(tb))
    cu = torch.tensor([0, T // 3, T // 3, T - 5, T], dtype=torch.int32, device="cuda")
    state = torch.randn(4, 1, C, generator=g).cuda()

    def at(t, by):
        buf = torch.full((t.numel() + 64,), float("nan"), dtype=t.dtype, device="cuda")
        buf[by:by + t.numel()] = t.reshape(-1).cuda()
        return buf[by:by + t.numel()].view(t.shape)

    got = []
    for by in (32, 33):
        a, b, dh = (at(vals[k], by) for k in ("a", "b", "dh"))
        h, out = la.la_gated_scan(a, b, cu, state_in=state, return_state=True)
        got.append((h, out) + la.la_gated_scan_backward(a, at(h, by), dh, cu, state_in=state, dstate_out=state,
                                                       return_dstate=True))
    for x, y in zip(*got):
        assert bool(torch.isfinite(x).all()) and torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,H,d", [(9, 1, 1), (40, 3, 5), (37, 2, 7), (300, 7, 33), (77, 5, 129), (31, 1, 515), (19, 3, 1030),
                                      (401, 1, 2051), (6, 2, 4097), (3, 1, 9001), (2, 1, 16383)])
def test_layer_norm_rows_that_start_anywhere(la, rows, H, d, dtype):
    # arrays on 16 bytes whose rows are not, among neighbours that keep their values
    x, w, b, dy = _norm_inputs((rows, H), d, dtype, 33, True)
    n, pad = x.numel(), 64
    ref, rm, rr = ops.layer_norm(_np(x), _np(w), _np(b), 1e-5)

    def among(t):
        buf = torch.full((n + 2 * pad,), float("nan"), dtype=t.dtype, device="cuda")
        buf[pad:pad + n] = t.reshape(-1)
        return buf, buf[pad:pad + n].view(t.shape)

    (_, xs), (_, dys), (yb, y), (gb, dx) = among(x), among(dy), among(x), among(x)
    _, mean, rstd = la.la_layer_norm(xs, w, b, return_stats=True, y=y)
    check(_np(y), ref, layer_norm_bounds(_np(x), _np(w), _np(b), rm, rr, 1e-5)[0], dtype, "y")
    grads = la.la_layer_norm_backward(xs, dys, mean, rstd, w, dx=dx)
    refs = ops.layer_norm_backward(_np(x), _np(dy), _np(mean), _np(rstd), _np(w))
    bounds = layer_norm_backward_bounds(_np(x), _np(dy), _np(mean), _np(rstd), _np(w), min(rows, 256))
    for g, r, bd, t in zip(grads, refs, bounds, (dtype, "f32", "f32")):
        check(_np(g), r, bd, t, "gradient")
    for buf in (yb, gb):
        assert bool(torch.isnan(buf[:pad]).all()) and bool(torch.isnan(buf[pad + n:]).all())


def test_layer_norm_large_constant_rows_of_odd_length(la):
    # deviations are zero although the mean times rstd is beyond fp32
    x = torch.full((24, 77), 1e36, device="cuda")
    w, b = torch.ones(77, device="cuda"), torch.full((77,), 0.5, device="cuda")
    y, mean, rstd = la.la_layer_norm(x, w, b, eps=1e-12, return_stats=True)
    assert bool((y == 0.5).all()) and bool((mean == x[0, 0]).all())
    dx, dw, db = la.la_layer_norm_backward(x, torch.ones_like(x), mean, rstd, w)
    assert bool((dw == 0.0).all()) and bool((db == 24.0).all()) and bool(torch.isfinite(dx).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layer_norm_gradients_without_a_weight(la, dtype):
    x, w, b, dy = _norm_inputs((30, 2), 64, dtype, 31, True)
    _, mean, rstd = la.la_layer_norm(x, return_stats=True)
    full = la.la_layer_norm_backward(x, dy, mean, rstd, torch.ones_like(w))    # a product with 1 is exact
    dx, dw, db = la.la_layer_norm_backward(x, dy, mean, rstd)
    # rows are given out by the groups of the weight, which change no row's own sums
    assert dw is None and db is None and torch.equal(dx, full[0])
    dx, dw, db = la.la_layer_norm_backward(x, dy, mean, rstd, dbias=torch.full_like(b, 9.0))
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), full))
    with pytest.raises(ValueError):
        la.la_layer_norm_backward(x, dy, mean, rstd, dweight=torch.empty(3, 64, device="cuda"))


def test_layer_norm_refuses(la):
    x, w, b, dy = _norm_inputs((6, 2), 64, "bf16", 32, True)
    y, mean, rstd = la.la_layer_norm(x, w, b, return_stats=True)
    for bad in (dict(weight=w[:, :32].contiguous()), dict(weight=w.bfloat16()), dict(weight=w[0], bias=b), dict(eps=-1.0),
                dict(y=x), dict(weight=w.t()), dict(weight=torch.ones(3, 64, device="cuda"))):
        with pytest.raises((ValueError, la.LinAttnError)):
            la.la_layer_norm(x, **bad)
    for bad in ((x, dy.float(), mean, rstd, w), (x, dy, mean[:, 0].contiguous(), rstd, w), (x, dy[1:], mean, rstd, w)):
        with pytest.raises(ValueError):
            la.la_layer_norm_backward(*bad)
    with pytest.raises(la.LinAttnError):
        la.la_layer_norm(torch.zeros(2, 16385, device="cuda"))


# --------------------------------------------------------------------------- rotary positions

ROTARY = [(1, 1, 2, (1,)), (5, 2, 3, (1,)), (7, 3, 64, (32,)), (33, 4, 64, (8, 12, 12)), (9, 2, 64, (16, 0, 8)),
          (300, 16, 64, (8, 12, 12)), (10, 5, 83, (20, 19)), (6, 1, 128, (1, 2, 3, 4)), (12, 3, 80, (24,)), (4, 2, 1024, (512,)),
          (3, 70, 6, (1, 1)), (65, 1, 96, (16, 16))]


def _rotary_inputs(T, H, d, pairs, dtype, seed, far=1000):
    g = torch.Generator().manual_seed(seed)
    q, k = _randn(g, (T, H, d), dtype), _randn(g, (T, H, d), dtype)
    freq = torch.cat([10000.0 ** (-torch.arange(p, dtype=torch.float64) / max(p, 1)) for p in pairs]).float().cuda()
    pos = torch.randint(-far, far, (T, len(pairs)), generator=g).to(torch.int32).cuda()
    return q, k, freq, pos


def _check_rotary(la, q, k, freq, pos, pairs, interleaved, inverse, dtype, extra=0.0):
    out = la.la_rotary(q, k, freq, pos, pairs, interleaved=interleaved, inverse=inverse)
    for x, y in zip((q, k), out):
        ref = ops.rotary(_np(x), _np(freq), _np(pos), pairs, interleaved, inverse)
        bound = rotary_bound(_np(x), pairs, interleaved)
        check(_np(y), ref, bound * (1 + extra / (8 * U)), dtype, "rotary")
        P = sum(pairs)
        assert torch.equal(x[..., 2 * P:], y[..., 2 * P:])
    return out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,d,pairs", [(1, 1, 3, (1,)), (2501, 9, 77, (20, 18)), (1003, 8, 128, (20, 23)), (333, 1, 255, (127,)),
                                         (4099, 3, 7, (1, 0, 1)), (61, 25, 201, (50,)), (19, 301, 5, (2,))])
def test_rotary_rows_of_any_length_among_neighbours(la, T, H, d, pairs, interleaved, dtype):
    q, k, freq, pos = _rotary_inputs(T, H, d, pairs, dtype, 71)
    n, pad = q.numel(), 64

    def among(t, by):
        buf = torch.full((n + 2 * pad,), float("nan"), dtype=t.dtype, device="cuda")
        buf[by:by + n] = t.reshape(-1)
        return buf, buf[by:by + n].view(t.shape)

    (qb, q1), (kb, k1) = among(q, pad), among(k, pad)
    ref_q, ref_k = (ops.rotary(_np(x), _np(freq), _np(pos), pairs, interleaved, False) for x in (q, k))
    la.la_rotary(q1, k1, freq, pos, pairs, interleaved=interleaved, q_out=q1, k_out=k1)      # in place
    check(_np(q1), ref_q, rotary_bound(_np(q), pairs, interleaved), dtype, "q")
    check(_np(k1), ref_k, rotary_bound(_np(k), pairs, interleaved), dtype, "k")
    for buf in (qb, kb):
        assert bool(torch.isnan(buf[:pad]).all()) and bool(torch.isnan(buf[pad + n:]).all())
    # arrays that do not start on 16 bytes, and q alone, turn alike
    (_, q2), (_, k2) = among(q, pad + 1), among(k, pad + 1)
    o2 = la.la_rotary(q2, k2, freq, pos, pairs, interleaved=interleaved)
    assert torch.equal(o2[0], q1) and torch.equal(o2[1], k1)
    assert torch.equal(la.la_rotary(q, None, freq, pos, pairs, interleaved=interleaved), q1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,d,pairs", ROTARY, ids=str)
def test_rotary(la, T, H, d, pairs, interleaved, dtype):
    q, k, freq, pos = _rotary_inputs(T, H, d, pairs, dtype, 41)
    out = _check_rotary(la, q, k, freq, pos, pairs, interleaved, False, dtype)
    _check_rotary(la, q, k, freq, pos, pairs, interleaved, True, dtype)
    assert torch.equal(la.la_rotary(q, None, freq, pos, pairs, interleaved=interleaved), out[0])
    q2, k2 = q.clone(), k.clone()
    la.la_rotary(q2, k2, freq, pos, pairs, interleaved=interleaved, q_out=q2, k_out=k2)         # in place
    assert torch.equal(q2, out[0]) and torch.equal(k2, out[1])
    q3 = q.clone()
    mixed = la.la_rotary(q3, k, freq, pos, pairs, interleaved=interleaved, q_out=q3)            # q alone in place
    assert torch.equal(q3, out[0]) and torch.equal(mixed[1], out[1])
    for by in (1, 2, 3):
        un = la.la_rotary(_off(q, by), _off(k, by), _off(freq, by), _off(pos, by), pairs, interleaved=interleaved,
                          q_out=_off(torch.zeros_like(q), by))
        assert torch.equal(un[0], out[0]) and torch.equal(un[1], out[1])


def test_rotary_far_positions_and_odd_frequencies(la):
    T, H, d, pairs = 64, 2, 16, (8,)
    q, k, freq, pos = _rotary_inputs(T, H, d, pairs, "f32", 42)
    pos[:, 0] = torch.tensor([0, 1, -1, 2 ** 20, 2 ** 27, -2 ** 27 - 3] + [2 ** 28 - 1 - 7 * i for i in range(58)])
    _check_rotary(la, q, k, freq, pos, pairs, False, False, "f32")
    freq[:] = torch.tensor([-1.0, 1e-8, 3.14159274, 6.28318548, 100.5, 0.0, -0.3, 1e-3])
    pos.remainder_(1 << 20)         # 100.5 radians at 2^20: below 2^25 turns
    _check_rotary(la, q, k, freq, pos, pairs, True, False, "f32")
    # the ends of the position's range: the fixed-point fraction of a turn is off by 2^-54 of a turn a position
    freq[:] = torch.rand(8)
    pos[:, 0] = torch.tensor([2 ** 31 - 1, -2 ** 31] * 32)
    # and the oracle's own fp64 product by half a step of an angle of 2^31 (2^-22 radians)
    _check_rotary(la, q, k, freq, pos, pairs, False, False, "f32", extra=2 ** -22 + 2 * np.pi * 2 ** -23)


def test_rotary_zero_positions_are_exact_and_bad_frequencies_are_nan(la):
    q, k, freq, pos = _rotary_inputs(40, 3, 64, (16, 16), "bf16", 43)
    pos.zero_()
    for il in (False, True):
        out = la.la_rotary(q, k, freq, pos, (16, 16), interleaved=il)
        assert torch.equal(out[0], q) and torch.equal(out[1], k)
    freq[3], freq[20] = float("nan"), float("inf")
    y = la.la_rotary(q, None, freq, pos, (16, 16))
    bad = torch.zeros(64, dtype=torch.bool)
    bad[[3, 35, 20, 52]] = True
    assert torch.isnan(y[..., bad.cuda()]).all() and torch.equal(y[..., ~bad.cuda()], q[..., ~bad.cuda()])


def test_rotary_turning_back_is_its_gradient(la):
    q, k, freq, pos = _rotary_inputs(30, 2, 24, (5, 6), "f32", 44)
    w = torch.randn_like(q)
    y = la.la_rotary(q, None, freq, pos, (5, 6))
    dq = la.la_rotary(w, None, freq, pos, (5, 6), inverse=True)
    # <w, R q> = <R^T w, q>: both sums in fp64 of fp32 values within 8 u (|x0| + |x1|)
    lhs, rhs = (w.double() * y.double()).sum().item(), (dq.double() * q.double()).sum().item()
    bound = (rotary_bound(_np(q), (5, 6), False) * np.abs(_np(w))).sum() + \
            (rotary_bound(_np(w), (5, 6), False) * np.abs(_np(q))).sum() + \
            HALF["f32"] * (np.abs(_np(y) * _np(w)).sum() + np.abs(_np(dq) * _np(q)).sum())
    assert abs(lhs - rhs) <= bound


def test_rotary_refuses(la):
    q, k, freq, pos = _rotary_inputs(10, 2, 16, (4, 4), "f32", 45)
    for bad in (dict(pairs=(4, 5)), dict(pairs=(8,)), dict(positions=pos.long()), dict(freq=freq.double()),
                dict(k=k.bfloat16()), dict(k=k[:5]), dict(q_out=k), dict(positions=pos[:5]), dict(k=None, k_out=k.clone()),
                dict(q_out=q.view(10, 16, 2)), dict(freq=freq.cpu())):
        kw = dict(q=q, k=k, freq=freq, positions=pos, pairs=(4, 4))
        kw.update(bad)
        with pytest.raises((ValueError, la.LinAttnError)):
            la.la_rotary(**kw)


# --------------------------------------------------------------------------- graphs and streams

@pytest.mark.parametrize("d", [1024, 1001])
def test_layer_norm_offsets_beyond_32_bits(la, d):
    # 64 rows over and over: rows that many apart start at the same place in their 16 bytes, so they give the same bits
    n = (1 << 31) // (64 * d) + 200
    x, w, b, dy = _norm_inputs((64,), d, "bf16", 81, False)
    small, mean, rstd = la.la_layer_norm(x, w, b, return_stats=True)
    dsmall = la.la_layer_norm_backward(x, dy, mean, rstd, w)[0]
    big = x.repeat(n, 1)
    y, mean, rstd = la.la_layer_norm(big, w, b, return_stats=True)
    assert bool((y.view(n, 64, d) == small).all())
    del y
    assert bool((la.la_layer_norm_backward(big, dy.repeat(n, 1), mean, rstd, w)[0].view(n, 64, d) == dsmall).all())
    del big
    torch.cuda.empty_cache()


@pytest.mark.parametrize("H,d,pairs", [(16, 64, (20, 12)), (8, 77, (38,)), (64, 877, (400,))])
def test_rotary_offsets_beyond_32_bits(la, H, d, pairs):
    n = (1 << 31) // (64 * H * d) + 20
    q, _, freq, pos = _rotary_inputs(64, H, d, pairs, "bf16", 82)
    small = la.la_rotary(q, None, freq, pos, pairs)
    big = q.repeat(n, 1, 1)
    la.la_rotary(big, None, freq, pos.repeat(n, 1), pairs, q_out=big)
    assert bool((big.view(n, 64, H, d) == small).all())
    del big
    torch.cuda.empty_cache()


def test_gated_scan_odd_rows_beyond_32_bits(la):
    T, d = 64000, 33793                                   # 2.2 G elements per tensor
    a = torch.full((T, 1, d), 0.5, dtype=torch.bfloat16, device="cuda")
    b = torch.ones((T, 1, d), dtype=torch.bfloat16, device="cuda")
    b[T - 3:] = 3.0
    h, out = la.la_gated_scan(a, b, return_state=True)
    assert bool((h[100:T - 3] == 2.0).all()) and bool((out == 5.5).all())
    assert bool((h[T - 3:, 0] == torch.tensor([[4.0], [5.0], [5.5]], device="cuda")).all())
    da, db = la.la_gated_scan_backward(a, h, b)
    assert bool((db[T - 3:, 0] == torch.tensor([[5.25], [4.5], [3.0]], device="cuda")).all())
    assert bool((db[:T - 100] == 2.0).all()) and bool((da[200:T - 100] == 4.0).all())
    del a, b, h, da, db
    torch.cuda.empty_cache()


def test_captured_calls_replay_on_new_inputs(la):
    c = _scan_case([900, 0, 333], 2, 64, "f32", "bf16", 51)
    q, k, freq, pos = _rotary_inputs(200, 2, 64, (8, 12, 12), "bf16", 52)
    w, bias = torch.ones(2, 64, device="cuda"), torch.zeros(2, 64, device="cuda")

    def calls():
        h, st = la.la_gated_scan(c["a"], c["b"], cu_seqlens=c["cu_t"], state_in=c["s"], return_state=True)
        g = la.la_gated_scan_backward(c["a"], h, c["dh"], cu_seqlens=c["cu_t"], state_in=c["s"], dstate_out=c["ds"],
                                      return_dstate=True)
        y, mean, rstd = la.la_layer_norm(h, w, bias, return_stats=True)
        n = la.la_layer_norm_backward(h, c["dh"], mean, rstd, w)
        s1 = torch.empty_like(c["s"])
        hs = la.la_gated_step(c["a"][:3], c["b"][:3], c["s"], state_out=s1)
        return (h, st, *g, y, mean, rstd, *n, hs, s1, *la.la_rotary(q, k, freq, pos, (8, 12, 12)))

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls()
    for seed in (53, 54):
        n = _scan_case([900, 0, 333], 2, 64, "f32", "bf16", seed)
        for key in ("a", "b", "dh", "s", "ds"):
            c[key].copy_(n[key])
        q.normal_()
        pos.add_(17)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        assert all(torch.equal(x, y) for x, y in zip(got, calls()))


def test_calls_on_two_streams_at_once(la):
    cases = [_scan_case([20000 + 100 * i], 4, 64, "f32", "bf16", 60 + i) for i in range(2)]
    want = [la.la_gated_scan(c["a"], c["b"], return_state=True) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(10):
        got = [la.la_gated_scan(c["a"], c["b"], return_state=True, stream=s) for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])
    # a raw handle and the default stream's zero
    h = la.la_gated_scan(cases[0]["a"], cases[0]["b"], stream=streams[0].cuda_stream)
    h0 = la.la_gated_scan(cases[0]["a"], cases[0]["b"], stream=0)
    torch.cuda.synchronize()
    assert torch.equal(h, want[0][0]) and torch.equal(h0, want[0][0])


# --------------------------------------------------------------------------- a layer of them

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_linear_attention_layer_forward_and_backward(la, dtype):
    """Gated values, rotated q and k, unnormalised causal attention over the identity map, a norm
    per head; and back through every one of them.  Each stage is held against the oracle on the
    stage's own inputs, so that every tolerance is that stage's."""
    lengths, H, d, pairs = [70, 1, 0, 200], 2, 64, (8, 12, 12)
    c = _scan_case(lengths, H, d, "f32", dtype, 71)
    T = sum(lengths)
    q, k, freq, pos = _rotary_inputs(T, H, d, pairs, dtype, 72)
    w, bias = 1 + 0.1 * torch.randn(H, d, device="cuda"), 0.1 * torch.randn(H, d, device="cuda")
    cu = c["cu_t"]
    v, _ = _check_scan(la, c, "f32", dtype, False)
    qr, kr = _check_rotary(la, q, k, freq, pos, pairs, False, False, dtype)
    out = la.la_forward(qr, kr, v, "identity", causal=True, norm="none", cu_seqlens=cu)
    ref = oracle.forward(_np(qr), _np(kr), _np(v), "identity", True, cu_seqlens=c["cu"], norm="none")
    rms = np.sqrt((ref ** 2).mean(-1, keepdims=True))
    assert (np.abs(_np(out) - ref) <= (1e-4 if dtype == "f32" else 2e-2) * rms + HALF[dtype] * np.abs(ref)).all()
    y, mean, rstd = la.la_layer_norm(out, w, bias, return_stats=True)
    _check_norm(la, out, w, bias, c["dh"], dtype)
    dout, dw, db = la.la_layer_norm_backward(out, c["dh"], mean, rstd, w)
    dq, dk, dv = la.la_backward(qr, kr, v, dout, "identity", causal=True, norm="none", cu_seqlens=cu)
    refs = oracle.backward(_np(qr), _np(kr), _np(v), _np(dout), "identity", True, cu_seqlens=c["cu"], norm="none")
    for g, r in zip((dq, dk, dv), refs):
        rms = np.sqrt((r ** 2).mean())
        assert (np.abs(_np(g) - r) <= (1e-4 if dtype == "f32" else 2e-2) * np.maximum(np.abs(r), rms)).all()
    _check_rotary(la, dq, dk, freq, pos, pairs, False, True, dtype)
    c["dh"] = dv
    _check_scan_backward(la, c, v, "f32", dtype, False)


def test_one_token_at_a_time_equals_the_whole_sequence(la):
    """Serving: rotary, gated step, decode step and norm for every token, against the same layer
    over the whole sequence."""
    T, H, d, pairs = 20, 2, 64, (32,)
    c = _scan_case([T], H, d, "f32", "f32", 73)
    q, k, freq, pos = _rotary_inputs(T, H, d, pairs, "f32", 74)
    pos[:, 0] = torch.arange(T)
    w = torch.ones(H, d, device="cuda")
    v = la.la_gated_scan(c["a"], c["b"])
    qr, kr = la.la_rotary(q, k, freq, pos, pairs)
    y = la.la_layer_norm(la.la_forward(qr, kr, v, "elu1", causal=True), w)
    state, memory = torch.zeros(1, H, d, device="cuda"), torch.zeros(1, H, d, d + 1, device="cuda")
    for t in range(T):
        vt = la.la_gated_step(c["a"][t:t + 1], c["b"][t:t + 1], state)
        qt, kt = la.la_rotary(q[t:t + 1], k[t:t + 1], freq, pos[t:t + 1], pairs)
        assert torch.equal(qt[0], qr[t]) and torch.equal(kt[0], kr[t])
        yt = la.la_layer_norm(la.la_decode_step(qt, kt, vt, memory, "elu1"), w)
        # the attention output within 1e-4 of its row's size on both sides, which the norm scales to one
        assert (yt[0] - y[t]).abs().max().item() <= 4e-4 * max(1.0, y[t].abs().max().item())


def test_gated_scan_wait_that_runs_out_is_reported(la):
    """The hook makes every tile's look back wait 1 ms for a state that nothing publishes: the call
    ends, reports it, and the next one is whole again."""
    c = _scan_case([700], 1, 64, "f32", "f32", 19)
    nb = la.la_gated_scan_workspace_bytes(False, 1, 700, 1, 64)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    la.la_test_force_wait_timeout(True)
    try:
        la.la_gated_scan(c["a"], c["b"], workspace=ws)
        code = la.la_workspace_error(ws)
        la.la_gated_scan_backward(c["a"], c["b"], c["dh"], workspace=ws)
        code_b = la.la_workspace_error(ws)
    finally:
        la.la_test_force_wait_timeout(False)
    assert (code, code_b) == (2, 2)
    h, _ = _check_scan(la, c, "f32", "f32", True)
    _check_scan_backward(la, c, h, "f32", "f32", True)
    la.la_gated_scan(c["a"], c["b"], workspace=ws)
    assert la.la_workspace_error(ws) == 0


def test_first_calls_of_a_process_can_be_captured(la):
    """Nothing has to run once before a capture: a fresh process captures its very first calls."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch, kernelized_linear_attention_gb300 as la
a = torch.rand(700, 2, 64, device="cuda"); b = torch.randn(700, 2, 64, device="cuda"); w = torch.ones(2, 64, device="cuda")
f = torch.rand(32, device="cuda"); p = torch.arange(700, dtype=torch.int32, device="cuda"); big = torch.randn(3, 8192, device="cuda")
w2 = torch.ones(8192, device="cuda")
g = torch.cuda.CUDAGraph()
def calls():
    h = la.la_gated_scan(a, b)
    da, db = la.la_gated_scan_backward(a, h, b)
    y, m, r = la.la_layer_norm(h, w, return_stats=True)
    n = la.la_layer_norm_backward(h, b, m, r, w)
    y2, m2, r2 = la.la_layer_norm(big, w2, return_stats=True)
    n2 = la.la_layer_norm_backward(big, b.new_ones(3, 8192), m2, r2, w2)
    return (h, da, db, y, *n, y2, *n2, *la.la_rotary(a, b, f, p, [32]))
with torch.cuda.graph(g):
    outs = calls()
g.replay()
torch.cuda.synchronize()
got = [o.clone() for o in outs]
assert all(torch.equal(x, y) for x, y in zip(got, calls()))
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr
