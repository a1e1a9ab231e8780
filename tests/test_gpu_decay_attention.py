"""GPU parity of linear attention with a decay for each head (prompts, gradients, single tokens)
against the fp64 oracle; tolerances in decay_util.py."""
import numpy as np
import pytest

from decay_util import U, backward_bounds, check, forward_bounds
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


def _off(t, by):
    """The same values in memory whose address is `by` elements off a 256-byte boundary."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    out = buf[by:].view(t.shape)
    out.copy_(t)
    return out


def _case(lengths, H, dk, dv, dtype, seed=1, log_decay=None):
    g = torch.Generator().manual_seed(seed)
    T, n = sum(lengths), len(lengths)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g) * scale).to(TYPES[dtype]).cuda()

    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    if log_decay is None:
        log_decay = torch.log1p(-(2.0 ** -(1 + 9 * torch.rand(H, generator=g).double()))).float()
    return dict(q=normal(T, H, dk, scale=dk ** -0.25), k=normal(T, H, dk, scale=dk ** -0.25), v=normal(T, H, dv),
                do=normal(T, H, dv), s=torch.randn(n, H, dk, dv, generator=g).cuda(),
                ds=torch.randn(n, H, dk, dv, generator=g).cuda(), ld=torch.as_tensor(log_decay).cuda(), cu=cu,
                cu_t=torch.from_numpy(cu).cuda(), spans=list(zip(cu[:-1].tolist(), cu[1:].tolist())), dtype=dtype,
                scale=0.37)


def _forward(la, c, state, **kw):
    return la.la_decay_attention(c["q"], c["k"], c["v"], c["ld"], scale=c["scale"], state_in=c["s"] if state else None,
                                 **(kw or dict(cu_seqlens=c["cu_t"], return_state=True)))


def _backward(la, c, state, **kw):
    return la.la_decay_attention_backward(c["q"], c["k"], c["v"], c["do"], c["ld"], scale=c["scale"],
                                          state_in=c["s"] if state else None, dstate_out=c["ds"] if state else None,
                                          **(kw or dict(cu_seqlens=c["cu_t"], return_dstate=True)))


def _check_forward(la, c, state, what=""):
    q, k, v, ld, s = (_np(c[x]) for x in ("q", "k", "v", "ld", "s"))
    s = s if state else None
    out, new = _forward(la, c, state)
    ref, ref_new = ops.decay_attention(q, k, v, ld, c["scale"], c["cu"], state_in=s)
    b_out, b_new = forward_bounds(q, k, v, ld, c["scale"], c["spans"], s, c["dtype"])
    check(_np(out), ref, b_out, c["dtype"], f"{what} out")
    check(_np(new), ref_new, b_new, "f32", f"{what} state_out")
    return out, new


def _check_backward(la, c, state, what=""):
    q, k, v, do, ld, s, ds = (_np(c[x]) for x in ("q", "k", "v", "do", "ld", "s", "ds"))
    s, ds = (s, ds) if state else (None, None)
    got = _backward(la, c, state)
    ref = ops.decay_attention_backward(q, k, v, do, ld, c["scale"], c["cu"], state_in=s, dstate_out=ds)
    bounds = backward_bounds(q, k, v, do, ld, c["scale"], c["spans"], s, ds, c["dtype"])
    for name, x, y, b in zip(("dq", "dk", "dv", "dstate_in"), got, ref, bounds):
        check(_np(x), y, b, "f32" if name == "dstate_in" else c["dtype"], f"{what} {name}")
    return got


LENGTHS = [[1], [2, 1], [0, 0, 3, 0], [31, 32, 33, 0, 65], [127], [128], [129], [0, 128, 0, 256, 0], [1] * 300,
           [255, 257, 1, 640], [900], [0, 0, 0]]


@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda l: "x".join(map(str, l[:5])))
def test_packed(la, lengths, dtype, state):
    c = _case(lengths, 2, 64, 64, dtype)
    _check_forward(la, c, state)
    _check_backward(la, c, state)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(1, 1), (3, 5), (16, 16), (37, 53), (64, 24), (40, 72), (96, 80), (128, 128), (64, 128),
                                   (128, 64), (65, 64), (130, 256), (256, 16), (256, 256)])
def test_widths(la, dk, dv, dtype):
    c = _case([150, 0, 277], 2, dk, dv, dtype, seed=2)
    _check_forward(la, c, True)
    _check_backward(la, c, True)


@pytest.mark.parametrize("dtype,H,dk,dv", [("f32", 70, 24, 24), ("bf16", 70, 24, 24), ("bf16", 48, 64, 64), ("bf16", 33, 128, 128),
                                           ("bf16", 400, 16, 8), ("bf16", 300, 8, 72)])
def test_segments_of_several_chunks(la, dtype, H, dk, dv):
    """Enough tokens that a segment has several chunks, in the sequences' middle and at their ends."""
    c = _case([1500, 3, 901], H, dk, dv, dtype, seed=3)
    _check_forward(la, c, True)
    _check_backward(la, c, True)


@pytest.mark.parametrize("dk,dv", [(16, 16), (8, 72)])
def test_one_segment_of_many_chunks(la, dk, dv):
    """Each of so many heads is one segment: no state between segments, 30 chunks after one another."""
    c = _case([3800], 200, dk, dv, "bf16", seed=23)
    q, k, v, do, ld = (_np(c[x]) for x in ("q", "k", "v", "do", "ld"))
    out, new = _forward(la, c, False, nseq=1, return_state=True)
    ref, ref_new = ops.decay_attention(q, k, v, ld, c["scale"], c["cu"])
    b_out, b_new = forward_bounds(q, k, v, ld, c["scale"], c["spans"], None, "bf16")
    check(_np(out), ref, b_out, "bf16", "out")
    check(_np(new), ref_new, b_new, "f32", "state_out")
    got = _backward(la, c, False, nseq=1)
    refs = ops.decay_attention_backward(q, k, v, do, ld, c["scale"], c["cu"])
    for x, y, b in zip(got, refs, backward_bounds(q, k, v, do, ld, c["scale"], c["spans"], None, None, "bf16")):
        check(_np(x), y, b, "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decays_from_nothing_to_everything(la, dtype):
    ld = torch.tensor([0.0, -float("inf"), -1e-7, -1e-3, -0.7, -5.0, -60.0, -1e4, -1e30, -3e38])
    c = _case([700, 130], 10, 64, 64, dtype, seed=4, log_decay=ld)
    c["scale"] = 1.0
    for state in (False, True):
        _check_forward(la, c, state)
        _check_backward(la, c, state)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_growing_states(la, dtype):
    c = _case([300], 2, 64, 64, dtype, seed=5, log_decay=torch.tensor([0.01, 0.002]))
    _check_forward(la, c, True)
    _check_backward(la, c, True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("nseq,n", [(1, 700), (5, 129), (3, 1), (4, 128)])
def test_equal_lengths_without_cu_seqlens(la, nseq, n, dtype):
    c = _case([n] * nseq, 3, 64, 64, dtype, seed=6)
    assert all(torch.equal(x, y) for x, y in zip(_forward(la, c, True),
                                                 _forward(la, c, True, nseq=nseq, return_state=True)))
    assert all(torch.equal(x, y) for x, y in zip(_backward(la, c, True),
                                                 _backward(la, c, True, nseq=nseq, return_dstate=True)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_operands_anywhere(la, dtype):
    """Operands and outputs that start on no vector's boundary."""
    c = _case([200, 90], 2, 64, 64, dtype, seed=7)
    for by in (1, 2, 3):
        o = dict(c, **{x: _off(c[x], by) for x in ("q", "k", "v", "do", "s", "ds", "ld")})
        _check_forward(la, o, True, f"off by {by}")
        _check_backward(la, o, True, f"off by {by}")
    one = dict(c, v=_off(c["v"], 1))
    _check_forward(la, one, True, "v off")
    out = _off(torch.zeros_like(c["v"]), 1)
    la.la_decay_attention(c["q"], c["k"], c["v"], c["ld"], scale=c["scale"], cu_seqlens=c["cu_t"], out=out)
    ref, _ = ops.decay_attention(_np(c["q"]), _np(c["k"]), _np(c["v"]), _np(c["ld"]), c["scale"], c["cu"])
    check(_np(out), ref, forward_bounds(_np(c["q"]), _np(c["k"]), _np(c["v"]), _np(c["ld"]), c["scale"], c["spans"], None,
                                        dtype)[0], dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,dk,dv", [(1, 1, 1, 1), (3, 2, 64, 64), (5, 3, 37, 53), (2, 4, 128, 128), (7, 1, 256, 256),
                                       (4, 2, 256, 3), (300, 5, 16, 8), (2, 2, 96, 132)])
def test_step(la, B, H, dk, dv, dtype):
    c = _case([1] * B, H, dk, dv, dtype, seed=8)
    q, k, v, ld, s = (_np(c[x]) for x in ("q", "k", "v", "ld", "s"))
    ref, ref_new = ops.decay_attention(q, k, v, ld, c["scale"], c["cu"], state_in=s)
    b_out, b_new = forward_bounds(q, k, v, ld, c["scale"], c["spans"], s, "f32")
    for by in (0, 1):
        state, new = _off(c["s"], by), _off(torch.zeros_like(c["s"]), by)
        keep = state.clone()
        out = la.la_decay_step(c["q"], c["k"], c["v"], c["ld"], state, scale=c["scale"], state_out=new)
        assert torch.equal(state, keep)
        check(_np(out), ref, b_out, dtype, "out")
        check(_np(new), ref_new, b_new, "f32", "state_out")
        out2 = la.la_decay_step(_off(c["q"], by), _off(c["k"], by), _off(c["v"], by), c["ld"], state, scale=c["scale"])
        assert torch.equal(out, out2) and torch.equal(state, new)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_then_single_tokens(la, dtype):
    """A prompt's state goes on token by token; the same as one call over all of it."""
    c = _case([200, 200], 2, 64, 64, dtype, seed=9)
    first = torch.cat([torch.arange(0, 190), torch.arange(200, 390)]).cuda()
    part = dict(c, **{x: c[x][first].contiguous() for x in ("q", "k", "v")})
    out, state = la.la_decay_attention(part["q"], part["k"], part["v"], c["ld"], scale=c["scale"], nseq=2,
                                       return_state=True)
    rows = [out.view(2, 190, 2, 64)]
    for t in range(190, 200):
        at = [t, 200 + t]
        rows.append(la.la_decay_step(c["q"][at], c["k"][at], c["v"][at], c["ld"], state, scale=c["scale"])[:, None])
    got = torch.cat(rows, 1).reshape(400, 2, 64)
    q, k, v, ld = (_np(c[x]) for x in ("q", "k", "v", "ld"))
    ref, ref_new = ops.decay_attention(q, k, v, ld, c["scale"], c["cu"])
    b_out, b_new = forward_bounds(q, k, v, ld, c["scale"], c["spans"], None, dtype)
    check(_np(got), ref, b_out, dtype, "out")
    check(_np(state), ref_new, b_new, "f32", "state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_states_in_place(la, dtype):
    c = _case([300, 0, 5, 128], 2, 64, 64, dtype, seed=10)
    out, new = _forward(la, c, True)
    s = c["s"].clone()
    out2 = la.la_decay_attention(c["q"], c["k"], c["v"], c["ld"], scale=c["scale"], cu_seqlens=c["cu_t"], state_in=s,
                                 state_out=s)
    assert torch.equal(out, out2) and torch.equal(new, s)
    got = _backward(la, c, True)
    ds = c["ds"].clone()
    got2 = la.la_decay_attention_backward(c["q"], c["k"], c["v"], c["do"], c["ld"], scale=c["scale"],
                                          cu_seqlens=c["cu_t"], state_in=c["s"], dstate_out=ds, dstate_in=ds)
    assert all(torch.equal(x, y) for x, y in zip(got, got2 + (ds,)))
    # what is not asked for changes nothing
    assert torch.equal(out, la.la_decay_attention(c["q"], c["k"], c["v"], c["ld"], scale=c["scale"],
                                                  cu_seqlens=c["cu_t"], state_in=c["s"]))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which", ["q", "k", "v", "do"])
def test_values_that_are_not_finite_stay_where_they_belong(la, which, dtype, bad):
    """A token's value reaches neither the tokens that do not see it nor other sequences."""
    c = _case([150, 210, 140], 2, 64, 64, dtype, seed=11)
    at = 150 + 77
    d = dict(c, **{which: c[which].clone()})
    d[which][at, 1, 5] = bad
    clean, dirty = _forward(la, c, False), _forward(la, d, False)
    seen = torch.zeros(500, 2, dtype=torch.bool, device="cuda")
    if which in ("k", "v"):
        seen[at:360, 1] = True
    elif which == "q":
        seen[at, 1] = True
    assert torch.equal(clean[0][~seen], dirty[0][~seen])
    keep = torch.ones(3, 2, dtype=torch.bool, device="cuda")
    if which in ("k", "v"):
        keep[1, 1] = False
    assert torch.equal(clean[1][keep], dirty[1][keep])
    if which == "v" and bad != 3e38:      # its own channel has it from there on, the others do not
        assert not torch.isfinite(dirty[0][at:360, 1, 5]).any()
        others = torch.arange(64, device="cuda") != 5
        assert torch.equal(clean[0][..., others], dirty[0][..., others])
    clean, dirty = _backward(la, c, False), _backward(la, d, False)
    after, before = torch.zeros_like(seen), torch.zeros_like(seen)
    after[at:360, 1], before[150:at + 1, 1] = True, True
    own = torch.zeros_like(seen)
    own[at, 1] = True
    # dq_i needs do_i and k_j, v_j of j <= i; dk_j needs v_j and q_i, do_i of i >= j; dv_j needs k_j and the same
    reach = {"q": (None, before, before), "k": (after, None, own), "v": (after, own, None), "do": (own, before, before)}
    for x, y, r in zip(clean, dirty, reach[which]):
        assert torch.equal(x, y) if r is None else torch.equal(x[~r], y[~r])


@pytest.mark.parametrize("d", [64, 128])
def test_neighbours_full_of_nan(la, d):
    """Sequences of many chunks that end in the middle of one, between others that hold nothing finite."""
    H, n = 150, [700, 40, 3, 900, 61]
    T = sum(n)
    g = torch.Generator(device="cuda").manual_seed(24)
    x = {k: torch.randn(T, H, d, generator=g, device="cuda", dtype=torch.bfloat16) for k in ("q", "k", "v", "do")}
    ld = torch.full((H,), -0.02, device="cuda")
    cu = torch.tensor(np.cumsum([0] + n), dtype=torch.int32).cuda()
    alive = torch.cat([torch.full((m,), i % 2 == 0) for i, m in enumerate(n)]).cuda()
    y = {k: torch.where(alive[:, None, None], v, torch.full_like(v, float("nan"))) for k, v in x.items()}
    for _ in range(3):
        a, b = (la.la_decay_attention(z["q"], z["k"], z["v"], ld, cu_seqlens=cu, return_state=True) for z in (x, y))
        assert torch.equal(a[0][alive], b[0][alive]) and torch.equal(a[1][::2], b[1][::2])
        a, b = (la.la_decay_attention_backward(z["q"], z["k"], z["v"], z["do"], ld, cu_seqlens=cu) for z in (x, y))
        assert all(torch.equal(u[alive], w[alive]) for u, w in zip(a, b))


def test_large_values_beside_small_ones(la):
    """Tokens whose values differ by many powers of two: the small ones' outputs keep their digits."""
    c = _case([300], 2, 64, 64, "bf16", seed=12)
    size = torch.exp2(torch.randint(-60, 30, (300, 1, 1), generator=torch.Generator().manual_seed(3)).float()).cuda()
    c["v"] = (c["v"].float() * size.sort(0).values).bfloat16()
    c["k"] = (c["k"].float() * torch.exp2(torch.arange(300) % 7 - 3.0).cuda()[:, None, None]).bfloat16()
    _check_forward(la, c, False)
    _check_backward(la, c, False)


@pytest.mark.parametrize("cu", [[0, 50, 40, 100], [1, 50, 60, 100], [0, 50, 60, 99], [0, -5, 60, 100], [0, 50, 200, 100]])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_malformed_cu_seqlens_are_reported(la, cu, dtype):
    c = _case([100], 2, 64, 64, dtype, seed=13)
    cu = torch.tensor(cu, dtype=torch.int32).cuda()
    ws = torch.empty(max(la.la_decay_attention_workspace_bytes(c["q"].dtype, True, 3, 100, 2, 64, 64),
                         la.la_decay_attention_backward_workspace_bytes(c["q"].dtype, True, 3, 100, 2, 64, 64)),
                     dtype=torch.uint8, device="cuda")
    out, new = torch.full_like(c["v"], 7.0), torch.full((3, 2, 64, 64), 7.0, device="cuda")
    la.la_decay_attention(c["q"], c["k"], c["v"], c["ld"], cu_seqlens=cu, out=out, state_out=new, workspace=ws)
    assert la.la_workspace_error(ws) == 1
    grads = [torch.full_like(c["q"], 7.0) for _ in range(3)]
    la.la_decay_attention_backward(c["q"], c["k"], c["v"], c["do"], c["ld"], cu_seqlens=cu, dq=grads[0], dk=grads[1],
                                   dv=grads[2], dstate_in=new, workspace=ws)
    assert la.la_workspace_error(ws) == 1
    assert all(bool((x == 7.0).all()) for x in [out, new] + grads)
    la.la_decay_attention(c["q"], c["k"], c["v"], c["ld"], nseq=1, out=out, workspace=ws)     # and the next call is right
    assert la.la_workspace_error(ws) == 0
    check(_np(out), ops.decay_attention(_np(c["q"]), _np(c["k"]), _np(c["v"]), _np(c["ld"]))[0],
          forward_bounds(_np(c["q"]), _np(c["k"]), _np(c["v"]), _np(c["ld"]), 1.0, c["spans"], None, dtype)[0], dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_same_bits_every_time(la, dtype):
    c = _case([1000, 3, 700], 4, 64, 64, dtype, seed=14)
    first = _forward(la, c, True) + _backward(la, c, True)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(first, _forward(la, c, True) + _backward(la, c, True)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_and_replayed_with_other_values(la, dtype):
    c, d = _case([400, 129], 2, 64, 64, dtype, seed=15), _case([129, 400], 2, 64, 64, dtype, seed=16)
    want = _forward(la, d, True) + _backward(la, d, True)
    held = {x: c[x].clone() for x in ("q", "k", "v", "do", "s", "ds", "ld", "cu_t")}
    h = dict(c, **held)
    _forward(la, h, True), _backward(la, h, True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _forward(la, h, True) + _backward(la, h, True)
    for x in held:
        held[x].copy_(d[x])
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_two_streams_at_once(la):
    cases = [_case([2000, 77], 8, 64, 64, "bf16", seed=s) for s in (17, 18)]
    want = [_forward(la, c, True) + _backward(la, c, True) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        got = []
        for c, s in zip(cases, streams):
            kw = dict(cu_seqlens=c["cu_t"], stream=s)
            got.append(_forward(la, c, True, return_state=True, **kw) + _backward(la, c, True, return_dstate=True, **kw))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(g, w))


@pytest.mark.parametrize("d", [64, 128])
def test_a_wait_that_runs_out_is_reported(la, d):
    """(The state sums' kernel and the products', one launch each: every role's own wait takes two seconds.)"""
    c = _case([500, 100], 2, d, d, "bf16", seed=22)
    kw = dict(cu_seqlens=c["cu_t"])
    want = _forward(la, c, True, **kw)
    ws = torch.empty(la.la_decay_attention_workspace_bytes(torch.bfloat16, True, 2, 600, 2, d, d), dtype=torch.uint8,
                     device="cuda")
    la.la_test_force_wait_timeout(True)
    try:
        _forward(la, c, True, workspace=ws, **kw)
        assert la.la_workspace_error(ws) == 2
    finally:
        la.la_test_force_wait_timeout(False)
    got = _forward(la, c, True, workspace=ws, **kw)
    assert la.la_workspace_error(ws) == 0
    assert torch.equal(got, want)


def test_no_tokens(la):
    c = _case([0, 0], 2, 64, 64, "bf16", seed=19)
    out, new = _forward(la, c, True)
    assert out.shape == (0, 2, 64) and torch.equal(new, c["s"])
    assert torch.equal(_backward(la, c, True)[3], c["ds"])
    out, new = _forward(la, c, False, nseq=2, return_state=True)
    assert not new.any()
    assert la.la_decay_step(c["q"], c["k"], c["v"], c["ld"], torch.empty(0, 2, 64, 64, device="cuda")).shape == (0, 2, 64)


def test_rows_beyond_32_bits(la):
    """More than 2^32 bytes and 2^31 elements of rows, without the memory for an oracle of all: the last
    sequence alone, which starts beyond them, has the same bits in a call of its own."""
    H, d, n, T = 512, 64, 300, 68000
    g = torch.Generator(device="cuda").manual_seed(20)
    x = [torch.randn(T, H, d, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
    ld = torch.full((H,), -0.01, device="cuda")
    cu = torch.tensor([0, T - n, T], dtype=torch.int32).cuda()
    assert T * H * d > 2 ** 31
    out, new = la.la_decay_attention(*x, ld, cu_seqlens=cu, return_state=True)
    tail = [y[-n:].contiguous() for y in x]
    s = torch.zeros(1, H, d, d, device="cuda")
    q, k, v = (_np(y[:, -1:]) for y in tail)
    ref, ref_new = ops.decay_attention(q, k, v, _np(ld[-1:]))
    b_out, b_new = forward_bounds(q, k, v, _np(ld[-1:]), 1.0, [(0, n)], None, "bf16")
    check(_np(out[-n:, -1:]), ref, b_out, "bf16")
    check(_np(new[1:, -1:]), ref_new, b_new, "f32")


def test_gradients_against_differences(la):
    """Directional derivatives of the 64-bit forward along random directions."""
    c = _case([130, 40], 2, 24, 40, "f32", seed=21)
    names = ("q", "k", "v", "s")
    x = {n: _np(c[n]) for n in names}
    do, ds, ld = _np(c["do"]), _np(c["ds"]), _np(c["ld"])

    def loss(**moved):
        y = {**x, **moved}
        out, new = ops.decay_attention(y["q"], y["k"], y["v"], ld, c["scale"], c["cu"], state_in=y["s"])
        return (out * do).sum() + (new * ds).sum()

    s0, ds0 = _np(c["s"]), _np(c["ds"])
    bounds = backward_bounds(x["q"], x["k"], x["v"], do, ld, c["scale"], c["spans"], s0, ds0, "f32")
    rng = np.random.default_rng(0)
    # linear in each operand: the differences are exact but for the 64-bit rounding of two losses over a step of 2e-4
    size = (np.abs(do) * np.abs(ops.decay_attention(*(np.abs(x[n]) for n in "qkv"), ld, c["scale"], c["cu"],
                                                    state_in=np.abs(s0))[0])).sum() + (np.abs(ds0)).sum() * 1e3
    for name, grad, bound in zip(names, _backward(la, c, True), bounds):
        way = rng.normal(size=x[name].shape)
        slope = (loss(**{name: x[name] + 1e-4 * way}) - loss(**{name: x[name] - 1e-4 * way})) / 2e-4
        off = ((bound + U * np.abs(_np(grad))) * np.abs(way)).sum() + 2 ** -44 * size / 2e-4
        assert abs((_np(grad) * way).sum() - slope) <= off


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[1], [31], [32], [33], [127], [128], [129], [256], [1000], [64, 0, 64]])
def test_states_that_nobody_asks_for_change_nothing(la, lengths, dtype):
    c = _case(lengths, 3, 64, 64, dtype, seed=21)
    for state in (False, True):
        out, _ = _forward(la, c, state)
        assert torch.equal(out, _forward(la, c, state, cu_seqlens=c["cu_t"]))
        if len(lengths) == 1:
            assert torch.equal(out, _forward(la, c, state, nseq=1))
        got = _backward(la, c, state)
        for kw in [dict(cu_seqlens=c["cu_t"])] + [dict(nseq=1)] * (len(lengths) == 1):
            assert all(torch.equal(x, y) for x, y in zip(got[:3], _backward(la, c, state, **kw)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_calls_behind_one_another_share_a_workspace(la, dtype):
    # each call's first kernel has to wait for the last one of the call ahead: nothing but the stream orders them
    cases = [_case(lengths, 8, 64, 64, dtype, seed=22 + i) for i, lengths in enumerate([[3000, 77], [40] * 60, [129]])]
    want = [_forward(la, c, True) + _backward(la, c, True) for c in cases]
    need = max(max(la.la_decay_attention_backward_workspace_bytes(TYPES[dtype], True, len(c["spans"]), c["q"].shape[0], 8,
                                                                  64, 64) for c in cases), 256)
    w = torch.empty(need, dtype=torch.uint8, device="cuda")
    got = [tuple(torch.empty_like(x) for x in r) for r in want]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, (out, state, dq, dk, dv, ds) in zip(cases, got):
            la.la_decay_attention(c["q"], c["k"], c["v"], c["ld"], scale=c["scale"], cu_seqlens=c["cu_t"],
                                  state_in=c["s"], state_out=state, out=out, workspace=w)
            la.la_decay_attention_backward(c["q"], c["k"], c["v"], c["do"], c["ld"], scale=c["scale"],
                                           cu_seqlens=c["cu_t"], state_in=c["s"], dstate_out=c["ds"], dq=dq, dk=dk,
                                           dv=dv, dstate_in=ds, workspace=w)
        kept = [tuple(x.clone() for x in r) for r in got]
        for r in got:
            for x in r:
                x.zero_()
        assert all(torch.equal(x, y) for r, s in zip(kept, want) for x, y in zip(r, s))


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (37, 53)])
def test_many_heads_and_short_sequences(la, dk, dv):
    c = _case([5, 0, 130, 64, 1, 300, 128] * 3, 40, dk, dv, "bf16", seed=25)
    _check_forward(la, c, True)
    _check_backward(la, c, True)


@pytest.mark.parametrize("dv", [1, 2, 4, 129, 250, 251, 256])
def test_step_of_any_width(la, dv):
    g = torch.Generator().manual_seed(dv)
    q, k = (torch.randn(3, 2, 33, generator=g).cuda() for _ in range(2))
    v, s = torch.randn(3, 2, dv, generator=g).cuda(), torch.randn(3, 2, 33, dv, generator=g).cuda()
    ld = torch.tensor([-0.1, -2.0]).cuda()
    new = torch.empty_like(s)
    out = la.la_decay_step(q, k, v, ld, s, scale=0.5, state_out=new)
    want = s.double() * ld.double().exp()[None, :, None, None] + k.double()[..., None] * v.double()[..., None, :]
    # a product, a sum and a rounding of the decay: 2^-22 of the terms; then 33 terms more
    size = s.double().abs() + (k.double()[..., None] * v.double()[..., None, :]).abs()
    assert ((new.double() - want).abs() <= 2.0 ** -21 * size).all()
    terms = (q.double().abs()[..., None] * size).sum(2)
    assert ((out.double() - 0.5 * (q.double()[..., None] * want).sum(2)).abs() <= 40 * 2.0 ** -23 * terms).all()


def test_more_chunks_than_a_state_takes(la):
    """So many heads that each would be one segment, and more tokens than one segment has; nothing is forgotten."""
    c = _case([33000], 160, 8, 8, "bf16", seed=26, log_decay=torch.tensor([0.0, -1e-6, -1e-4, -1e-2] * 40))
    _check_forward(la, c, False)
    out, new = _forward(la, c, False, nseq=1, return_state=True)
    q, k, v, ld = (_np(c[x]) for x in ("q", "k", "v", "ld"))
    ref, ref_new = ops.decay_attention(q, k, v, ld, c["scale"], c["cu"])
    b_out, b_new = forward_bounds(q, k, v, ld, c["scale"], c["spans"], None, "bf16")
    check(_np(out), ref, b_out, "bf16", "out")
    check(_np(new), ref_new, b_new, "f32", "state_out")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_an_equal_batch_captured_twice_and_replayed(la, dtype):
    c = _case([400, 400], 3, 64, 64, dtype, seed=27)
    want = _forward(la, c, True, nseq=2, return_state=True) + _backward(la, c, True, nseq=2, return_dstate=True)
    torch.cuda.synchronize()
    graphs, got = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for graph in graphs:
        with torch.cuda.graph(graph):
            got.append(_forward(la, c, True, nseq=2, return_state=True) +
                       _backward(la, c, True, nseq=2, return_dstate=True))
    for _ in range(3):
        for r in got:
            for x in r:
                x.zero_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for r in got for x, y in zip(r, want))
