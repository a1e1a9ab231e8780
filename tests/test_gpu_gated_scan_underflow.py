"""GPU: states of the gated recurrence that outlive their gates' product in fp32 (strong forgetting with large or
infinite states, or nothing added), forward and adjoint, against the fp64 oracle."""
import numpy as np
import pytest

from layer_ops_util import U, check
from oracle import layer_ops as ops

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
KINDS = [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")]


@pytest.fixture(scope="module")
def la():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kernelized_linear_attention_gb300 as m
    m.load_library()
    return m


# Half of the smallest step of a stored type: fp32 has 24 bits from 2^-126 on (smallest step 2^-149), bf16 8 bits
# (2^-133); a value below 2^-126 is rounded to a multiple of that, whatever its size.
SMALLEST = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134}


def _np(t):
    return t.detach().cpu().double().numpy()


def bound(a, b, spans, state, reverse=False):
    """scan_bound's recurrence of errors (five roundings of the majorant M_t a token), with what the range of fp32 takes.
    A result below its normal range is off by at most half its smallest step, 2^-150, for each of four roundings a
    token.  A product of gates of at most one below that range is off by 2^-150 for each product of 32 tokens, 4
    warps and 8 tiles: less than 2^-144; it scales a state of up to 2^20 (a larger one goes token by token), and
    what one run leaves the next ones only shrink: 2^-124 in all."""
    a, b = np.abs(a), np.abs(b)
    E, edge = np.zeros_like(b), np.zeros((len(spans),) + b.shape[1:])
    for s, (lo, hi) in enumerate(spans):
        M = np.abs(state[s])
        M = np.where(np.isfinite(M), M, 0.0)      # (an infinite state: nothing finite follows)
        e = np.zeros(b.shape[1:])
        for t in (range(hi - 1, lo - 1, -1) if reverse else range(lo, hi)):
            g = 1.0 if reverse and t == hi - 1 else a[t + 1] if reverse else a[t]
            M = g * M + b[t]
            e = g * e + 5 * U * M + 4 * 2.0 ** -150
            E[t] = e + 2.0 ** -124
        edge[s] = (a[lo] * (e + U * M) if reverse else e) + 2.0 ** -124 if hi > lo else 0.0
    return E, edge


def _case(lengths, d, ta, tb, gates, added, states, seed):
    g = torch.Generator().manual_seed(seed)
    T, n = sum(lengths), len(lengths)
    a = torch.tensor(gates)[torch.randint(0, len(gates), (T, 1, d), generator=g)]
    b = added * torch.randn(T, 1, d, generator=g)
    s = torch.tensor(states)[torch.randint(0, len(states), (n, 1, d), generator=g)]
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    return dict(a=a.to(TYPES[ta]).cuda(), b=b.to(TYPES[tb]).cuda(), s=s.cuda(), cu=torch.from_numpy(cu).cuda(),
                spans=list(zip(cu[:-1].tolist(), cu[1:].tolist())))


def _check(la, c, ta, tb):
    a, b, s = _np(c["a"]), _np(c["b"]), _np(c["s"])
    cu = np.array([lo for lo, _ in c["spans"]] + [c["spans"][-1][1]])
    h, out = la.la_gated_scan(c["a"], c["b"], cu_seqlens=c["cu"], state_in=c["s"], return_state=True)
    with np.errstate(invalid="ignore", over="ignore"):
        ref, ref_out = ops.gated_scan(a, b, cu, state_in=s)
        E, edge = bound(a, b, c["spans"], s)
        check(_np(h), ref, E + SMALLEST[tb], tb, "h")
        check(_np(out), ref_out, edge, "f32", "state_out")
        # the adjoint: b is what reaches h, the state what reaches the last token
        ones = torch.ones_like(c["b"])
        da, db, ds = la.la_gated_scan_backward(c["a"], ones, c["b"], cu_seqlens=c["cu"], state_in=torch.ones_like(c["s"]),
                                               dstate_out=c["s"], return_dstate=True)
        ra, rb, rs = ops.gated_scan_backward(a, np.ones_like(b), b, cu, state_in=np.ones_like(s), dstate_out=s)
        E, edge = bound(a, b, c["spans"], s, reverse=True)
        check(_np(db), rb, E + SMALLEST[tb], tb, "db")
        check(_np(da), ra, E + SMALLEST[ta], ta, "da")              # times a state of one
        check(_np(ds), rs, edge, "f32", "dstate_in")


@pytest.mark.parametrize("ta,tb", KINDS)
@pytest.mark.parametrize("gates", [(0.1,), (0.2,), (0.5,), (0.05, 0.5, 0.9), (1e-3, -0.25), (1e-30,)], ids=str)
@pytest.mark.parametrize("d", [64, 63, 62])
def test_infinite_states_stay_infinite(la, d, gates, ta, tb):
    inf = float("inf")
    _check(la, _case([1300, 0, 90, 700], d, ta, tb, gates, 1.0, (inf, -inf, 1.0), d), ta, tb)
    c = _case([1300, 0, 90, 700], d, ta, tb, gates, 1.0, (0.0,), d + 1)
    c["b"][5, 0, 1] = inf
    c["b"][70, 0, 2] = -inf
    c["b"][1389, 0, 3] = inf
    c["b"][2089, 0, 4] = -inf
    _check(la, c, ta, tb)


@pytest.mark.parametrize("ta,tb", KINDS)
@pytest.mark.parametrize("added", [0.0, 1e-25, 1.0])
@pytest.mark.parametrize("gates", [(0.1,), (0.2,), (0.25, 0.3), (0.5,), (0.8, 0.9), (1e-3, 0.5, -0.5)], ids=str)
@pytest.mark.parametrize("d", [64, 63, 62])
def test_large_states_decay_gate_by_gate(la, d, gates, added, ta, tb):
    _check(la, _case([1300, 0, 90, 700], d, ta, tb, gates, added, (1e30, -3e38, 1.0, 0.0), d), ta, tb)


@pytest.mark.parametrize("T", [1, 17, 33, 60, 100, 128, 129])
def test_short_sequences(la, T):
    for ta, tb in KINDS:
        _check(la, _case([T, T, 1], 37, ta, tb, (0.1, 0.02), 0.0, (1e30, -3e38, float("inf")), T), ta, tb)
        _check(la, _case([3 * T], 40, ta, tb, (1e-3,), 0.0, (1e30, -3e38, float("inf")), T), ta, tb)


@pytest.mark.parametrize("ta,tb", KINDS)
def test_gates_above_one_within_the_range(la, ta, tb):
    # 12 gates of 2^-10 and 12 of 2^10, over and over: the state goes from 2^100 to 2^-20 and back, products of consecutive
    # gates from 2^-120 to 2^120; powers of two, so that every step is exact
    T, d = 2000, 64
    up = torch.arange(T) // 12 % 2 == 1
    a = torch.where(up, 2.0 ** 10, 2.0 ** -10)[:, None, None].expand(T, 1, d).contiguous().to(TYPES[ta]).cuda()
    b = torch.zeros(T, 1, d, dtype=TYPES[tb], device="cuda")
    s = (2.0 ** 100 * torch.sign(torch.randn(1, 1, d))).cuda()
    h, out = la.la_gated_scan(a, b, state_in=s, return_state=True)
    e = 100 + torch.cumsum(torch.where(up, 10, -10), 0)
    want = torch.ldexp(torch.ones(T), e)[:, None, None].cuda() * torch.sign(s)
    assert torch.equal(h.float(), want) and torch.equal(out, want[-1:])


@pytest.mark.parametrize("ta,tb", KINDS)
def test_states_of_ordinary_size_with_strong_forgetting(la, ta, tb):
    # what every row with a zero input and a gate of 0.5 does to a state, up to the size that takes the products
    for d in (64, 63):
        c = _case([1300, 0, 90, 700], d, ta, tb, (0.5, 0.3, 0.05), 0.0, (2.0 ** 20, -3e5, 64.0, 1e-3), 3)
        c["b"][100:130] = 1.0            # a few inputs, then nothing again
        _check(la, c, ta, tb)
        zero = torch.zeros_like(c["a"])
        h = la.la_gated_scan(zero, torch.zeros_like(c["b"]), cu_seqlens=c["cu"], state_in=c["s"])
        assert bool((h == 0).all())      # gates of zero forget everything


@pytest.mark.parametrize("ta,tb", KINDS)
@pytest.mark.parametrize("added", [1e8, 1e30])
def test_large_values_with_strong_forgetting(la, added, ta, tb):
    # large states beside inputs of their size: the products are enough (their 2^-144 |s| is 2^-44 of such an input)
    for d in (64, 63):
        c = _case([1300, 0, 90, 700], d, ta, tb, (0.2, 0.05), added, (1e9, -1e31, 1.0), 5)
        c["b"][200:205] = 0.0
        _check(la, c, ta, tb)


@pytest.mark.parametrize("ta,tb", KINDS)
def test_infinite_states_over_many_tiles(la, ta, tb):
    # every tile goes token by token through all that lies before it in its block of 64 tiles: slow, but no wait runs out
    T, d = 30000, 512
    a = torch.full((T, 1, d), 0.5, dtype=TYPES[ta], device="cuda")
    b = torch.randn(T, 1, d, device="cuda").to(TYPES[tb])
    s = torch.full((1, 1, d), float("inf"), device="cuda")
    s[..., ::2] *= -1
    ws = torch.empty(la.la_gated_scan_workspace_bytes(False, 1, T, 1, d), dtype=torch.uint8, device="cuda")
    h, out = la.la_gated_scan(a, b, state_in=s, return_state=True, workspace=ws)
    assert la.la_workspace_error(ws) == 0
    assert torch.equal(h, s.to(h.dtype).expand_as(h)) and torch.equal(out, s)
    da, db, ds = la.la_gated_scan_backward(a, torch.ones_like(b), b, dstate_out=s, return_dstate=True, workspace=ws)
    assert la.la_workspace_error(ws) == 0
    assert torch.equal(db, s.to(db.dtype).expand_as(db)) and torch.equal(ds, s)
