"""Accuracy of the decayed attention on the tensor cores: errors as norms over a head, and of the state that queries read
(limits and bounds derived in decay_limits.py)."""
import numpy as np
import pytest

from decay_limits import limits, relative, rows_that_differ_little
from oracle import layer_ops as ops

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def la():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kernelized_linear_attention_gb300 as m
    m.load_library()
    return m


def _np(t):
    return t.detach().cpu().double().numpy()


def _normal(shape, seed, scale=1.0, dtype=torch.bfloat16):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


def _operands(T, H, dk, dv, seed):
    return (_normal((T, H, dk), seed, dk ** -0.25), _normal((T, H, dk), seed + 1, dk ** -0.25),
            _normal((T, H, dv), seed + 2), _normal((T, H, dv), seed + 3))


@pytest.mark.parametrize("lengths,H,dk,dv,decays", [
    ([1500, 3, 901], 48, 64, 64, [-0.5, -0.05, -0.004, 0.0]), ([1500, 3, 901], 33, 128, 128, [-0.3, -0.01, 0.0]),
    ([1500, 3, 901], 300, 8, 72, [-0.5, -0.05, -0.004, 0.0]), ([3800], 200, 16, 16, [-1e-2, -1e-4, 0.0]),
    ([130, 257], 2, 64, 64, [-0.05, 0.0]), ([33000], 160, 8, 8, [0.0, -1e-6, -1e-4, -1e-2])],
    ids=lambda v: str(v).replace(" ", ""))
def test_errors_of_whole_heads(la, lengths, H, dk, dv, decays):
    T, scale = sum(lengths), 0.37
    q, k, v, do = _operands(T, H, dk, dv, T)
    ld = torch.tensor((decays * H)[:H]).cuda()
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    spans, chunks = list(zip(cu[:-1].tolist(), cu[1:].tolist())), min(64, -(-max(lengths) // 128))
    seqs = dict(nseq=1) if len(lengths) == 1 else dict(cu_seqlens=torch.from_numpy(cu).cuda())
    a, g = [_np(x) for x in (q, k, v, do)], _np(ld)
    out = la.la_decay_attention(q, k, v, ld, scale=scale, **seqs)
    ref, _ = ops.decay_attention(*a[:3], g, scale, cu)
    got, lim = relative(_np(out), ref), limits(*a[:3], ref, g, scale, spans, chunks)
    assert (got <= lim).all(), (got / lim).max()
    if T > 10000:
        return
    grads = la.la_decay_attention_backward(q, k, v, do, ld, scale=scale, **seqs)
    refs = ops.decay_attention_backward(*a, g, scale, cu)
    for name, x, (i, j, l), back, y in zip(("dq", "dk", "dv"), grads, ((3, 2, 1), (2, 3, 0), (1, 0, 3)), (False, True, True),
                                           refs):
        got, lim = relative(_np(x), y), limits(a[i], a[j], a[l], y, g, scale, spans, chunks, back)
        assert (got <= lim).all(), (name, (got / lim).max())


@pytest.mark.parametrize("d", [64, 128])
def test_the_state_that_queries_read(la, d):
    """Rows of a carried state that differ by less than one bf16 holds, one token in 200 asks for the difference; nothing
    is added and nothing decays, so that every chunk has the same state."""
    H, T = 160, 1500
    q1, s, ref, bound = rows_that_differ_little(H, d, d, d)
    zero = torch.zeros(T, H, d, dtype=torch.bfloat16, device="cuda")
    q = zero.clone()
    at = list(range(3, T, 200))
    q[at] = torch.from_numpy(q1).bfloat16().cuda()
    out, new = la.la_decay_attention(q, zero, zero, torch.zeros(H, device="cuda"), state_in=torch.from_numpy(s)[None].cuda(),
                                     nseq=1, return_state=True)
    got = _np(out)
    assert (np.abs(got[at] - ref) <= bound).all()
    assert torch.equal(new[0].cpu(), torch.from_numpy(s))
    others = np.setdiff1d(np.arange(T), at)
    assert not got[others].any()
    # the gradient of q reads the state's transpose
    st = np.ascontiguousarray(s.transpose(0, 2, 1))
    do = zero.clone()
    do[at] = q[at]
    dq = la.la_decay_attention_backward(zero, zero, zero, do, torch.zeros(H, device="cuda"), nseq=1,
                                        state_in=torch.from_numpy(st)[None].cuda())[0]
    assert (np.abs(_np(dq)[at] - ref) <= bound).all()
    # gradients of k and v read what comes from behind
    ds = torch.from_numpy(s)[None].cuda()
    dv = la.la_decay_attention_backward(zero, q, zero, zero, torch.zeros(H, device="cuda"), nseq=1, dstate_out=ds)[2]
    assert (np.abs(_np(dv)[at] - ref) <= bound).all()
    dk = la.la_decay_attention_backward(zero, zero, q, zero, torch.zeros(H, device="cuda"), nseq=1,
                                        dstate_out=torch.from_numpy(st)[None].cuda())[1]
    assert (np.abs(_np(dk)[at] - ref) <= bound).all()
