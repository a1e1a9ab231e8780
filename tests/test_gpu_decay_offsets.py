"""Rows of the decayed attention behind 2^31 elements, all heads of them, and their gradients."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def la():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kernelized_linear_attention_gb300 as m
    m.load_library()
    return m


def test_rows_of_all_heads_beyond_32_bits(la):
    """A sequence behind more than 2^31 elements of rows: all its heads, its state and its gradients, against the same
    sequence in a call of its own (as norms: the segments differ)."""
    H, d, n, T = 512, 64, 300, 66000
    g = torch.Generator(device="cuda").manual_seed(20)
    x = [torch.randn(T, H, d, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(4)]
    ld = torch.full((H,), -0.01, device="cuda")
    cu = torch.tensor([0, T - n, T], dtype=torch.int32).cuda()
    assert (T - n) * H * d > 2 ** 31
    tail = [y[-n:].clone() for y in x]

    def near(got, want, limit):
        got, want = got.double(), want.double()
        off = ((got - want) ** 2).sum((0, 2)).sqrt() / (want ** 2).sum((0, 2)).sqrt()
        assert (off <= limit).all(), off.max()

    out, new = la.la_decay_attention(*x[:3], ld, cu_seqlens=cu, return_state=True)
    want, want_new = la.la_decay_attention(*tail[:3], ld, nseq=1, return_state=True)
    # two results of the same sums, each off by at most 0.0035 (limits of decay_limits.py)
    near(out[-n:], want, 0.005)
    near(new[1].transpose(0, 1), want_new[0].transpose(0, 1), 1e-5)
    del out
    grads = la.la_decay_attention_backward(*x, ld, cu_seqlens=cu, return_dstate=True)
    wants = la.la_decay_attention_backward(*tail, ld, nseq=1, return_dstate=True)
    for a, b in zip(grads[:3], wants[:3]):
        near(a[-n:], b, 0.005)
    near(grads[3][1].transpose(0, 1), wants[3][0].transpose(0, 1), 1e-5)


@pytest.mark.parametrize("dtype,T", [(torch.float32, 66000), (torch.bfloat16, 66000)])
def test_rows_beyond_32_bits_on_cuda_cores(la, dtype, T):
    """The same on CUDA cores: fp32 rows, and bf16 rows whose width is no multiple of 8."""
    H, n = 512, 65
    d = 64 if dtype == torch.float32 else 66
    g = torch.Generator(device="cuda").manual_seed(21)
    ld = torch.full((H,), -0.05, device="cuda")
    cu = torch.tensor([0, T - n, T], dtype=torch.int32).cuda()
    x = [torch.randn(T, H, d, generator=g, device="cuda", dtype=dtype) for _ in range(4)]
    assert (T - n) * H * d > 2 ** 31
    tail = [y[-n:].clone() for y in x]
    limit = 1e-5 if dtype == torch.float32 else 0.005      # fp32 sums of 65 tokens and 64 channels; two bf16 roundings

    def near(got, want):
        got, want = got.double(), want.double()
        off = ((got - want) ** 2).sum((0, 2)).sqrt() / (want ** 2).sum((0, 2)).sqrt()
        assert (off <= limit).all(), off.max()

    near(la.la_decay_attention(*x[:3], ld, cu_seqlens=cu)[-n:], la.la_decay_attention(*tail[:3], ld, nseq=1))
    grads = la.la_decay_attention_backward(*x, ld, cu_seqlens=cu)
    for a, b in zip(grads, la.la_decay_attention_backward(*tail, ld, nseq=1)):
        near(a[-n:], b)
