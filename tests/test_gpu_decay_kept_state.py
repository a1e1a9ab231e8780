"""What the state of the decayed attention loses while it stays in one segment on the tensor cores."""
import numpy as np
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


@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("chunks", [1, 2, 64, 65, 256])
def test_what_a_kept_state_loses(la, chunks, up):
    """As many heads as make a sequence of that many chunks one segment, or as few as it takes; every token adds a little to
    the state, and the last one takes the first state off again, so that its output is what was added and what was lost.

    A product of 16 tokens cuts 16 terms off below 2^-25 and their sum with the state below 2^-23 of the state's power of two
    (1: the state stays in [1/2, 2)): 5 2^-23, eight times a chunk, over 64 chunks at most.  What enters a segment is summed
    1024 tokens at a time, 64 such products of the added terms alone, in fp32.  The state is read to 2^-16 of itself, keys and
    values are bf16 and unweighted; 20 roundings of fp32; the output is a bf16."""
    T, H, d = 128 * chunks, 152, 8
    rng = np.random.default_rng(chunks)
    s = torch.from_numpy(rng.uniform(1.0, 1.9, (H, d, d))).bfloat16()
    k = torch.zeros(T, H, d)
    k[:-1] = 2.0 ** -22 * torch.from_numpy(rng.uniform(0.5, 1.0, (T - 1, H, d))) * (1.0 if up else -1.0)
    v = torch.from_numpy(rng.uniform(0.5, 1.0, (T, H, d))).float()
    q = torch.zeros(T, H, d)
    q[-1, :, 0] = k[-1, :, 0] = 1.0
    v[-1] = -s[:, 0].float()
    q, k, v = (x.bfloat16() for x in (q, k, v))
    out = la.la_decay_attention(q.cuda(), k.cuda(), v.cuda(), torch.zeros(H, device="cuda"),
                                state_in=s.float()[None].cuda(), nseq=1)
    kv = (k[:-1, :, :1].double() * v[:-1].double()).sum(0).numpy()
    got, terms = out[-1].double().cpu().numpy(), np.abs(kv)
    bound = 40 * 2.0 ** -23 * min(chunks, 64) + 2.0 ** -14 * terms + (2.0 ** -16 + 20 * 2.0 ** -24) * 2.0
    print(f"up {up} chunks {chunks}: lost {(kv - got).min():.2e} .. {(kv - got).max():.2e} of 1 .. 2, bound {bound.max():.2e}")
    assert (np.abs(got - kv) <= bound + 2.0 ** -8 * (np.abs(kv) + bound)).all()


def test_a_segment_has_64_chunks_at_most(la):
    """However many heads there are, longer sequences have a state between segments."""
    for cu in (False, True):
        for T, H in ((1 << 20, 400), (1 << 20, 7), (33000, 400), (8320, 1000)):
            few = la.la_decay_attention_workspace_bytes(torch.bfloat16, cu, 1, T, H, 64, 64)
            assert few >= (-(-T // 8192) - 1) * H * 64 * 64 * 4
