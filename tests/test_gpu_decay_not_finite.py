"""What values that are not finite reach in segments of several chunks."""
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


def _columns(clean, dirty, channel, rows):
    """Only `channel`'s rows [(head, rows)] may differ, and none of them is finite."""
    same = torch.ones_like(clean, dtype=torch.bool)
    for h, where in rows:
        same[where, h, channel] = False
        assert not torch.isfinite(dirty[where, h, channel]).any()
    assert torch.equal(clean[same], dirty[same])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("d", [64, 128])
def test_values_that_are_not_finite_in_segments_of_many_chunks(la, d, bad):
    """Sequences of up to 12 chunks that are one segment each: a value of v (in dq, of k; in dk, of q; in dv, of dout) reaches
    its channel from its token on (to it, from the end) and nothing else; tokens in the first, a middle, the last chunk."""
    n, H = [1500, 70, 901], 456
    T = sum(n)
    g = torch.Generator(device="cuda").manual_seed(d)
    x = [torch.randn(T, H, d, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(4)]
    ld = torch.full((H,), -0.01, device="cuda")
    cu = torch.tensor(np.cumsum([0] + n), dtype=torch.int32).cuda()
    places = [(0, 1500, 1, [0]), (0, 1500, 7, [700]), (0, 1500, 8, [1499]), (1570, 2471, 3, [1570 + 5, 1570 + 130, 2470]),
              (1500, 1570, 5, [1530])]
    channel = d - 3

    def call(*a):
        out, new = la.la_decay_attention(*a[:3], ld, scale=0.5, cu_seqlens=cu, return_state=True)
        return [out] + list(la.la_decay_attention_backward(*a, ld, scale=0.5, cu_seqlens=cu)) + [new]

    clean = call(*x)
    # operand that is z of the pass -> which result, and whether it runs from the end
    for which, result, back in ((2, 0, False), (1, 1, False), (0, 2, True), (3, 3, True)):
        y = [t.clone() for t in x]
        for lo, hi, h, tokens in places:
            y[which][tokens, h, channel] = bad
        rows = [(h, slice(lo, max(tokens) + 1) if back else slice(min(tokens), hi)) for lo, hi, h, tokens in places]
        dirty = call(*y)
        _columns(clean[result], dirty[result], channel, rows)
        if which == 2:
            keep = torch.ones(len(n), H, dtype=torch.bool, device="cuda")
            for s, h in ((0, 1), (0, 7), (0, 8), (2, 3), (1, 5)):
                keep[s, h] = False
                assert not torch.isfinite(dirty[4][s, h, :, channel]).any()
            assert torch.equal(clean[4][keep], dirty[4][keep])
