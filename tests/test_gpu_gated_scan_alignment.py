"""GPU: the gated scan and its adjoint with any of their arrays a few elements off: whatever way tiles come in and rows go
out, the results are the same bits, and what lies around the outputs keeps its values."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
PAD = 64


@pytest.fixture(scope="module")
def la():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kernelized_linear_attention_gb300 as m
    m.load_library()
    return m


def _among(t, by):
    """t `by` elements off a 256-byte boundary, among NaN."""
    buf = torch.full((t.numel() + 2 * PAD + by,), float("nan"), dtype=t.dtype, device="cuda")
    at = buf[PAD + by:PAD + by + t.numel()]
    at.copy_(t.reshape(-1))
    return buf, at.view(t.shape)


@pytest.mark.parametrize("ta,tb", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("T,d", [(100, 64), (300, 62), (300, 63), (1000, 64), (1000, 72), (513, 130), (700, 1)])
def test_any_array_anywhere(la, T, d, ta, tb):
    g = torch.Generator().manual_seed(T + d)
    a = torch.rand(T, 1, d, generator=g).to(TYPES[ta]).cuda()
    b, dh = (torch.randn(T, 1, d, generator=g).to(TYPES[tb]).cuda() for _ in range(2))
    cu = torch.tensor([0, T // 3, T // 3, T], dtype=torch.int32, device="cuda")
    s = torch.randn(3, 1, d, generator=g).cuda()
    h, out = la.la_gated_scan(a, b, cu, state_in=s, return_state=True)
    da, db, ds = la.la_gated_scan_backward(a, h, dh, cu, state_in=s, dstate_out=s, return_dstate=True)
    for by in (1, 2, 3, 4):
        for off in ("a", "b", "y", "da", "h", "ab", "aby", "all"):
            def at(t, name):
                return _among(t, by if off == "all" or name in off.replace("da", "D") else 0)
            (yb, y), (dab, dag), (dbb, dbg) = at(b, "y"), at(a, "D"), at(b, "y")
            yb.fill_(float("nan")), dab.fill_(float("nan")), dbb.fill_(float("nan"))
            x = {"a": at(a, "a")[1], "b": at(b, "b")[1], "h": at(h, "h")[1], "dh": at(dh, "b")[1]}
            _, out2 = la.la_gated_scan(x["a"], x["b"], cu, state_in=s, return_state=True, h=y)
            ds2 = la.la_gated_scan_backward(x["a"], x["h"], x["dh"], cu, state_in=s, dstate_out=s, return_dstate=True,
                                            da=dag, db=dbg)[2]
            for got, want in ((y, h), (out2, out), (dag, da), (dbg, db), (ds2, ds)):
                assert torch.equal(got, want), (by, off)
            for buf, n in ((yb, y), (dab, dag), (dbb, dbg)):
                first = (n.data_ptr() - buf.data_ptr()) // buf.element_size()
                assert bool(torch.isnan(buf[:first]).all()) and bool(torch.isnan(buf[first + n.numel():]).all()), (by, off)
