"""Refusals of the operators around the attention call, made on the host before anything is enqueued."""
import ctypes
import os

import pytest

torch = pytest.importorskip("torch")

P = [i << 28 for i in range(1, 16)]   # pointers that are never read: far apart, well aligned


@pytest.fixture(scope="module")
def lib():
    import kernelized_linear_attention_gb300 as la
    if not os.path.exists(la.library_path()):
        from kernelized_linear_attention_gb300 import build
        build.build()
    return la.load_library()


def _scan(lib, **kw):
    a = dict(a=P[0], b=P[1], at=0, bt=1, cu=None, nseq=1, T=128, H=2, d=64, si=None, so=None, h=P[2], ws=P[3],
             bytes=1 << 26, stream=None)
    a.update(kw)
    return lib.la_gated_scan(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(at=2), 1), (dict(bt=-1), 1), (dict(nseq=0), 1), (dict(nseq=65536), 1), (dict(T=-1), 1), (dict(T=1 << 31), 1),
    (dict(H=0), 1), (dict(d=0), 1), (dict(T=130, nseq=4), 1), (dict(a=None), 1), (dict(b=None), 1), (dict(h=None), 1),
    (dict(ws=None), 1), (dict(ws=P[3] + 16), 1), (dict(a=P[0] + 2), 1), (dict(b=P[1] + 1), 1), (dict(h=P[2] + 1), 1),
    (dict(si=P[4] + 2), 1), (dict(so=P[4] + 2), 1), (dict(cu=P[4] + 2), 1),
    (dict(H=1 << 15, d=64), 2), (dict(bytes=255), 3),
    (dict(h=P[0]), 1), (dict(h=P[1]), 1), (dict(h=P[1] + 2), 1), (dict(so=P[0] + 4), 1),      # outputs on inputs
    (dict(si=P[4], so=P[4] + 4), 1), (dict(h=P[3] + 256), 1), (dict(cu=P[2]), 1),
])
def test_gated_scan_rejects_bad_arguments(lib, bad, code):
    assert _scan(lib, **bad) == code


def _scan_bwd(lib, **kw):
    a = dict(a=P[0], h=P[1], dh=P[2], at=0, bt=1, cu=None, nseq=1, T=128, H=2, d=64, si=None, dso=None, da=P[3],
             db=P[4], dsi=None, ws=P[5], bytes=1 << 26, stream=None)
    a.update(kw)
    return lib.la_gated_scan_backward(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(at=2), 1), (dict(bt=3), 1), (dict(nseq=0), 1), (dict(T=130, nseq=4), 1), (dict(a=None), 1), (dict(h=None), 1),
    (dict(dh=None), 1), (dict(da=None), 1), (dict(db=None), 1), (dict(ws=None), 1), (dict(da=P[3] + 2), 1),
    (dict(dsi=P[6] + 1), 1), (dict(dso=P[6] + 1), 1), (dict(H=1 << 15, d=64), 2), (dict(bytes=0), 3),
    (dict(da=P[0]), 1), (dict(db=P[2]), 1), (dict(da=P[4]), 1), (dict(dso=P[6], dsi=P[6] + 8), 1),
    (dict(si=P[6], dsi=P[6]), 1),
])
def test_gated_scan_backward_rejects_bad_arguments(lib, bad, code):
    assert _scan_bwd(lib, **bad) == code


def test_gated_scan_workspace_query(lib):
    import kernelized_linear_attention_gb300 as la
    assert la.la_gated_scan_workspace_bytes(False, 3, 100, 2, 64) == 0
    assert la.la_gated_scan_workspace_bytes(True, 3, 100, 2, 64) > 0
    assert la.la_gated_scan_workspace_bytes(True, 1, 0, 1, 1) > 0
    assert la.la_gated_scan_workspace_bytes(True, 1, 10, 1 << 15, 64) == 0


def _step(lib, **kw):
    a = dict(a=P[0], b=P[1], at=0, bt=1, B=4, H=2, d=64, si=P[2], so=P[2], h=P[3], stream=None)
    a.update(kw)
    return lib.la_gated_step(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(at=5), 1), (dict(bt=5), 1), (dict(B=-1), 1), (dict(H=0), 1), (dict(d=0), 1), (dict(a=None), 1),
    (dict(si=None), 1), (dict(so=None), 1), (dict(h=None), 1), (dict(si=P[2] + 2), 1), (dict(h=P[1]), 1),
    (dict(so=P[2] + 4), 1), (dict(so=P[0]), 1), (dict(H=1 << 15, d=64), 2), (dict(B=0), 0), (dict(B=0, a=None), 0),
])
def test_gated_step_rejects_bad_arguments(lib, bad, code):
    assert _step(lib, **bad) == code


def _norm(lib, **kw):
    a = dict(x=P[0], w=P[1], b=P[2], dt=1, rows=128, groups=2, d=64, eps=1e-5, y=P[3], mean=P[4], rstd=P[5],
             stream=None)
    a.update(kw)
    return lib.la_layer_norm(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(dt=2), 1), (dict(rows=-1), 1), (dict(groups=0), 1), (dict(groups=3), 1), (dict(d=0), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(x=None), 1), (dict(y=None), 1),
    (dict(x=P[0] + 1), 1), (dict(w=P[1] + 2), 1), (dict(mean=P[4] + 2), 1), (dict(y=P[0]), 1), (dict(mean=P[3]), 1),
    (dict(rstd=P[4] + 4), 1), (dict(d=16385), 2), (dict(groups=1 << 14, rows=1 << 14, d=128), 2), (dict(rows=0), 0),
    (dict(rows=0, x=None, y=None), 0),
])
def test_layer_norm_rejects_bad_arguments(lib, bad, code):
    assert _norm(lib, **bad) == code


def _norm_bwd(lib, **kw):
    a = dict(x=P[0], dy=P[1], w=P[2], mean=P[3], rstd=P[4], dt=1, rows=128, groups=2, d=64, dx=P[5], dw=P[6], db=P[7],
             ws=P[8], bytes=1 << 26, stream=None)
    a.update(kw)
    return lib.la_layer_norm_backward(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(dt=2), 1), (dict(rows=-2), 1), (dict(groups=3), 1), (dict(d=0), 1), (dict(d=16385), 2), (dict(ws=None), 1),
    (dict(ws=P[8] + 8), 1), (dict(x=None), 1), (dict(dy=None), 1), (dict(mean=None), 1), (dict(rstd=None), 1),
    (dict(dx=None), 1), (dict(dx=P[5] + 1), 1), (dict(dw=P[6] + 2), 1),
])
def test_layer_norm_backward_rejects_bad_arguments(lib, bad, code):
    assert _norm_bwd(lib, **bad) == code


def _rotary(lib, pairs=(16, 16), **kw):
    a = dict(q=P[0], k=P[1], freq=P[2], pos=P[3], dt=1, T=128, H=2, d=64,
             pairs=(ctypes.c_int * max(1, len(pairs)))(*pairs), naxes=len(pairs), il=0, inv=0, qo=P[4], ko=P[5],
             stream=None)
    a.update(kw)
    return lib.la_rotary(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(dt=2), 1), (dict(T=-1), 1), (dict(T=1 << 31), 1), (dict(H=0), 1), (dict(d=1), 1), (dict(naxes=0), 1),
    (dict(pairs=(0, 0)), 1), (dict(pairs=(-1, 4)), 1), (dict(pairs=(16, 17)), 1), (dict(pairs=(2 ** 30, 2 ** 30)), 1),
    (dict(il=2), 1), (dict(inv=-1), 1), (dict(q=None), 1), (dict(qo=None), 1), (dict(freq=None), 1), (dict(pos=None), 1),
    (dict(ko=None), 1), (dict(k=None), 1), (dict(q=P[0] + 1), 1), (dict(freq=P[2] + 2), 1), (dict(pos=P[3] + 1), 1),
    (dict(qo=P[0] + 2), 1), (dict(qo=P[1]), 1), (dict(ko=P[4]), 1), (dict(qo=P[2]), 1),
    (dict(pairs=(1,) * 5), 2), (dict(d=1025), 2), (dict(T=0), 0), (dict(T=0, q=None, qo=None), 0),
])
def test_rotary_rejects_bad_arguments(lib, bad, code):
    assert _rotary(lib, **bad) == code


def test_rotary_rejects_a_missing_list_of_pairs(lib):
    a = (P[0], P[1], P[2], P[3], 1, 128, 2, 64, None, 1, 0, 0, P[4], P[5], None)
    assert lib.la_rotary(*a) == 1


def _decay(lib, **kw):
    a = dict(q=P[0], k=P[1], v=P[2], ld=P[3], dt=1, cu=None, nseq=1, T=128, H=2, dk=64, dv=32, scale=1.0, si=None, so=None,
             out=P[4], ws=P[5], bytes=1 << 26, stream=None)
    a.update(kw)
    return lib.la_decay_attention(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(dt=2), 1), (dict(nseq=0), 1), (dict(nseq=65536), 1), (dict(T=-1), 1), (dict(T=1 << 31), 1), (dict(H=0), 1),
    (dict(H=65536), 1), (dict(dk=0), 1), (dict(dv=0), 1), (dict(dk=257), 2), (dict(dv=257), 2), (dict(T=130, nseq=4), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(ld=None), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(ws=P[5] + 16), 1), (dict(bytes=255), 3),
    (dict(q=P[0] + 1), 1), (dict(v=P[2] + 1), 1), (dict(ld=P[3] + 2), 1), (dict(si=P[6] + 2), 1), (dict(so=P[6] + 2), 1),
    (dict(cu=P[6] + 2), 1), (dict(out=P[0]), 1), (dict(out=P[2]), 1), (dict(so=P[1] + 4), 1), (dict(out=P[3] - 2), 1),
    (dict(si=P[6], so=P[6] + 4), 1), (dict(out=P[5] + 64), 1), (dict(cu=P[4]), 1),
])
def test_decay_attention_rejects_bad_arguments(lib, bad, code):
    assert _decay(lib, **bad) == code


def _decay_bwd(lib, **kw):
    a = dict(q=P[0], k=P[1], v=P[2], do=P[3], ld=P[4], dt=1, cu=None, nseq=1, T=128, H=2, dk=64, dv=32, scale=1.0, si=None,
             dso=None, dq=P[5], dk_=P[6], dv_=P[7], dsi=None, ws=P[8], bytes=1 << 26, stream=None)
    a.update(kw)
    return lib.la_decay_attention_backward(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(dt=-1), 1), (dict(nseq=0), 1), (dict(T=1 << 31), 1), (dict(H=0), 1), (dict(dk=257), 2), (dict(dv=0), 1),
    (dict(T=130, nseq=4), 1), (dict(scale=float("inf")), 1), (dict(q=None), 1), (dict(do=None), 1), (dict(ld=None), 1),
    (dict(dq=None), 1), (dict(dk_=None), 1), (dict(dv_=None), 1), (dict(ws=None), 1), (dict(ws=P[8] + 8), 1),
    (dict(bytes=255), 3), (dict(do=P[3] + 1), 1), (dict(dv_=P[7] + 1), 1), (dict(dso=P[9] + 2), 1), (dict(dsi=P[9] + 1), 1),
    (dict(dq=P[0]), 1), (dict(dk_=P[5]), 1), (dict(dv_=P[3]), 1), (dict(dso=P[9], dsi=P[9] + 4), 1),
    (dict(si=P[9], dsi=P[9]), 1), (dict(dq=P[8] + 64), 1),
])
def test_decay_attention_backward_rejects_bad_arguments(lib, bad, code):
    assert _decay_bwd(lib, **bad) == code


def _decay_step(lib, **kw):
    a = dict(q=P[0], k=P[1], v=P[2], ld=P[3], dt=1, B=4, H=2, dk=64, dv=32, scale=1.0, si=P[4], so=P[4], out=P[5],
             stream=None)
    a.update(kw)
    return lib.la_decay_step(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(dt=3), 1), (dict(B=-1), 1), (dict(H=0), 1), (dict(dk=0), 1), (dict(dk=257), 2), (dict(dv=257), 2),
    (dict(B=1 << 20, H=1 << 12), 2), (dict(scale=float("nan")), 1), (dict(q=None), 1), (dict(ld=None), 1),
    (dict(si=None), 1), (dict(so=None), 1), (dict(out=None), 1), (dict(si=P[4] + 2), 1), (dict(k=P[1] + 1), 1),
    (dict(so=P[4] + 4), 1), (dict(out=P[0]), 1), (dict(so=P[0]), 1), (dict(B=0), 0), (dict(B=0, q=None), 0),
])
def test_decay_step_rejects_bad_arguments(lib, bad, code):
    assert _decay_step(lib, **bad) == code


def test_decay_workspace_queries(lib):
    import kernelized_linear_attention_gb300 as la
    for query in (la.la_decay_attention_workspace_bytes, la.la_decay_attention_backward_workspace_bytes):
        assert query(torch.bfloat16, False, 3, 100, 2, 64, 64) == 0
        assert query(torch.bfloat16, True, 3, 100, 2, 64, 64) > 0
        assert query(torch.bfloat16, True, 1, 0, 1, 1, 1) > 0
        assert query(torch.bfloat16, True, 1, 10, 2, 300, 64) == 0
        # states are kept between segments only, not for each of many short sequences
        assert query(torch.bfloat16, True, 60000, 60000, 16, 64, 64) < 1 << 30
    assert (la.la_decay_attention_backward_workspace_bytes(torch.float32, True, 1, 100000, 2, 64, 64)
            > la.la_decay_attention_workspace_bytes(torch.float32, True, 1, 100000, 2, 64, 64))


def _qk(lib, pairs=(16, 16), **kw):
    a = dict(q=P[0], k=P[1], qw=P[2], kw_=P[3], freq=P[4], pos=P[5], dt=1, T=128, Hq=4, Hk=2, d=64, qs=256, ks=128,
             pairs=(ctypes.c_int * max(1, len(pairs)))(*pairs), naxes=len(pairs), il=0, per=0, eps=1e-6, qo=P[6], ko=P[7],
             qr=P[8], kr=P[9], stream=None)
    a.update(kw)
    return lib.la_qk_norm_rotary(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(dt=2), 1), (dict(T=-1), 1), (dict(T=1 << 31), 1), (dict(Hq=0), 1), (dict(Hk=-1), 1), (dict(d=1), 1), (dict(per=2), 1),
    (dict(qs=255), 1), (dict(ks=127), 1), (dict(qs=1 << 31), 2), (dict(naxes=0), 1), (dict(pairs=(0, 0)), 1),
    (dict(pairs=(16, 17)), 1), (dict(pairs=(-1, 4)), 1), (dict(pairs=(1,) * 5), 2), (dict(d=1025, qs=4100, ks=2050), 2),
    (dict(Hq=20000, d=64, qs=1280000), 2), (dict(il=2), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(q=None), 1), (dict(k=None), 1), (dict(qo=None), 1), (dict(ko=None), 1), (dict(freq=None), 1), (dict(pos=None), 1),
    (dict(Hk=0, ks=0), 1), (dict(q=P[0] + 1), 1), (dict(qw=P[2] + 2), 1), (dict(kr=P[9] + 2), 1), (dict(pos=P[5] + 2), 1),
    (dict(qo=P[0] + 2), 1), (dict(qo=P[1]), 1), (dict(ko=P[6]), 1), (dict(qo=P[2]), 1), (dict(qr=P[6]), 1),
    (dict(qo=P[0], qs=512), 1),                                  # in place only where rows are contiguous
    (dict(q=P[6] - 100 * 512, qs=512), 1),                       # the output inside a strided input
    (dict(T=0), 0), (dict(T=0, q=None, qo=None), 0),
])
def test_qk_norm_rotary_rejects_bad_arguments(lib, bad, code):
    assert _qk(lib, **bad) == code


def _qk_bwd(lib, pairs=(16, 16), **kw):
    a = dict(q=P[0], k=P[1], qr=P[2], kr=P[3], dqo=P[4], dko=P[5], qw=P[6], kw_=P[7], freq=P[8], pos=P[9], dt=1, T=128, Hq=4,
             Hk=2, d=64, qs=256, ks=128, pairs=(ctypes.c_int * max(1, len(pairs)))(*pairs), naxes=len(pairs), il=0, per=0,
             dq=P[10], dk=P[11], dqw=P[12], dkw=P[13], ws=P[14], bytes=1 << 27, stream=None)
    a.update(kw)
    return lib.la_qk_norm_rotary_backward(*a.values())


@pytest.mark.parametrize("bad,code", [
    (dict(dt=-1), 1), (dict(T=-1), 1), (dict(Hq=0), 1), (dict(d=1), 1), (dict(qs=200), 1), (dict(per=-1), 1),
    (dict(pairs=(16, 17)), 1), (dict(il=3), 1), (dict(ws=None), 1), (dict(ws=P[14] + 8), 1), (dict(q=None), 1),
    (dict(qr=None), 1), (dict(kr=None), 1), (dict(dqo=None), 1), (dict(dk=None), 1), (dict(Hk=0, ks=0), 1),
    (dict(dq=P[10] + 1), 1), (dict(dqw=P[12] + 2), 1), (dict(d=1025, qs=4100, ks=2050), 2),
])
def test_qk_norm_rotary_backward_rejects_bad_arguments(lib, bad, code):
    assert _qk_bwd(lib, **bad) == code


def test_decay_binding_refuses_what_does_not_fit():
    import kernelized_linear_attention_gb300 as la
    x, ld = torch.zeros(4, 2, 8), torch.zeros(2)
    for call in (lambda: la.la_decay_attention(x, x, x, ld), lambda: la.la_decay_attention_backward(x, x, x, x, ld),
                 lambda: la.la_decay_step(x, x, x, ld, torch.zeros(4, 2, 8, 8)),
                 lambda: la.la_decay_attention(x[0], x, x, ld),
                 lambda: la.la_decay_attention(x, x, x, ld, cu_seqlens=torch.zeros(3, dtype=torch.int32), nseq=5)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        la.la_decay_attention(None, x, x, ld)


def test_binding_refuses_cpu_tensors_and_wrong_ranks():
    import kernelized_linear_attention_gb300 as la
    x = torch.zeros(4, 2, 8)
    with pytest.raises(ValueError):
        la.la_gated_scan(x, x)
    with pytest.raises(ValueError):
        la.la_gated_scan_backward(x, x, x)
    with pytest.raises(ValueError):
        la.la_gated_step(x, x, x)
    with pytest.raises(ValueError):
        la.la_layer_norm(x)
    with pytest.raises(ValueError):
        la.la_layer_norm_backward(x, x, x[..., 0].contiguous(), x[..., 0].contiguous(), x[0, 0])
    with pytest.raises(ValueError):
        la.la_rotary(x, x, torch.zeros(4), torch.zeros(4, 1, dtype=torch.int32), [4])
    with pytest.raises(ValueError):
        la.la_gated_scan(x[0], x[0])
    with pytest.raises(TypeError):
        la.la_gated_scan(None, None)
    with pytest.raises(ValueError):
        la.la_gated_scan(x, x, cu_seqlens=torch.zeros(3, dtype=torch.int32), nseq=5)


def test_decay_attention_of_the_most_tokens(lib):
    # chunks end behind the last token: their ends are 32-bit numbers too
    import kernelized_linear_attention_gb300 as la
    most = (1 << 31) - 1025
    for T, code, some in ((most, 3, True), (most + 1, 2, False), ((1 << 31) - 1, 2, False)):
        assert _decay(lib, T=T, H=1, dk=1, dv=1, q=P[0], k=P[0], v=P[0], out=P[0] + (1 << 40), bytes=0) == code
        for cu in (False, True):
            assert (la.la_decay_attention_workspace_bytes(torch.float32, cu, 1, T, 1, 1, 1) > 0) == some
            assert (la.la_decay_attention_backward_workspace_bytes(torch.bfloat16, cu, 1, T, 1, 8, 8) > 0) == some


def test_decay_segments_end(lib):
    """A state on the tensor cores takes 32768 tokens at most before it is begun anew, however many heads there are."""
    import kernelized_linear_attention_gb300 as la
    for cu in (False, True):
        for T, H in ((1 << 20, 400), (1 << 20, 7), (33000, 400)):
            few = la.la_decay_attention_workspace_bytes(torch.bfloat16, cu, 1, T, H, 64, 64)
            assert few >= (-(-T // 32768) - 1) * H * 64 * 64 * 4
