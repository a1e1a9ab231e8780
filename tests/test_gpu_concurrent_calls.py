"""Two host threads call the same entry point at once, each on a stream and in a workspace of its own, with sizes that
need different amounts of shared memory of the same kernel: both succeed, however they interleave."""
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

CALLS = 5000


@pytest.fixture(scope="module")
def la():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import kernelized_linear_attention_gb300 as m
    m.load_library()
    return m


def _normal(*shape, dtype=torch.float32, scale=0.3):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(sum(shape)))).to(dtype).cuda()


def _decay(la, d):
    q, k, v = (_normal(40, 1, d) for _ in range(3))
    ld, out = torch.full((1,), -0.1, device="cuda"), torch.empty_like(q)
    w = torch.empty(la.la_decay_attention_workspace_bytes(torch.float32, False, 1, 40, 1, d, d), dtype=torch.uint8,
                    device="cuda")
    return lambda: [la.la_decay_attention(q, k, v, ld, nseq=1, out=out, workspace=w)]


def _decay_backward(la, d):
    q, k, v, do = (_normal(40, 1, d) for _ in range(4))
    ld, grads = torch.full((1,), -0.1, device="cuda"), [torch.empty_like(q) for _ in range(3)]
    w = torch.empty(la.la_decay_attention_backward_workspace_bytes(torch.float32, False, 1, 40, 1, d, d),
                    dtype=torch.uint8, device="cuda")
    return lambda: list(la.la_decay_attention_backward(q, k, v, do, ld, nseq=1, dq=grads[0], dk=grads[1], dv=grads[2],
                                                       workspace=w))


def _qk(la, d):
    q, out = _normal(40, 1, d), torch.empty(40, 1, d, device="cuda")
    freq, pos = torch.ones(d // 2, device="cuda"), torch.arange(40, dtype=torch.int32, device="cuda")
    return lambda: [la.la_qk_norm_rotary(q, None, None, None, freq, pos, (d // 2,), q_out=out)[0]]


def _qk_backward(la, d):
    q, dy, dq = _normal(40, 1, d), _normal(40, 1, d), torch.empty(40, 1, d, device="cuda")
    freq, pos = torch.ones(d // 2, device="cuda"), torch.arange(40, dtype=torch.int32, device="cuda")
    rstd = torch.ones(40, 1, device="cuda")
    w = torch.empty(la.la_qk_norm_rotary_backward_workspace_bytes(torch.float32, 40, 1, 0, d), dtype=torch.uint8,
                    device="cuda")
    return lambda: [la.la_qk_norm_rotary_backward(q, None, rstd, None, dy, None, None, None, freq, pos, (d // 2,), dq=dq,
                                                  workspace=w)[0]]


def _forward(la, d):
    q, k, v = (_normal(40, 1, d) for _ in range(3))
    out = torch.empty_like(q)
    w = torch.empty(la.la_workspace_bytes(True, "elu1", torch.float32, False, 1, 40, 1, d, d, d), dtype=torch.uint8,
                    device="cuda")
    return lambda: [la.la_forward_causal(q, k, v, "elu1", nseq=1, out=out, workspace=w)]


def _backward(la, d):
    q, k, v, do = (_normal(40, 1, d) for _ in range(4))
    grads = [torch.empty_like(q) for _ in range(3)]
    w = torch.empty(la.la_backward_workspace_bytes(True, "elu1", torch.float32, False, 1, 40, 1, d, d, d),
                    dtype=torch.uint8, device="cuda")
    return lambda: list(la.la_backward(q, k, v, do, "elu1", nseq=1, dq=grads[0], dk=grads[1], dv=grads[2], workspace=w))


def _feature_map(la, d):
    x, omega, phi = _normal(40, 1, d), _normal(64, d), torch.empty(40, 1, 64, device="cuda")
    return lambda: [la.la_feature_map(x, "favor", omega, phi=phi)]


def _decode(la, r):
    q, k, v, omega = _normal(4, 1, 256), _normal(4, 1, 256), _normal(4, 1, 256), _normal(r, 256, scale=0.1)
    state, out = torch.zeros(4, 1, r, 257, device="cuda"), torch.empty(4, 1, 256, device="cuda")
    return lambda: [la.la_decode_step(q, k, v, state, "favor", omega, out=out)]


def _features(la, d):
    g = torch.Generator().manual_seed(d)
    blocks = torch.randn(1, d, d, generator=g, dtype=torch.float64).cuda()
    lengths = torch.randn(1, d, d, generator=g, dtype=torch.float64).cuda()
    omega = torch.empty(d, d, device="cuda")
    return lambda: [la.la_orthogonal_features(blocks, lengths, d, omega=omega)]


class _Recorder:
    """The library with its calls written down: entry point and arguments as it gets them."""

    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        fn = getattr(self.lib, name)

        def call(*a):
            self.calls.append((fn, a))
            return fn(*a)
        return call


@pytest.mark.parametrize("make,narrow,wide", [
    (_decay, 32, 256), (_decay_backward, 32, 256), (_qk, 1000, 1024), (_qk_backward, 1000, 1024), (_forward, 16, 128),
    (_backward, 16, 112), (_feature_map, 16, 128), (_decode, 320, 512), (_features, 16, 128)],
    ids=lambda v: getattr(v, "__name__", str(v)))
def test_calls_of_two_threads(la, monkeypatch, make, narrow, wide):
    """The calls as the binding makes them, without its own time between them."""
    from kernelized_linear_attention_gb300 import _binding
    streams, calls, results, want = [torch.cuda.Stream() for _ in range(2)], [], [], []
    torch.cuda.synchronize()
    for size, stream in zip((narrow, wide), streams):
        with torch.cuda.stream(stream):
            call = make(la, size)
            stream.synchronize()
            lib = _Recorder(_binding.load_library())
            with monkeypatch.context() as m:
                m.setattr(_binding, "_lib", lib)
                results.append(call())
            calls.append([c for c in lib.calls if not c[0].__name__.endswith("_bytes")][-1])
            stream.synchronize()
            want.append([x.clone() for x in results[-1]])
    torch.cuda.synchronize()
    failures, start = [], threading.Barrier(2)

    def work(fn, args):
        start.wait()
        for _ in range(CALLS):
            status = fn(*args)
            if status != 0:
                failures.append(f"{fn.__name__}: status {status}")
                return

    threads = [threading.Thread(target=work, args=c) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failures, failures
    if make is not _decode:              # (whose state goes on from call to call)
        assert all(torch.equal(x, y) for r, w in zip(results, want) for x, y in zip(r, w))
