"""ctypes binding of liblinattn.so (argument marshalling only)."""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "lib", "liblinattn.so")

MAP_IDS = {"identity": 0, "elu1": 1, "favor": 2, "dpfp": 3}
DTYPE_IDS = {torch.float32: 0, torch.bfloat16: 1}
NORM_IDS = {"attention": 0, "none": 1, "sum": 2}

LA_OK = 0
_c_i64, _c_int, _c_float, _c_size, _vp = ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_void_p

_lib = None


class LinAttnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status} ({la_status_string(status)})")
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load liblinattn.so once.  Raises if it was not built: there is no fallback."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(
            f"{_LIB_PATH} is missing: build it with `python -c \"import __graft_entry__ as g; g.build()\"` "
            "(kernelized linear attention has no CPU fallback)")
    lib = ctypes.CDLL(_LIB_PATH)
    fwd_args = [_vp, _vp, _vp, _vp, _c_int, _c_int, _vp, _c_int, _c_i64, _c_int, _c_int, _c_int, _c_int,
                _c_float, _vp, _vp, _c_size, _vp]
    sigs = {
        "la_feature_map": ([_vp, _vp, _c_int, _c_int, _c_i64, _c_int, _c_int, _c_int, _vp, _vp], _c_int),
        "la_forward_bidir": (fwd_args, _c_int),
        "la_forward_causal": (fwd_args, _c_int),
        "la_forward_phase": ([_c_int, _c_int, _c_int] + fwd_args[:14] + [_vp, _vp] + fwd_args[14:]
                             + [ctypes.POINTER(_c_int)], _c_int),
        "la_forward": ([_c_int, _c_int] + fwd_args[:14] + [_vp, _vp] + fwd_args[14:], _c_int),
        "la_backward": ([_c_int, _c_int] + fwd_args[:14] + [_vp, _vp, _vp, _vp] + fwd_args[15:], _c_int),
        "la_backward_workspace_bytes": ([_c_int, _c_int, _c_int, _c_int, _c_int, _c_i64, _c_int, _c_int, _c_int,
                                         _c_int], _c_size),
        "la_decode_step": ([_vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                            _c_float, _vp, _vp, _vp], _c_int),
        "la_forward_causal_noalloc": (fwd_args[:15] + [_vp], _c_int),
        "la_noalloc_error": ([ctypes.POINTER(_c_int), _vp], _c_int),
        "la_test_force_wait_timeout": ([_c_int], _c_int),
        "la_test_segment_plan": ([_c_i64, _c_i64, _c_int, _c_i64, ctypes.POINTER(_c_i64)], _c_i64),
        "la_workspace_bytes": ([_c_int, _c_int, _c_int, _c_int, _c_int, _c_i64, _c_int, _c_int, _c_int, _c_int],
                               _c_size),
        "la_check_cu_seqlens": ([_vp, _c_int, _c_i64, _vp], _c_int),
        "la_workspace_error": ([_vp, ctypes.POINTER(_c_int), _vp], _c_int),
        "la_orthogonal_features": ([_vp, _vp, _c_int, _c_int, _vp, _vp], _c_int),
        "la_selected_path": ([_c_int, _c_int, _c_int, _c_int, _c_int, _c_int], _c_int),
        "la_gated_scan": ([_vp, _vp, _c_int, _c_int, _vp, _c_int, _c_i64, _c_int, _c_int, _vp, _vp, _vp, _vp, _c_size,
                           _vp], _c_int),
        "la_gated_scan_backward": ([_vp, _vp, _vp, _c_int, _c_int, _vp, _c_int, _c_i64, _c_int, _c_int, _vp, _vp, _vp,
                                    _vp, _vp, _vp, _c_size, _vp], _c_int),
        "la_gated_scan_workspace_bytes": ([_c_int, _c_int, _c_i64, _c_int, _c_int], _c_size),
        "la_gated_step": ([_vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp], _c_int),
        "la_layer_norm": ([_vp, _vp, _vp, _c_int, _c_i64, _c_int, _c_int, _c_float, _vp, _vp, _vp, _vp], _c_int),
        "la_layer_norm_backward": ([_vp, _vp, _vp, _vp, _vp, _c_int, _c_i64, _c_int, _c_int, _vp, _vp, _vp, _vp,
                                    _c_size, _vp], _c_int),
        "la_layer_norm_backward_workspace_bytes": ([_c_int, _c_i64, _c_int, _c_int], _c_size),
        "la_rotary": ([_vp, _vp, _vp, _vp, _c_int, _c_i64, _c_int, _c_int, ctypes.POINTER(_c_int), _c_int, _c_int,
                       _c_int, _vp, _vp, _vp], _c_int),
        "la_qk_norm_rotary": ([_vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_i64, _c_int, _c_int, _c_int, _c_i64, _c_i64,
                               ctypes.POINTER(_c_int), _c_int, _c_int, _c_int, _c_float, _vp, _vp, _vp, _vp, _vp], _c_int),
        "la_qk_norm_rotary_backward": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_int, _c_i64, _c_int, _c_int,
                                        _c_int, _c_i64, _c_i64, ctypes.POINTER(_c_int), _c_int, _c_int, _c_int, _vp, _vp,
                                        _vp, _vp, _vp, _c_size, _vp], _c_int),
        "la_qk_norm_rotary_backward_workspace_bytes": ([_c_int, _c_i64, _c_int, _c_int, _c_int], _c_size),
        "la_decay_attention": ([_vp, _vp, _vp, _vp, _c_int, _vp, _c_int, _c_i64, _c_int, _c_int, _c_int, _c_float, _vp,
                                _vp, _vp, _vp, _c_size, _vp], _c_int),
        "la_decay_attention_workspace_bytes": ([_c_int, _c_int, _c_int, _c_i64, _c_int, _c_int, _c_int], _c_size),
        "la_decay_attention_backward": ([_vp, _vp, _vp, _vp, _vp, _c_int, _vp, _c_int, _c_i64, _c_int, _c_int, _c_int,
                                         _c_float, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_size, _vp], _c_int),
        "la_decay_attention_backward_workspace_bytes": ([_c_int, _c_int, _c_int, _c_i64, _c_int, _c_int, _c_int],
                                                        _c_size),
        "la_decay_step": ([_vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _c_float, _vp, _vp, _vp, _vp],
                          _c_int),
        "la_status_string": ([_c_int], ctypes.c_char_p),
        "la_version": ([], _c_int),
    }
    for name, (argtypes, restype) in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = argtypes
        fn.restype = restype
    _lib = lib
    return lib


def _check(fn: str, status: int):
    if status != LA_OK:
        raise LinAttnError(fn, status)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype=None, cuda=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _holds(n: int, **tensors):
    """Every tensor that is given has the n elements that the call reads or writes."""
    for name, t in tensors.items():
        if t is not None and t.numel() < n:
            raise ValueError(f"{name} must have {n} elements, got {tuple(t.shape)}")


def _map_id(m) -> int:
    """Map id from a name ("identity", "elu1", "favor", "dpfp<nu>") or an id."""
    if isinstance(m, str):
        return MAP_IDS["dpfp"] if m.startswith("dpfp") else MAP_IDS[m]
    return int(m)


def _norm_id(n) -> int:
    """Normalisation id from a name ("attention", "none", "sum") or an id."""
    return NORM_IDS[n] if isinstance(n, str) else int(n)


def _feature_dim(m, d_k: int, omega) -> int:
    """r of a map: Omega's rows (FAVOR+), 2 d_k nu (DPFP-nu, named "dpfp<nu>"), else d_k."""
    if _map_id(m) == MAP_IDS["favor"]:
        return omega.shape[0]
    if _map_id(m) == MAP_IDS["dpfp"]:
        if not (isinstance(m, str) and m[4:].isdigit()):
            raise ValueError('the DPFP map is named "dpfp<nu>", e.g. "dpfp2"')
        return 2 * d_k * int(m[4:])
    return d_k


def la_status_string(status: int) -> str:
    return load_library().la_status_string(int(status)).decode()


def la_version() -> int:
    return load_library().la_version()


def la_selected_path(causal: bool, map, dtype, d_k: int, d_v: int, r: int) -> int:
    dt = DTYPE_IDS[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return load_library().la_selected_path(int(causal), _map_id(map), dt, d_k, d_v, r)


def la_workspace_bytes(causal: bool, map, dtype, has_cu_seqlens: bool, nseq: int, T: int, H: int,
                       d_k: int, d_v: int, r: int) -> int:
    dt = DTYPE_IDS[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return load_library().la_workspace_bytes(int(causal), _map_id(map), dt, int(has_cu_seqlens), nseq, T, H,
                                             d_k, d_v, r)


def la_feature_map(x: torch.Tensor, map, omega: Optional[torch.Tensor] = None,
                   phi: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """phi(x) for x [T, H, d] (fp32 or bf16) -> fp32 [T, H, r]."""
    lib = load_library()
    _need(x, "x")
    m = _map_id(map)
    T, H, d = x.shape
    r = _feature_dim(map, d, omega)
    if omega is not None:
        _need(omega, "omega", torch.float32)
    if phi is None:
        phi = torch.empty((T, H, r), dtype=torch.float32, device=x.device)
    _need(phi, "phi", torch.float32)
    _holds(T * H * r, phi=phi)
    _holds(r * d, omega=omega if m == MAP_IDS["favor"] else None)
    _check("la_feature_map", lib.la_feature_map(_ptr(x), _ptr(omega), m, DTYPE_IDS[x.dtype], T, H, d, r,
                                                _ptr(phi), _stream(stream)))
    return phi


def forward_ptrs(causal: bool, q, k, v, omega, map, dtype, cu_seqlens, nseq, T, H, d_k, d_v, r, eps,
                 out, workspace, workspace_bytes, stream) -> None:
    """Raw call with integer device pointers (for callers that manage memory)."""
    lib = load_library()
    fn = lib.la_forward_causal if causal else lib.la_forward_bidir
    dt = DTYPE_IDS[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    _check(fn.__name__, fn(q, k, v, omega, _map_id(map), dt, cu_seqlens, nseq, T, H, d_k, d_v, r, eps,
                           out, workspace, workspace_bytes, _stream(stream)))


def forward_general_ptrs(causal: bool, q, k, v, omega, map, dtype, cu_seqlens, nseq, T, H, d_k, d_v, r, eps,
                         out, workspace, workspace_bytes, stream, norm="attention", state_in=None,
                         state_out=None) -> None:
    """Raw la_forward call with integer device pointers (state_in / state_out too)."""
    dt = DTYPE_IDS[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    _check("la_forward", load_library().la_forward(int(causal), _norm_id(norm), q, k, v, omega, _map_id(map), dt,
                                                   cu_seqlens, nseq, T, H, d_k, d_v, r, eps, state_in, state_out,
                                                   out, workspace, workspace_bytes, _stream(stream)))


def la_forward_phase(causal: bool, phase: int, q, k, v, omega, map, dtype, cu_seqlens, nseq, T, H, d_k, d_v, r,
                     eps, out, workspace, workspace_bytes, stream=None, norm="attention", state_in=None,
                     state_out=None) -> int:
    """One phase (0 plan, 1 state, 2 scan, 3 output) with integer device
    pointers (state_in / state_out too); returns the number of kernels it
    enqueued."""
    lib = load_library()
    dt = DTYPE_IDS[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    n = _c_int(0)
    _check("la_forward_phase", lib.la_forward_phase(int(causal), int(phase), _norm_id(norm), q, k, v, omega,
                                                    _map_id(map), dt, cu_seqlens, nseq, T, H, d_k, d_v, r, eps,
                                                    state_in, state_out, out, workspace, workspace_bytes,
                                                    _stream(stream), ctypes.byref(n)))
    return n.value


def la_forward_causal_noalloc(q, k, v, map, omega=None, cu_seqlens=None, nseq=None, eps=1e-6, out=None,
                              stream=None) -> torch.Tensor:
    """Causal forward whose scratch is the library's fixed device array (no
    workspace, no device allocation inside the library); see
    include/linattn.h for the sharing rules."""
    _need(q, "q"); _need(k, "k"); _need(v, "v")
    T, H, d_k = q.shape
    d_v = v.shape[2]
    m = _map_id(map)
    r = _feature_dim(map, d_k, omega)
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32)
        nseq = cu_seqlens.numel() - 1
    elif nseq is None:
        nseq = 1
    if out is None:
        out = torch.empty((T, H, d_v), dtype=q.dtype, device=q.device)
    _need(out, "out", q.dtype)
    _holds(T * H * d_k, k=k)
    _holds(T * H * d_v, v=v, out=out)
    _holds(r * d_k, omega=omega if m == MAP_IDS["favor"] else None)
    _check("la_forward_causal_noalloc", load_library().la_forward_causal_noalloc(
        _ptr(q), _ptr(k), _ptr(v), _ptr(omega), m, DTYPE_IDS[q.dtype], _ptr(cu_seqlens), nseq, T, H, d_k, d_v, r,
        eps, _ptr(out), _stream(stream)))
    return out


def la_test_force_wait_timeout(enable: bool) -> None:
    """Test hook: while enabled, the causal tensor-core output kernel's bounded waits are made
    to run out (it records LA_DEVERR_WAIT_TIMEOUT and returns); see include/linattn.h."""
    st = load_library().la_test_force_wait_timeout(1 if enable else 0)
    if st != LA_OK:
        raise LinAttnError("la_test_force_wait_timeout", st)


def la_test_segment_plan(nchunks: int, pairs: int, nsm: int, force_chunks: int = 0):
    """Test hook (host only): (segment length in chunks, simulated makespan in chunk times)
    the tensor-core planner chooses, or evaluates for force_chunks; see include/linattn.h."""
    ms = _c_i64(0)
    lc = load_library().la_test_segment_plan(nchunks, pairs, nsm, force_chunks, ctypes.byref(ms))
    if lc < 0:
        raise ValueError("la_test_segment_plan: nchunks, pairs and nsm must be at least 1")
    return int(lc), int(ms.value)


def la_noalloc_error(stream=None) -> int:
    """Device error code the latest la_forward_causal_noalloc call on the current
    device recorded in the library's scratch array (0 = none; synchronises)."""
    code = _c_int(0)
    st = load_library().la_noalloc_error(ctypes.byref(code), _stream(stream))
    if st not in (LA_OK, 5):
        raise LinAttnError("la_noalloc_error", st)
    return code.value


def _forward(causal, q, k, v, map, omega, cu_seqlens, nseq, eps, out, workspace, stream, norm="attention",
             state_in=None, state_out=None):
    _need(q, "q"); _need(k, "k"); _need(v, "v")
    if q.dtype not in DTYPE_IDS or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share dtype float32 or bfloat16")
    T, H, d_k = q.shape
    d_v = v.shape[2]
    m = _map_id(map)
    r = _feature_dim(map, d_k, omega)
    if omega is not None:
        _need(omega, "omega", torch.float32)
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32)
        nseq = cu_seqlens.numel() - 1
    elif nseq is None:
        nseq = 1
    for name, st in (("state_in", state_in), ("state_out", state_out)):
        if st is not None:
            _need(st, name, torch.float32)
            if tuple(st.shape) != (nseq, H, r, d_v + 1):
                raise ValueError(f"{name} must have shape {(nseq, H, r, d_v + 1)}, got {tuple(st.shape)}")
    if out is None:
        out = torch.empty((T, H, d_v), dtype=q.dtype, device=q.device)
    _need(out, "out", q.dtype)
    _holds(T * H * d_k, k=k)
    _holds(T * H * d_v, v=v, out=out)
    _holds(r * d_k, omega=omega if m == MAP_IDS["favor"] else None)
    need = la_workspace_bytes(causal, m, q.dtype, cu_seqlens is not None, nseq, T, H, d_k, d_v, r)
    if workspace is None:
        # a size of 0 means the call will be rejected: let the library say why
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    nid = _norm_id(norm)
    if nid == NORM_IDS["attention"] and state_in is None and state_out is None:
        forward_ptrs(causal, _ptr(q), _ptr(k), _ptr(v), _ptr(omega), m, q.dtype, _ptr(cu_seqlens), nseq, T, H,
                     d_k, d_v, r, eps, _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                     stream)
    else:
        _check("la_forward", load_library().la_forward(
            int(causal), nid, _ptr(q), _ptr(k), _ptr(v), _ptr(omega), m, DTYPE_IDS[q.dtype], _ptr(cu_seqlens),
            nseq, T, H, d_k, d_v, r, eps, _ptr(state_in), _ptr(state_out), _ptr(out), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream)))
    return out, workspace


def la_forward_bidir(q, k, v, map, omega=None, cu_seqlens=None, nseq=None, eps=1e-6, out=None,
                     workspace=None, stream=None) -> torch.Tensor:
    """Bidirectional kernelized attention; returns out [T, H, d_v] (dtype of q)."""
    return _forward(False, q, k, v, map, omega, cu_seqlens, nseq, eps, out, workspace, stream)[0]


def la_forward_causal(q, k, v, map, omega=None, cu_seqlens=None, nseq=None, eps=1e-6, out=None,
                      workspace=None, stream=None) -> torch.Tensor:
    """Causal kernelized attention; returns out [T, H, d_v] (dtype of q)."""
    return _forward(True, q, k, v, map, omega, cu_seqlens, nseq, eps, out, workspace, stream)[0]


def la_forward(q, k, v, map, omega=None, causal=True, norm="attention", cu_seqlens=None, nseq=None, eps=1e-6,
               state_in=None, state_out=None, return_state=False, out=None, workspace=None, stream=None):
    """General forward: norm "attention" | "none" | "sum", optional carried
    state.  state_in / state_out: fp32 [nseq, H, r, d_v + 1] (row f: S[f, :]
    then z[f]).  With return_state=True a state_out is allocated when none is
    given and (out, state_out) is returned."""
    if return_state and state_out is None:
        T, H, d_k = q.shape
        nn = cu_seqlens.numel() - 1 if cu_seqlens is not None else (nseq or 1)
        r = _feature_dim(map, d_k, omega)
        state_out = torch.empty((nn, H, r, v.shape[2] + 1), dtype=torch.float32, device=q.device)
    o = _forward(bool(causal), q, k, v, map, omega, cu_seqlens, nseq, eps, out, workspace, stream, norm=norm,
                 state_in=state_in, state_out=state_out)[0]
    return (o, state_out) if return_state else o


def la_decode_step(q, k, v, state, map, omega=None, norm="attention", eps=1e-6, out=None, stream=None):
    """One token per sequence: q, k [B, H, d_k], v [B, H, d_v]; state fp32
    [B, H, r, d_v + 1] is updated in place; returns out [B, H, d_v]."""
    _need(q, "q"); _need(k, "k"); _need(v, "v"); _need(state, "state", torch.float32)
    if q.dtype not in DTYPE_IDS or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share dtype float32 or bfloat16")
    B, H, d_k = q.shape
    d_v = v.shape[2]
    r = _feature_dim(map, d_k, omega)
    if tuple(state.shape) != (B, H, r, d_v + 1):
        raise ValueError(f"state must have shape {(B, H, r, d_v + 1)}, got {tuple(state.shape)}")
    if omega is not None:
        _need(omega, "omega", torch.float32)
    if out is None:
        out = torch.empty((B, H, d_v), dtype=q.dtype, device=q.device)
    _need(out, "out", q.dtype)
    _holds(B * H * d_k, k=k)
    _holds(B * H * d_v, v=v, out=out)
    _holds(r * d_k, omega=omega if _map_id(map) == MAP_IDS["favor"] else None)
    _check("la_decode_step", load_library().la_decode_step(
        _ptr(q), _ptr(k), _ptr(v), _ptr(omega), _map_id(map), DTYPE_IDS[q.dtype], _norm_id(norm), B, H, d_k, d_v,
        r, eps, _ptr(state), _ptr(out), _stream(stream)))
    return out


def la_backward_workspace_bytes(causal: bool, map, dtype, has_cu_seqlens: bool, nseq: int, T: int, H: int,
                                d_k: int, d_v: int, r: int) -> int:
    dt = DTYPE_IDS[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return load_library().la_backward_workspace_bytes(int(causal), _map_id(map), dt, int(has_cu_seqlens), nseq, T,
                                                      H, d_k, d_v, r)


def la_backward(q, k, v, dout, map, omega=None, causal=True, norm="attention", cu_seqlens=None, nseq=None,
                eps=1e-6, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients (dq, dk, dv) of sum(dout * out) for the forward with the same
    arguments; allocates what is not given."""
    _need(q, "q"); _need(k, "k"); _need(v, "v"); _need(dout, "dout")
    if q.dtype not in DTYPE_IDS or any(t.dtype != q.dtype for t in (k, v, dout)):
        raise ValueError("q, k, v, dout must share dtype float32 or bfloat16")
    T, H, d_k = q.shape
    d_v = v.shape[2]
    m = _map_id(map)
    r = _feature_dim(map, d_k, omega)
    if omega is not None:
        _need(omega, "omega", torch.float32)
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32)
        nseq = cu_seqlens.numel() - 1
    elif nseq is None:
        nseq = 1
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _need(t, name, q.dtype)
    _holds(T * H * d_k, k=k, dq=dq, dk=dk)
    _holds(T * H * d_v, v=v, dout=dout, dv=dv)
    _holds(r * d_k, omega=omega if m == MAP_IDS["favor"] else None)
    need = la_backward_workspace_bytes(causal, m, q.dtype, cu_seqlens is not None, nseq, T, H, d_k, d_v, r)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _check("la_backward", load_library().la_backward(
        int(causal), _norm_id(norm), _ptr(q), _ptr(k), _ptr(v), _ptr(omega), m, DTYPE_IDS[q.dtype],
        _ptr(cu_seqlens), nseq, T, H, d_k, d_v, r, eps, _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return dq, dk, dv


def attention(q, k, v, map="favor", omega=None, causal=True, cu_seqlens=None, nseq=None, eps=1e-6,
              out=None, workspace=None, stream=None, return_workspace=False, norm="attention"):
    """Convenience wrapper: allocates out/workspace with torch, calls the library."""
    o, ws = _forward(bool(causal), q, k, v, map, omega, cu_seqlens, nseq, eps, out, workspace, stream, norm=norm)
    return (o, ws) if return_workspace else o


def la_check_cu_seqlens(cu_seqlens: torch.Tensor, T: int, stream=None) -> bool:
    """True when cu_seqlens obeys the packing rules (synchronises)."""
    _need(cu_seqlens, "cu_seqlens", torch.int32)
    st = load_library().la_check_cu_seqlens(_ptr(cu_seqlens), cu_seqlens.numel() - 1, T, _stream(stream))
    if st not in (LA_OK, 1):
        raise LinAttnError("la_check_cu_seqlens", st)
    return st == LA_OK


def la_workspace_error(workspace: torch.Tensor, stream=None) -> int:
    """Device error code recorded in a workspace (0 = none; synchronises)."""
    code = _c_int(0)
    st = load_library().la_workspace_error(_ptr(workspace), ctypes.byref(code), _stream(stream))
    if st not in (LA_OK, 5):
        raise LinAttnError("la_workspace_error", st)
    return code.value


def la_orthogonal_features(gauss_blocks: torch.Tensor, gauss_lengths: torch.Tensor, r: int,
                           omega: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Orthogonal random-feature matrix [r, d] fp32 from fp64 Gaussian draws."""
    _need(gauss_blocks, "gauss_blocks", torch.float64)
    _need(gauss_lengths, "gauss_lengths", torch.float64)
    d = gauss_blocks.shape[-1]
    if omega is None:
        omega = torch.empty((r, d), dtype=torch.float32, device=gauss_blocks.device)
    _need(omega, "omega", torch.float32)
    _holds(-(-r // max(d, 1)) * d * d, gauss_blocks=gauss_blocks)
    _holds(r * d, gauss_lengths=gauss_lengths, omega=omega)
    _check("la_orthogonal_features", load_library().la_orthogonal_features(
        _ptr(gauss_blocks), _ptr(gauss_lengths), r, d, _ptr(omega), _stream(stream)))
    return omega


# --------------------------------------------------------------------------- operators around the attention call
#
# These calls are short enough that their checks count: an operand is tested as a whole and looked
# at in detail only when something is wrong with it.

def _first(t, name) -> int:
    """The device index of a call's first operand, a CUDA tensor of float32 or bfloat16."""
    _need(t, name)
    if t.dtype not in DTYPE_IDS:
        raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return t.get_device()


def _addr(t, name, dtype, shape, index) -> int:
    """Address of an operand: contiguous, on CUDA device `index`, of the given dtype (None: float32 or
    bfloat16) and shape (None: any)."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() == index and t.is_contiguous()
            and (t.dtype is dtype if dtype is not None else t.dtype in DTYPE_IDS)
            and (shape is None or t.shape == shape)):
        _need(t, name, dtype)
        if dtype is None and t.dtype not in DTYPE_IDS:
            raise ValueError(f"{name} must be float32 or bfloat16, got {t.dtype}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        raise ValueError(f"{name} is on {t.device}, other operands on cuda:{index}")
    return t.data_ptr()


def _addr_or_none(t, name, dtype, shape, index):
    return None if t is None else _addr(t, name, dtype, shape, index)


def _out(t, name, dtype, shape, like):
    """(output, its address): the caller's, or a new one on the device of `like`."""
    if t is not None:
        return t, _addr(t, name, dtype, shape, like.get_device())
    t = torch.empty(shape, dtype=dtype, device=like.device)
    return t, t.data_ptr()


class _On:
    """Makes an operand's device current for a call and, where a stream is given, that stream: what the
    call allocates belongs to it."""

    def __init__(self, index, stream):
        dev = torch.device("cuda", index)
        self.guards = []
        if index != torch.cuda.current_device():
            self.guards.append(torch.cuda.device(dev))
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                stream = (torch.cuda.ExternalStream(int(stream), device=dev) if int(stream)
                          else torch.cuda.default_stream(dev))
            elif stream.device != dev:
                raise ValueError(f"the stream is on {stream.device}, the operands on {dev}")
            self.guards.append(torch.cuda.stream(stream))

    def __enter__(self):
        for g in self.guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


_current_stream = torch._C._cuda_getCurrentRawStream   # of a device index, as a handle


def _elsewhere(index, stream) -> bool:
    """Whether a call has to change the current device or stream first (it then calls itself under _On)."""
    return stream is not None or index != torch._C._cuda_getDevice()


def _workspace(workspace, nbytes, index):
    """(workspace, its address, its bytes); allocates one of `nbytes` where none is given."""
    if workspace is None:
        # a size of 0 means the call will be rejected: let the library say why
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=torch.device("cuda", index))
        return workspace, workspace.data_ptr(), workspace.numel()
    _addr(workspace, "workspace", workspace.dtype, None, index)
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _sequences(cu_seqlens, nseq) -> int:
    if cu_seqlens is not None:
        if not isinstance(cu_seqlens, torch.Tensor):
            raise TypeError("cu_seqlens must be a torch.Tensor")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be a vector of at least two entries")
        if nseq is not None and nseq != cu_seqlens.numel() - 1:
            raise ValueError(f"nseq is {nseq}, cu_seqlens has {cu_seqlens.numel() - 1} sequences")
        return cu_seqlens.numel() - 1
    return 1 if nseq is None else int(nseq)


def _rows3(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [T, H, d], got shape {tuple(t.shape)}")
    return t.shape


def la_gated_scan_workspace_bytes(has_cu_seqlens: bool, nseq: int, T: int, H: int, d: int) -> int:
    return load_library().la_gated_scan_workspace_bytes(int(has_cu_seqlens), nseq, T, H, d)


def la_gated_scan(a, b, cu_seqlens=None, nseq=None, state_in=None, state_out=None, return_state=False, h=None,
                  workspace=None, stream=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + b_t of packed rows a, b [T, H, d] (fp32 or
    bf16 each); returns h [T, H, d] (dtype of b).  state_in / state_out: fp32 [nseq, H, d],
    state_out may be state_in.  With return_state=True a state_out is allocated when none is
    given and (h, state_out) is returned."""
    lib = load_library()
    T, H, d = shape = _rows3(b, "b")
    nseq = _sequences(cu_seqlens, nseq)
    states, f32, dev = (nseq, H, d), torch.float32, _first(b, "b")
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return la_gated_scan(a, b, cu_seqlens, nseq, state_in, state_out, return_state, h, workspace)
    pa = _addr(a, "a", None, shape, dev)
    pc = _addr_or_none(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
    pi = _addr_or_none(state_in, "state_in", f32, states, dev)
    if h is None:
        h = torch.empty_like(b)
    if return_state and state_out is None:
        state_out = torch.empty(states, dtype=f32, device=b.device)
    workspace, pw, nw = _workspace(
        workspace, 0 if workspace is not None else
        lib.la_gated_scan_workspace_bytes(cu_seqlens is not None, nseq, T, H, d), dev)
    _check("la_gated_scan", lib.la_gated_scan(
        pa, b.data_ptr(), DTYPE_IDS[a.dtype], DTYPE_IDS[b.dtype], pc, nseq, T, H, d, pi,
        _addr_or_none(state_out, "state_out", f32, states, dev), _addr(h, "h", b.dtype, shape, dev), pw, nw,
        _current_stream(dev)))
    return (h, state_out) if return_state else h


def la_gated_scan_backward(a, h, dh, cu_seqlens=None, nseq=None, state_in=None, dstate_out=None, return_dstate=False,
                           da=None, db=None, dstate_in=None, workspace=None, stream=None):
    """Gradients (da, db) of sum(dh * h) + sum(dstate_out * state_out) for la_gated_scan, whose
    output h is read; with return_dstate=True (da, db, dstate_in)."""
    lib = load_library()
    T, H, d = shape = _rows3(h, "h")
    nseq = _sequences(cu_seqlens, nseq)
    states, f32, dev = (nseq, H, d), torch.float32, _first(h, "h")
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return la_gated_scan_backward(a, h, dh, cu_seqlens, nseq, state_in, dstate_out, return_dstate, da, db,
                                          dstate_in, workspace)
    pa, pd = _addr(a, "a", None, shape, dev), _addr(dh, "dh", h.dtype, shape, dev)
    pc = _addr_or_none(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
    pi = _addr_or_none(state_in, "state_in", f32, states, dev)
    po = _addr_or_none(dstate_out, "dstate_out", f32, states, dev)
    if da is None:
        da = torch.empty_like(a)
    if db is None:
        db = torch.empty_like(h)
    if return_dstate and dstate_in is None:
        dstate_in = torch.empty(states, dtype=f32, device=h.device)
    workspace, pw, nw = _workspace(
        workspace, 0 if workspace is not None else
        lib.la_gated_scan_workspace_bytes(cu_seqlens is not None, nseq, T, H, d), dev)
    _check("la_gated_scan_backward", lib.la_gated_scan_backward(
        pa, h.data_ptr(), pd, DTYPE_IDS[a.dtype], DTYPE_IDS[h.dtype], pc, nseq, T, H, d, pi, po,
        _addr(da, "da", a.dtype, shape, dev), _addr(db, "db", h.dtype, shape, dev),
        _addr_or_none(dstate_in, "dstate_in", f32, states, dev), pw, nw, _current_stream(dev)))
    return (da, db, dstate_in) if return_dstate else (da, db)


def la_gated_step(a, b, state, state_out=None, h=None, stream=None):
    """One token for each of B sequences of the gated recurrence: a, b [B, H, d]; state fp32
    [B, H, d] is updated in place, or written to state_out when given; returns h [B, H, d]."""
    lib = load_library()
    B, H, d = shape = _rows3(b, "b")
    f32, dev = torch.float32, _first(b, "b")
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return la_gated_step(a, b, state, state_out, h)
    pa, ps = _addr(a, "a", None, shape, dev), _addr(state, "state", f32, shape, dev)
    po = ps if state_out is None else _addr(state_out, "state_out", f32, shape, dev)
    if h is None:
        h = torch.empty_like(b)
    _check("la_gated_step", lib.la_gated_step(pa, b.data_ptr(), DTYPE_IDS[a.dtype], DTYPE_IDS[b.dtype], B, H, d, ps, po,
                                              _addr(h, "h", b.dtype, shape, dev), _current_stream(dev)))
    return h


def _norm_shape(x, weight, bias):
    """(rows, groups, d) of x [..., d] with weight and bias [d] (shared) or [G, d] (G: x's
    second dimension from the right, each index with its own)."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    shape = x.shape
    if len(shape) < 1 or shape[-1] < 1:
        raise ValueError(f"x must be [..., d], got shape {tuple(shape)}")
    d, groups = shape[-1], 1
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if len(t.shape) == 2 and len(shape) >= 2 and t.shape == shape[-2:]:
            groups = shape[-2]
        elif t.shape != shape[-1:]:
            raise ValueError(f"{name} must have shape {(d,)} or x's last two dimensions, got {tuple(t.shape)}")
    if weight is not None and bias is not None and weight.shape != bias.shape:
        raise ValueError("weight and bias must have the same shape")
    return x.numel() // d, groups, d


def la_layer_norm(x, weight=None, bias=None, eps=1e-5, return_stats=False, y=None, mean=None, rstd=None, stream=None):
    """Layer norm over the last dimension of x [..., d] (fp32 or bf16): (x - mean) rstd weight +
    bias.  weight, bias: fp32 [d], or [H, d] for x [..., H, d].  Returns y, or with
    return_stats=True (y, mean, rstd), the statistics fp32 of x's shape without its last
    dimension, as la_layer_norm_backward reads them."""
    lib = load_library()
    rows, groups, d = _norm_shape(x, weight, bias)
    f32, dev, shape = torch.float32, _first(x, "x"), x.shape
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return la_layer_norm(x, weight, bias, eps, return_stats, y, mean, rstd)
    stats = shape[:-1]
    pw, pb = _addr_or_none(weight, "weight", f32, None, dev), _addr_or_none(bias, "bias", f32, None, dev)
    if y is None:
        y = torch.empty_like(x)
    if return_stats:
        mean = torch.empty(stats, dtype=f32, device=x.device) if mean is None else mean
        rstd = torch.empty(stats, dtype=f32, device=x.device) if rstd is None else rstd
    _check("la_layer_norm", lib.la_layer_norm(
        x.data_ptr(), pw, pb, DTYPE_IDS[x.dtype], rows, groups, d, eps, _addr(y, "y", x.dtype, shape, dev),
        _addr_or_none(mean, "mean", f32, stats, dev), _addr_or_none(rstd, "rstd", f32, stats, dev),
        _current_stream(dev)))
    return (y, mean, rstd) if return_stats else y


def la_layer_norm_backward_workspace_bytes(dtype, rows: int, groups: int, d: int) -> int:
    dt = DTYPE_IDS[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return load_library().la_layer_norm_backward_workspace_bytes(dt, rows, groups, d)


def la_layer_norm_backward(x, dy, mean, rstd, weight=None, dx=None, dweight=None, dbias=None, workspace=None, stream=None):
    """Gradients (dx, dweight, dbias) of sum(dy * y) for la_layer_norm; weight [d] or [H, d] gives
    the shape of dweight and dbias (fp32).  weight None is 1, and without a dweight or dbias to tell
    their shape these gradients are None."""
    lib = load_library()
    like = weight if weight is not None else dweight if dweight is not None else dbias
    rows, groups, d = _norm_shape(x, like, None)
    f32, dev, shape = torch.float32, _first(x, "x"), x.shape
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return la_layer_norm_backward(x, dy, mean, rstd, weight, dx, dweight, dbias, workspace)
    stats = shape[:-1]
    pd = _addr(dy, "dy", x.dtype, shape, dev)
    pm, pr = _addr(mean, "mean", f32, stats, dev), _addr(rstd, "rstd", f32, stats, dev)
    pw = _addr_or_none(weight, "weight", f32, None, dev)
    dx = torch.empty_like(x) if dx is None else dx
    wshape = None if like is None else like.shape
    if like is not None:
        dweight = torch.empty(wshape, dtype=f32, device=x.device) if dweight is None else dweight
        dbias = torch.empty(wshape, dtype=f32, device=x.device) if dbias is None else dbias
    workspace, pws, nws = _workspace(
        workspace, 0 if workspace is not None else
        lib.la_layer_norm_backward_workspace_bytes(DTYPE_IDS[x.dtype], rows, groups, d), dev)
    _check("la_layer_norm_backward", lib.la_layer_norm_backward(
        x.data_ptr(), pd, pw, pm, pr, DTYPE_IDS[x.dtype], rows, groups, d, _addr(dx, "dx", x.dtype, shape, dev),
        _addr_or_none(dweight, "dweight", f32, wshape, dev), _addr_or_none(dbias, "dbias", f32, wshape, dev), pws, nws,
        _current_stream(dev)))
    return dx, dweight, dbias


def la_rotary(q, k, freq, positions, pairs, interleaved=False, inverse=False, q_out=None, k_out=None, stream=None):
    """Rotary positions on q and k [T, H, d] (k may be None): pair p turns by positions[t, axis(p)]
    freq[p].  freq: fp32 [P]; positions: int32 [T, naxes] (or [T] for one axis); pairs: how many
    pairs each axis turns, sum(pairs) = P.  interleaved: channels (2p, 2p + 1) instead of (p, p + P).
    inverse=True turns back (the gradient).  q_out may be q, k_out k.  Returns (q_out, k_out), or
    q_out alone when k is None."""
    lib = load_library()
    T, H, d = shape = _rows3(q, "q")
    dev, n = _first(q, "q"), len(pairs)
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return la_rotary(q, k, freq, positions, pairs, interleaved, inverse, q_out, k_out)
    pk = _addr_or_none(k, "k", q.dtype, shape, dev)
    pf = _addr(freq, "freq", torch.float32, (sum(pairs),), dev)
    if not isinstance(positions, torch.Tensor):
        raise TypeError("positions must be a torch.Tensor")
    pp = _addr(positions, "positions", torch.int32, (T,) if n == 1 and positions.dim() == 1 else (T, n), dev)
    if k is None and k_out is not None:
        raise ValueError("k_out is given without k")
    if q_out is None:
        q_out = torch.empty_like(q)
    if k is not None and k_out is None:
        k_out = torch.empty_like(k)
    _check("la_rotary", lib.la_rotary(
        q.data_ptr(), pk, pf, pp, DTYPE_IDS[q.dtype], T, H, d, (_c_int * n)(*pairs), n, bool(interleaved),
        bool(inverse), _addr(q_out, "q_out", q.dtype, shape, dev),
        _addr_or_none(k_out, "k_out", q.dtype, shape, dev), _current_stream(dev)))
    return q_out if k is None else (q_out, k_out)


def _strided(t, name, dtype, index):
    """(address, elements between tokens) of rows [T, H, d] whose tokens may be any distance apart, a token's
    rows next to one another: a slice of a fused projection's output."""
    T, H, d = _rows3(t, name)
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, other operands on cuda:{index}")
    if t.is_contiguous() or t.numel() == 0:
        return t.data_ptr(), H * d
    st, sh, sd = t.stride()
    if sd != 1 or (H > 1 and sh != d) or (T > 1 and st < H * d):
        raise ValueError(f"{name}: a token's rows must lie next to one another, got strides {(st, sh, sd)}")
    return t.data_ptr(), st if T > 1 else H * d


def _qk_operands(q, k, q_weight, k_weight, freq, positions, pairs):
    """Device index, addresses and sizes that la_qk_norm_rotary and its gradients share."""
    T, Hq, d = _rows3(q, "q")
    if not q.is_cuda or q.dtype not in DTYPE_IDS:
        raise ValueError(f"q must be a CUDA tensor of float32 or bfloat16, got {q.dtype} on {q.device}")
    dev, n, Hk = q.get_device(), len(pairs), 0
    pq, sq = _strided(q, "q", q.dtype, dev)
    pk, sk = None, 0
    if k is not None:
        Tk, Hk, dk = _rows3(k, "k")
        if Tk != T or dk != d:
            raise ValueError(f"k must have shape {(T, 'Hk', d)}, got {tuple(k.shape)}")
        pk, sk = _strided(k, "k", q.dtype, dev)
    elif k_weight is not None:
        raise ValueError("k_weight is given without k")
    per_head, ws = False, []
    for w, name, H in ((q_weight, "q_weight", Hq), (k_weight, "k_weight", Hk)):
        if w is not None and isinstance(w, torch.Tensor) and w.dim() == 2:
            per_head = True
    for w, name, H in ((q_weight, "q_weight", Hq), (k_weight, "k_weight", Hk)):
        ws.append(_addr_or_none(w, name, torch.float32, (H, d) if per_head else (d,), dev))
    pf = _addr(freq, "freq", torch.float32, (sum(pairs),), dev)
    if not isinstance(positions, torch.Tensor):
        raise TypeError("positions must be a torch.Tensor")
    pp = _addr(positions, "positions", torch.int32, (T,) if n == 1 and positions.dim() == 1 else (T, n), dev)
    return dev, T, Hq, Hk, d, pq, sq, pk, sk, ws[0], ws[1], per_head, pf, pp, (_c_int * n)(*pairs), n


def _device_of(t, name) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def la_qk_norm_rotary(q, k, q_weight, k_weight, freq, positions, pairs, eps=1e-6, interleaved=False, return_rstd=False,
                      q_out=None, k_out=None, q_rstd=None, k_rstd=None, stream=None):
    """Norm of every head's queries and keys (x / sqrt(mean(x^2) + eps) weight) and their rotation (as
    la_rotary) in one pass.  q [T, Hq, d], k [T, Hk, d] (fp32 or bf16, k may be None), tokens any
    distance apart: slices of a fused projection need no copy.  q_weight, k_weight: fp32 [d], or both
    per head ([Hq, d], [Hk, d]), or None.  Returns (q_out, k_out), contiguous, or with return_rstd=True
    (q_out, k_out, q_rstd, k_rstd), as la_qk_norm_rotary_backward reads them.  q_out may be q, k_out k."""
    lib = load_library()
    if _elsewhere(_device_of(q, "q"), stream):
        with _On(q.get_device(), stream):
            return la_qk_norm_rotary(q, k, q_weight, k_weight, freq, positions, pairs, eps, interleaved, return_rstd,
                                     q_out, k_out, q_rstd, k_rstd)
    dev, T, Hq, Hk, d, pq, sq, pk, sk, wq, wk, per_head, pf, pp, pa, n = _qk_operands(q, k, q_weight, k_weight, freq,
                                                                                      positions, pairs)
    if k is None and (k_out is not None or k_rstd is not None):
        raise ValueError("k_out or k_rstd is given without k")
    dt, f32 = q.dtype, torch.float32
    q_out, pqo = _out(q_out, "q_out", dt, (T, Hq, d), q)
    k_out, pko = (None, None) if k is None else _out(k_out, "k_out", dt, (T, Hk, d), q)
    pqr = pkr = None
    if return_rstd or q_rstd is not None:
        q_rstd, pqr = _out(q_rstd, "q_rstd", f32, (T, Hq), q)
    if k is not None and (return_rstd or k_rstd is not None):
        k_rstd, pkr = _out(k_rstd, "k_rstd", f32, (T, Hk), q)
    _check("la_qk_norm_rotary", lib.la_qk_norm_rotary(
        pq, pk, wq, wk, pf, pp, DTYPE_IDS[dt], T, Hq, Hk, d, sq, sk, pa, n, bool(interleaved), per_head, eps, pqo, pko,
        pqr, pkr, _current_stream(dev)))
    return (q_out, k_out, q_rstd, k_rstd) if return_rstd else (q_out, k_out)


def la_qk_norm_rotary_backward_workspace_bytes(dtype, T: int, Hq: int, Hk: int, d: int) -> int:
    dt = DTYPE_IDS[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return load_library().la_qk_norm_rotary_backward_workspace_bytes(dt, T, Hq, Hk, d)


def la_qk_norm_rotary_backward(q, k, q_rstd, k_rstd, dq_out, dk_out, q_weight, k_weight, freq, positions, pairs,
                               interleaved=False, dq=None, dk=None, dq_weight=None, dk_weight=None, workspace=None,
                               stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of sum(dq_out * q_out) + sum(dk_out * k_out) for
    la_qk_norm_rotary; dq, dk contiguous, those of the weights fp32 of the weights' shapes (None where a
    weight is None)."""
    lib = load_library()
    if _elsewhere(_device_of(q, "q"), stream):
        with _On(q.get_device(), stream):
            return la_qk_norm_rotary_backward(q, k, q_rstd, k_rstd, dq_out, dk_out, q_weight, k_weight, freq, positions,
                                              pairs, interleaved, dq, dk, dq_weight, dk_weight, workspace)
    dev, T, Hq, Hk, d, pq, sq, pk, sk, wq, wk, per_head, pf, pp, pa, n = _qk_operands(q, k, q_weight, k_weight, freq,
                                                                                      positions, pairs)
    dt, f32 = q.dtype, torch.float32
    for w, dw, name in ((q_weight, dq_weight, "dq_weight"), (k_weight, dk_weight, "dk_weight")):
        if w is None and dw is not None:
            raise ValueError(f"{name} is given without its weight")
    if k is None and any(x is not None for x in (k_rstd, dk_out, dk)):
        raise ValueError("k_rstd, dk_out or dk is given without k")
    pqr, pdq = _addr(q_rstd, "q_rstd", f32, (T, Hq), dev), _addr(dq_out, "dq_out", dt, (T, Hq, d), dev)
    pkr = pdk = None
    if k is not None:
        pkr, pdk = _addr(k_rstd, "k_rstd", f32, (T, Hk), dev), _addr(dk_out, "dk_out", dt, (T, Hk, d), dev)
    dq, po = _out(dq, "dq", dt, (T, Hq, d), q)
    dk, pko = (None, None) if k is None else _out(dk, "dk", dt, (T, Hk, d), q)
    pqw = pkw = None
    if q_weight is not None:
        dq_weight, pqw = _out(dq_weight, "dq_weight", f32, q_weight.shape, q)
    if k_weight is not None:
        dk_weight, pkw = _out(dk_weight, "dk_weight", f32, k_weight.shape, q)
    workspace, pw, nw = _workspace(
        workspace, 0 if workspace is not None else
        lib.la_qk_norm_rotary_backward_workspace_bytes(DTYPE_IDS[dt], T, Hq, Hk, d), dev)
    _check("la_qk_norm_rotary_backward", lib.la_qk_norm_rotary_backward(
        pq, pk, pqr, pkr, pdq, pdk, wq, wk, pf, pp, DTYPE_IDS[dt], T, Hq, Hk, d, sq, sk, pa, n, bool(interleaved),
        per_head, po, pko, pqw, pkw, pw, nw, _current_stream(dev)))
    return dq, dk, dq_weight, dk_weight


# --------------------------------------------------------------------------- linear attention with a decay for each head

def _decay_operands(q, k, v, log_decay):
    """(T, H, d_k, d_v, shape of v, device index, addresses of q, k, v, log_decay)."""
    T, H, dk = shape = _rows3(q, "q")
    dv, dev = _rows3(v, "v")[2], _first(q, "q")
    vshape = (T, H, dv)
    return (T, H, dk, dv, vshape, dev, q.data_ptr(), _addr(k, "k", q.dtype, shape, dev),
            _addr(v, "v", q.dtype, vshape, dev), _addr(log_decay, "log_decay", torch.float32, (H,), dev))


def la_decay_attention_workspace_bytes(dtype, has_cu_seqlens: bool, nseq: int, T: int, H: int, d_k: int, d_v: int) -> int:
    dt = DTYPE_IDS[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return load_library().la_decay_attention_workspace_bytes(dt, int(has_cu_seqlens), nseq, T, H, d_k, d_v)


def la_decay_attention(q, k, v, log_decay, scale=1.0, cu_seqlens=None, nseq=None, state_in=None, state_out=None,
                       return_state=False, out=None, workspace=None, stream=None):
    """Causal linear attention with a decay for each head: S_t = exp(log_decay) S_{t-1} + k_t v_t^T,
    out_t = scale q_t^T S_t.  q, k [T, H, d_k], v [T, H, d_v] (fp32 or bf16); log_decay fp32 [H], at
    most 0; returns out [T, H, d_v].  state_in / state_out: fp32 [nseq, H, d_k, d_v], state_out may be
    state_in.  With return_state=True a state_out is allocated when none is given and (out, state_out)
    is returned."""
    lib = load_library()
    nseq = _sequences(cu_seqlens, nseq)
    if _elsewhere(_first(q, "q"), stream):
        with _On(q.get_device(), stream):
            return la_decay_attention(q, k, v, log_decay, scale, cu_seqlens, nseq, state_in, state_out, return_state,
                                      out, workspace)
    T, H, dk, dv, shape, dev, pq, pk, pv, pl = _decay_operands(q, k, v, log_decay)
    states, f32, dt = (nseq, H, dk, dv), torch.float32, DTYPE_IDS[q.dtype]
    pc = _addr_or_none(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
    pi = _addr_or_none(state_in, "state_in", f32, states, dev)
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=q.device)
    if return_state and state_out is None:
        state_out = torch.empty(states, dtype=f32, device=q.device)
    workspace, pw, nw = _workspace(
        workspace, 0 if workspace is not None else
        lib.la_decay_attention_workspace_bytes(dt, cu_seqlens is not None, nseq, T, H, dk, dv), dev)
    _check("la_decay_attention", lib.la_decay_attention(
        pq, pk, pv, pl, dt, pc, nseq, T, H, dk, dv, scale, pi, _addr_or_none(state_out, "state_out", f32, states, dev),
        _addr(out, "out", q.dtype, shape, dev), pw, nw, _current_stream(dev)))
    return (out, state_out) if return_state else out


def la_decay_attention_backward_workspace_bytes(dtype, has_cu_seqlens: bool, nseq: int, T: int, H: int, d_k: int,
                                                d_v: int) -> int:
    dt = DTYPE_IDS[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return load_library().la_decay_attention_backward_workspace_bytes(dt, int(has_cu_seqlens), nseq, T, H, d_k, d_v)


def la_decay_attention_backward(q, k, v, dout, log_decay, scale=1.0, cu_seqlens=None, nseq=None, state_in=None,
                                dstate_out=None, return_dstate=False, dq=None, dk=None, dv=None, dstate_in=None,
                                workspace=None, stream=None):
    """Gradients (dq, dk, dv) of sum(dout * out) + sum(dstate_out * state_out) for la_decay_attention
    with the same arguments (log_decay a constant); with return_dstate=True (dq, dk, dv, dstate_in)."""
    lib = load_library()
    nseq = _sequences(cu_seqlens, nseq)
    if _elsewhere(_first(q, "q"), stream):
        with _On(q.get_device(), stream):
            return la_decay_attention_backward(q, k, v, dout, log_decay, scale, cu_seqlens, nseq, state_in, dstate_out,
                                               return_dstate, dq, dk, dv, dstate_in, workspace)
    T, H, d_k, d_v, shape, dev, pq, pk, pv, pl = _decay_operands(q, k, v, log_decay)
    states, f32, dt = (nseq, H, d_k, d_v), torch.float32, DTYPE_IDS[q.dtype]
    pd = _addr(dout, "dout", q.dtype, shape, dev)
    pc = _addr_or_none(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
    pi = _addr_or_none(state_in, "state_in", f32, states, dev)
    po = _addr_or_none(dstate_out, "dstate_out", f32, states, dev)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if return_dstate and dstate_in is None:
        dstate_in = torch.empty(states, dtype=f32, device=q.device)
    workspace, pw, nw = _workspace(
        workspace, 0 if workspace is not None else
        lib.la_decay_attention_backward_workspace_bytes(dt, cu_seqlens is not None, nseq, T, H, d_k, d_v), dev)
    _check("la_decay_attention_backward", lib.la_decay_attention_backward(
        pq, pk, pv, pd, pl, dt, pc, nseq, T, H, d_k, d_v, scale, pi, po, _addr(dq, "dq", q.dtype, q.shape, dev),
        _addr(dk, "dk", q.dtype, q.shape, dev), _addr(dv, "dv", q.dtype, shape, dev),
        _addr_or_none(dstate_in, "dstate_in", f32, states, dev), pw, nw, _current_stream(dev)))
    return (dq, dk, dv, dstate_in) if return_dstate else (dq, dk, dv)


def la_decay_step(q, k, v, log_decay, state, scale=1.0, state_out=None, out=None, stream=None):
    """One token for each of B sequences of la_decay_attention: q, k [B, H, d_k], v [B, H, d_v]; state
    fp32 [B, H, d_k, d_v] is updated in place, or written to state_out when given; returns out
    [B, H, d_v]."""
    lib = load_library()
    if _elsewhere(_first(q, "q"), stream):
        with _On(q.get_device(), stream):
            return la_decay_step(q, k, v, log_decay, state, scale, state_out, out)
    B, H, dk, dv, shape, dev, pq, pk, pv, pl = _decay_operands(q, k, v, log_decay)
    states, f32 = (B, H, dk, dv), torch.float32
    ps = _addr(state, "state", f32, states, dev)
    po = ps if state_out is None else _addr(state_out, "state_out", f32, states, dev)
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=q.device)
    _check("la_decay_step", lib.la_decay_step(pq, pk, pv, pl, DTYPE_IDS[q.dtype], B, H, dk, dv, scale, ps, po,
                                              _addr(out, "out", q.dtype, shape, dev), _current_stream(dev)))
    return out
