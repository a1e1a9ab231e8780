// C entry points of the operators around the attention call (gated linear
// recurrence, layer norm, rotary positions): argument checks and dispatch.
#include <cmath>

#include "ops/ops.h"

namespace la {

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool dtype_ok(int dtype) { return dtype == LA_F32 || dtype == LA_BF16; }
size_t esize(int dtype) { return dtype == LA_F32 ? 4 : 2; }

struct Span {
    const void* p;
    size_t bytes;
};

bool overlap(const Span& x, const Span& y) {
    if (!x.p || !y.p || x.bytes == 0 || y.bytes == 0) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
    return a < b + y.bytes && b < a + x.bytes;
}

// No output overlaps an input or another output.
template <int NO, int NI>
bool disjoint(const Span (&out)[NO], const Span (&in)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (overlap(out[i], in[j])) return false;
        for (int j = i + 1; j < NO; ++j)
            if (overlap(out[i], out[j])) return false;
    }
    return true;
}

la_status gated_dims(bool has_cu, int nseq, int64_t T, int H, int d) {
    if (nseq < 1 || nseq > 65535 || H < 1 || H > 65535 || d < 1) return LA_ERR_INVALID_ARG;
    if (T < 0 || T > (int64_t)INT32_MAX) return LA_ERR_INVALID_ARG;
    if (!has_cu && T % nseq != 0) return LA_ERR_INVALID_ARG;
    if ((int64_t)H * d > LA_MAX_CHANNELS) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

la_status norm_dims(int dtype, int64_t rows, int groups, int d) {
    if (!dtype_ok(dtype) || rows < 0 || groups < 1 || d < 1 || rows % groups != 0) return LA_ERR_INVALID_ARG;
    if (d > LA_MAX_NORM_D || (int64_t)groups * d > LA_MAX_CHANNELS || rows > (int64_t)1 << 40)
        return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

la_status result(cudaError_t e) { return e == cudaSuccess ? LA_OK : LA_ERR_CUDA; }

}  // namespace

}  // namespace la

using namespace la;

extern "C" {

size_t la_gated_scan_workspace_bytes(int has_cu_seqlens, int nseq, int64_t T, int H, int d) {
    if (gated_dims(has_cu_seqlens != 0, nseq, T, H, d) != LA_OK) return 0;
    return gated_workspace_bytes(T, H * d);
}

la_status la_gated_scan(const void* a, const void* b, int a_dtype, int dtype, const int32_t* cu_seqlens, int nseq,
                        int64_t T, int H, int d, const float* state_in, float* state_out, void* h, void* workspace,
                        size_t workspace_bytes, void* stream) {
    if (!dtype_ok(a_dtype) || !dtype_ok(dtype)) return LA_ERR_INVALID_ARG;
    la_status st = gated_dims(cu_seqlens != nullptr, nseq, T, H, d);
    if (st != LA_OK) return st;
    if (workspace == nullptr || !aligned(workspace, kAlign)) return LA_ERR_INVALID_ARG;
    if (T > 0 && (!a || !b || !h)) return LA_ERR_INVALID_ARG;
    if (!aligned(a, esize(a_dtype)) || !aligned(b, esize(dtype)) || !aligned(h, esize(dtype)) ||
        !aligned(state_in, 4) || !aligned(state_out, 4) || !aligned(cu_seqlens, 4))
        return LA_ERR_INVALID_ARG;
    const int C = H * d;
    if (workspace_bytes < gated_workspace_bytes(T, C)) return LA_ERR_WORKSPACE;
    const size_t n = (size_t)T * C, ns = sizeof(float) * (size_t)nseq * C;
    const Span out[] = {{h, n * esize(dtype)}, {state_out, ns}, {workspace, gated_workspace_bytes(T, C)}};
    const Span in[] = {{a, n * esize(a_dtype)}, {b, n * esize(dtype)}, {state_in == state_out ? nullptr : state_in, ns},
                       {cu_seqlens, sizeof(int32_t) * ((size_t)nseq + 1)}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    GatedParams p{};
    p.a = a; p.x = b; p.y = h;
    p.state_in = p.edge_in = state_in; p.edge_out = state_out;
    p.cu_seqlens = cu_seqlens; p.nseq = nseq; p.T = T; p.C = C;
    return result(gated_scan(p, a_dtype, dtype, 0, workspace, static_cast<cudaStream_t>(stream)));
}

la_status la_gated_scan_backward(const void* a, const void* h, const void* dh, int a_dtype, int dtype,
                                 const int32_t* cu_seqlens, int nseq, int64_t T, int H, int d,
                                 const float* state_in, const float* dstate_out, void* da, void* db,
                                 float* dstate_in, void* workspace, size_t workspace_bytes, void* stream) {
    if (!dtype_ok(a_dtype) || !dtype_ok(dtype)) return LA_ERR_INVALID_ARG;
    la_status st = gated_dims(cu_seqlens != nullptr, nseq, T, H, d);
    if (st != LA_OK) return st;
    if (workspace == nullptr || !aligned(workspace, kAlign)) return LA_ERR_INVALID_ARG;
    if (T > 0 && (!a || !h || !dh || !da || !db)) return LA_ERR_INVALID_ARG;
    for (const void* q : {h, dh, static_cast<const void*>(db)})
        if (!aligned(q, esize(dtype))) return LA_ERR_INVALID_ARG;
    if (!aligned(a, esize(a_dtype)) || !aligned(da, esize(a_dtype)) || !aligned(state_in, 4) ||
        !aligned(dstate_out, 4) || !aligned(dstate_in, 4) || !aligned(cu_seqlens, 4))
        return LA_ERR_INVALID_ARG;
    const int C = H * d;
    if (workspace_bytes < gated_workspace_bytes(T, C)) return LA_ERR_WORKSPACE;
    const size_t n = (size_t)T * C, na = n * esize(a_dtype), nx = n * esize(dtype);
    const size_t ns = sizeof(float) * (size_t)nseq * C;
    const Span out[] = {{da, na}, {db, nx}, {dstate_in, ns}, {workspace, gated_workspace_bytes(T, C)}};
    const Span in[] = {{a, na}, {h, nx}, {dh, nx}, {state_in, ns}, {dstate_out == dstate_in ? nullptr : dstate_out, ns},
                       {cu_seqlens, sizeof(int32_t) * ((size_t)nseq + 1)}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    GatedParams p{};
    p.a = a; p.x = dh; p.h = h; p.y = db; p.da = da;
    p.state_in = state_in; p.edge_in = dstate_out; p.edge_out = dstate_in;
    p.cu_seqlens = cu_seqlens; p.nseq = nseq; p.T = T; p.C = C;
    return result(gated_scan(p, a_dtype, dtype, 1, workspace, static_cast<cudaStream_t>(stream)));
}

la_status la_gated_step(const void* a, const void* b, int a_dtype, int dtype, int B, int H, int d,
                        const float* state_in, float* state_out, void* h, void* stream) {
    if (!dtype_ok(a_dtype) || !dtype_ok(dtype) || B < 0) return LA_ERR_INVALID_ARG;
    la_status st = gated_dims(true, 1, B, H, d);
    if (st != LA_OK) return st;
    if (B == 0) return LA_OK;
    if (!a || !b || !state_in || !state_out || !h) return LA_ERR_INVALID_ARG;
    if (!aligned(a, esize(a_dtype)) || !aligned(b, esize(dtype)) || !aligned(h, esize(dtype)) ||
        !aligned(state_in, 4) || !aligned(state_out, 4))
        return LA_ERR_INVALID_ARG;
    const int64_t n = (int64_t)B * H * d;
    const Span out[] = {{h, n * esize(dtype)}, {state_out, (size_t)n * 4}};
    const Span in[] = {{a, n * esize(a_dtype)}, {b, n * esize(dtype)},
                       {state_in == state_out ? nullptr : state_in, (size_t)n * 4}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    return result(gated_step(a, b, a_dtype, dtype, n, state_in, state_out, h, static_cast<cudaStream_t>(stream)));
}

la_status la_layer_norm(const void* x, const float* weight, const float* bias, int dtype, int64_t rows, int groups,
                        int d, float eps, void* y, float* mean, float* rstd, void* stream) {
    la_status st = norm_dims(dtype, rows, groups, d);
    if (st != LA_OK) return st;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return LA_ERR_INVALID_ARG;
    if (rows == 0) return LA_OK;
    if (!x || !y) return LA_ERR_INVALID_ARG;
    if (!aligned(x, esize(dtype)) || !aligned(y, esize(dtype)) || !aligned(weight, 4) || !aligned(bias, 4) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return LA_ERR_INVALID_ARG;
    const size_t n = (size_t)rows * d * esize(dtype), np = sizeof(float) * (size_t)groups * d;
    const Span out[] = {{y, n}, {mean, (size_t)rows * 4}, {rstd, (size_t)rows * 4}};
    const Span in[] = {{x, n}, {weight, np}, {bias, np}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    return result(layer_norm(x, weight, bias, dtype, rows, groups, d, eps, y, mean, rstd,
                             static_cast<cudaStream_t>(stream)));
}

size_t la_layer_norm_backward_workspace_bytes(int dtype, int64_t rows, int groups, int d) {
    if (norm_dims(dtype, rows, groups, d) != LA_OK) return 0;
    return layer_norm_backward_workspace_bytes(dtype, rows, groups, d);
}

la_status la_layer_norm_backward(const void* x, const void* dy, const float* weight, const float* mean,
                                 const float* rstd, int dtype, int64_t rows, int groups, int d, void* dx,
                                 float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    la_status st = norm_dims(dtype, rows, groups, d);
    if (st != LA_OK) return st;
    if (workspace == nullptr || !aligned(workspace, kAlign)) return LA_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !dy || !mean || !rstd || !dx)) return LA_ERR_INVALID_ARG;
    for (const void* q : {x, dy, static_cast<const void*>(dx)})
        if (!aligned(q, esize(dtype))) return LA_ERR_INVALID_ARG;
    for (const float* q : {weight, mean, rstd, static_cast<const float*>(dweight), static_cast<const float*>(dbias)})
        if (!aligned(q, 4)) return LA_ERR_INVALID_ARG;
    const size_t need = layer_norm_backward_workspace_bytes(dtype, rows, groups, d);
    if (need == 0) return LA_ERR_CUDA;
    if (workspace_bytes < need) return LA_ERR_WORKSPACE;
    const size_t n = (size_t)rows * d * esize(dtype), np = sizeof(float) * (size_t)groups * d, nr = (size_t)rows * 4;
    const Span out[] = {{dx, n}, {dweight, np}, {dbias, np}, {workspace, need}};
    const Span in[] = {{x, n}, {dy, n}, {weight, np}, {mean, nr}, {rstd, nr}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    return result(layer_norm_backward(x, dy, weight, mean, rstd, dtype, rows, groups, d, dx, dweight, dbias, workspace,
                                      static_cast<cudaStream_t>(stream)));
}

la_status la_rotary(const void* q, const void* k, const float* freq, const int32_t* positions, int dtype, int64_t T,
                    int H, int d, const int* pairs, int naxes, int interleaved, int inverse, void* q_out, void* k_out,
                    void* stream) {
    if (!dtype_ok(dtype) || T < 0 || T > (int64_t)INT32_MAX || H < 1 || H > 65535 || d < 2) return LA_ERR_INVALID_ARG;
    if (naxes < 1 || pairs == nullptr || (interleaved & ~1) || (inverse & ~1)) return LA_ERR_INVALID_ARG;
    if (naxes > LA_MAX_AXES || d > LA_MAX_ROTARY_D) return LA_ERR_UNSUPPORTED;
    RotaryParams p{};
    int64_t P = 0;
    for (int i = 0; i < naxes; ++i) {
        if (pairs[i] < 0) return LA_ERR_INVALID_ARG;
        p.first[i] = (int)P;
        P += pairs[i];
        if (2 * P > d) return LA_ERR_INVALID_ARG;
    }
    for (int i = naxes; i <= LA_MAX_AXES; ++i) p.first[i] = (int)P;
    if (P < 1) return LA_ERR_INVALID_ARG;
    if ((k == nullptr) != (k_out == nullptr)) return LA_ERR_INVALID_ARG;
    if (T == 0) return LA_OK;
    if (!q || !q_out || !freq || !positions) return LA_ERR_INVALID_ARG;
    for (const void* x : {q, k, static_cast<const void*>(q_out), static_cast<const void*>(k_out)})
        if (!aligned(x, esize(dtype))) return LA_ERR_INVALID_ARG;
    if (!aligned(freq, 4) || !aligned(positions, 4)) return LA_ERR_INVALID_ARG;
    const size_t n = (size_t)T * H * d * esize(dtype);
    const Span out[] = {{q_out, n}, {k_out, n}};
    const Span in[] = {{q == q_out ? nullptr : q, n}, {k == k_out ? nullptr : k, n}, {freq, (size_t)P * 4},
                       {positions, (size_t)T * naxes * 4}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    p.q = q; p.k = k; p.q_out = q_out; p.k_out = k_out;
    p.freq = freq; p.positions = positions;
    p.T = T; p.H = H; p.d = d; p.P = (int)P; p.naxes = naxes;
    p.interleaved = interleaved; p.inverse = inverse;
    return result(rotary(p, dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
