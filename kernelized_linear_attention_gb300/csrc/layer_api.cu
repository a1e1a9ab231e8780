// C entry points of the operators around the attention call (gated linear
// recurrence, layer norm, rotary positions, norm of queries and keys) and of
// linear attention with a decay for each head: argument checks and dispatch.
#include <cmath>

#include "ops/decay.h"
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

la_status decay_dims(int dtype, bool has_cu, int nseq, int64_t T, int H, int dk, int dv) {
    if (!dtype_ok(dtype) || nseq < 1 || nseq > 65535 || H < 1 || H > 65535 || dk < 1 || dv < 1) return LA_ERR_INVALID_ARG;
    if (T < 0 || T > (int64_t)INT32_MAX) return LA_ERR_INVALID_ARG;
    if (!has_cu && T % nseq != 0) return LA_ERR_INVALID_ARG;
    // (tokens of a chunk behind the last one are counted in 32 bits)
    if (dk > LA_MAX_DK || dv > LA_MAX_DV || T > (int64_t)INT32_MAX - 1024) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

DecayCall decay_call(const float* log_decay, const int32_t* cu_seqlens, int nseq, int64_t T, int H, int dk, int dv,
                     float scale) {
    DecayCall c{};
    c.log_decay = log_decay;
    c.cu_seqlens = cu_seqlens;
    c.nseq = nseq;
    c.T = T;
    c.H = H;
    c.dk = dk;
    c.dv = dv;
    c.scale = scale;
    return c;
}

la_status turns(Turns& p, const float* freq, const int32_t* positions, int d, const int* pairs, int naxes,
                int interleaved, int inverse) {
    if (naxes < 1 || pairs == nullptr || (interleaved & ~1) || (inverse & ~1)) return LA_ERR_INVALID_ARG;
    if (naxes > LA_MAX_AXES || d > LA_MAX_ROTARY_D) return LA_ERR_UNSUPPORTED;
    int64_t P = 0;
    for (int i = 0; i < naxes; ++i) {
        if (pairs[i] < 0) return LA_ERR_INVALID_ARG;
        p.first[i] = (int)P;
        P += pairs[i];
        if (2 * P > d) return LA_ERR_INVALID_ARG;
    }
    for (int i = naxes; i <= LA_MAX_AXES; ++i) p.first[i] = (int)P;
    if (P < 1) return LA_ERR_INVALID_ARG;
    p.freq = freq;
    p.positions = positions;
    p.P = (int)P;
    p.naxes = naxes;
    p.interleaved = interleaved;
    p.inverse = inverse;
    return LA_OK;
}

// Rows [T][H][d] whose tokens are `stride` elements apart: q and k of the norm with rotation.
la_status qk_dims(int dtype, int64_t T, int Hq, int Hk, int d, int64_t q_stride, int64_t k_stride, int per_head) {
    if (!dtype_ok(dtype) || T < 0 || T > (int64_t)INT32_MAX || Hq < 1 || Hq > 65535 || Hk < 0 || Hk > 65535 || d < 2 ||
        (per_head & ~1))
        return LA_ERR_INVALID_ARG;
    if (q_stride < (int64_t)Hq * d || k_stride < (int64_t)Hk * d) return LA_ERR_INVALID_ARG;
    if ((int64_t)(Hq + Hk) * d > LA_MAX_CHANNELS || q_stride > INT32_MAX || k_stride > INT32_MAX) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}
size_t strided_bytes(int64_t T, int H, int d, int64_t stride, int dtype) {
    return T < 1 ? 0 : ((size_t)(T - 1) * stride + (size_t)H * d) * esize(dtype);
}

// Bytes of workspace; `some` stands for a cu_seqlens that is not read.
size_t decay_bytes(int dtype, bool has_cu, int nseq, int64_t T, int H, int dk, int dv, bool backward) {
    static const int32_t some = 0;
    if (decay_dims(dtype, has_cu, nseq, T, H, dk, dv) != LA_OK) return 0;
    DecayCall c = decay_call(nullptr, has_cu ? &some : nullptr, nseq, T, H, dk, dv, 1.f);
    return decay_layout(c, dtype, backward, nullptr);
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

size_t la_decay_attention_workspace_bytes(int dtype, int has_cu_seqlens, int nseq, int64_t T, int H, int d_k, int d_v) {
    return decay_bytes(dtype, has_cu_seqlens != 0, nseq, T, H, d_k, d_v, false);
}

la_status la_decay_attention(const void* q, const void* k, const void* v, const float* log_decay, int dtype,
                             const int32_t* cu_seqlens, int nseq, int64_t T, int H, int d_k, int d_v, float scale,
                             const float* state_in, float* state_out, void* out, void* workspace,
                             size_t workspace_bytes, void* stream) {
    la_status st = decay_dims(dtype, cu_seqlens != nullptr, nseq, T, H, d_k, d_v);
    if (st != LA_OK) return st;
    if (!std::isfinite(scale) || !log_decay || !aligned(log_decay, 4)) return LA_ERR_INVALID_ARG;
    if (workspace == nullptr || !aligned(workspace, kAlign)) return LA_ERR_INVALID_ARG;
    if (T > 0 && (!q || !k || !v || !out)) return LA_ERR_INVALID_ARG;
    for (const void* x : {q, k, v, static_cast<const void*>(out)})
        if (!aligned(x, esize(dtype))) return LA_ERR_INVALID_ARG;
    if (!aligned(state_in, 4) || !aligned(state_out, 4) || !aligned(cu_seqlens, 4)) return LA_ERR_INVALID_ARG;
    DecayCall c = decay_call(log_decay, cu_seqlens, nseq, T, H, d_k, d_v, scale);
    const size_t need = decay_layout(c, dtype, false, workspace);
    if (workspace_bytes < need) return LA_ERR_WORKSPACE;
    const size_t nk = (size_t)T * H * d_k * esize(dtype), nv = (size_t)T * H * d_v * esize(dtype);
    const size_t ns = sizeof(float) * (size_t)nseq * H * d_k * d_v;
    const Span outs[] = {{out, nv}, {state_out, ns}, {workspace, need}};
    const Span ins[] = {{q, nk}, {k, nk}, {v, nv}, {log_decay, (size_t)H * 4},
                        {state_in == state_out ? nullptr : state_in, ns},
                        {cu_seqlens, sizeof(int32_t) * ((size_t)nseq + 1)}};
    if (!disjoint(outs, ins)) return LA_ERR_INVALID_ARG;
    return result(decay_forward(c, q, k, v, dtype, state_in, state_out, out, static_cast<cudaStream_t>(stream)));
}

size_t la_decay_attention_backward_workspace_bytes(int dtype, int has_cu_seqlens, int nseq, int64_t T, int H, int d_k,
                                                   int d_v) {
    return decay_bytes(dtype, has_cu_seqlens != 0, nseq, T, H, d_k, d_v, true);
}

la_status la_decay_attention_backward(const void* q, const void* k, const void* v, const void* dout,
                                      const float* log_decay, int dtype, const int32_t* cu_seqlens, int nseq, int64_t T,
                                      int H, int d_k, int d_v, float scale, const float* state_in,
                                      const float* dstate_out, void* dq, void* dk, void* dv, float* dstate_in,
                                      void* workspace, size_t workspace_bytes, void* stream) {
    la_status st = decay_dims(dtype, cu_seqlens != nullptr, nseq, T, H, d_k, d_v);
    if (st != LA_OK) return st;
    if (!std::isfinite(scale) || !log_decay || !aligned(log_decay, 4)) return LA_ERR_INVALID_ARG;
    if (workspace == nullptr || !aligned(workspace, kAlign)) return LA_ERR_INVALID_ARG;
    if (T > 0 && (!q || !k || !v || !dout || !dq || !dk || !dv)) return LA_ERR_INVALID_ARG;
    for (const void* x : {q, k, v, dout, static_cast<const void*>(dq), static_cast<const void*>(dk),
                          static_cast<const void*>(dv)})
        if (!aligned(x, esize(dtype))) return LA_ERR_INVALID_ARG;
    if (!aligned(state_in, 4) || !aligned(dstate_out, 4) || !aligned(dstate_in, 4) || !aligned(cu_seqlens, 4))
        return LA_ERR_INVALID_ARG;
    DecayCall c = decay_call(log_decay, cu_seqlens, nseq, T, H, d_k, d_v, scale);
    const size_t need = decay_layout(c, dtype, true, workspace);
    if (workspace_bytes < need) return LA_ERR_WORKSPACE;
    const size_t nk = (size_t)T * H * d_k * esize(dtype), nv = (size_t)T * H * d_v * esize(dtype);
    const size_t ns = sizeof(float) * (size_t)nseq * H * d_k * d_v;
    const Span outs[] = {{dq, nk}, {dk, nk}, {dv, nv}, {dstate_in, ns}, {workspace, need}};
    const Span ins[] = {{q, nk}, {k, nk}, {v, nv}, {dout, nv}, {log_decay, (size_t)H * 4}, {state_in, ns},
                        {dstate_out == dstate_in ? nullptr : dstate_out, ns},
                        {cu_seqlens, sizeof(int32_t) * ((size_t)nseq + 1)}};
    if (!disjoint(outs, ins)) return LA_ERR_INVALID_ARG;
    return result(decay_backward(c, q, k, v, dout, dtype, state_in, dstate_out, dq, dk, dv, dstate_in,
                                 static_cast<cudaStream_t>(stream)));
}

la_status la_decay_step(const void* q, const void* k, const void* v, const float* log_decay, int dtype, int B, int H,
                        int d_k, int d_v, float scale, const float* state_in, float* state_out, void* out,
                        void* stream) {
    if (B < 0) return LA_ERR_INVALID_ARG;
    la_status st = decay_dims(dtype, true, 1, B, H, d_k, d_v);
    if (st != LA_OK) return st;
    if (!std::isfinite(scale)) return LA_ERR_INVALID_ARG;
    if ((int64_t)B * H > (int64_t)INT32_MAX) return LA_ERR_UNSUPPORTED;
    if (B == 0) return LA_OK;
    if (!q || !k || !v || !log_decay || !state_in || !state_out || !out) return LA_ERR_INVALID_ARG;
    for (const void* x : {q, k, v, static_cast<const void*>(out)})
        if (!aligned(x, esize(dtype))) return LA_ERR_INVALID_ARG;
    if (!aligned(log_decay, 4) || !aligned(state_in, 4) || !aligned(state_out, 4)) return LA_ERR_INVALID_ARG;
    const size_t nk = (size_t)B * H * d_k * esize(dtype), nv = (size_t)B * H * d_v * esize(dtype);
    const size_t ns = sizeof(float) * (size_t)B * H * d_k * d_v;
    const Span outs[] = {{out, nv}, {state_out, ns}};
    const Span ins[] = {{q, nk}, {k, nk}, {v, nv}, {log_decay, (size_t)H * 4},
                        {state_in == state_out ? nullptr : state_in, ns}};
    if (!disjoint(outs, ins)) return LA_ERR_INVALID_ARG;
    return result(decay_step(q, k, v, log_decay, dtype, B, H, d_k, d_v, scale, state_in, state_out, out,
                             static_cast<cudaStream_t>(stream)));
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
    RotaryParams p{};
    const la_status st = turns(p, freq, positions, d, pairs, naxes, interleaved, inverse);
    if (st != LA_OK) return st;
    if ((k == nullptr) != (k_out == nullptr)) return LA_ERR_INVALID_ARG;
    if (T == 0) return LA_OK;
    if (!q || !q_out || !freq || !positions) return LA_ERR_INVALID_ARG;
    for (const void* x : {q, k, static_cast<const void*>(q_out), static_cast<const void*>(k_out)})
        if (!aligned(x, esize(dtype))) return LA_ERR_INVALID_ARG;
    if (!aligned(freq, 4) || !aligned(positions, 4)) return LA_ERR_INVALID_ARG;
    const size_t n = (size_t)T * H * d * esize(dtype);
    const Span out[] = {{q_out, n}, {k_out, n}};
    const Span in[] = {{q == q_out ? nullptr : q, n}, {k == k_out ? nullptr : k, n}, {freq, (size_t)p.P * 4},
                       {positions, (size_t)T * naxes * 4}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    p.q = q; p.k = k; p.q_out = q_out; p.k_out = k_out;
    p.T = T; p.H = H; p.d = d;
    return result(rotary(p, dtype, static_cast<cudaStream_t>(stream)));
}

la_status la_qk_norm_rotary(const void* q, const void* k, const float* q_weight, const float* k_weight,
                            const float* freq, const int32_t* positions, int dtype, int64_t T, int Hq, int Hk, int d,
                            int64_t q_stride, int64_t k_stride, const int* pairs, int naxes, int interleaved,
                            int per_head, float eps, void* q_out, void* k_out, float* q_rstd, float* k_rstd,
                            void* stream) {
    la_status st = qk_dims(dtype, T, Hq, Hk, d, q_stride, k_stride, per_head);
    if (st != LA_OK) return st;
    QkNormParams p{};
    st = turns(p, freq, positions, d, pairs, naxes, interleaved, 0);
    if (st != LA_OK) return st;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return LA_ERR_INVALID_ARG;
    if (T == 0) return LA_OK;
    if (!q || !q_out || !freq || !positions || (Hk > 0 && (!k || !k_out)) || (Hk == 0 && (k || k_out || k_rstd)))
        return LA_ERR_INVALID_ARG;
    for (const void* x : {q, k, static_cast<const void*>(q_out), static_cast<const void*>(k_out)})
        if (!aligned(x, esize(dtype))) return LA_ERR_INVALID_ARG;
    for (const float* x : {q_weight, k_weight, freq, static_cast<const float*>(q_rstd), static_cast<const float*>(k_rstd)})
        if (!aligned(x, 4)) return LA_ERR_INVALID_ARG;
    if (!aligned(positions, 4)) return LA_ERR_INVALID_ARG;
    const size_t nq = (size_t)T * Hq * d * esize(dtype), nk = (size_t)T * Hk * d * esize(dtype);
    const size_t wq = (size_t)(per_head ? Hq : 1) * d * 4, wk = (size_t)(per_head ? Hk : 1) * d * 4;
    const bool q_place = q == q_out && q_stride == (int64_t)Hq * d, k_place = k == k_out && k_stride == (int64_t)Hk * d;
    const Span out[] = {{q_out, nq}, {k_out, nk}, {q_rstd, (size_t)T * Hq * 4}, {k_rstd, (size_t)T * Hk * 4}};
    const Span in[] = {{q_place ? nullptr : q, strided_bytes(T, Hq, d, q_stride, dtype)},
                       {k_place ? nullptr : k, strided_bytes(T, Hk, d, k_stride, dtype)}, {q_weight, wq}, {k_weight, wk},
                       {freq, (size_t)p.P * 4}, {positions, (size_t)T * naxes * 4}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    p.x[0] = q; p.x[1] = k;
    p.y[0] = q_out; p.y[1] = k_out;
    p.w[0] = q_weight; p.w[1] = k_weight;
    p.rstd[0] = q_rstd; p.rstd[1] = k_rstd;
    p.stride[0] = q_stride; p.stride[1] = k_stride;
    p.T = T; p.H[0] = Hq; p.H[1] = Hk; p.d = d; p.per_head = per_head; p.eps = eps;
    return result(qk_norm_rotary(p, dtype, static_cast<cudaStream_t>(stream)));
}

size_t la_qk_norm_rotary_backward_workspace_bytes(int dtype, int64_t T, int Hq, int Hk, int d) {
    if (qk_dims(dtype, T, Hq, Hk, d, (int64_t)Hq * d, (int64_t)Hk * d, 0) != LA_OK || d > LA_MAX_ROTARY_D) return 0;
    return qk_norm_rotary_backward_workspace_bytes(T, Hq + Hk, d);
}

la_status la_qk_norm_rotary_backward(const void* q, const void* k, const float* q_rstd, const float* k_rstd,
                                     const void* dq_out, const void* dk_out, const float* q_weight,
                                     const float* k_weight, const float* freq, const int32_t* positions, int dtype,
                                     int64_t T, int Hq, int Hk, int d, int64_t q_stride, int64_t k_stride,
                                     const int* pairs, int naxes, int interleaved, int per_head, void* dq, void* dk,
                                     float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                                     void* stream) {
    la_status st = qk_dims(dtype, T, Hq, Hk, d, q_stride, k_stride, per_head);
    if (st != LA_OK) return st;
    QkNormParams p{};
    st = turns(p, freq, positions, d, pairs, naxes, interleaved, 1);
    if (st != LA_OK) return st;
    if (workspace == nullptr || !aligned(workspace, kAlign)) return LA_ERR_INVALID_ARG;
    if (Hk == 0 && (k || dk_out || dk || k_rstd || k_weight || dk_weight)) return LA_ERR_INVALID_ARG;
    if (T > 0 && (!q || !q_rstd || !dq_out || !dq || !freq || !positions ||
                  (Hk > 0 && (!k || !k_rstd || !dk_out || !dk))))
        return LA_ERR_INVALID_ARG;
    for (const void* x : {q, k, dq_out, dk_out, static_cast<const void*>(dq), static_cast<const void*>(dk)})
        if (!aligned(x, esize(dtype))) return LA_ERR_INVALID_ARG;
    for (const float* x : {q_rstd, k_rstd, q_weight, k_weight, freq, static_cast<const float*>(dq_weight),
                           static_cast<const float*>(dk_weight)})
        if (!aligned(x, 4)) return LA_ERR_INVALID_ARG;
    if (!aligned(positions, 4)) return LA_ERR_INVALID_ARG;
    const size_t need = qk_norm_rotary_backward_workspace_bytes(T, Hq + Hk, d);
    if (need == 0) return LA_ERR_CUDA;
    if (workspace_bytes < need) return LA_ERR_WORKSPACE;
    const size_t nq = (size_t)T * Hq * d * esize(dtype), nk = (size_t)T * Hk * d * esize(dtype);
    const size_t wq = (size_t)(per_head ? Hq : 1) * d * 4, wk = (size_t)(per_head ? Hk : 1) * d * 4;
    const Span out[] = {{dq, nq}, {dk, nk}, {dq_weight, wq}, {dk_weight, wk}, {workspace, need}};
    const Span in[] = {{q, strided_bytes(T, Hq, d, q_stride, dtype)}, {k, strided_bytes(T, Hk, d, k_stride, dtype)},
                       {q_rstd, (size_t)T * Hq * 4}, {k_rstd, (size_t)T * Hk * 4}, {dq_out, nq}, {dk_out, nk},
                       {q_weight, wq}, {k_weight, wk}, {freq, (size_t)p.P * 4}, {positions, (size_t)T * naxes * 4}};
    if (!disjoint(out, in)) return LA_ERR_INVALID_ARG;
    p.x[0] = q; p.x[1] = k;
    p.dy[0] = dq_out; p.dy[1] = dk_out;
    p.y[0] = dq; p.y[1] = dk;
    p.w[0] = q_weight; p.w[1] = k_weight;
    p.rstd[0] = const_cast<float*>(q_rstd); p.rstd[1] = const_cast<float*>(k_rstd);
    p.dw[0] = dq_weight; p.dw[1] = dk_weight;
    p.partial = dq_weight || dk_weight ? static_cast<float*>(workspace) : nullptr;
    p.stride[0] = q_stride; p.stride[1] = k_stride;
    p.T = T; p.H[0] = Hq; p.H[1] = Hk; p.d = d; p.per_head = per_head;
    return result(qk_norm_rotary_backward(p, dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
