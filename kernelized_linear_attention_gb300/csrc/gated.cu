// Gated linear recurrence h_t = a_t h_{t-1} + b_t per channel over packed
// sequences, and its adjoint g_t = dh_t + a_{t+1} g_{t+1}.
//
// Tokens are cut into tiles.  A first pass gives, per tile and channel, the
// product of the gates and the state from zero; a second carries the state
// over the tiles; a third runs the recurrence inside each tile from the state
// that enters it.  A tile that holds a sequence boundary passes nothing on
// from before it, so no value crosses from one sequence to another.
#include "internal.h"

namespace la {

namespace {

constexpr int kTile = 128;         // tokens per tile
constexpr int kPrepThreads = 256;
constexpr int kScanThreads = 128;  // one channel per thread

// Clears the header, checks the packing rules and finds the sequence that
// holds each tile's first token.
__global__ void __launch_bounds__(kPrepThreads) gated_prep_kernel(GatedParams p, int tiles) {
    if (blockIdx.x == 0) {
        __shared__ int bad;
        if (threadIdx.x == 0) {
            bad = 0;
            p.hdr->n_units = 0;
            p.hdr->range = 0;
        }
        __syncthreads();
        if (p.cu_seqlens) {
            bool b = false;
            for (int s = threadIdx.x; s < p.nseq; s += kPrepThreads) b |= p.cu_seqlens[s + 1] < p.cu_seqlens[s];
            if (threadIdx.x == 0) b |= p.cu_seqlens[0] != 0 || p.cu_seqlens[p.nseq] != p.T;
            if (b) bad = 1;
            __syncthreads();
        }
        if (threadIdx.x == 0) p.hdr->error = bad ? LA_DEVERR_CU_SEQLENS : LA_DEVERR_NONE;
    }
    for (int i = blockIdx.x * kPrepThreads + threadIdx.x; i < tiles; i += gridDim.x * kPrepThreads) {
        const int64_t t = (int64_t)i * kTile;
        int s;
        if (p.cu_seqlens) {
            int lo = 0, hi = p.nseq;   // largest s in [0, nseq) with cu[s] <= t
            while (hi - lo > 1) {
                const int m = (lo + hi) >> 1;
                if (p.cu_seqlens[m] <= t) lo = m; else hi = m;
            }
            s = lo;
        } else {
            s = (int)(t / (p.T / p.nseq));
        }
        p.tile_seq[i] = s;
    }
}

__device__ __forceinline__ int64_t seq_begin(const GatedParams& p, int s) {
    return p.cu_seqlens ? (int64_t)p.cu_seqlens[s] : (int64_t)s * (p.T / p.nseq);
}

// first[i] / last[i]: the sequence whose first / last token is row t0 + i, else -1.
__device__ void mark_rows(const GatedParams& p, int tile, int64_t t0, int n, int* first, int* last) {
    for (int i = threadIdx.x; i < kTile; i += blockDim.x) first[i] = last[i] = -1;
    __syncthreads();
    for (int base = p.tile_seq[tile]; base < p.nseq && seq_begin(p, base) < t0 + n; base += blockDim.x) {
        const int s = base + threadIdx.x;
        if (s < p.nseq) {
            const int64_t lo = seq_begin(p, s), hi = seq_begin(p, s + 1);
            if (hi > lo) {
                if (lo >= t0 && lo < t0 + n) first[lo - t0] = s;
                if (hi - 1 >= t0 && hi - 1 < t0 + n) last[hi - 1 - t0] = s;
            }
        }
    }
    __syncthreads();
}

template <typename TA, typename TX, bool Rev>
__global__ void __launch_bounds__(kScanThreads) gated_tile_kernel(GatedParams p) {
    __shared__ int first[kTile], last[kTile];
    if (p.hdr->error) return;
    const int tile = blockIdx.x;
    const int64_t t0 = (int64_t)tile * kTile;
    const int n = (int)min64(kTile, p.T - t0);
    mark_rows(p, tile, t0, n, first, last);
    const int c = blockIdx.y * kScanThreads + threadIdx.x;
    if (c >= p.C) return;
    const TA* a = static_cast<const TA*>(p.a);
    const TX* x = static_cast<const TX*>(p.x);
    float prod = 1.f, state = 0.f, head = 0.f;
    for (int i = 0; i < n; ++i) {
        const int j = Rev ? n - 1 - i : i;
        const int64_t at = (t0 + j) * p.C + c;
        const int s = Rev ? last[j] : first[j];
        const float in = load_elem(x, at);
        if (s >= 0) {
            prod = 0.f;
            state = in;
            if (p.edge_in) {
                const float e = p.edge_in[(int64_t)s * p.C + c];
                head = state = Rev ? in + e : fmaf(load_elem(a, at), e, in);
            }
        } else {
            const float g = load_elem(a, Rev ? at + p.C : at);
            prod *= g;
            state = fmaf(g, state, in);
        }
    }
    p.agg[(int64_t)tile * p.C + c] = make_float2(prod, state);
    p.head[(int64_t)tile * p.C + c] = head;
}

template <bool Rev>
__global__ void __launch_bounds__(kScanThreads) gated_carry_kernel(GatedParams p, int tiles) {
    if (p.hdr->error) return;
    const int c = blockIdx.x * kScanThreads + threadIdx.x;
    if (c >= p.C) return;
    float state = 0.f;
    for (int i = 0; i < tiles; ++i) {
        const int tile = Rev ? tiles - 1 - i : i;
        const int64_t at = (int64_t)tile * p.C + c;
        p.carry[at] = state;
        // a sequence that begins (adjoint: ends) in the tile cuts the carry
        const int64_t t0 = (int64_t)tile * kTile, t1 = min64(t0 + kTile, p.T);
        const int s = p.tile_seq[tile];
        const bool cut = Rev ? (t1 == p.T || p.tile_seq[tile + 1] != s || seq_begin(p, s + 1) <= t1)
                             : (seq_begin(p, s) == t0 || seq_begin(p, s + 1) < t1);
        const float2 ag = p.agg[at];
        state = cut ? ag.y : fmaf(ag.x, state, ag.y);
    }
}

template <typename TA, typename TX, bool Rev>
__global__ void __launch_bounds__(kScanThreads) gated_apply_kernel(GatedParams p) {
    __shared__ int first[kTile], last[kTile];
    if (p.hdr->error) return;
    const int tile = blockIdx.x;
    const int64_t t0 = (int64_t)tile * kTile;
    const int n = (int)min64(kTile, p.T - t0);
    mark_rows(p, tile, t0, n, first, last);
    const int c = blockIdx.y * kScanThreads + threadIdx.x;
    if (c >= p.C) return;
    const TA* a = static_cast<const TA*>(p.a);
    const TX* x = static_cast<const TX*>(p.x);
    float state = p.carry[(int64_t)tile * p.C + c];
    // edge_out may be edge_in: where the tile's last boundary opens a sequence that another tile
    // closes, its first state comes from the first pass (the others are read before this thread
    // writes them)
    int open = -1;
    for (int i = 0; i < n; ++i) {
        const int j = Rev ? n - 1 - i : i;
        if ((Rev ? last[j] : first[j]) >= 0) open = j;
    }
    for (int i = 0; i < n; ++i) {
        const int j = Rev ? n - 1 - i : i;
        const int64_t at = (t0 + j) * p.C + c;
        const float in = load_elem(x, at);
        const int s = Rev ? last[j] : first[j];
        if (s >= 0) {
            state = in;
            if (p.edge_in && j == open) {
                state = p.head[(int64_t)tile * p.C + c];
            } else if (p.edge_in) {
                const float e = p.edge_in[(int64_t)s * p.C + c];
                state = Rev ? in + e : fmaf(load_elem(a, at), e, in);
            }
        } else {
            state = fmaf(load_elem(a, Rev ? at + p.C : at), state, in);
        }
        store_elem(static_cast<TX*>(p.y), at, state);
        if (Rev) {
            const int f = first[j];
            float before;
            if (f >= 0) before = p.state_in ? p.state_in[(int64_t)f * p.C + c] : 0.f;
            else before = load_elem(static_cast<const TX*>(p.h), at - p.C);
            store_elem(static_cast<TA*>(p.da), at, state * before);
            if (f >= 0 && p.edge_out) p.edge_out[(int64_t)f * p.C + c] = load_elem(a, at) * state;
        } else if (last[j] >= 0 && p.edge_out) {
            p.edge_out[(int64_t)last[j] * p.C + c] = state;
        }
    }
}

// An empty sequence passes its state on.
__global__ void __launch_bounds__(kScanThreads) gated_empty_kernel(GatedParams p) {
    if (p.hdr->error) return;
    for (int s = blockIdx.x; s < p.nseq; s += gridDim.x)
        if (seq_begin(p, s) == seq_begin(p, s + 1))
            for (int c = threadIdx.x; c < p.C; c += kScanThreads)
                p.edge_out[(int64_t)s * p.C + c] = p.edge_in ? p.edge_in[(int64_t)s * p.C + c] : 0.f;
}

template <typename TA, typename TX>
__global__ void __launch_bounds__(kPrepThreads) gated_step_kernel(const TA* a, const TX* b, int64_t n,
                                                                  const float* state_in, float* state_out, TX* h) {
    const int64_t i = (int64_t)blockIdx.x * kPrepThreads + threadIdx.x;
    if (i >= n) return;
    const float s = fmaf(load_elem(a, i), state_in[i], load_elem(b, i));
    state_out[i] = s;
    store_elem(h, i, s);
}

struct GatedLayout {
    size_t tile_seq, agg, carry, head, total;
    int tiles;
};

GatedLayout gated_layout(int64_t T, int C) {
    GatedLayout lo{};
    lo.tiles = (int)ceil_div(T, kTile);
    size_t o = align_up(sizeof(WsHeader), kAlign);
    lo.tile_seq = o; o = align_up(o + sizeof(int) * (size_t)lo.tiles, kAlign);
    lo.agg = o;      o = align_up(o + sizeof(float2) * (size_t)lo.tiles * C, kAlign);
    lo.carry = o;    o = align_up(o + sizeof(float) * (size_t)lo.tiles * C, kAlign);
    lo.head = o;     o = align_up(o + sizeof(float) * (size_t)lo.tiles * C, kAlign);
    lo.total = o;
    return lo;
}

template <typename TA, typename TX, bool Rev>
cudaError_t run_scan(const GatedParams& p, int tiles, cudaStream_t s) {
    const int prep = (int)min64(ceil_div(tiles, kPrepThreads) + 1, 64);
    gated_prep_kernel<<<prep, kPrepThreads, 0, s>>>(p, tiles);
    if (tiles > 0) {
        const dim3 grid((unsigned)tiles, (unsigned)ceil_div(p.C, kScanThreads));
        gated_tile_kernel<TA, TX, Rev><<<grid, kScanThreads, 0, s>>>(p);
        gated_carry_kernel<Rev><<<(unsigned)ceil_div(p.C, kScanThreads), kScanThreads, 0, s>>>(p, tiles);
        gated_apply_kernel<TA, TX, Rev><<<grid, kScanThreads, 0, s>>>(p);
    }
    if (p.edge_out && (p.cu_seqlens || p.T == 0))
        gated_empty_kernel<<<(unsigned)min64(p.nseq, 1024), kScanThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename TA, typename TX>
cudaError_t step(const void* a, const void* b, int64_t n, const float* state_in, float* state_out, void* h,
                 cudaStream_t s) {
    gated_step_kernel<TA, TX><<<(unsigned)ceil_div(n, kPrepThreads), kPrepThreads, 0, s>>>(
        static_cast<const TA*>(a), static_cast<const TX*>(b), n, state_in, state_out, static_cast<TX*>(h));
    return cudaGetLastError();
}

}  // namespace

size_t gated_workspace_bytes(int64_t T, int C) { return gated_layout(T, C).total; }

cudaError_t gated_scan(GatedParams p, int a_dtype, int dtype, int reverse, void* workspace, cudaStream_t s) {
    const GatedLayout lo = gated_layout(p.T, p.C);
    char* ws = static_cast<char*>(workspace);
    p.hdr = reinterpret_cast<WsHeader*>(ws);
    p.tile_seq = reinterpret_cast<int*>(ws + lo.tile_seq);
    p.agg = reinterpret_cast<float2*>(ws + lo.agg);
    p.carry = reinterpret_cast<float*>(ws + lo.carry);
    p.head = reinterpret_cast<float*>(ws + lo.head);
    auto go = [&](auto ta, auto tx) -> cudaError_t {
        using TA = decltype(ta);
        using TX = decltype(tx);
        return reverse ? run_scan<TA, TX, true>(p, lo.tiles, s) : run_scan<TA, TX, false>(p, lo.tiles, s);
    };
    const float f = 0.f;
    const __nv_bfloat16 h{};
    if (a_dtype == LA_F32) return dtype == LA_F32 ? go(f, f) : go(f, h);
    return dtype == LA_F32 ? go(h, f) : go(h, h);
}

cudaError_t gated_step(const void* a, const void* b, int a_dtype, int dtype, int64_t n, const float* state_in,
                       float* state_out, void* h, cudaStream_t s) {
    if (a_dtype == LA_F32)
        return dtype == LA_F32 ? step<float, float>(a, b, n, state_in, state_out, h, s)
                               : step<float, __nv_bfloat16>(a, b, n, state_in, state_out, h, s);
    return dtype == LA_F32 ? step<__nv_bfloat16, float>(a, b, n, state_in, state_out, h, s)
                           : step<__nv_bfloat16, __nv_bfloat16>(a, b, n, state_in, state_out, h, s);
}

}  // namespace la
