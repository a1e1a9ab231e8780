// Gated linear recurrence h_t = a_t h_{t-1} + b_t per channel over packed
// sequences, and its adjoint g_t = dh_t + a_{t+1} g_{t+1} with db = g and
// da_t = g_t h_{t-1}.
//
// The work is two (adjoint: three) flops per element, so the floor is one read
// of every input and one write of every output.  One pass does that: a tile of
// tokens x 64 channels is read into registers once; composing tokens
//     (A, B) o (a, b) = (a A, a B + b)
// gives each warp's and then the tile's product of gates A and state from zero
// B, and once the state that enters the tile is known the recurrence itself
// runs over the registers and the outputs are written.
//
// The entering state comes from the tiles before it.  Every tile publishes its
// (A, B) as soon as it has them and its leaving state once it knows the
// entering one; a tile walks back over at most 32 tiles to the nearest
// published state and applies the (A, B) in between in token order, which are
// the same fused multiply-adds as those of the tiles themselves: the result
// does not depend on which tile was how far.  Tiles are handed out by a ticket in token order, so the
// tiles that a block waits for are held by blocks already running.
//
// A tile that holds a sequence boundary publishes its leaving state at once
// and nothing from before the boundary enters what follows it: no value
// crosses from one sequence to another.  For the adjoint, token order is
// reversed and a boundary is a last token.
#include "internal.h"

namespace la {

namespace {

constexpr int kPrepThreads = 256;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kSlice = 64;           // channels per tile: two per lane
constexpr int kMinTile = kWarps * 8;
constexpr int kMarked = 1, kCut = 2;   // tile_seq: the tile holds a first or last row; one that cuts the recurrence
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kForcedLimitNs = 1000000ull;

// Set by the test hook: look backs then wait for a state that nothing publishes, for 1 ms.
__device__ int g_force_timeout;

__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ int load_acquire(const int* p) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void store_release(int* p, int v) {
    asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

__device__ __forceinline__ int64_t seq_begin(const GatedParams& p, int s) {
    return p.cu_seqlens ? (int64_t)p.cu_seqlens[s] : (int64_t)s * (p.T / p.nseq);
}

// Whether cu_seqlens breaks the packing rules; the whole block takes part.
__device__ bool malformed(const GatedParams& p) {
    bool b = false;
    if (p.cu_seqlens) {
        for (int s = threadIdx.x; s < p.nseq; s += blockDim.x) b |= p.cu_seqlens[s + 1] < p.cu_seqlens[s];
        if (threadIdx.x == 0) b |= p.cu_seqlens[0] != 0 || p.cu_seqlens[p.nseq] != p.T;
    }
    return __syncthreads_or(b) != 0;
}

// Largest s with cu[s] <= t.
__device__ int seq_of(const GatedParams& p, int64_t t) {
    if (!p.cu_seqlens) return (int)(t / (p.T / p.nseq));
    int lo = 0, hi = p.nseq;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (p.cu_seqlens[m] <= t) lo = m; else hi = m;
    }
    return lo;
}

// Clears the header, the ticket and the flags, checks the packing rules and
// notes for each tile the sequence of its first token and whether a boundary
// lies in it.
__global__ void __launch_bounds__(kPrepThreads) gated_prep_kernel(GatedParams p, int tile_tokens, int tiles, int nflags,
                                                                  int reverse) {
    asm volatile("griddepcontrol.launch_dependents;");
    if (blockIdx.x == 0) {
        const bool bad = malformed(p);
        if (threadIdx.x == 0) {
            p.hdr->error = bad ? LA_DEVERR_CU_SEQLENS : LA_DEVERR_NONE;
            p.hdr->n_units = 0;
            p.hdr->range = 0;
            *p.ticket = 0;
        }
    }
    const int step = gridDim.x * kPrepThreads, at = blockIdx.x * kPrepThreads + threadIdx.x;
    for (int i = at; i < nflags; i += step) p.flags[i] = 0;
    for (int i = at; i < tiles; i += step) {
        const int64_t t0 = (int64_t)i * tile_tokens, t1 = min64(t0 + tile_tokens, p.T);
        const int s = seq_of(p, t0);
        const int64_t lo = seq_begin(p, s), hi = seq_begin(p, s + 1);
        const bool first = lo == t0 || hi < t1, last = hi <= t1;   // of some sequence, in the tile
        const bool cut = reverse ? last : first;
        p.tile_seq[i] = s * 4 + (first || last ? kMarked : 0) + (cut ? kCut : 0);
    }
}

// Two neighbouring channels of a row: one vector access where every row is
// aligned for it (Vec), else two.
template <typename T> struct Two;
template <> struct Two<float> {
    float2 v;
    __device__ float2 get() const { return v; }
    __device__ void set(float2 f) { v = f; }
};
template <> struct Two<__nv_bfloat16> {
    __nv_bfloat162 v;
    __device__ float2 get() const { return __bfloat1622float2(v); }
    __device__ void set(float2 f) { v = __floats2bfloat162_rn(f.x, f.y); }
};
template <bool Vec, typename T>
__device__ __forceinline__ Two<T> load_two(const T* p, int left) {   // left: channels of the row from p on
    Two<T> r;
    if (Vec) {
        if (left > 0) r = *reinterpret_cast<const Two<T>*>(p);
        else r.set(make_float2(0.f, 0.f));
    } else {
        r.v.x = left > 0 ? p[0] : T(0.f);
        r.v.y = left > 1 ? p[1] : T(0.f);
    }
    return r;
}
template <bool Vec, typename T>
__device__ __forceinline__ void store_two(T* p, int left, float2 f) {
    Two<T> r;
    r.set(f);
    if (Vec) {
        if (left > 0) *reinterpret_cast<Two<T>*>(p) = r;
    } else {
        if (left > 0) p[0] = r.v.x;
        if (left > 1) p[1] = r.v.y;
    }
}
__device__ __forceinline__ float2 edge_two(const float* p, int left) {
    return make_float2(left > 0 ? p[0] : 0.f, left > 1 ? p[1] : 0.f);
}
__device__ __forceinline__ void store_edge(float* p, int left, float2 f) {
    if (left > 0) p[0] = f.x;
    if (left > 1) p[1] = f.y;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y));
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return make_float2(a.x * b.x, a.y * b.y); }

// (A, B) of a run of tokens for a lane's two channels; a boundary inside it
// makes B the leaving state whatever entered.
struct Run {
    float2 A, B;
};

template <int K>
struct Shared {
    float4 run[kWarps][32];          // (A.x, A.y, B.x, B.y) of each warp's tokens
    int cut[kWarps];                 // a boundary among them
    float2 carry[32];                // state that enters the tile
    int first[kWarps * K], last[kWarps * K];   // the sequence that begins / ends at a row, else -1
    int ticket, next;
};

// Waits (bounded) until a state is published within the 32 tiles before `tile` and every tile after it has its (A, B), and returns the state that
// enters `tile` for the lane's two channels.  One warp.
__device__ float2 look_back(const GatedParams& p, int tile, int slice, int tiles, int lane, bool forced) {
    const int* flags = p.flags + (int64_t)slice * tiles;
    const int mine = tile - 1 - lane;                        // lane 0: the tile just before
    const uint64_t start = now_ns(), limit = forced ? kForcedLimitNs : kWaitLimitNs;
    int back;                                                // tiles between the state found and this one
    for (;;) {
        const int f = forced ? 0 : mine >= 0 ? load_acquire(flags + mine) : 2;
        const unsigned have = __ballot_sync(0xffffffffu, f >= 1), state = __ballot_sync(0xffffffffu, f == 2);
        if (state) {
            back = __ffs(state) - 1;
            const unsigned between = (1u << back) - 1;       // back <= 31
            if ((have & between) == between) break;
        }
        if (__any_sync(0xffffffffu, now_ns() - start > limit)) {
            if (lane == 0) record_error(p.hdr, LA_DEVERR_WAIT_TIMEOUT);
            return make_float2(0.f, 0.f);
        }
    }
    __syncwarp();
    const int c = slice * kSlice + 2 * lane;
    float2 s = make_float2(0.f, 0.f);
    const int from = tile - 1 - back;
    const int Cp = p.Cpad;
    if (from >= 0) s = __ldcg(reinterpret_cast<const float2*>(p.state + (int64_t)from * Cp + c));
#pragma unroll 8
    for (int i = from + 1; i < tile; ++i) {
        const float4 r = __ldcg(reinterpret_cast<const float4*>(p.run + (int64_t)i * Cp + c));
        s = fma2(make_float2(r.x, r.y), s, make_float2(r.z, r.w));
    }
    return s;
}

template <typename TA, typename TX, bool Rev, bool Vec, int K>
__global__ void __launch_bounds__(kThreads, 2) gated_scan_kernel(GatedParams p, int tiles, int slices, int solo) {
    __shared__ Shared<K> sh;
    constexpr int kTile = kWarps * K;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const TA* a = static_cast<const TA*>(p.a);
    const TX* x = static_cast<const TX*>(p.x);
    const TX* h = static_cast<const TX*>(p.h);
    const int64_t C = p.C;

    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (solo) {
        // a single tile of tokens: no other kernel has looked at the arguments
        const bool bad = malformed(p);
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            p.hdr->error = bad ? LA_DEVERR_CU_SEQLENS : LA_DEVERR_NONE;
            p.hdr->n_units = 0;
            p.hdr->range = 0;
        }
        if (bad) return;
    } else if (p.hdr->error == LA_DEVERR_CU_SEQLENS) {
        return;
    }
    const bool forced = !solo && *(volatile int*)&g_force_timeout != 0;

    // an empty sequence passes its state on
    if (p.edge_out && (p.cu_seqlens || p.T == 0)) {
        for (int s0 = blockIdx.x * 32; s0 < p.nseq; s0 += gridDim.x * 32) {
            const int s = s0 + lane;
            unsigned empty = __ballot_sync(0xffffffffu, s < p.nseq && seq_begin(p, s) == seq_begin(p, s + 1));
            for (; empty; empty &= empty - 1) {
                const int64_t at = (int64_t)(s0 + __ffs(empty) - 1) * C;
                for (int c = threadIdx.x; c < p.C; c += kThreads) p.edge_out[at + c] = p.edge_in ? p.edge_in[at + c] : 0.f;
            }
        }
    }

    const int total = tiles * slices;
    int ticket = solo ? blockIdx.x : 0;
    if (!solo) {
        if (threadIdx.x == 0) sh.ticket = atomicAdd(p.ticket, 1);
        __syncthreads();
        ticket = sh.ticket;
    }
    while (ticket < total) {
        const int order = ticket / slices, slice = ticket - order * slices;
        const int tile = Rev ? tiles - 1 - order : order;
        const int64_t t0 = (int64_t)tile * kTile;
        const int n = (int)min64(kTile, p.T - t0);
        const int c = slice * kSlice + 2 * lane, left = p.C - c;
        // the warp's tokens: j = row within the tile, descending for the adjoint
        const int j0 = (Rev ? kWarps - 1 - warp : warp) * K;

        // --- every load of the tile in flight
        Two<TA> ra[K];
        Two<TX> rx[K];
        {
            const int64_t row = (t0 + j0) * C + c;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const bool in = j0 + k < n;
                // the gate into token t of the adjoint is a_{t+1}; a last row has none
                const bool gate = Rev ? t0 + j0 + k + 1 < p.T : in;
                ra[k] = load_two<Vec>(a + row + (k + (Rev ? 1 : 0)) * C, gate ? left : 0);
                rx[k] = load_two<Vec>(x + row + k * C, in ? left : 0);
            }
        }
        int next = 0;
        if (!solo && threadIdx.x == 0) next = atomicAdd(p.ticket, 1);

        // --- boundaries
        const int ts = solo ? kMarked | kCut : p.tile_seq[tile];
        const bool cut_tile = ts & kCut, marked = ts & kMarked;
        if (marked) {
            for (int i = threadIdx.x; i < kTile; i += kThreads) sh.first[i] = sh.last[i] = -1;
            __syncthreads();
            for (int base = ts >> 2; base < p.nseq && seq_begin(p, base) < t0 + n; base += kThreads) {
                const int s = base + threadIdx.x;
                if (s < p.nseq) {
                    const int64_t lo = seq_begin(p, s), hi = seq_begin(p, s + 1);
                    if (hi > lo) {
                        if (lo >= t0 && lo < t0 + n) sh.first[lo - t0] = s;
                        if (hi - 1 >= t0 && hi - 1 < t0 + n) sh.last[hi - 1 - t0] = s;
                    }
                }
            }
            __syncthreads();
        }
        // bit k: a boundary that cuts the recurrence at row j0 + k; and the rows whose state leaves
        unsigned cuts = 0, ends = 0;
        if (marked) {
            const bool f = lane < K && sh.first[j0 + lane] >= 0, l = lane < K && sh.last[j0 + lane] >= 0;
            const unsigned fm = __ballot_sync(0xffffffffu, f), lm = __ballot_sync(0xffffffffu, l);
            cuts = Rev ? lm : fm;
            ends = Rev ? fm : lm;
        }

        // --- the warp's (A, B)
        // The state after the warp's last boundary is kept: edge_out may be edge_in, and the
        // sequence that begins there may be closed by another warp before this one comes back to
        // it.  Sequences of earlier boundaries are closed by this warp itself, after its reads.
        Run r{make_float2(1.f, 1.f), make_float2(0.f, 0.f)};
        float2 open = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int k = Rev ? K - 1 - i : i;
            const float2 g = ra[k].get(), in = rx[k].get();
            if ((cuts >> k) & 1) {
                float2 s = in;
                if (p.edge_in) {
                    const float2 e = edge_two(p.edge_in + (int64_t)(Rev ? sh.last : sh.first)[j0 + k] * C + c, left);
                    s = Rev ? make_float2(in.x + e.x, in.y + e.y) : fma2(g, e, in);
                }
                r.A = make_float2(0.f, 0.f);
                r.B = open = s;
            } else if (j0 + k < n) {
                r.A = mul2(r.A, g);
                r.B = fma2(g, r.B, in);
            }
        }
        sh.run[warp][lane] = make_float4(r.A.x, r.A.y, r.B.x, r.B.y);
        if (lane == 0) sh.cut[warp] = cuts != 0;
        if (threadIdx.x == 0) sh.next = next;
        __syncthreads();

        // --- what stands before the warp within the tile
        Run before{make_float2(1.f, 1.f), make_float2(0.f, 0.f)};
        bool cut_before = false;
        for (int w = 0; w < warp; ++w) {
            const float4 q = sh.run[w][lane];
            if (sh.cut[w]) {
                before.B = make_float2(q.z, q.w);
                cut_before = true;
            } else {
                before.A = mul2(before.A, make_float2(q.x, q.y));
                before.B = fma2(make_float2(q.x, q.y), before.B, make_float2(q.z, q.w));
            }
        }

        // --- the last warp publishes the tile's (A, B), or its leaving state where a boundary cuts it
        Run whole = before;
        if (!solo && warp == kWarps - 1) {
            if (cuts) {
                whole.B = r.B;
            } else {
                whole.A = mul2(whole.A, r.A);
                whole.B = fma2(r.A, whole.B, r.B);
            }
            const int64_t at = (int64_t)order * p.Cpad + c;
            const bool final = cut_tile || order == 0;
            if (final) __stcg(reinterpret_cast<float2*>(p.state + at), whole.B);
            else __stcg(reinterpret_cast<float4*>(p.run + at), make_float4(whole.A.x, whole.A.y, whole.B.x, whole.B.y));
            __threadfence();
            __syncwarp();
            int* flag = p.flags + (int64_t)slice * tiles + order;
            if (lane == 0) store_release(flag, final ? 2 : 1);
            // --- and finds the state that enters it
            float2 s = make_float2(0.f, 0.f);
            const bool fresh = marked && (Rev ? sh.last[n - 1] : sh.first[0]) >= 0;   // nothing enters
            if (!fresh) s = look_back(p, order, slice, tiles, lane, forced);
            sh.carry[lane] = s;
            if (!final) {
                __stcg(reinterpret_cast<float2*>(p.state + at), fma2(whole.A, s, whole.B));
                __threadfence();
                __syncwarp();
                if (lane == 0) store_release(flag, 2);
            }
        }
        if (solo && threadIdx.x < 32) sh.carry[lane] = make_float2(0.f, 0.f);
        Two<TX> rh[Rev ? K : 1];
        if (Rev) {
            const int64_t row = (t0 + j0) * C + c;
#pragma unroll
            for (int k = 0; k < K; ++k)
                rh[k] = load_two<Vec>(h + row + (k - 1) * C, j0 + k < n && t0 + j0 + k > 0 ? left : 0);
        }
        __syncthreads();

        // --- the recurrence from the state that enters the warp
        float2 s = cut_before ? before.B : fma2(before.A, sh.carry[lane], before.B);
        const int64_t row = (t0 + j0) * C + c;
        const unsigned open_at = cuts ? (Rev ? __ffs(cuts) - 1 : 31 - __clz(cuts)) : 32;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int k = Rev ? K - 1 - i : i;
            if (j0 + k >= n) continue;
            const float2 g = ra[k].get(), in = rx[k].get();
            if ((cuts >> k) & 1) {
                s = in;
                if (k == open_at) {
                    s = open;
                } else if (p.edge_in) {
                    const float2 e = edge_two(p.edge_in + (int64_t)(Rev ? sh.last : sh.first)[j0 + k] * C + c, left);
                    s = Rev ? make_float2(in.x + e.x, in.y + e.y) : fma2(g, e, in);
                }
            } else {
                s = fma2(g, s, in);
            }
            store_two<Vec>(static_cast<TX*>(p.y) + row + k * C, left, s);
            float2 leaving = s;
            if (Rev) {
                float2 prev = rh[k].get();
                if ((ends >> k) & 1) {
                    const int q = sh.first[j0 + k];
                    prev = p.state_in ? edge_two(p.state_in + (int64_t)q * C + c, left) : make_float2(0.f, 0.f);
                    if (p.edge_out) leaving = mul2(load_two<Vec>(a + row + k * C, left).get(), s);
                }
                store_two<Vec>(static_cast<TA*>(p.da) + row + k * C, left, mul2(s, prev));
            }
            if (((ends >> k) & 1) && p.edge_out)
                store_edge(p.edge_out + (int64_t)(Rev ? sh.first : sh.last)[j0 + k] * C + c, left, leaving);
        }
        if (solo) return;
        ticket = sh.next;
        __syncthreads();      // the next tile overwrites the shared runs and marks
    }
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
    size_t ticket, flags, tile_seq, run, state, total;
    int slices, Cpad;
};

GatedLayout gated_layout(int64_t T, int C) {
    GatedLayout lo{};
    lo.slices = (int)ceil_div(C, kSlice);
    lo.Cpad = lo.slices * kSlice;
    const size_t tiles = T <= kMinTile ? 0 : (size_t)ceil_div(T, kMinTile);
    size_t o = align_up(sizeof(WsHeader), kAlign);
    lo.ticket = o;   o = align_up(o + sizeof(int), kAlign);
    lo.flags = o;    o = align_up(o + sizeof(int) * tiles * lo.slices, kAlign);
    lo.tile_seq = o; o = align_up(o + sizeof(int) * tiles, kAlign);
    lo.run = o;      o = align_up(o + sizeof(float2) * tiles * lo.Cpad, kAlign);
    lo.state = o;    o = align_up(o + sizeof(float) * tiles * lo.Cpad, kAlign);
    lo.total = o;
    return lo;
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return n;
}

template <typename TA, typename TX, bool Rev, bool Vec, int K>
cudaError_t run_scan(const GatedParams& p, int slices, cudaStream_t s) {
    constexpr int kTile = kWarps * K;
    const int tiles = (int)ceil_div(p.T, kTile);
    const bool solo = tiles <= 1;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    if (solo) {
        cfg.gridDim = dim3((unsigned)slices);
    } else {
        const int nsm = sm_count();
        if (nsm <= 0) return cudaErrorInvalidDevice;
        const int64_t nflags = (int64_t)tiles * slices;
        if (nflags > INT32_MAX / 2) return cudaErrorInvalidValue;
        const int prep = (int)min64(ceil_div(nflags > tiles ? nflags : tiles, kPrepThreads), nsm);
        gated_prep_kernel<<<prep, kPrepThreads, 0, s>>>(p, kTile, tiles, (int)nflags, Rev ? 1 : 0);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3((unsigned)min64(nflags, (int64_t)nsm * 4));
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, gated_scan_kernel<TA, TX, Rev, Vec, K>, p, tiles, slices, solo ? 1 : 0);
}

bool two_aligned(const void* p, size_t esize) { return reinterpret_cast<uintptr_t>(p) % (2 * esize) == 0; }

template <typename TA, typename TX, bool Rev>
cudaError_t dispatch(const GatedParams& p, int slices, cudaStream_t s) {
    const bool vec = p.C % 2 == 0 && two_aligned(p.a, sizeof(TA)) && two_aligned(p.da, sizeof(TA)) &&
                     two_aligned(p.x, sizeof(TX)) && two_aligned(p.h, sizeof(TX)) && two_aligned(p.y, sizeof(TX));
    constexpr int K = 16;
    return vec ? run_scan<TA, TX, Rev, true, K>(p, slices, s) : run_scan<TA, TX, Rev, false, K>(p, slices, s);
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

cudaError_t gated_force_wait_timeout(int enable) { return cudaMemcpyToSymbol(g_force_timeout, &enable, sizeof(int)); }

cudaError_t gated_scan(GatedParams p, int a_dtype, int dtype, int reverse, void* workspace, cudaStream_t s) {
    const GatedLayout lo = gated_layout(p.T, p.C);
    char* ws = static_cast<char*>(workspace);
    p.hdr = reinterpret_cast<WsHeader*>(ws);
    p.ticket = reinterpret_cast<int*>(ws + lo.ticket);
    p.flags = reinterpret_cast<int*>(ws + lo.flags);
    p.tile_seq = reinterpret_cast<int*>(ws + lo.tile_seq);
    p.run = reinterpret_cast<float2*>(ws + lo.run);
    p.state = reinterpret_cast<float*>(ws + lo.state);
    p.Cpad = lo.Cpad;
    auto go = [&](auto ta, auto tx) -> cudaError_t {
        using TA = decltype(ta);
        using TX = decltype(tx);
        return reverse ? dispatch<TA, TX, true>(p, lo.slices, s) : dispatch<TA, TX, false>(p, lo.slices, s);
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
