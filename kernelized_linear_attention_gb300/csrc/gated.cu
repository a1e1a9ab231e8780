// Gated linear recurrence h_t = a_t h_{t-1} + b_t per channel over packed
// sequences, and its adjoint g_t = dh_t + a_{t+1} g_{t+1} with db = g and
// da_t = g_t h_{t-1}.
//
// The work is two (adjoint: three) flops per element, so the floor is one read
// of every input and one write of every output.  One pass does that: a tile of
// tokens x 64 channels is read once; composing tokens
//     (A, B) o (a, b) = (a A, a B + b)
// gives each warp's and then the tile's product of gates A and state from zero
// B, and once the state that enters the tile is known the recurrence itself
// runs over the tile and the outputs are written.
//
// The entering state comes from the tiles before it.  Every tile publishes its
// (A, B) as soon as it has them, which waits for nothing.  Eight tiles in scan
// order form a group, whose last tile publishes the group's joint (A, B) as
// soon as it sees the others', and eight groups a block of 64 tiles, whose last
// tile publishes the state that leaves it.  A tile applies the groups before it
// in its block and the tiles before it in its group to the state that left the
// block before, always in token order, so the result does not depend on timing;
// the only serial chain is one trip to L2 per 64 tiles.  (With a state per tile
// and a walk back to the nearest one the chain took 0.17 us a tile, 190 us for
// 65536 tokens; with a state per 16 tiles 107 us.)  A published word says
// itself that it is there (it is no longer kUnset), so a publication needs no
// fence.  Tiles are handed out by a ticket in token order: the tiles that a
// thread block waits for are held by thread blocks already running, and the
// earliest unfinished tile never waits.
//
// A product of gates (up to one) below fp32's normal range is off by up to 2^-150 for each of at most 32 tokens of a
// warp, 4 warps and 8 tiles, so by less than 2^-144, and what a state of up to 2^20 adds through it by less than
// 2^-124.  A larger state that outweighs what the run's tokens add (an infinite one stays infinite however often it is
// halved) goes through them one by one (Channel).  Looking out for these runs costs 1 to 2.5 percent, 6 with odd bf16
// rows; states beyond 2^20 with products below the range take the slower way that looks at every run (65536 x 1024
// with inputs of 1e8 and gates below 0.3 0.5 ms, with an infinite state in every channel 15 ms).
//
// A tile that holds a sequence boundary publishes kCutTag for A: B is the state
// that leaves it whatever entered, so no value crosses from one sequence to
// another.  For the adjoint, token order is reversed and a boundary is a last
// token.
//
// Measured (GB300, 6.76 TB/s copies): 65536 x 1024 with fp32 gates and bf16 rows 111 us, 4.8 TB/s; all
// bf16 97 us; 40009 x 512 fp32 in 64 sequences 63 us, 3.9 TB/s; the adjoint of 8 x 4096 x 512 bf16
// 47 us, 3.6 TB/s, of 65536 x 512 with fp32 gates 93 us, 5.0 TB/s.  About 12 us of each are the preparation,
// the first copies and the last tiles.  Beyond that the stages are what bounds it: a tile keeps its
// place in shared memory while its entering state is on the way (with states that are at once there the
// first of these takes 91 us).
#include <float.h>

#include "ops/ops.h"
#include "ops/vec.cuh"
#include "tc_ptx.cuh"

namespace la {

namespace {

constexpr int kPrepThreads = 256;
constexpr int kSlice = 64;           // channels per tile: two per lane
constexpr int kMinTile = 32;         // fewest tokens per tile: what the workspace is sized for
constexpr int kGroup = 8;            // tiles per group, and groups per published state
constexpr int kSuper = kGroup * kGroup;
constexpr int kMarked = 1, kCut = 2;   // tile_seq: the tile holds a first or last row; one that cuts the recurrence
constexpr uint32_t kUnset = 0xffffffffu;   // not published yet: a NaN that no arithmetic gives
constexpr uint32_t kCutTag = 0xfffffffeu;  // as A: a boundary lies in the tile; another such NaN
// Limits of the waits in SM clocks: 2 s and 1 ms at 2 GHz.
constexpr long long kWaitClocks = 4000000000ll;
constexpr long long kForcedClocks = 2000000ll;

// Set by the test hook: look backs then wait for a state that nothing publishes, for 1 ms.
__device__ int g_force_timeout;

// Published words are written and read as they are (relaxed, past L1); a value with one of the two
// reserved patterns, a NaN from the inputs, goes out as another NaN.
__device__ __forceinline__ float settable(float x) {
    return __float_as_uint(x) >= kCutTag ? __uint_as_float(0x7fffffffu) : x;
}
__device__ __forceinline__ bool is_set(float x) { return __float_as_uint(x) != kUnset; }
__device__ __forceinline__ void publish(float2* p, float2 v) {
    asm volatile("st.relaxed.gpu.global.v2.f32 [%0], {%1, %2};" ::"l"(p), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ void publish(float* p, float v) {
    asm volatile("st.relaxed.gpu.global.f32 [%0], %1;" ::"l"(p), "f"(v) : "memory");
}
__device__ __forceinline__ float2 peek(const float2* p) {
    float2 v;
    asm volatile("ld.relaxed.gpu.global.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ float peek(const float* p) {
    float v;
    asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ bool is_set(float2 v) { return is_set(v.x) && is_set(v.y); }

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

// Clears the header, the ticket and what tiles publish, checks the packing rules and
// notes for each tile the sequence of its first token and whether a boundary
// lies in it.
__global__ void __launch_bounds__(kPrepThreads) gated_prep_kernel(GatedParams p, int tile_tokens, int tiles,
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
    const uint4 unset = make_uint4(kUnset, kUnset, kUnset, kUnset);
    const int64_t states = (int64_t)(tiles / kSuper) * (p.Cpad / 4), joints = (int64_t)(tiles / kGroup) * (p.Cpad / 2),
                  runs = (int64_t)tiles * (p.Cpad / 2);
    for (int64_t i = at; i < states; i += step) reinterpret_cast<uint4*>(p.state)[i] = unset;
    for (int64_t i = at; i < joints; i += step) reinterpret_cast<uint4*>(p.joint)[i] = unset;
    for (int64_t i = at; i < runs; i += step) reinterpret_cast<uint4*>(p.run)[i] = unset;
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

// (A, B) of a run of tokens, for a lane's two channels.
struct Run {
    float2 A, B;
};

template <int W, int K>
struct Shared {
    float4 run[W][32];               // (A.x, A.y, B.x, B.y) of each warp's tokens; then the state that enters them
    int cut[W];                      // a boundary among them
    int first[W * K], last[W * K];   // the sequence that begins / ends at a row, else -1
    int ticket, next;
};

// A published run cuts when a boundary lies in it: what enters does not reach what leaves.
__device__ __forceinline__ bool cuts_off(float2 run) { return __float_as_uint(run.x) == kCutTag; }
__device__ __forceinline__ float through(float2 run, float s) { return cuts_off(run) ? run.y : fmaf(run.x, s, run.y); }
// Whether a product A of gates says too little about a state s that enters: below the normal range, with a large s.
// (NaN stays NaN.)
__device__ __forceinline__ bool inexact(float smallest_a, float largest_s) {
    return smallest_a < FLT_MIN && !(largest_s <= 0x1p20f);
}
// The same for several runs at once: no run of them is inexact where this is not.
struct Extremes {
    float a = FLT_MAX, s = 0.f;
    __device__ __forceinline__ void add(float2 run, float s_enters) {
        a = fminf(a, fabsf(run.x));            // (kCutTag is a NaN, which neither takes)
        s = fmaxf(s, fabsf(s_enters));
    }
    __device__ __forceinline__ bool inexact() const { return la::inexact(a, s); }
};

// A channel's rows in scan order, counted in places from the first tile's first (the adjoint: from the last tile's
// end, which may lie behind the last row).
template <typename TA, typename TX, bool Rev>
struct Channel {
    const TA* a;
    const TX* x;
    int64_t C, T, places;
    int c;

    // The recurrence from s over n places from `at` on, none of which cuts.
    __device__ __forceinline__ float walk(float s, int64_t at, int n) const {
        const int64_t lo = Rev ? places - at - n : at, end = min64(lo + n, T);
        if (c >= C) return s;
        constexpr int kAhead = 2;             // rows whose loads are under way together (eight take registers from the
                                              // callers: the adjoint of 32768 x 512 in bf16 52 us instead of 48)
        for (int64_t i = 0; lo + i < end; i += kAhead) {
            float gate[kAhead], in[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int64_t t = Rev ? end - 1 - i - k : lo + i + k;
                const bool there = t >= lo && t < end;
                // (the array's last row cuts: the adjoint's gate of a row that does not, a_{t+1}, is there)
                gate[k] = there ? (float)a[(t + (Rev ? 1 : 0)) * C + c] : 0.f;
                in[k] = there ? (float)x[t * C + c] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (lo + i + k < end) s = fmaf(gate[k], s, in[k]);
        }
        return s;
    }
    // The state after a run from place `at` on that s enters.  What A s may be off by, 2^-144 |s|, does not show beside a B
    // of more than 2^-100 |s| either: no row has to be walked for large values as such.
    __device__ __forceinline__ float exactly(float2 run, float s, int64_t at, int n) const {
        const bool off = !cuts_off(run) && inexact(fabsf(run.x), fabsf(s)) && !isnan(s) &&
                         !(fabsf(s) * 0x1p-100f <= fminf(fabsf(run.y), FLT_MAX));
        return off ? walk(s, at, n) : through(run, s);
    }
};
template <typename TA, typename TX, bool Rev>
__device__ __forceinline__ Channel<TA, TX, Rev> channel_of(const GatedParams& p, int c, int64_t places) {
    return {static_cast<const TA*>(p.a), static_cast<const TX*>(p.x), p.C, p.T, places, c};
}

// The word of warp w's run (two channels each) that holds A of channel ch; B is two words on.
__device__ __forceinline__ float* run_word(float4 (*run)[32], int w, int ch) {
    return reinterpret_cast<float*>(&run[w][ch >> 1]) + (ch & 1);
}

// s through the runs of a tile's W warps of K tokens each, the tile at place `at`, in channel ch; Leave: the state that
// enters each warp is left in the place of its A.
template <typename TA, typename TX, bool Rev, int W, int K, bool Leave>
__device__ __noinline__ float exactly_warps(const GatedParams& p, float4 (*run)[32], const int* warp_cut, bool cut_tile,
                                            int tiles, int slice, int ch, float s, int64_t at) {
    const auto channel = channel_of<TA, TX, Rev>(p, slice * kSlice + ch, (int64_t)tiles * (W * K));
#pragma unroll 1
    for (int w = 0; w < W; ++w) {
        const float a = run_word(run, w, ch)[0], b = run_word(run, w, ch)[2];
        if (Leave) run_word(run, w, ch)[0] = s;
        s = cut_tile && warp_cut[w] ? b : channel.exactly(make_float2(a, b), s, at + w * K, K);
    }
    return s;
}

// The tile's run in channel ch as it is published, from those of its warps.
template <typename TA, typename TX, bool Rev, int W, int K>
__device__ __forceinline__ float2 tile_run(const GatedParams& p, float4 (*run)[32], const int* warp_cut, bool cut_tile,
                                           int tiles, int order, int slice, int ch) {
    float2 own = make_float2(1.f, 0.f);
    Extremes of;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const float a = run_word(run, w, ch)[0], b = run_word(run, w, ch)[2];
        if (w > 0) of.add(make_float2(a, b), own.y);      // (zero enters the first)
        own.y = cut_tile && warp_cut[w] ? b : fmaf(a, own.y, b);
        own.x *= a;
    }
    if (__builtin_expect(of.inexact(), 0))
        own.y = exactly_warps<TA, TX, Rev, W, K, false>(p, run, warp_cut, cut_tile, tiles, slice, ch, 0.f,
                                                        (int64_t)order * (W * K));
    return make_float2(cut_tile ? __uint_as_float(kCutTag) : settable(own.x), settable(own.y));
}

// What look_back has found to be inexact, once more from what is published: all that its lane leaves and publishes.
template <typename TA, typename TX, bool Rev, int W, int K>
__device__ __noinline__ void look_back_exactly(const GatedParams& p, float4 (*run)[32], const int* warp_cut,
                                               bool cut_tile, bool fresh, float2 own, int tiles, int order, int slice,
                                               int ch) {
    constexpr int kTile = W * K, kGroupTokens = kGroup * kTile;
    const auto channel = channel_of<TA, TX, Rev>(p, slice * kSlice + ch, (int64_t)tiles * kTile);
    const int q = order % kGroup, group = order / kGroup, g = group % kGroup, super = group / kGroup;
    const int64_t at = (int64_t)order * kTile;
    const float2* tile_runs = p.run + (int64_t)(order - q) * p.Cpad + channel.c;
    float A = 1.f, B = 0.f, s = 0.f;
    bool cut = false;
#pragma unroll 1
    for (int i = 0; i < q; ++i) {
        const float2 r = peek(tile_runs + (int64_t)i * p.Cpad);
        cut |= cuts_off(r);
        B = channel.exactly(r, B, at + (i - q) * kTile, kTile);
        A *= r.x;
    }
    if (q == kGroup - 1) {
        B = channel.exactly(own, B, at, kTile);
        A = cut || cut_tile ? __uint_as_float(kCutTag) : settable(A * own.x);
        publish(p.joint + (int64_t)group * p.Cpad + channel.c, make_float2(A, settable(B)));
    }
    if (!fresh) {
        if (!cut) {
            if (super > 0) s = peek(p.state + (int64_t)(super - 1) * p.Cpad + channel.c);
#pragma unroll 1
            for (int i = 0; i < g; ++i)
                s = channel.exactly(peek(p.joint + (int64_t)(group - g + i) * p.Cpad + channel.c), s,
                                    (int64_t)(group - g + i) * kGroupTokens, kGroupTokens);
        }
#pragma unroll 1
        for (int i = 0; i < q; ++i)
            s = channel.exactly(peek(tile_runs + (int64_t)i * p.Cpad), s, at + (i - q) * kTile, kTile);
    }
    const float left = exactly_warps<TA, TX, Rev, W, K, true>(p, run, warp_cut, cut_tile, tiles, slice, ch, s, at);
    if (order % kSuper == kSuper - 1) publish(p.state + (int64_t)super * p.Cpad + channel.c, settable(left));
}

// What a look-back lane does for its channel ch of a tile whose run `own` is published: finds the
// state that enters the tile and leaves in the place of each warp's A the state that enters that
// warp.  `fresh`: nothing enters.  Every wait is bounded; a lane whose wait runs out records it and
// takes zero.
template <typename TA, typename TX, bool Rev, int W, int K>
__device__ __forceinline__ void look_back(const GatedParams& p, float4 (*run)[32], const int* warp_cut, bool cut_tile,
                                          bool fresh, float2 own, int tiles, int order, int slice, int ch,
                                          bool forced) {
    const int c = slice * kSlice + ch;
    const int q = order % kGroup, group = order / kGroup, g = group % kGroup, super = group / kGroup;
    const bool joins = q == kGroup - 1, leaves = order % kSuper == kSuper - 1;
    float s = 0.f;
    Extremes of;                         // of all the runs below
    bool late = false;                   // a wait has run out
    if (!fresh || joins) {
        const long long start = clock64(), limit = forced ? kForcedClocks : kWaitClocks;
        const float2* tile_runs = p.run + (int64_t)(order - q) * p.Cpad + c;
        const float2* group_run = p.joint + (int64_t)(group - g) * p.Cpad + c;
        const float* state = p.state + (int64_t)(super - 1) * p.Cpad + c;
        float2 r[kGroup - 1], j[kGroup - 1];
        float sup = __uint_as_float(kUnset);
        unsigned polls = 0;
        auto run_out = [&]() {
            if ((++polls & 15) == 0 && (clock64() - start > limit ||
                                        *(volatile int*)&p.hdr->error == LA_DEVERR_WAIT_TIMEOUT)) {
                record_error(p.hdr, LA_DEVERR_WAIT_TIMEOUT);
                late = true;
            }
            return late;
        };
        // one trip for everything that may be there already
        if (super > 0) sup = peek(state);
#pragma unroll
        for (int i = 0; i < kGroup - 1; ++i) {
            r[i] = i < q ? peek(tile_runs + (int64_t)i * p.Cpad) : make_float2(0.f, 0.f);
            j[i] = i < g ? peek(group_run + (int64_t)i * p.Cpad) : make_float2(0.f, 0.f);
        }
        // the tiles of the group: their runs come without waiting for anything
        bool cut = false;
        for (;;) {
            bool missing = forced;
            cut = false;
#pragma unroll
            for (int i = 0; i < kGroup - 1; ++i)
                if (i < q) {
                    missing |= !is_set(r[i]);
                    cut |= cuts_off(r[i]);
                }
            if (!missing || run_out()) break;
#pragma unroll
            for (int i = 0; i < kGroup - 1; ++i)
                if (i < q && !is_set(r[i])) r[i] = peek(tile_runs + (int64_t)i * p.Cpad);
        }
        if (joins) {
            float A = 1.f, B = 0.f;
#pragma unroll
            for (int i = 0; i < kGroup - 1; ++i) {
                if (i > 0) of.add(r[i], B);
                B = through(r[i], B);
                A *= r[i].x;
            }
            of.add(own, B);
            B = through(own, B);
            A = cut || cut_tile ? __uint_as_float(kCutTag) : settable(A * own.x);
            if (!of.inexact() || late) publish(p.joint + (int64_t)group * p.Cpad + c, make_float2(A, settable(B)));
        }
        // the groups of the block, needed unless a boundary lies in the group
        if (!fresh && !cut) {
            for (;;) {
                bool missing = forced, far = super > 0;
#pragma unroll
                for (int i = 0; i < kGroup - 1; ++i)
                    if (i < g) {
                        missing |= !is_set(j[i]);
                        far &= !cuts_off(j[i]);
                    }
                if (!(missing || (far && !is_set(sup))) || run_out()) break;
                if (far && !is_set(sup)) sup = peek(state);
#pragma unroll
                for (int i = 0; i < kGroup - 1; ++i)
                    if (i < g && !is_set(j[i])) j[i] = peek(group_run + (int64_t)i * p.Cpad);
            }
            s = super > 0 ? sup : 0.f;
#pragma unroll
            for (int i = 0; i < kGroup - 1; ++i)
                if (i < g) {
                    of.add(j[i], s);
                    s = through(j[i], s);
                }
        }
        if (!fresh) {
#pragma unroll
            for (int i = 0; i < kGroup - 1; ++i)
                if (i < q) {
                    of.add(r[i], s);
                    s = through(r[i], s);
                }
        }
        if (late) s = 0.f;
    }
    float e[W + 1];                      // the states that enter the warps
    e[0] = s;
    if (leaves) of.add(own, s);
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const float a = run_word(run, w, ch)[0], b = run_word(run, w, ch)[2];
        of.add(make_float2(a, b), e[w]);
        e[w + 1] = cut_tile && warp_cut[w] ? b : fmaf(a, e[w], b);
    }
    if (__builtin_expect(of.inexact() && !late, 0)) {
        look_back_exactly<TA, TX, Rev, W, K>(p, run, warp_cut, cut_tile, fresh, own, tiles, order, slice, ch);
        return;
    }
    if (leaves) publish(p.state + (int64_t)super * p.Cpad + c, settable(through(own, s)));
#pragma unroll
    for (int w = 0; w < W; ++w) run_word(run, w, ch)[0] = e[w];
}

// first[i] / last[i]: the sequence whose first / last token is row t0 + i, else -1; n rows, and
// the marks of `rows` rows are reset.  Called by `threads` threads that then synchronise.
__device__ __forceinline__ void clear_marks(int rows, int* first, int* last, int thread, int threads) {
    for (int i = thread; i < rows; i += threads) first[i] = last[i] = -1;
}
__device__ __forceinline__ void set_marks(const GatedParams& p, int seq, int64_t t0, int n, int* first, int* last,
                                          int thread, int threads) {
    for (int base = seq; base < p.nseq && seq_begin(p, base) < t0 + n; base += threads) {
        const int s = base + thread;
        if (s < p.nseq) {
            const int64_t lo = seq_begin(p, s), hi = seq_begin(p, s + 1);
            if (hi > lo) {
                if (lo >= t0 && lo < t0 + n) first[lo - t0] = s;
                if (hi - 1 >= t0 && hi - 1 < t0 + n) last[hi - 1 - t0] = s;
            }
        }
    }
}

// An empty sequence passes its state on.  The block's first `threads` threads call it.
__device__ void pass_empty(const GatedParams& p, int threads) {
    if (!p.edge_out || !(p.cu_seqlens || p.T == 0)) return;
    const int lane = threadIdx.x & 31;
    for (int s0 = blockIdx.x * 32; s0 < p.nseq; s0 += gridDim.x * 32) {
        const int s = s0 + lane;
        unsigned empty = __ballot_sync(0xffffffffu, s < p.nseq && seq_begin(p, s) == seq_begin(p, s + 1));
        for (; empty; empty &= empty - 1) {
            const int64_t at = (int64_t)(s0 + __ffs(empty) - 1) * p.C;
            for (int c = threadIdx.x; c < p.C; c += threads) p.edge_out[at + c] = p.edge_in ? p.edge_in[at + c] : 0.f;
        }
    }
}

// Tiles held in registers, one at a time per block: a single tile of tokens (Solo), and bf16 arrays that do not start on
// four bytes, whose elements no asynchronous copy can fetch (32768 x 1002: 273 us, bound by loads of two bytes).
// The same warps, tokens and order of operations as the ring's: the same results.
constexpr int kRegisterBlocks = 2;       // per SM
template <typename TA, typename TX, bool Rev, bool Vec, bool Solo, int W, int K>
__global__ void __launch_bounds__((W + 2) * 32, Solo ? 1 : kRegisterBlocks)
gated_scan_kernel(const __grid_constant__ GatedParams p, int tiles, int slices) {
    __shared__ Shared<W, K> sh;
    constexpr int kTile = W * K, kThreads = (W + 2) * 32;   // the last two warps look back
    static_assert(kTile >= kMinTile, "the workspace holds ceil(T / kMinTile) tiles");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const TA* a = static_cast<const TA*>(p.a);
    const TX* x = static_cast<const TX*>(p.x);
    const TX* h = static_cast<const TX*>(p.h);
    const int64_t C = p.C;

    asm volatile("griddepcontrol.wait;" ::: "memory");
    if constexpr (Solo) {
        // no other kernel has looked at the arguments
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
    const bool forced = !Solo && *(volatile int*)&g_force_timeout != 0;

    pass_empty(p, kThreads);

    const int total = tiles * slices;
    int ticket = blockIdx.x;
    if constexpr (!Solo) {
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
        const bool work = warp < W;
        const int j0 = work ? (Rev ? W - 1 - warp : warp) * K : kTile;

        // --- every load of the tile in flight
        Two<TA> ra[K];
        Two<TX> rx[K];
        if (work) {
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
        if (!Solo && threadIdx.x == 0) next = atomicAdd(p.ticket, 1);

        // --- boundaries
        const int ts = Solo ? kMarked | kCut : p.tile_seq[tile];
        const bool cut_tile = ts & kCut, marked = ts & kMarked;
        if (marked) {
            clear_marks(kTile, sh.first, sh.last, threadIdx.x, kThreads);
            __syncthreads();
            set_marks(p, ts >> 2, t0, n, sh.first, sh.last, threadIdx.x, kThreads);
            __syncthreads();
        }
        // bit k: a boundary that cuts the recurrence at row j0 + k; and the rows whose state leaves
        unsigned cuts = 0, ends = 0;
        if (marked) {
            const bool f = work && lane < K && sh.first[j0 + lane] >= 0;
            const bool l = work && lane < K && sh.last[j0 + lane] >= 0;
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
        if (work) {
#pragma unroll
            for (int i = 0; i < K; ++i) {
                const int k = Rev ? K - 1 - i : i;
                const float2 g = ra[k].get(), in = rx[k].get();
                if ((cuts >> k) & 1) {
                    float2 s = in;
                    if (p.edge_in) {
                        const int q = (Rev ? sh.last : sh.first)[j0 + k];
                        const float2 e = edge_two(p.edge_in + (int64_t)q * C + c, left);
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
        }
        if (threadIdx.x == 0) sh.next = next;
        __syncthreads();

        // --- the tile's run goes out, and the state that enters it is found
        if (!work && !Solo) {
            const bool fresh = marked && (Rev ? sh.last[n - 1] : sh.first[0]) >= 0;   // nothing enters
            const int ch = threadIdx.x - W * 32;
            const float2 own = tile_run<TA, TX, Rev, W, K>(p, sh.run, sh.cut, cut_tile, tiles, order, slice, ch);
            publish(p.run + (int64_t)order * p.Cpad + slice * kSlice + ch, own);
            look_back<TA, TX, Rev, W, K>(p, sh.run, sh.cut, cut_tile, fresh, own, tiles, order, slice, ch, forced);
        } else if (!work) {
            const int ch = threadIdx.x - W * 32;
            exactly_warps<TA, TX, Rev, W, K, true>(p, sh.run, sh.cut, true, tiles, slice, ch, 0.f, 0);
        }
        Two<TX> rh[Rev ? K : 1];
        if (Rev && work) {
            const int64_t row = (t0 + j0) * C + c;
#pragma unroll
            for (int k = 0; k < K; ++k)
                rh[k] = load_two<Vec>(h + row + (k - 1) * C, j0 + k < n && t0 + j0 + k > 0 ? left : 0);
        }
        __syncthreads();

        // --- the recurrence from the state that enters the warp
        if (work) {
            float2 s = *reinterpret_cast<const float2*>(&sh.run[warp][lane]);
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
                        const int q = (Rev ? sh.last : sh.first)[j0 + k];
                        const float2 e = edge_two(p.edge_in + (int64_t)q * C + c, left);
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
        }
        if (Solo) return;
        ticket = sh.next;
        __syncthreads();      // the next tile overwrites the shared runs and marks
    }
}

__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, long long limit) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    const long long start = clock64();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 256; ++i)
            if (tc::mbar_try_wait(bar, parity)) return true;
        if (clock64() - start > limit) return false;
    }
}

// --------------------------------------------------------------------------
// Tiles that TMA brings into a ring in shared memory.  One warp takes tickets, one starts the copies,
// compute warps form the tile's runs, a publishing pair of warps sends them out without
// waiting for other tiles, look-back warps find the entering state, and the compute warps come back to
// the tile when it is there to run the recurrence.  A compute warp takes whichever of the two it can do
// next, so stages are neither held for a fixed number of tiles nor idle: the trips to L2 are hidden
// behind the tiles that follow.
//
// Tile copies (kTiles) need rows that start on 16 bytes.  Other rows of four-byte steps are copied by four
// warps, four bytes a lane, into the same places (kWords: 32768 x 1023 in fp32 119 us; with tiles in registers
// 182 us).  bf16 rows of odd length, every other of which starts inside four bytes, are copied as the words that
// hold them, one more a row than they fill, and put together by the lanes that read them (kHalves: 32768 x 1001
// 121 us; in registers 243 us).
// --------------------------------------------------------------------------
enum Copies { kTiles, kWords, kHalves };

// A lane's two channels of the tile's rows from j0 on, row `token` of the array first (its parity tells where the
// row starts where rows are of odd length).
template <typename T, bool Halves>
struct TileRows {
    static constexpr bool kOdd = Halves && sizeof(T) == 2;
    static constexpr int kPitch = kSlice * (int)sizeof(T) + (kOdd ? 4 : 0);     // bytes of a row
    const uint8_t* at;
    int parity;
    __device__ __forceinline__ TileRows(const uint8_t* tile, int j0, int lane, int token)
        : at(tile + j0 * kPitch + lane * 2 * (int)sizeof(T)), parity(token & 1) {}
    __device__ __forceinline__ float2 operator[](int k) const {
        if constexpr (kOdd) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(at + k * kPitch);
            const uint32_t v = __byte_perm(w[0], w[1], (parity ^ k) & 1 ? 0x5432 : 0x3210);
            return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
        } else {
            return reinterpret_cast<const Two<T>*>(at + k * kPitch)->get();
        }
    }
};

template <typename TA, typename TX, bool Rev, Copies Copy, int W, int K, int S>
struct Ring {
    static constexpr int kTeams = 2;                    // compute teams, taking tiles in turn: W warps of K tokens
    static constexpr int kRows = W * K;
    static constexpr int kLookers = S % 4 == 0 ? 4 : S % 5 == 0 ? 5 : 3;   // pairs of look-back warps, in turn
    static constexpr int kCopiers = Copy == kTiles ? 1 : 4;
    static constexpr int kThreads = (kTeams * W + 2 * kLookers + 2 + 1 + kCopiers) * 32;
    using A = TileRows<TA, Copy == kHalves>;
    using X = TileRows<TX, Copy == kHalves>;
    static constexpr int kA = kRows * A::kPitch, kX = kRows * X::kPitch;
    static constexpr int kStage = kA + kX + (Rev ? kX : 0);
    struct Small {
        float4 run[S][W][32];              // each warp's run; then, in its first half, the state that enters it
        float2 own[S][kSlice];             // the tile's run as it is published
        float2 open[S][W][32];             // the state after the last boundary among the warp's tokens
        int first[S][kRows], last[S][kRows];
        int cut[S][W];
        int order[S], slice[S], seq[S];    // order < 0: no more tiles
        uint64_t known[S], full[S], runs[S], sent[S], carried[S], empty[S];
        int gave_up;
    };
    static constexpr size_t kBytes = (size_t)S * kStage + sizeof(Small) + 128;
};

__device__ __forceinline__ void copy_word(uint32_t to, const void* from, int bytes) {   // the rest of the word as zero
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
// Copies Rows rows x kSlice channels of [tokens][C] from row t0 and channel c0 on to `place`, rows and channels
// outside as zeros: the share of one of `warps` warps.
template <typename T, int Rows, bool Halves>
__device__ __forceinline__ void copy_rows(uint8_t* place, const void* from, int64_t t0, int c0, int64_t tokens, int C,
                                          int warp, int warps, int lane) {
    constexpr int kRowWords = kSlice * (int)sizeof(T) / 4, kEach = 4 / (int)sizeof(T);   // of a row; elements in a word
    constexpr int kPitch = TileRows<T, Halves>::kPitch;
    const uint32_t to = tc::smem_u32(place);
    const T* base = static_cast<const T*>(from);
    auto word = [&](int r, int w) {
        const int64_t t = t0 + r, end = t * C + C;
        int64_t e = t * C + c0 + w * kEach;
        if constexpr (TileRows<T, Halves>::kOdd) e &= ~1ll;            // the word that holds it
        int there = t >= 0 && t < tokens && e < end ? 4 : 0;
        if constexpr (TileRows<T, Halves>::kOdd)
            if (there && e + 1 == tokens * C) there = 2;               // the array's last element, alone in its word
        copy_word(to + r * kPitch + w * 4, there ? base + e : base, there);
    };
    for (int r = warp; r < Rows; r += warps)
#pragma unroll
        for (int w = 0; w < kRowWords / 32; ++w) word(r, w * 32 + lane);
    if constexpr (TileRows<T, Halves>::kOdd)
        for (int r = warp + lane * warps; r < Rows; r += 32 * warps) word(r, kRowWords);
}

// over_slices: 2^64 / slices, rounded up; 0 for one slice.
// Vec: outputs that take two channels of every row in one store.
template <typename TA, typename TX, bool Rev, Copies Copy, bool Vec, int W, int K, int S>
__global__ void __launch_bounds__(Ring<TA, TX, Rev, Copy, W, K, S>::kThreads, 1)
gated_ring_kernel(const __grid_constant__ GatedParams p, int tiles, int slices, unsigned long long over_slices,
                  const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_x,
                  const __grid_constant__ CUtensorMap map_h) {
    using R = Ring<TA, TX, Rev, Copy, W, K, S>;
    constexpr bool Tma = Copy == kTiles, kOdd = Copy == kHalves;
    static_assert(R::kRows >= kMinTile, "the workspace holds ceil(T / kMinTile) tiles");
    constexpr int kLookers = R::kLookers, kTeams = R::kTeams;
    // Who takes every n-th tile waits for phases of its own tiles only, one after the other, when n
    // divides S (another's tile may still be loading when its own later one is there, and a phase is
    // told by its parity alone).  And the marks of the end need a stage for everyone.
    static_assert(S % kLookers == 0 && S % kTeams == 0, "teams and look-back pairs stay with their stages");
    // aligned by an offset: through an integer the compiler would lose that it is shared memory, and
    // every access would be a generic one (twice the time per tile)
    extern __shared__ __align__(128) uint8_t raw[];
    uint8_t* data = raw + (-tc::smem_u32(raw) & 127u);
    typename R::Small& sh = *reinterpret_cast<typename R::Small*>(data + (size_t)S * R::kStage);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            tc::mbar_init(&sh.known[i], 1);
            tc::mbar_init(&sh.full[i], 1 + (Tma ? 1 : 32 * R::kCopiers));   // the tile's marks, and the copies
            tc::mbar_init(&sh.runs[i], W);
            tc::mbar_init(&sh.sent[i], 2);
            tc::mbar_init(&sh.carried[i], 2);
            tc::mbar_init(&sh.empty[i], W);
        }
        sh.gave_up = 0;
        tc::fence_mbar_init();
    }
    __syncthreads();
    // up to here beside the preparation; what each warp then needs of it, it reads for itself
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // A wait that runs out (which takes a fault elsewhere) is recorded, and every role leaves.
    auto wait = [&](uint64_t* bar, int i) {
        if (wait_phase(bar, (i / S) & 1, 4 * kWaitClocks) && !*(volatile int*)&sh.gave_up) return true;
        record_error(p.hdr, LA_DEVERR_WAIT_TIMEOUT);
        *(volatile int*)&sh.gave_up = 1;
        return false;
    };

    if (warp >= kTeams * W + 2 * kLookers + 3) {
        // ---------------- copies of the tiles that the ticket warp names
        const int copier = warp - (kTeams * W + 2 * kLookers + 3);
        if (!Tma || lane == 0) {
            int copied = 0;
            for (int i = 0;; ++i) {
                const int st = i % S;
                if (!wait(&sh.known[st], i)) break;
                const int order = sh.order[st];
                if (order < 0) {
                    const bool last = sh.slice[st];       // the last mark of the end
                    tc::mbar_arrive(&sh.full[st]);
                    if (last) return;
                    continue;
                }
                const int c0 = sh.slice[st] * kSlice, t0 = (Rev ? tiles - 1 - order : order) * R::kRows;
                uint8_t* at = data + (size_t)st * R::kStage;
                // rows before the first and behind the last one come as zeros
                if (Tma) {
                    tc::mbar_arrive_expect_tx(&sh.full[st], R::kStage);
                    tc::tma_load_2d(at, &map_a, c0, t0 + (Rev ? 1 : 0), &sh.full[st]);
                    tc::tma_load_2d(at + R::kA, &map_x, c0, t0, &sh.full[st]);
                    if (Rev) tc::tma_load_2d(at + R::kA + R::kX, &map_h, c0, t0 - 1, &sh.full[st]);
                } else {
                    copy_rows<TA, R::kRows, kOdd>(at, p.a, (int64_t)t0 + (Rev ? 1 : 0), c0, p.T, p.C, copier,
                                                  R::kCopiers, lane);
                    copy_rows<TX, R::kRows, kOdd>(at + R::kA, p.x, t0, c0, p.T, p.C, copier, R::kCopiers, lane);
                    if (Rev)
                        copy_rows<TX, R::kRows, kOdd>(at + R::kA + R::kX, p.h, (int64_t)t0 - 1, c0, p.T, p.C, copier,
                                                      R::kCopiers, lane);
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                                     tc::smem_u32(&sh.full[st]))
                                 : "memory");
                }
                copied = i + 1;
            }
            // no copy is in flight when the block ends
            if (Tma)
                for (int j = copied > S ? copied - S : 0; j < copied; ++j)
                    wait_phase(&sh.full[j % S], (j / S) & 1, kWaitClocks);
            else
                asm volatile("cp.async.wait_all;" ::: "memory");
        }
        return;
    }

    if (warp == kTeams * W + 2 * kLookers + 2) {
        // ---------------- tickets (none where the boundaries are malformed)
        const int refused = *(volatile int*)&p.hdr->error;
        // A ticket is asked for two tiles ahead and its sequence one tile ahead: neither trip to L2
        // stands between two copies.
        constexpr int kAhead = 2;
        auto order_of = [&](int t) { return over_slices ? (int)__umul64hi((unsigned long long)t, over_slices) : t; };
        auto seq_of_ticket = [&](int t) {
            const int order = order_of(t);
            return t < tiles * slices ? p.tile_seq[Rev ? tiles - 1 - order : order] : 0;
        };
        int asked[kAhead], ticket[kAhead], seq[kAhead];
        const int first = lane == 0 ? atomicAdd(p.ticket, kAhead) : 0;
        const int total = refused == LA_DEVERR_CU_SEQLENS ? 0 : tiles * slices;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) asked[u] = first + u;
#pragma unroll
        for (int u = 0; u < kAhead / 2; ++u) {
            ticket[u] = __shfl_sync(0xffffffffu, asked[u], 0);
            seq[u] = seq_of_ticket(ticket[u]);
        }
        int i = 0, over = 0;
        bool ok = true, done = false;
        while (!done) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (done) continue;
                constexpr int kHalf = kAhead / 2;
                const int v = (u + kHalf) % kAhead, st = i % S;
                ticket[v] = __shfl_sync(0xffffffffu, asked[v], 0);
                seq[v] = seq_of_ticket(ticket[v]);
                asked[u] = lane == 0 && ticket[v] < total ? atomicAdd(p.ticket, 1) : total;
                if (i >= S) ok = __all_sync(0xffffffffu, wait(&sh.empty[st], i - S));
                if (!ok) {
                    done = true;
                } else if (ticket[u] >= total) {
                    if (++over == kLookers) done = true;      // every look-back pair and team meets one
                    if (lane == 0) {
                        sh.order[st] = -1;
                        sh.slice[st] = done;
                        tc::mbar_arrive(&sh.known[st]);
                        tc::mbar_arrive(&sh.full[st]);
                    }
                    ++i;
                } else {
                    const int order = order_of(ticket[u]), slice = ticket[u] - order * slices;
                    if (lane == 0) {
                        sh.order[st] = order;
                        sh.slice[st] = slice;
                        sh.seq[st] = seq[u];
                        tc::mbar_arrive(&sh.known[st]);
                    }
                    if (seq[u] & kMarked) {
                        const int64_t t0 = (int64_t)(Rev ? tiles - 1 - order : order) * R::kRows;
                        clear_marks(R::kRows, sh.first[st], sh.last[st], lane, 32);
                        __syncwarp();
                        set_marks(p, seq[u] >> 2, t0, (int)min64(R::kRows, p.T - t0), sh.first[st], sh.last[st], lane,
                                  32);
                    }
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&sh.full[st]);
                    ++i;
                }
            }
        }
        return;
    }

    if (warp >= kTeams * W) {
        // ---------------- two warps publish every tile's run; pairs look back for the tiles in turn
        const bool forced = *(volatile int*)&g_force_timeout != 0;
        const int pair = (warp - kTeams * W) / 2, ch = (warp - kTeams * W) % 2 * 32 + lane;
        const bool publisher = pair == kLookers;
        for (int i = publisher ? 0 : pair;; i += publisher ? 1 : kLookers) {
            const int st = i % S;
            if (!wait(&sh.full[st], i) || sh.order[st] < 0) return;
            if (!wait(publisher ? &sh.runs[st] : &sh.sent[st], i)) return;
            const int order = sh.order[st], slice = sh.slice[st];
            const bool cut_tile = sh.seq[st] & kCut;
            if (publisher) {
                const float2 own =
                    tile_run<TA, TX, Rev, W, K>(p, sh.run[st], sh.cut[st], cut_tile, tiles, order, slice, ch);
                publish(p.run + (int64_t)order * p.Cpad + slice * kSlice + ch, own);
                sh.own[st][ch] = own;
            } else {
                // a boundary at the tile's first row (adjoint: its last): nothing enters
                const int64_t t0 = (int64_t)(Rev ? tiles - 1 - order : order) * R::kRows;
                const int edge = Rev ? (int)min64(R::kRows, p.T - t0) - 1 : 0;
                const bool fresh = cut_tile && (Rev ? sh.last[st] : sh.first[st])[edge] >= 0;
                look_back<TA, TX, Rev, W, K>(p, sh.run[st], sh.cut[st], cut_tile, fresh, sh.own[st][ch], tiles, order,
                                             slice, ch, forced);
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(publisher ? &sh.sent[st] : &sh.carried[st]);
        }
    }

    // ---------------- compute
    if (p.edge_out && p.cu_seqlens && *(volatile int*)&p.hdr->error != LA_DEVERR_CU_SEQLENS)
        pass_empty(p, kTeams * W * 32);
    const int team = warp / W, member = warp % W;
    const int j0 = (Rev ? W - 1 - member : member) * K;       // the warp's rows; descending for the adjoint
    // The state after the warp's last boundary is kept until it comes back to the tile: edge_out may
    // be edge_in, and the sequence that begins there may be closed by another warp before.  Sequences
    // of earlier boundaries are closed by this warp itself, after its reads.
    int ahead = team, b = team;           // the next tile to form the run of; the next to come back to
    int end = INT32_MAX;                  // the team's first tile that is none, once known
    for (;;) {
        if (b >= end) return;
        bool form = false;
        const long long start = clock64();
        for (unsigned spins = 1;; ++spins) {
            // a run first: other tiles wait for it
            form = ahead < end && __any_sync(0xffffffffu, tc::mbar_test_wait(&sh.full[ahead % S], (ahead / S) & 1));
            if (form) break;
            if (b < ahead && __any_sync(0xffffffffu, tc::mbar_test_wait(&sh.carried[b % S], (b / S) & 1))) break;
            if ((spins & 255) == 0 &&
                __any_sync(0xffffffffu, *(volatile int*)&sh.gave_up || clock64() - start > 4 * kWaitClocks)) {
                record_error(p.hdr, LA_DEVERR_WAIT_TIMEOUT);
                *(volatile int*)&sh.gave_up = 1;
                return;
            }
        }
        if (form) {
            const int i = ahead, st = i % S;
            ahead += kTeams;
            if (!wait(&sh.full[st], i)) return;
            const int order = sh.order[st];
            if (order < 0) {
                end = i;
            } else {
                const uint8_t* at = data + (size_t)st * R::kStage;
                const typename R::A sa(at, j0, lane, Rev ? 1 : 0);        // tiles and j0 are even
                const typename R::X sx(at + R::kA, j0, lane, 0);
                const int64_t t0 = (int64_t)(Rev ? tiles - 1 - order : order) * R::kRows;
                const int n = (int)min64(R::kRows, p.T - t0), c = sh.slice[st] * kSlice + 2 * lane, left = p.C - c;
                unsigned cuts = 0;
                if (sh.seq[st] & kCut) {
                    const int* m = Rev ? sh.last[st] : sh.first[st];
                    cuts = __ballot_sync(0xffffffffu, lane < K && m[j0 + lane] >= 0);
                }
                Run r{make_float2(1.f, 1.f), make_float2(0.f, 0.f)};
                float2 o = make_float2(0.f, 0.f);
                if (cuts == 0 && n == R::kRows) {
#pragma unroll
                    for (int q = 0; q < K; ++q) {
                        const int k = Rev ? K - 1 - q : q;
                        const float2 g = sa[k], in = sx[k];
                        r.A = mul2(r.A, g);
                        r.B = fma2(g, r.B, in);
                    }
                } else {
#pragma unroll 1
                    for (int q = 0; q < K; ++q) {
                        const int k = Rev ? K - 1 - q : q;
                        const float2 g = sa[k], in = sx[k];
                        if ((cuts >> k) & 1) {
                            float2 s = in;
                            if (p.edge_in) {
                                const int sq = (Rev ? sh.last[st] : sh.first[st])[j0 + k];
                                const float2 e = edge_two(p.edge_in + (int64_t)sq * p.C + c, left);
                                s = Rev ? make_float2(in.x + e.x, in.y + e.y) : fma2(g, e, in);
                            }
                            r.A = make_float2(0.f, 0.f);
                            r.B = o = s;
                        } else if (j0 + k < n) {
                            r.A = mul2(r.A, g);
                            r.B = fma2(g, r.B, in);
                        }
                    }
                }
                if (cuts) sh.open[st][member][lane] = o;
                sh.run[st][member][lane] = make_float4(r.A.x, r.A.y, r.B.x, r.B.y);
                if (lane == 0) sh.cut[st][member] = cuts != 0;
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sh.runs[st]);
            }
        }
        if (!form) {
            const int st = b % S;
            if (!wait(&sh.carried[st], b)) return;
            b += kTeams;
            const int order = sh.order[st], seq = sh.seq[st];
            const uint8_t* at = data + (size_t)st * R::kStage;
            const typename R::A sa(at, j0, lane, Rev ? 1 : 0);
            const typename R::X sx(at + R::kA, j0, lane, 0), sh_h(at + R::kA + R::kX, j0, lane, 1);
            const int64_t t0 = (int64_t)(Rev ? tiles - 1 - order : order) * R::kRows;
            const int n = (int)min64(R::kRows, p.T - t0), c = sh.slice[st] * kSlice + 2 * lane, left = p.C - c;
            const int64_t row = (t0 + j0) * p.C + c;
            unsigned cuts = 0, ends = 0;
            if (seq & kMarked) {
                const unsigned fm = __ballot_sync(0xffffffffu, lane < K && sh.first[st][j0 + lane] >= 0);
                const unsigned lm = __ballot_sync(0xffffffffu, lane < K && sh.last[st][j0 + lane] >= 0);
                cuts = Rev ? lm : fm;
                ends = Rev ? fm : lm;
            }
            float2 s = *reinterpret_cast<const float2*>(&sh.run[st][member][lane]);
            TX* y = static_cast<TX*>(p.y) + row;
            TA* da = Rev ? static_cast<TA*>(p.da) + row : nullptr;
            if ((cuts | ends) == 0 && n == R::kRows) {
#pragma unroll
                for (int q = 0; q < K; ++q) {
                    const int k = Rev ? K - 1 - q : q;
                    s = fma2(sa[k], s, sx[k]);
                    store_two<Vec>(y + k * (int64_t)p.C, left, s);
                    if (Rev) store_two<Vec>(da + k * (int64_t)p.C, left, mul2(s, sh_h[k]));
                }
            } else {
                const int open_at = cuts ? (Rev ? __ffs(cuts) - 1 : 31 - __clz(cuts)) : 32;
#pragma unroll 1
                for (int q = 0; q < K; ++q) {
                    const int k = Rev ? K - 1 - q : q;
                    if (j0 + k >= n) continue;
                    const float2 g = sa[k], in = sx[k];
                    if ((cuts >> k) & 1) {
                        s = in;
                        if (k == open_at) {
                            s = sh.open[st][member][lane];
                        } else if (p.edge_in) {
                            const int sq = (Rev ? sh.last[st] : sh.first[st])[j0 + k];
                            const float2 e = edge_two(p.edge_in + (int64_t)sq * p.C + c, left);
                            s = Rev ? make_float2(in.x + e.x, in.y + e.y) : fma2(g, e, in);
                        }
                    } else {
                        s = fma2(g, s, in);
                    }
                    store_two<Vec>(y + k * (int64_t)p.C, left, s);
                    float2 leaving = s;
                    if (Rev) {
                        float2 prev = sh_h[k];
                        if ((ends >> k) & 1) {
                            const int sq = sh.first[st][j0 + k];
                            prev = p.state_in ? edge_two(p.state_in + (int64_t)sq * p.C + c, left)
                                              : make_float2(0.f, 0.f);
                            const TA* gate = static_cast<const TA*>(p.a) + row + k * (int64_t)p.C;
                            if (p.edge_out) leaving = mul2(load_two<false>(gate, left).get(), s);
                        }
                        store_two<Vec>(da + k * (int64_t)p.C, left, mul2(s, prev));
                    }
                    if (((ends >> k) & 1) && p.edge_out)
                        store_edge(p.edge_out + (int64_t)(Rev ? sh.first[st] : sh.last[st])[j0 + k] * p.C + c, left,
                                   leaving);
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sh.empty[st]);
        }
    }
}

// One token: N neighbouring elements a thread (four where the operands' alignment allows vectors).  Bound by
// the launch: 3 x 16 x 64 take about 3 us.
template <typename TA, typename TX, int N>
__global__ void __launch_bounds__(kPrepThreads) gated_step_kernel(const TA* a, const TX* b, int64_t n,
                                                                  const float* state_in, float* state_out, TX* h) {
    const int64_t i = ((int64_t)blockIdx.x * kPrepThreads + threadIdx.x) * N;
    if (i >= n) return;
    float fa[N], fb[N], fs[N];
    unpack(fa, *reinterpret_cast<const Vec<TA, N>*>(a + i));
    unpack(fb, *reinterpret_cast<const Vec<TX, N>*>(b + i));
    unpack(fs, *reinterpret_cast<const Vec<float, N>*>(state_in + i));
#pragma unroll
    for (int k = 0; k < N; ++k) fs[k] = fmaf(fa[k], fs[k], fb[k]);
    Vec<float, N> s;
    Vec<TX, N> o;
    pack(s, fs);
    pack(o, fs);
    *reinterpret_cast<Vec<float, N>*>(state_out + i) = s;
    *reinterpret_cast<Vec<TX, N>*>(h + i) = o;
}

struct GatedLayout {
    size_t ticket, tile_seq, run, joint, state, total;
    int slices, Cpad;
};

GatedLayout gated_layout(int64_t T, int C) {
    GatedLayout lo{};
    lo.slices = (int)ceil_div(C, kSlice);
    lo.Cpad = lo.slices * kSlice;
    const size_t tiles = T <= kMinTile ? 0 : (size_t)ceil_div(T, kMinTile);
    size_t o = align_up(sizeof(WsHeader), kAlign);
    lo.ticket = o;   o = align_up(o + sizeof(int), kAlign);
    lo.tile_seq = o; o = align_up(o + sizeof(int) * tiles, kAlign);
    lo.run = o;      o = align_up(o + sizeof(float2) * tiles * lo.Cpad, kAlign);
    lo.joint = o;    o = align_up(o + sizeof(float2) * (tiles / kGroup) * lo.Cpad, kAlign);
    lo.state = o;    o = align_up(o + sizeof(float) * (tiles / kSuper) * lo.Cpad, kAlign);
    lo.total = o;
    return lo;
}

// More than one tile: the preparation, then a persistent kernel that may start while it ends.
template <typename F, typename... Args>
cudaError_t launch_tiles(F kernel, const GatedParams& p, int reverse, int tile_tokens, int tiles, int slices,
                         int per_sm, int threads, size_t smem, cudaStream_t s, Args... args) {
    const int nsm = sm_count();
    if (nsm <= 0) return cudaErrorInvalidDevice;
    const int64_t work = (int64_t)tiles * slices;
    if (work > INT32_MAX / 2) return cudaErrorInvalidValue;
    const int prep = (int)min64(ceil_div((int64_t)tiles * p.Cpad, 16 * kPrepThreads), 4 * nsm);
    gated_prep_kernel<<<prep, kPrepThreads, 0, s>>>(p, tile_tokens, tiles, reverse);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)min64(work, (int64_t)nsm * per_sm));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, kernel, p, tiles, slices, args...);
}

template <typename TA, typename TX, bool Rev, bool Vec, bool Solo, int W, int K>
cudaError_t run_registers(const GatedParams& p, int slices, cudaStream_t s) {
    constexpr int kTile = W * K, kThreads = (W + 2) * 32;
    const int tiles = (int)ceil_div(p.T, kTile);
    auto kernel = gated_scan_kernel<TA, TX, Rev, Vec, Solo, W, K>;
    if constexpr (Solo) {
        kernel<<<slices, kThreads, 0, s>>>(p, tiles, slices);
        return cudaGetLastError();
    } else {
        return launch_tiles(kernel, p, Rev ? 1 : 0, kTile, tiles, slices, kRegisterBlocks, kThreads, 0, s);
    }
}

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);
// The driver's encoder of tile maps, looked up once (the library is not linked with the driver's).
EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e =
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
        return e == cudaSuccess && found == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeTiled>(f) : nullptr;
    }();
    return fn;
}

// [T][C] rows -> boxes of `rows` tokens x kSlice channels, unswizzled.
template <typename T>
bool row_map(CUtensorMap* m, const void* base, int64_t tokens, int C, int rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)C, (cuuint64_t)tokens}, strides[1] = {(cuuint64_t)C * sizeof(T)};
    const cuuint32_t box[2] = {kSlice, (cuuint32_t)rows}, steps[2] = {1, 1};
    const EncodeTiled encode = encode_tiled();
    return encode && encode(m, sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                            const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename TA, typename TX, bool Rev, Copies Copy, bool Vec, int W, int K, int S>
cudaError_t run_ring(const GatedParams& p, int slices, cudaStream_t s) {
    using R = Ring<TA, TX, Rev, Copy, W, K, S>;
    static_assert(R::kRows % 2 == 0 && K % 2 == 0, "a row's parity is that of its place in the tile");
    static_assert(R::kBytes <= 227 * 1024, "a block's shared memory");
    CUtensorMap ma{}, mx{}, mh{};
    if (Copy == kTiles && (!row_map<TA>(&ma, p.a, p.T, p.C, R::kRows) || !row_map<TX>(&mx, p.x, p.T, p.C, R::kRows) ||
                !row_map<TX>(&mh, Rev ? p.h : p.x, p.T, p.C, R::kRows)))
        return cudaErrorInvalidValue;
    auto kernel = gated_ring_kernel<TA, TX, Rev, Copy, Vec, W, K, S>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)R::kBytes);
    if (e != cudaSuccess) return e;
    return launch_tiles(kernel, p, Rev ? 1 : 0, R::kRows, (int)ceil_div(p.T, R::kRows), slices, 1, R::kThreads,
                        R::kBytes, s, slices > 1 ? ~0ull / (unsigned)slices + 1 : 0ull, ma, mx, mh);
}

bool two_aligned(const void* p, size_t esize) { return reinterpret_cast<uintptr_t>(p) % (2 * esize) == 0; }

bool tile_aligned(const void* p, int C, size_t esize) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (size_t)C * esize % 16 == 0;
}

// Every row in words of four bytes.
bool word_aligned(const void* p, int C, size_t esize) {
    return reinterpret_cast<uintptr_t>(p) % 4 == 0 && (size_t)C * esize % 4 == 0;
}

// The inputs' places choose how tiles come in, the outputs' how rows go out.
template <typename TA, typename TX, bool Rev>
cudaError_t dispatch(const GatedParams& p, int slices, cudaStream_t s) {
    constexpr size_t ea = sizeof(TA), ex = sizeof(TX);
    const bool out = p.C % 2 == 0 && two_aligned(p.y, ex) && two_aligned(p.da, ea);
    // stages that fill shared memory
    constexpr int kBytes = (int)(ea + (Rev ? 2 : 1) * ex);   // of a token and channel
    constexpr int W = 4, K = kBytes <= 4 ? 32 : kBytes <= 10 ? 16 : 8;
    constexpr int S = kBytes <= 4 ? 6 : kBytes <= 6 ? 8 : kBytes <= 8 ? 6 : kBytes <= 10 ? 4 : 8;
    if (p.T <= W * K) {
        const bool vec = out && two_aligned(p.a, ea) && two_aligned(p.x, ex) && two_aligned(p.h, ex);
        return vec ? run_registers<TA, TX, Rev, true, true, W, K>(p, slices, s)
                   : run_registers<TA, TX, Rev, false, true, W, K>(p, slices, s);
    }
    if (out && tile_aligned(p.a, p.C, ea) && tile_aligned(p.x, p.C, ex) && tile_aligned(p.h, p.C, ex))
        return run_ring<TA, TX, Rev, kTiles, true, W, K, S>(p, slices, s);
    if constexpr (ea == 4 && ex == 4) {
        return run_ring<TA, TX, Rev, kWords, false, W, K, S>(p, slices, s);
    } else {
        if (word_aligned(p.a, p.C, ea) && word_aligned(p.x, p.C, ex) && word_aligned(p.h, p.C, ex))
            return out ? run_ring<TA, TX, Rev, kWords, true, W, K, S>(p, slices, s)
                       : run_ring<TA, TX, Rev, kWords, false, W, K, S>(p, slices, s);
        // (rows of even length start on four bytes with their array)
        const bool starts = word_aligned(p.a, 2, ea) && word_aligned(p.x, 2, ex) && word_aligned(p.h, 2, ex);
        if (p.C % 2 == 1 && starts)
            return run_ring<TA, TX, Rev, kHalves, false, W, K, Rev && kBytes == 6 ? 6 : S>(p, slices, s);
        return run_registers<TA, TX, Rev, false, false, W, K>(p, slices, s);
    }
}

template <typename TA, typename TX>
cudaError_t step(const void* a, const void* b, int64_t n, const float* state_in, float* state_out, void* h,
                 cudaStream_t s) {
    auto aligned = [](const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; };
    const TA* ta = static_cast<const TA*>(a);
    const TX* tb = static_cast<const TX*>(b);
    TX* th = static_cast<TX*>(h);
    if (n % 4 == 0 && aligned(a, 4 * sizeof(TA)) && aligned(b, 4 * sizeof(TX)) && aligned(h, 4 * sizeof(TX)) &&
        aligned(state_in, 16) && aligned(state_out, 16))
        gated_step_kernel<TA, TX, 4><<<(unsigned)ceil_div(n / 4, kPrepThreads), kPrepThreads, 0, s>>>(
            ta, tb, n, state_in, state_out, th);
    else
        gated_step_kernel<TA, TX, 1><<<(unsigned)ceil_div(n, kPrepThreads), kPrepThreads, 0, s>>>(
            ta, tb, n, state_in, state_out, th);
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
    p.tile_seq = reinterpret_cast<int*>(ws + lo.tile_seq);
    p.run = reinterpret_cast<float2*>(ws + lo.run);
    p.joint = reinterpret_cast<float2*>(ws + lo.joint);
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
