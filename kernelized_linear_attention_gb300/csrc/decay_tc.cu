// Linear attention with a decay for each head on the tensor cores: bf16 rows of up to 128 channels.
//
// A chunk is 128 tokens of one head; a block walks the chunks of one segment in order (from the end in a reverse pass).
// Per chunk, with x, y, z as in ops/decay.h, n tokens, and S the state before the chunk:
//
//     A = x y^T                       P = A decayed and masked (scale g^(i-j), j <= i)
//     O = x S                         O scaled per row (scale g^(i+1)), then O += P z
//     S = g^n S + (w y)^T z           w_j = g^(n-1-j)
//
// Every product is tcgen05.mma kind::f16 on bf16 with fp32 accumulators in tensor memory.  What is computed here enters
// a product rounded: P and w y to bf16 (2^-8; P of a segment of one chunk in two parts), like the outputs that come of
// them; the state as a bf16 and what that leaves (2^-16); the weighted y of the state sums, which calls return, in
// three parts (2^-24).  Values keep bf16's range, so nothing is scaled or clamped.  Rows of operands lie in shared
// memory as in tc_ptx.cuh ([rows][64] blocks with the 128-byte
// swizzle); D is 64 or 128, the channels of both sides rounded up (missing ones are filled with zeros by TMA).
//
// P z with a masked P of 0 would spread a z that is not finite to tokens that do not see it.  Such values are found
// while the chunk waits for its products, set to zero after the state has taken them, and written as NaN to the
// channel's outputs that see them.
#include "ops/decay.h"
#include "tc_ptx.cuh"

namespace la {

namespace {

using namespace tc;

constexpr int kC = 128;                       // tokens of a chunk
constexpr uint32_t kTile = kC * 128;          // [128][64] bf16
constexpr uint64_t kDrainNs = 100000000ull;   // bound of the waits before an early exit
__device__ int g_force_wait_timeout = 0;      // test hook: a wait that nothing ends

// ---------------------------------------------------------------------------
// Pieces
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Bytes to the next multiple of 1024 (as an offset, so that what lies there is known to be shared memory: through a
// pointer that went through an integer every access is a generic one).
__device__ __forceinline__ uint32_t to_1024(const void* p) { return (0u - smem_u32(p)) & 1023u; }

// A pair of fp32 as bf16 and the rest.
__device__ __forceinline__ uint32_t split(uint64_t& v) {
    const uint32_t h = f32x2_to_bf16x2(v);
    v = f32x2_fma(f32x2_of(h << 16, h & 0xffff0000u), f32x2_splat(-1.f), v);
    return h;
}
__device__ __forceinline__ uint64_t pair_of(uint32_t w) { return f32x2_of(w << 16, w & 0xffff0000u); }

// The loops of all roles have to stay in the instruction caches together (unrolled and with every wait's retries in
// place the products took 128 us for 65536 x 16 x 64, code of 78 KB): waits that are not over at once, and what only
// values that are not finite need, are calls.
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity); }
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
    return mbar_try_wait(bar, parity) || wait_long(bar, parity);
}
// After a wait for tensor memory: values that were on their way are not used before it.
template <int N>
__device__ __forceinline__ void arrived(uint32_t (&v)[N]) {
#pragma unroll
    for (int j = 0; j < N; ++j) asm volatile("" : "+r"(v[j]));
}
// A whole warp's wait: true for every lane or for none.
__device__ __forceinline__ bool wait_w(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(bar, parity));
}
// A warp's arrival, behind what its lanes have written to shared memory for the async proxy.
__device__ __forceinline__ void arrive_w(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
__device__ __forceinline__ void init_all(uint64_t* bars, int n, uint32_t count) {
    for (int i = 0; i < n; ++i) mbar_init(bars + i, count);
}

// Powers 0 .. 128 of the decay.
__device__ __forceinline__ void fill_powers(float* pw, const DecayBase& base) {
    for (int i = threadIdx.x; i <= kC; i += blockDim.x) pw[i] = decay_power(base, i);
}

// A channel that is not finite at token `row` of the chunk.
__device__ inline void move_edge(unsigned short* edge, int row, bool reverse) {
    unsigned short held = *edge;
    while (reverse ? row + 1 > held : row < held) {
        const unsigned short seen = atomicCAS(edge, held, (unsigned short)(reverse ? row + 1 : row));
        if (seen == held) break;
        held = seen;
    }
}

// Waits, like mbar_wait, until a count in shared memory has got to `least`.
__device__ __noinline__ bool wait_count(const int* count, int least) {
    const uint64_t began = globaltimer_ns();
    while (*reinterpret_cast<const volatile int*>(count) < least)
        if (globaltimer_ns() - began > 2000000000ull) return false;
    __threadfence_block();
    return true;
}
// Sets a row's values that are not finite to zero in four of its 16-byte chunks (row -1: nothing).
__device__ __noinline__ void clear_strange(unsigned char* tile, unsigned short* edge, int* strange, int row, int c0, bool reverse) {
    if (row < 0) return;
#pragma unroll 1
    for (int i = 0; i < 32; ++i) {
        uint16_t* const at = reinterpret_cast<uint16_t*>(tile + sw128_chunk(row, c0 + (i >> 3))) + (i & 7);
        if ((*at & 0x7f80u) != 0x7f80u) continue;
        *at = 0;
        move_edge(edge + 8 * c0 + i, row, reverse);
        *strange = 1;
    }
}
// Channel i of a row's 32 (pairs in o) from the token on that made it strange is NaN.
__device__ __noinline__ uint32_t mark_strange(uint32_t o, const unsigned short* edge, int row, bool reverse) {
    if (reverse ? row < edge[0] : row >= edge[0]) o = (o & 0xffff0000u) | 0x7fc0u;
    if (reverse ? row < edge[1] : row >= edge[1]) o = (o & 0xffffu) | 0x7fc00000u;
    return o;
}

__device__ __forceinline__ void store_32(void* to, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// ---------------------------------------------------------------------------
// State sums of a segment
// ---------------------------------------------------------------------------
// Warp 0 loads, warp 1 issues the products, two groups of eight warps weight y, one the even tiles and one the odd ones.
// The tensor cores truncate when they accumulate: after 64 steps (1024 tokens) the sums go on in fp32 registers, rounded
// to nearest.  (Two parts of the weighted y instead of three, which outputs alone would not notice: 57 us instead of 60.)
// 65536 x 16 x 64 take 60 us, 40 for their bytes at the copy rate, and 16384 x 16 x 128 49 with tiles of 64 tokens (128
// leave no room for a second weighted tile): the weighting warps issue in 40% of the slots, each tile's in a row.
constexpr int kStatesThreads = 640;
template <int D> struct StatesShape {
    static constexpr int blocks = D / 64;                 // of 64 channels
    static constexpr int rows = D == 64 ? 128 : 64;       // tokens of a tile
    static constexpr int flush = 1024 / rows;             // tiles
    static constexpr int warps = D == 64 ? 8 : 16;        // that have the sums
    static constexpr int columns = D == 64 ? 128 : 256;   // of tensor memory a set of sums, of two
    static constexpr int stages = 4;                      // of y and z
    static constexpr uint32_t tile = rows * 128;          // bytes of a block
};
template <int D> struct __align__(1024) StatesSmem {
    using F = StatesShape<D>;
    unsigned char yw[2][3][F::blocks][F::tile];           // weighted y in three parts, two tiles
    unsigned char y[F::stages][F::blocks][F::tile], z[F::stages][F::blocks][F::tile];
    float pw[kC + 4];
    uint64_t full[F::stages], empty[F::stages];           // TMA -> weighting, products;  both -> TMA
    uint64_t yw_full[2], yw_empty[2];                     // weighting -> products;  products -> weighting
    uint64_t sum_full[2], sum_empty[2];                   // products -> registers;  registers -> products
    uint64_t drain, never;
    uint32_t tmem;
};

template <int D>
__global__ void __launch_bounds__(kStatesThreads, 1)
    decay_tc_states_kernel(const __grid_constant__ DecayCall c, const __grid_constant__ DecayStates p, DecayWhich which,
                           const __grid_constant__ CUtensorMap my, const __grid_constant__ CUtensorMap mz) {
    using F = StatesShape<D>;
    extern __shared__ __align__(1024) unsigned char raw[];
    StatesSmem<D>& s = *reinterpret_cast<StatesSmem<D>*>(raw + to_1024(raw));
    const int h = blockIdx.x, index = blockIdx.y + 65535 * blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    chain_wait();
    chain_go();
    DecaySegment g;
    if (index >= (which == kEnds ? c.nseq : c.segments)) return;
    if (decay_malformed(c)) return;
    const int64_t size = (int64_t)c.dk * c.dv;
    float* to;
    const float* enter = nullptr;
    if (which == kEnds) {
        to = p.edge_out + ((int64_t)index * c.H + h) * size;
        if (!decay_edge_segment(c, index, p.reverse, g)) {
            // an empty sequence: what enters it leaves it
            const float* from = p.edge_in ? p.edge_in + ((int64_t)index * c.H + h) * size : nullptr;
            for (int i = threadIdx.x; i < size; i += kStatesThreads) to[i] = from ? from[i] : 0.f;
            return;
        }
        enter = decay_entering(c, g, h, p.reverse, p.edge_in);
    } else {
        if (!decay_segment(c, index, g)) return;
        if (p.reverse ? decay_first(g) : decay_last(g)) {
            if (which == kInner) return;
            to = p.edge_out + ((int64_t)g.seq * c.H + h) * size;
        } else {
            to = c.states[p.reverse] + ((int64_t)(decay_slot(g) - (p.reverse ? 1 : 0)) * c.H + h) * size;
        }
    }
    const DecayBase base = decay_base(c.log_decay[h]);
    const int tiles = (g.end - g.start + F::rows - 1) / F::rows, groups = (tiles + F::flush - 1) / F::flush;
    if (threadIdx.x == 0) {
        init_all(s.full, F::stages, 1);
        init_all(s.empty, F::stages, 8 + 1);
        init_all(s.yw_full, 2, 8);
        init_all(s.yw_empty, 2, 1);
        init_all(s.sum_full, 2, 1);
        init_all(s.sum_empty, 2, F::warps);
        init_all(&s.drain, 1, 1);
        init_all(&s.never, 1, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&s.tmem, 2 * F::columns);
        tmem_relinquish();
    }
    fill_powers(s.pw, base);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s.tmem;
    bool ok = true;
    int loads = 0;
    // of the warps that have sums: 32 columns of a row
    const int w = warp - 4, q = w & 3, part = (D == 64 ? w & 7 : w) >> 2, row = 32 * q + lane, col = 32 * part;
    float sum[32];

    if (warp == 0) {
        if (lane == 0) {
            for (; loads < tiles; ++loads) {
                const int st = loads % F::stages;
                if (loads >= F::stages) ok = wait(&s.empty[st], (loads / F::stages - 1) & 1);
                if (!ok) break;
                mbar_arrive_expect_tx(&s.full[st], 2 * F::blocks * F::tile);
                for (int b = 0; b < F::blocks; ++b) {
                    tma_load_3d(s.y[st][b], &my, 64 * b, h, g.start + loads * F::rows, &s.full[st]);
                    tma_load_3d(s.z[st][b], &mz, 64 * b, h, g.start + loads * F::rows, &s.full[st]);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        for (int k = 0; k < tiles; ++k) {
            const int st = k % F::stages, b = k & 1, f = k / F::flush, a = f & 1;
            ok = wait_w(&s.yw_full[b], (k >> 1) & 1);
            if (ok && k % F::flush == 0 && f >= 2) ok = wait_w(&s.sum_empty[a], (f / 2 - 1) & 1);
            if (!ok) break;
            tc_fence_after();
            constexpr uint32_t id = idesc_bf16(128, D, true, true);
            const uint64_t dz = sdesc_sw128(smem_u32(s.z[st]), F::tile, 1024);
            // D = 64: the first two parts of y are one product's 128 rows; the third's other rows are whatever lies behind
            // it, not used.  D = 128: the first part has sums of its own, the small ones share theirs.
#pragma unroll 1
            for (int i = 0; i < (D == 64 ? 2 : 3); ++i) {
                const uint64_t dy = sdesc_sw128(smem_u32(s.yw[b][D == 64 ? 2 * i : i]), F::tile, 1024);
                const uint32_t acc = tm + a * F::columns + D * (i < 2 ? i : 1);
#pragma unroll 4
                for (int j = 0; j < F::rows / 16; ++j)
                    mma_ss_w(acc, sdesc_add(dy, 2048 * j), sdesc_add(dz, 2048 * j), id,
                             k % F::flush > 0 || j > 0 || i == 2 ? 1u : 0u);
            }
            mma_commit_w(&s.yw_empty[b]);
            mma_commit_w(&s.empty[st]);
            if (k % F::flush == F::flush - 1 || k + 1 == tiles) mma_commit_w(&s.sum_full[a]);
        }
    } else if (warp >= 4) {
        const int mine = w >> 3, w8 = w & 7;
        // of a tile: this thread's row, and its 32 channels' first 16 bytes (the j-th: place ^ 16 j)
        const int r = D == 64 ? 32 * (w8 & 3) + lane : 32 * (w8 & 1) + lane, p8 = D == 64 ? w8 >> 2 : w8 >> 1;
        const uint32_t place = sw128_chunk(r, (p8 & 1) * 4);
        const bool sums = D == 128 || mine == 0;
        if (g_force_wait_timeout) ok = __all_sync(0xffffffffu, mbar_wait(&s.never, 0, 1000000ull));
#pragma unroll
        for (int j = 0; j < 32; ++j) sum[j] = 0.f;
        int flushed = 0;
        for (int k = mine; ok && (k < tiles || (sums && flushed < groups)); k += 2) {
            if (k < tiles) {
                const int st = k % F::stages, b = k & 1, t0 = g.start + k * F::rows, n = min(F::rows, g.end - t0);
                ok = wait_w(&s.full[st], (k / F::stages) & 1);
                if (ok && k >= 2) ok = wait_w(&s.yw_empty[b], (k / 2 - 1) & 1);
                if (!ok) break;
                const float far = p.reverse ? c.scale * decay_power(base, t0 - g.start) : decay_power(base, g.end - t0 - n);
                const uint64_t weight = f32x2_splat(r < n ? far * s.pw[p.reverse ? r + 1 : n - 1 - r] : 0.f);
                uint4 in[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) in[j] = *reinterpret_cast<const uint4*>(s.y[st][p8 >> 1] + (place ^ (16 * j)));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t v[4] = {in[j].x, in[j].y, in[j].z, in[j].w};
                    uint32_t o[3][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint64_t e = f32x2_mul(pair_of(r < n ? v[i] : 0u), weight);
                        o[0][i] = split(e);
                        o[1][i] = split(e);
                        o[2][i] = f32x2_to_bf16x2(e);
                    }
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        *reinterpret_cast<uint4*>(s.yw[b][i][p8 >> 1] + (place ^ (16 * j))) =
                            make_uint4(o[i][0], o[i][1], o[i][2], o[i][3]);
                    // nothing from another sequence
                    if (r >= n) *reinterpret_cast<uint4*>(s.z[st][p8 >> 1] + (place ^ (16 * j))) = make_uint4(0, 0, 0, 0);
                }
                fence_async_smem();
                arrive_w(&s.yw_full[b]);
                arrive_w(&s.empty[st]);
            }
            if (!sums || flushed == groups || (k < tiles && k < F::flush * (flushed + 1))) continue;
            const int a = flushed & 1;
            ok = wait_w(&s.sum_full[a], (flushed >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            // D = 64: rows 64 .. 127 of the first columns are the second part's; the third part's rows are 0 .. 63
            const int sets = D == 64 && q >= 2 ? 1 : 2;
#pragma unroll 1
            for (int i = 0; i < sets; ++i)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t v[16];
                    tmem_ld16(tmem_addr(tm, 32 * q, a * F::columns + D * i + col + 16 * u), v);
                    tmem_ld_wait();
                    arrived(v);
#pragma unroll
                    for (int j = 0; j < 16; ++j) sum[16 * u + j] += __uint_as_float(v[j]);
                }
            tc_fence_before();
            arrive_w(&s.sum_empty[a]);
            ++flushed;
        }
    }
    if (__syncthreads_or(!ok)) {
        // copies and products on their way end before the block does
        if (threadIdx.x == 0) {
            record_error(c.hdr, LA_DEVERR_WAIT_TIMEOUT);
            for (int i = max(0, loads - F::stages); i < loads; ++i)
                mbar_wait(&s.full[i % F::stages], (i / F::stages) & 1, kDrainNs);
        }
        if (warp == 1) {
            mma_commit_w(&s.drain);
            mbar_wait(&s.drain, 0, kDrainNs);
        }
    } else {
        const bool on = warp >= 4 && (D == 128 || w < 8);
        const float keep = decay_power(base, g.end - g.start);
        if (D == 64) {
            float (*ex)[65] = reinterpret_cast<float (*)[65]>(s.yw);
            if (on && q >= 2) {
#pragma unroll
                for (int j = 0; j < 32; ++j) ex[row - 64][col + j] = sum[j];
            }
            __syncthreads();
            if (on && q < 2) {
#pragma unroll
                for (int j = 0; j < 32; ++j) sum[j] += ex[row][col + j];
            }
        }
        if (on && row < c.dk) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                if (col + j >= c.dv) break;
                const int64_t at = (int64_t)row * c.dv + col + j;
                to[at] = enter ? fmaf(keep, enter[at], sum[j]) : sum[j];
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tm, 2 * F::columns);
}

// ---------------------------------------------------------------------------
// Products of a segment
// ---------------------------------------------------------------------------
// Warp 0 loads; warps 1, 2 and 3 issue products (scores and P z; the state's update; x S: one warp for all was what the
// others waited for, a hundred cycles and more for each of its waits and commits); warps 4 .. 11 look z over and turn
// scores into P; 12 .. 19 weight y (in its place, once the scores have read it) and make an operand of the state;
// 20 .. 27 write the outputs.  Every barrier's waits are consecutive, or behind something that implies the phase before,
// and no phase can end twice before a waiter has seen it: a wait tells phases by parity alone.
// 65536 x 16 x 64 take 107 us, 79 for their bytes at the copy rate: a chunk 2.0 us, of which the products are 0.7; half of
// the issue slots are used, by the way of the scores through registers above all.  16384 x 16 x 128 take 82 us, one
// wave of 128 blocks.  A block begins and ends in 4 us.
constexpr int kPassThreads = 896;
template <int D> struct PassShape {
    static constexpr int blocks = D / 64;
    static constexpr int stages = D == 64 ? 4 : 2, z_stages = D == 64 ? 4 : 1;   // of x and y; of z
    static constexpr int scores = D == 64 ? 2 : 1;        // buffers of scores and P
    // operands of the state; D = 64: its two parts side by side, one product of twice the width
    static constexpr int states = D == 64 ? 2 : 1, width = 128;
    static constexpr int ring = 4;                        // chunks from the look at z to the outputs, at most
    // tensor memory: the state, scores (then P: for each 16 tokens eight columns, and eight of second parts), x S, P z
    static constexpr uint32_t state = 0, score = D, read = score + 128 * scores, out = read + width;
};
template <int D> struct __align__(1024) PassSmem {
    using F = PassShape<D>;
    unsigned char x[F::stages][F::blocks][kTile], y[F::stages][F::blocks][kTile], z[F::z_stages][F::blocks][kTile];
    unsigned char state[F::states][2][F::blocks][D * 128];   // [D][64] in blocks, in two parts
    float pw[kC + 4 + 32];                                // powers of the decay, then 0 .. 31 of them with the scale
    __align__(16) float in_block[32];                     // decay inside a block of 32 tokens
    // by chunk: the first token whose channel is not finite (or 128); reverse: one behind the last one (or 0).  What is left
    // of the chunk that had the place before need not go: that channel is not finite in the state any more, and so in no
    // output of a later chunk.
    unsigned short edge[F::ring][D];
    int strange[F::ring];                                 // by chunk: whether there is one
    uint64_t xy_full[F::stages], xy_empty[F::stages], z_full[F::z_stages], z_empty[F::z_stages];
    uint64_t a_full[2], p_full[2];                        // scores;  P, and z looked over
    uint64_t conv_full[2], state_full;                    // operands made;  state updated
    uint64_t r_full[2], r_empty, o_full, o_empty;         // x S, P z;  taken by the outputs' warps
    uint64_t drain, never;
    uint32_t tmem;
    int updated;                                          // chunks that the state has taken
};

template <int D, bool Reverse>
__global__ void __launch_bounds__(kPassThreads, 1)
    decay_tc_pass_kernel(const __grid_constant__ DecayCall c, const __grid_constant__ DecayPass p, bool wide,
                         const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap my,
                         const __grid_constant__ CUtensorMap mz) {
    using F = PassShape<D>;
    extern __shared__ __align__(1024) unsigned char raw[];
    PassSmem<D>& s = *reinterpret_cast<PassSmem<D>*>(raw + to_1024(raw));
    const int h = blockIdx.x, index = blockIdx.y + 65535 * blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, row = 32 * q + lane;
    chain_wait();
    chain_go();
    DecaySegment g;
    if (index >= c.segments || !decay_segment(c, index, g)) return;
    const DecayBase base = decay_base(c.log_decay[h]);
    const float* const enter = decay_entering(c, g, h, p.reverse, p.edge);
    const int chunks = (g.end - g.start + kC - 1) / kC;
    constexpr bool reverse = Reverse;
    auto token = [&](int it) { return g.start + (reverse ? chunks - 1 - it : it) * kC; };
    // P in two parts where the segment is one chunk: the outputs are then as exact as in 32 bits, for little.  In every
    // chunk the second part takes the warps that make P a fifth longer, and all wait for them (65536 x 16 x 64: 218 us
    // instead of 183), for 0.0021 of the outputs' norm instead of 0.0023, with 0.0017 their own rounding.
    const bool two = chunks == 1;
    if (threadIdx.x == 0) {
        init_all(s.xy_full, F::stages, 1);
        init_all(s.xy_empty, F::stages, 2);
        init_all(s.z_full, F::z_stages, 1);
        init_all(s.z_empty, F::z_stages, 2);
        init_all(s.a_full, 2, 1);
        init_all(s.p_full, 2, 8);
        init_all(s.conv_full, 2, 8);
        init_all(&s.state_full, 1, 1);
        init_all(s.r_full, 2, 1);
        init_all(&s.r_empty, 1, 8);
        init_all(&s.o_full, 1, 1);
        init_all(&s.o_empty, 1, 8);
        init_all(&s.drain, 1, 3);
        init_all(&s.never, 1, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&s.tmem, 512);
        tmem_relinquish();
    }
    fill_powers(s.pw, base);
    if (threadIdx.x < 32) s.in_block[threadIdx.x] = decay_power(base, reverse ? threadIdx.x : 31 - threadIdx.x);
    if (threadIdx.x < 32) s.pw[kC + 4 + threadIdx.x] = c.scale * decay_power(base, threadIdx.x);
    for (int i = threadIdx.x; i < F::ring * D; i += kPassThreads) s.edge[i / D][i % D] = reverse ? 0 : kC;
    if (threadIdx.x < F::ring) s.strange[threadIdx.x] = 0;
    if (threadIdx.x == 0) s.updated = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s.tmem, lanes = tmem_addr(tm, 32 * q, 0);
    bool ok = true;
    int xy_loads = 0, z_loads = 0;

    if (warp == 0) {
        // ---- loads
        if (lane == 0) {
            for (int it = 0; it < chunks; ++it) {
                const int st = it % F::stages, sz = it % F::z_stages;
                if (it >= F::stages) ok = wait(&s.xy_empty[st], (it / F::stages - 1) & 1);
                if (!ok) break;
                mbar_arrive_expect_tx(&s.xy_full[st], 2 * F::blocks * kTile);
                for (int b = 0; b < F::blocks; ++b) {
                    tma_load_3d(s.x[st][b], &mx, 64 * b, h, token(it), &s.xy_full[st]);
                    tma_load_3d(s.y[st][b], &my, 64 * b, h, token(it), &s.xy_full[st]);
                }
                ++xy_loads;
                if (it >= F::z_stages) ok = wait(&s.z_empty[sz], (it / F::z_stages - 1) & 1);
                if (!ok) break;
                mbar_arrive_expect_tx(&s.z_full[sz], F::blocks * kTile);
                for (int b = 0; b < F::blocks; ++b) tma_load_3d(s.z[sz][b], &mz, 64 * b, h, token(it), &s.z_full[sz]);
                ++z_loads;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- scores (a buffer ahead or two) and P z
        auto scores = [&](int it) {
            const int st = it % F::stages, b = it % F::scores;
            ok = wait_w(&s.xy_full[st], (it / F::stages) & 1);
            if (!ok) return;
            tc_fence_after();
            constexpr uint32_t id = idesc_bf16(128, 128, false, false);
            const uint64_t dx = sdesc_sw128(smem_u32(s.x[st]), 16, 1024), dy = sdesc_sw128(smem_u32(s.y[st]), 16, 1024);
#pragma unroll 4
            for (int j = 0; j < D / 16; ++j) {
                const uint32_t at = (j >> 2) * kTile + 32 * (j & 3);
                mma_ss_w(tm + F::score + 128 * b, sdesc_add(dx, at), sdesc_add(dy, at), id, j > 0 ? 1u : 0u);
            }
            mma_commit_w(&s.a_full[b]);
        };
        for (int it = 0; it < min(F::scores, chunks) && ok; ++it) scores(it);
        for (int it = 0; it < chunks && ok; ++it) {
            const int b = it % F::scores, sz = it % F::z_stages;
            // (a chunk that is not whole: rows behind its end are zero once the operands are made)
            ok = wait_w(&s.p_full[b], (it / F::scores) & 1) && wait_w(&s.z_full[sz], (it / F::z_stages) & 1) &&
                 (it == 0 || wait_w(&s.o_empty, (it - 1) & 1)) &&
                 (g.end - token(it) >= kC || wait_w(&s.conv_full[it & 1], (it >> 1) & 1));
            if (!ok) break;
            tc_fence_after();
            constexpr uint32_t id = idesc_bf16(128, D, false, true);
            const uint64_t dz = sdesc_sw128(smem_u32(s.z[sz]), kTile, 1024);
#pragma unroll 4
            for (int j = 0; j < (two ? 2 : 1) * kC / 16; ++j)
                mma_ts_w(tm + F::out, tm + F::score + 128 * b + (two ? 8 : 16) * j, sdesc_add(dz, 2048 * (two ? j >> 1 : j)), id,
                         j > 0 ? 1u : 0u);
            mma_commit_w(&s.o_full);
            mma_commit_w(&s.z_empty[sz]);
            // (the warps that weight y have seen this buffer's scores done, too)
            if (it + F::scores < chunks) ok = wait_w(&s.conv_full[it & 1], (it >> 1) & 1);
            if (ok && it + F::scores < chunks) scores(it + F::scores);
        }
    } else if (warp == 2) {
        // ---- the state's update; D = 64: rows 64 .. 127 are whatever lies behind the weighted y, nothing reads them
        for (int it = 0; it + 1 < chunks && ok; ++it) {
            const int st = it % F::stages, sz = it % F::z_stages;
            ok = wait_w(&s.conv_full[it & 1], (it >> 1) & 1) && wait_w(&s.z_full[sz], (it / F::z_stages) & 1);
            if (!ok) break;
            tc_fence_after();
            constexpr uint32_t id = idesc_bf16(128, D, true, true);
            const uint64_t dy = sdesc_sw128(smem_u32(s.y[st]), kTile, 1024), dz = sdesc_sw128(smem_u32(s.z[sz]), kTile, 1024);
#pragma unroll 4
            for (int j = 0; j < kC / 16; ++j)
                mma_ss_w(tm + F::state, sdesc_add(dy, 2048 * j), sdesc_add(dz, 2048 * j), id, it > 0 || enter || j > 0 ? 1u : 0u);
            mma_commit_w(&s.state_full);
            mma_commit_w(&s.xy_empty[st]);
            mma_commit_w(&s.z_empty[sz]);
            ok = wait_w(&s.state_full, it & 1);
            if (lane == 0) *reinterpret_cast<volatile int*>(&s.updated) = it + 1;
            __syncwarp();
        }
    } else if (warp == 3) {
        // ---- x S
        for (int it = 0; it < chunks && ok; ++it) {
            const int st = it % F::stages;
            ok = wait_w(&s.conv_full[it & 1], (it >> 1) & 1) && wait_w(&s.xy_full[st], (it / F::stages) & 1) &&
                 (it == 0 || wait_w(&s.r_empty, (it - 1) & 1));
            if (!ok) break;
            if (it > 0 || enter) {
                tc_fence_after();
                constexpr uint32_t id = idesc_bf16(128, F::width, false, true);
                const uint64_t dx = sdesc_sw128(smem_u32(s.x[st]), 16, 1024);
#pragma unroll 1
                for (int i = 0; i < (D == 64 ? 1 : 2); ++i) {
                    const uint64_t ds = sdesc_sw128(smem_u32(s.state[it % F::states][i]), D * 128, 1024);
#pragma unroll 4
                    for (int j = 0; j < D / 16; ++j)
                        mma_ss_w(tm + F::read, sdesc_add(dx, (j >> 2) * kTile + 32 * (j & 3)), sdesc_add(ds, 2048 * j), id,
                                 i > 0 || j > 0 ? 1u : 0u);
                }
            }
            mma_commit_w(&s.r_full[it & 1]);
            mma_commit_w(&s.xy_empty[st]);
        }
    } else if (warp >= 4 && warp < 12) {
        // ---- scores to P, 16 tokens at a time
        const int half = (warp - 4) >> 2, c0 = half * 4;           // of z: this thread's 32 channels of every 64
        const uint32_t place = sw128_chunk(row, c0);               // of their first 16 bytes; the j-th: place ^ 16 j
        if (g_force_wait_timeout) ok = __all_sync(0xffffffffu, mbar_wait(&s.never, 0, 1000000ull));
        for (int it = 0; it < chunks && ok; ++it) {
            const int b = it % F::scores, n = min(kC, g.end - token(it)), sz = it % F::z_stages;
            const uint32_t zpar = (it / F::z_stages) & 1;
            const bool last = it + 1 == chunks;
            // before the scores are there: is a value of z not finite?
            ok = wait_w(&s.z_full[sz], zpar);
            if (!ok) break;
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < F::blocks; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint4 w = *reinterpret_cast<const uint4*>(s.z[sz][k] + (place ^ (16 * j)));
                    if (row < n) top = __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                                 __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
                }
            if (__any_sync(0xffffffffu, (top & 0xffffu) >= 0x7f80u || (top >> 16) >= 0x7f80u)) {
                // once the state has taken them, they are set to zero
                if (!last) ok = __all_sync(0xffffffffu, wait_count(&s.updated, it + 1));
                if (!ok) break;
                for (int k = 0; k < F::blocks; ++k)
                    clear_strange(s.z[sz][k], s.edge[it % F::ring] + 64 * k, &s.strange[it % F::ring], row < n ? row : -1, c0, reverse);
                fence_async_smem();
            }
            ok = wait_w(&s.a_full[b], (it / F::scores) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t at = lanes + F::score + 128 * b;
#pragma unroll 1
            for (int jb = 2 * half; jb < 2 * half + 2; ++jb) {
                uint32_t v[32];
                if (reverse ? jb < q : jb > q) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0;
                } else {
                    tmem_ld32(at + 32 * jb, v);
                    tmem_ld_wait();
                    arrived(v);
                    if (jb != q) {
                        // decay to the block's nearest token, times that inside the block
                        const uint64_t f = f32x2_splat(c.scale * s.pw[reverse ? 32 * jb - row : row - 32 * jb - 31]);
                        const ulonglong2* const in = reinterpret_cast<const ulonglong2*>(s.in_block);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const ulonglong2 w = in[j];
                            const uint64_t e0 = f32x2_mul(f32x2_mul(f32x2_of(v[4 * j], v[4 * j + 1]), f), w.x);
                            const uint64_t e1 = f32x2_mul(f32x2_mul(f32x2_of(v[4 * j + 2], v[4 * j + 3]), f), w.y);
                            v[4 * j] = (uint32_t)e0;
                            v[4 * j + 1] = (uint32_t)(e0 >> 32);
                            v[4 * j + 2] = (uint32_t)e1;
                            v[4 * j + 3] = (uint32_t)(e1 >> 32);
                        }
                    } else {
                        const float* const w = s.pw + kC + 4 + (reverse ? -lane : lane);   // (masked ones lie in front)
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float e = w[reverse ? j : -j] * __uint_as_float(v[j]);
                            v[j] = (reverse ? j >= lane : j <= lane) ? __float_as_uint(e) : 0u;
                        }
                    }
                    if (reverse && 32 * jb + 32 > n) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (32 * jb + j >= n) v[j] = 0;
                    }
                }
                // for each 16 tokens eight columns, and eight of what these leave
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t o[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        o[j] = f32x2_to_bf16x2(f32x2_of(v[16 * u + 2 * j], v[16 * u + 2 * j + 1]));
                    tmem_st8(at + 32 * jb + 16 * u, o);
                    if (two) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            o[j] = f32x2_to_bf16x2(f32x2_fma(pair_of(o[j]), f32x2_splat(-1.f),
                                                             f32x2_of(v[16 * u + 2 * j], v[16 * u + 2 * j + 1])));
                        tmem_st8(at + 32 * jb + 16 * u + 8, o);
                    }
                }
            }
            tmem_st_wait();
            tc_fence_before();
            arrive_w(&s.p_full[b]);
        }
    } else if (warp >= 12 && warp < 20) {
        // ---- weighted y, the state as an operand, nothing in rows behind a chunk's end
        const int part = (warp - 12) >> 2;                         // this thread's 32 channels of every 64
        const uint32_t place = sw128_chunk(row, 4 * part);         // of their first 16 bytes; the j-th: place ^ 16 j
        const bool rows = D == 128 || q < 2;                       // tensor memory lanes that are rows of the state
        if (enter && rows) {
#pragma unroll 1
            for (int k = 0; k < F::blocks; ++k) {
                const int col = 64 * k + 32 * part;
                uint32_t v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    float f = 0.f;
                    if (row < p.ds && col + j < p.dz)
                        f = enter[p.transposed ? (int64_t)(col + j) * p.ds + row : (int64_t)row * p.dz + col + j];
                    v[j] = __float_as_uint(f);
                }
                tmem_st32(lanes + F::state + col, v);
            }
            tmem_st_wait();
        }
        for (int it = 0; it < chunks && ok; ++it) {
            const int st = it % F::stages, sz = it % F::z_stages, n = min(kC, g.end - token(it));
            const uint32_t zpar = (it / F::z_stages) & 1;
            const bool last = it + 1 == chunks, has = it > 0 || enter;
            // the scores have read y (in the last chunk too: conv_full must not get a phase ahead of the scores' warp)
            ok = wait_w(&s.a_full[it % F::scores], (it / F::scores) & 1);
            if (!ok) break;
            if (!last) {
                const uint64_t w = f32x2_splat(row < n ? (reverse ? c.scale * s.pw[row + 1] : s.pw[n - 1 - row]) : 0.f);
#pragma unroll
                for (int k = 0; k < F::blocks; ++k) {
                    uint32_t v[4][4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 in = *reinterpret_cast<const uint4*>(s.y[st][k] + (place ^ (16 * j)));
                        v[j][0] = in.x; v[j][1] = in.y; v[j][2] = in.z; v[j][3] = in.w;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[j][i] = row < n ? f32x2_to_bf16x2(f32x2_mul(pair_of(v[j][i]), w)) : 0u;
                        *reinterpret_cast<uint4*>(s.y[st][k] + (place ^ (16 * j))) =
                            make_uint4(v[j][0], v[j][1], v[j][2], v[j][3]);
                    }
                }
            }
            // the state is there, and the operand that its buffer held has been read
            if (it >= F::states) {
                const int then = it - F::states;
                ok = wait_w(&s.r_full[then & 1], (then >> 1) & 1);
            }
            if (ok && it > 0) ok = wait_w(&s.state_full, (it - 1) & 1);
            if (!ok) break;
            if (n < kC) {
                // nothing from another sequence (z of the chunk before has been there: the state has it; so this is not
                // taken for the one that the barrier's parity last stood for)
                ok = wait_w(&s.z_full[sz], zpar);
                if (!ok) break;
                if (row >= n)
                    for (int k = 0; k < F::blocks; ++k)
                        for (int j = 0; j < 4; ++j)
                            *reinterpret_cast<uint4*>(s.z[sz][k] + (place ^ (16 * j))) = make_uint4(0, 0, 0, 0);
            }
            if (has && rows) {
                tc_fence_after();
                const uint64_t keep = f32x2_splat(s.pw[n]);
#pragma unroll 1
                for (int k = 0; k < F::blocks; ++k) {
                    const uint32_t at = lanes + F::state + 64 * k + 32 * part;
                    uint32_t v[32];
                    tmem_ld32(at, v);
                    tmem_ld_wait();
                    arrived(v);
                    unsigned char* const hi = s.state[it % F::states][0][k];
                    unsigned char* const lo = s.state[it % F::states][1][k];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t oh[4], ol[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t& w0 = v[8 * j + 2 * i];
                            uint32_t& w1 = v[8 * j + 2 * i + 1];
                            uint64_t f = f32x2_of(w0, w1);
                            const uint64_t kept = f32x2_mul(f, keep);
                            w0 = (uint32_t)kept;
                            w1 = (uint32_t)(kept >> 32);
                            oh[i] = split(f);
                            ol[i] = f32x2_to_bf16x2(f);
                        }
                        *reinterpret_cast<uint4*>(hi + (place ^ (16 * j))) = make_uint4(oh[0], oh[1], oh[2], oh[3]);
                        *reinterpret_cast<uint4*>(lo + (place ^ (16 * j))) = make_uint4(ol[0], ol[1], ol[2], ol[3]);
                    }
                    if (!last) tmem_st32(at, v);
                }
                tmem_st_wait();
            }
            fence_async_smem();
            tc_fence_before();
            arrive_w(&s.conv_full[it & 1]);
        }
    } else if (warp >= 20) {
        // ---- outputs: this thread's 32 channels of every 64
        const int part = (warp - 20) >> 2;
        for (int it = 0; it < chunks && ok; ++it) {
            const int t0 = token(it), n = min(kC, g.end - t0);
            const bool has = it > 0 || enter;
            ok = wait_w(&s.r_full[it & 1], (it >> 1) & 1);
            if (!ok) break;
            const uint64_t f = f32x2_splat(reverse ? s.pw[max(n - 1 - row, 0)] : c.scale * s.pw[row + 1]);
            __nv_bfloat16* const to = static_cast<__nv_bfloat16*>(p.out) + ((int64_t)(t0 + row) * c.H + h) * p.dz + 32 * part;
            // what the state adds, while P z runs
            uint64_t held[16];
            auto take = [&](int k) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t r[16], t[16];
                    tmem_ld16(lanes + F::read + 64 * k + 32 * part + 16 * u, r);
                    if (D == 64) tmem_ld16(lanes + F::read + 64 + 32 * part + 16 * u, t);
                    tmem_ld_wait();
                    arrived(r);
                    if (D == 64) arrived(t);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        uint64_t a = f32x2_of(r[2 * j], r[2 * j + 1]);
                        if (D == 64) a = f32x2_add(a, f32x2_of(t[2 * j], t[2 * j + 1]));
                        held[8 * u + j] = f32x2_mul(a, f);
                    }
                }
            };
            if (has) {
                tc_fence_after();
                take(0);
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) held[j] = 0;
            }
            if (D == 64) {
                tc_fence_before();
                arrive_w(&s.r_empty);
            }
            ok = wait_w(&s.o_full, it & 1);
            if (!ok) break;
            tc_fence_after();
            const bool strange = *reinterpret_cast<volatile int*>(&s.strange[it % F::ring]);
#pragma unroll 1
            for (int k = 0; k < F::blocks; ++k) {
                if (k > 0 && has) take(k);
                if (k > 0 && !has) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) held[j] = 0;
                }
                uint32_t o[16];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t v[16];
                    tmem_ld16(lanes + F::out + 64 * k + 32 * part + 16 * u, v);
                    tmem_ld_wait();
                    arrived(v);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        o[8 * u + j] = f32x2_to_bf16x2(f32x2_add(held[8 * u + j], f32x2_of(v[2 * j], v[2 * j + 1])));
                }
                if (strange) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        o[j] = mark_strange(o[j], s.edge[it % F::ring] + 64 * k + 32 * part + 2 * j, row, reverse);
                }
                if (k + 1 == F::blocks) {
                    tc_fence_before();
                    if (D != 64) arrive_w(&s.r_empty);
                    arrive_w(&s.o_empty);
                }
                if (row < n) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int at = 64 * k + 16 * u;
                        if (wide) {
                            const uint32_t (&w)[8] = *reinterpret_cast<const uint32_t (*)[8]>(o + 8 * u);
                            if (at + 32 * part < p.dz) store_32(to + at, w);
                        } else {
                            if (at + 32 * part < p.dz)
                                *reinterpret_cast<uint4*>(to + at) = make_uint4(o[8 * u], o[8 * u + 1], o[8 * u + 2], o[8 * u + 3]);
                            if (at + 32 * part + 8 < p.dz)
                                *reinterpret_cast<uint4*>(to + at + 8) =
                                    make_uint4(o[8 * u + 4], o[8 * u + 5], o[8 * u + 6], o[8 * u + 7]);
                        }
                    }
                }
            }
        }
    }
    if (__syncthreads_or(!ok)) {
        // copies and products on their way end before the block does
        if (threadIdx.x == 0) {
            record_error(c.hdr, LA_DEVERR_WAIT_TIMEOUT);
            for (int i = max(0, xy_loads - F::stages); i < xy_loads; ++i)
                mbar_wait(&s.xy_full[i % F::stages], (i / F::stages) & 1, kDrainNs);
            for (int i = max(0, z_loads - F::z_stages); i < z_loads; ++i)
                mbar_wait(&s.z_full[i % F::z_stages], (i / F::z_stages) & 1, kDrainNs);
        }
        if (warp >= 1 && warp <= 3) {
            mma_commit_w(&s.drain);
            mbar_wait(&s.drain, 0, kDrainNs);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tm, 512);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            return static_cast<EncodeTiledFn>(nullptr);
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}

// [T][H][d] bf16 -> boxes of `rows` tokens x 64 channels of one head, zeros behind the last channel and token.
bool rows_map(CUtensorMap* m, const void* base, const DecayCall& c, int d, int rows = kC) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)c.H, (cuuint64_t)c.T};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)c.H * d * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)rows}, one[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

dim3 grid_of(int H, int n) { return dim3(H, n < 65535 ? n : 65535, (n + 65534) / 65535); }

template <typename K>
cudaError_t opt_in(K kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <int D>
cudaError_t states(const DecayCall& c, const DecayStates& p, DecayWhich which, Chain& chain) {
    CUtensorMap my{}, mz{};
    constexpr int rows = StatesShape<D>::rows;
    if (c.T > 0 && (!rows_map(&my, p.y, c, c.dk, rows) || !rows_map(&mz, p.z, c, c.dv, rows))) return cudaErrorInvalidValue;
    constexpr size_t smem = sizeof(StatesSmem<D>) + 1024;
    static_assert(smem <= 227 * 1024, "shared memory");
    const cudaError_t e = opt_in(decay_tc_states_kernel<D>, smem);
    if (e != cudaSuccess) return e;
    return launch_in(chain, decay_tc_states_kernel<D>, grid_of(c.H, which == kEnds ? c.nseq : c.segments), kStatesThreads,
                     smem, c, p, which, my, mz);
}

template <int D>
cudaError_t pass(const DecayCall& c, const DecayPass& p, Chain& chain) {
    CUtensorMap mx, my, mz;
    if (!rows_map(&mx, p.x, c, p.ds) || !rows_map(&my, p.y, c, p.ds) || !rows_map(&mz, p.z, c, p.dz)) return cudaErrorInvalidValue;
    constexpr size_t smem = sizeof(PassSmem<D>) + 1024;
    static_assert(smem <= 227 * 1024, "shared memory");
    auto kernel = p.reverse ? decay_tc_pass_kernel<D, true> : decay_tc_pass_kernel<D, false>;
    const cudaError_t e = opt_in(kernel, smem);
    if (e != cudaSuccess) return e;
    // 32-byte stores of 16 channels where every row allows them
    const bool wide = p.dz % 16 == 0 && reinterpret_cast<uintptr_t>(p.out) % 32 == 0;
    return launch_in(chain, kernel, grid_of(c.H, c.segments), kPassThreads, smem, c, p, wide, mx, my, mz);
}

}  // namespace

cudaError_t decay_force_wait_timeout(int enable) { return cudaMemcpyToSymbol(g_force_wait_timeout, &enable, sizeof(int)); }

// Sequences of up to 32 tokens on average, a quarter of a chunk, go to the CUDA cores, which have many blocks on an SM: 256
// of 32 x 8 x 64 take 68 us and 86 on the tensor cores, their gradients 176 and 250 (a single one 15 and 11, 14 and 25); 256
// of 64 tokens 132 and 89, and 362 and 259; one of 65536 x 16 x 64 1500 and 190.  Packed batches are judged by their
// average, since the host does not know their lengths.  Where these are mixed, a segment bound's blocks that find
// nothing to do count as much as the products: a prompt of 4096 with 256 single tokens 129 us and 130, gradients 286 and 316;
// 65536 with 4096 of them 1705 and 1701, 4249 and 4418; 2048 with 512 of four tokens 157 and 201, 369 and 531.  Empty sequences
// count as well: 4096 tokens with 256 of them 83 and 68, 165 and 125; 65536 with 4096 941 and 687, 2243 and 1342.
constexpr int64_t kShortest = 32;

bool decay_tc_fits(const DecayCall& c, int dtype) {
    return dtype == LA_BF16 && c.dk <= 128 && c.dv <= 128 && c.dk % 8 == 0 && c.dv % 8 == 0 &&
           c.T > kShortest * c.nseq;
}

cudaError_t decay_tc_states(const DecayCall& c, const DecayStates& p, DecayWhich which, Chain& chain) {
    return c.dk <= 64 && c.dv <= 64 ? states<64>(c, p, which, chain) : states<128>(c, p, which, chain);
}

cudaError_t decay_tc_pass(const DecayCall& c, const DecayPass& p, Chain& chain) {
    return c.dk <= 64 && c.dv <= 64 ? pass<64>(c, p, chain) : pass<128>(c, p, chain);
}

}  // namespace la
