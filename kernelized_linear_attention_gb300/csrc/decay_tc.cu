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
// a product as two bf16, the rounded value and what it leaves (P, S, w y: off by 2^-18 of the value together), in
// the state sums as three (2^-26): the sums are the states that calls return.  Values keep bf16's range, so nothing is
// scaled or clamped.  Rows of operands lie in shared memory as in tc_ptx.cuh ([rows][64] blocks with the 128-byte
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

template <int D> struct Shape {
    static constexpr int blocks = D / 64;                  // of 64 channels
    static constexpr int threads = D == 64 ? 256 : 512;
    static constexpr int parts = threads / 128;            // column groups of 32 (of D) or 128 / parts (of the scores)
    static constexpr int per_sm = D == 64 ? 2 : 1;
};

// ---------------------------------------------------------------------------
// Pieces
// ---------------------------------------------------------------------------
// A pair of fp32 as bf16 and the rest.
__device__ __forceinline__ uint32_t split(uint64_t& v) {
    const uint32_t h = f32x2_to_bf16x2(v);
    v = f32x2_fma(f32x2_of(h << 16, h & 0xffff0000u), f32x2_splat(-1.f), v);
    return h;
}
__device__ __forceinline__ uint64_t pair_of(uint32_t w) { return f32x2_of(w << 16, w & 0xffff0000u); }

// Powers 0 .. 128 of the decay.
__device__ __forceinline__ void fill_powers(float* pw, const DecayBase& base) {
    for (int i = threadIdx.x; i <= kC; i += blockDim.x) pw[i] = decay_power(base, i);
}

// Whether a value of 32 channels of this thread's row of a tile is not finite; rows from n on are set to zero.
template <int Blocks>
__device__ __forceinline__ bool inspect(unsigned char* tile, int row, int part, int n) {
    unsigned char* const block = tile + (part >> 1) * kTile;
    const int c0 = (part & 1) * 4;
    if (row >= n) {
#pragma unroll
        for (int c = 0; c < 4; ++c) *reinterpret_cast<uint4*>(block + sw128_chunk(row, c0 + c)) = make_uint4(0, 0, 0, 0);
        return false;
    }
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint4 w = *reinterpret_cast<const uint4*>(block + sw128_chunk(row, c0 + c));
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                     __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
    }
    return (top & 0xffffu) >= 0x7f80u || (top >> 16) >= 0x7f80u;
}

// ---------------------------------------------------------------------------
// State sums of a segment
// ---------------------------------------------------------------------------
template <int D> struct __align__(1024) StatesSmem {
    unsigned char yw[3][Shape<D>::blocks][kTile];          // weighted y in three parts
    unsigned char y[Shape<D>::blocks][kTile], z[2][Shape<D>::blocks][kTile];
    float pw[kC + 4];
    uint64_t full_y, full_z[2], mma, drain, never;
    uint32_t tmem;
};

template <int D>
__global__ void __launch_bounds__(Shape<D>::threads, Shape<D>::per_sm)
    decay_tc_states_kernel(const __grid_constant__ DecayCall c, const __grid_constant__ DecayStates p, bool final,
                           const __grid_constant__ CUtensorMap my, const __grid_constant__ CUtensorMap mz) {
    using F = Shape<D>;
    extern __shared__ __align__(1024) unsigned char raw[];
    StatesSmem<D>& s = *reinterpret_cast<StatesSmem<D>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const int h = blockIdx.x, index = blockIdx.y + 65535 * blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, part = warp >> 2, row = 32 * q + lane;
    DecaySegment g;
    if (index >= (final ? c.nseq : c.segments)) return;
    if (decay_malformed(c)) return;
    const int64_t size = (int64_t)c.dk * c.dv;
    float* to;
    const float* enter = nullptr;
    if (final) {
        to = p.edge_out + ((int64_t)index * c.H + h) * size;
        if (!decay_edge_segment(c, index, p.reverse, g)) {
            // an empty sequence: what enters it leaves it
            const float* from = p.edge_in ? p.edge_in + ((int64_t)index * c.H + h) * size : nullptr;
            for (int i = threadIdx.x; i < size; i += F::threads) to[i] = from ? from[i] : 0.f;
            return;
        }
        enter = decay_entering(c, g, h, p.reverse, p.edge_in);
    } else {
        if (!decay_segment(c, index, g) || (p.reverse ? decay_first(g) : decay_last(g))) return;
        to = c.states[p.reverse] + ((int64_t)(decay_slot(g) - (p.reverse ? 1 : 0)) * c.H + h) * size;
    }
    const DecayBase base = decay_base(c.log_decay[h]);
    const int chunks = (g.end - g.start + kC - 1) / kC;
    int y_loads = 0, z_loads = 0;             // of thread 0
    auto load_y = [&]() {
        mbar_arrive_expect_tx(&s.full_y, F::blocks * kTile);
        for (int b = 0; b < F::blocks; ++b) tma_load_3d(s.y[b], &my, 64 * b, h, g.start + y_loads * kC, &s.full_y);
        ++y_loads;
    };
    auto load_z = [&]() {
        uint64_t* const full = &s.full_z[z_loads & 1];
        mbar_arrive_expect_tx(full, F::blocks * kTile);
        for (int b = 0; b < F::blocks; ++b) tma_load_3d(s.z[z_loads & 1][b], &mz, 64 * b, h, g.start + z_loads * kC, full);
        ++z_loads;
    };
    if (threadIdx.x == 0) {
        for (uint64_t* b : {&s.full_y, &s.full_z[0], &s.full_z[1], &s.mma, &s.drain, &s.never}) mbar_init(b, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&s.tmem, 128);
        tmem_relinquish();
    }
    fill_powers(s.pw, base);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s.tmem;
    if (threadIdx.x == 0) {
        load_y();
        load_z();
        if (chunks > 1) load_z();
    }
    bool ok = true;
    if (g_force_wait_timeout) ok = mbar_wait(&s.never, 0, 1000000ull);

    for (int k = 0; k < chunks; ++k) {
        const int st = k & 1, t0 = g.start + k * kC, n = min(kC, g.end - t0);
        ok = ok && mbar_wait(&s.full_y, k & 1);
        if (k > 0) {
            // the products of the chunk before have read the weighted y and their z
            ok = ok && mbar_wait(&s.mma, (k - 1) & 1);
            if (ok && threadIdx.x == 0 && k + 1 < chunks) load_z();
        }
        ok = ok && mbar_wait(&s.full_z[st], (k >> 1) & 1);
        {
            const float far = p.reverse ? c.scale * decay_power(base, t0 - g.start) : decay_power(base, g.end - t0 - n);
            const float w = row < n ? far * s.pw[p.reverse ? row + 1 : n - 1 - row] : 0.f;
            const unsigned char* const from = s.y[part >> 1];
            const int c0 = (part & 1) * 4;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t at = sw128_chunk(row, c0 + j);
                const uint4 v = *reinterpret_cast<const uint4*>(from + at);
                const uint32_t in[4] = {v.x, v.y, v.z, v.w};
                uint32_t o[3][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint64_t f = f32x2_mul(pair_of(row < n ? in[i] : 0u), f32x2_splat(w));
                    o[0][i] = split(f);
                    o[1][i] = split(f);
                    o[2][i] = f32x2_to_bf16x2(f);
                }
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    *reinterpret_cast<uint4*>(s.yw[i][part >> 1] + at) = make_uint4(o[i][0], o[i][1], o[i][2], o[i][3]);
                // nothing from another sequence
                if (row >= n) *reinterpret_cast<uint4*>(s.z[st][part >> 1] + at) = make_uint4(0, 0, 0, 0);
            }
        }
        fence_async_smem();
        if (__syncthreads_or(!ok)) break;
        if (threadIdx.x == 0 && k + 1 < chunks) load_y();
        __syncwarp();
        if (warp == 0) {
            tc_fence_after();
            constexpr uint32_t id = idesc_bf16(128, D, true, true);
            const uint64_t dz = sdesc_sw128(smem_u32(s.z[st]), kTile, 1024);
            // D = 64: the first two parts of y are one product's 128 rows; the third's other rows are not used
#pragma unroll
            for (int i = 0; i < (D == 64 ? 2 : 3); ++i) {
                const uint64_t dy = sdesc_sw128(smem_u32(s.yw[D == 64 ? 2 * i : i]), kTile, 1024);
                const uint32_t acc = tm + (D == 64 ? 64 * i : 0);
#pragma unroll
                for (int j = 0; j < kC / 16; ++j)
                    mma_ss_w(acc, sdesc_add(dy, 2048 * j), sdesc_add(dz, 2048 * j), id,
                             k > 0 || j > 0 || (D != 64 && i > 0) ? 1u : 0u);
            }
            mma_commit_w(&s.mma);
        }
    }
    ok = ok && mbar_wait(&s.mma, (chunks - 1) & 1);
    if (__syncthreads_or(!ok)) {
        // copies and products on their way end before the block does
        if (threadIdx.x == 0) {
            record_error(c.hdr, LA_DEVERR_WAIT_TIMEOUT);
            mbar_wait(&s.full_y, (y_loads - 1) & 1, kDrainNs);
            for (int i = max(0, z_loads - 2); i < z_loads; ++i) mbar_wait(&s.full_z[i & 1], (i >> 1) & 1, kDrainNs);
        }
        __syncwarp();
        if (warp == 0) {
            mma_commit_w(&s.drain);
            mbar_wait(&s.drain, 0, kDrainNs);
        }
    } else {
        tc_fence_after();
        const float keep = decay_power(base, g.end - g.start);
        const int col = 32 * part;
        uint32_t v[32];
        if (D == 64) {
            // rows 64 .. 127 hold the second part of rows 0 .. 63
            float (*ex)[65] = reinterpret_cast<float (*)[65]>(s.yw);
            tmem_ld32(tmem_addr(tm, 32 * q, col), v);
            tmem_ld_wait();
            if (q >= 2) {
#pragma unroll
                for (int j = 0; j < 32; ++j) ex[row - 64][col + j] = __uint_as_float(v[j]);
            }
            __syncthreads();
            if (q < 2) {
                uint32_t lo[32];
                tmem_ld32(tmem_addr(tm, 32 * q, 64 + col), lo);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    v[j] = __float_as_uint(__uint_as_float(v[j]) + (ex[row][col + j] + __uint_as_float(lo[j])));
            }
        } else {
            tmem_ld32(tmem_addr(tm, 32 * q, col), v);
            tmem_ld_wait();
        }
        if (row < c.dk) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                if (col + j >= c.dv) break;
                const int64_t at = (int64_t)row * c.dv + col + j;
                const float f = __uint_as_float(v[j]);
                to[at] = enter ? fmaf(keep, enter[at], f) : f;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tm, 128);
}

// ---------------------------------------------------------------------------
// Products of a segment
// ---------------------------------------------------------------------------
template <int D> struct __align__(1024) PassSmem {
    unsigned char x[Shape<D>::blocks][kTile], y[Shape<D>::blocks][kTile], z[Shape<D>::blocks][kTile];
    unsigned char yw[2][Shape<D>::blocks][kTile];                     // weighted y in two parts; outputs on their way
    // the state [D][64] in blocks, in two parts; D = 64: and the second part's own sums (rows 64 .. 127 of tensor memory)
    unsigned char state[D == 64 ? 3 : 2][Shape<D>::blocks][D * 128];
    float pw[kC + 4];
    __align__(16) float in_block[32];                                 // decay inside a block of 32 tokens
    int edge[D];                                                      // first (last) token whose channel is not finite
    uint64_t full_xy, full_z, mma_a, mma_o, mma_s, mma_f, drain, never;
    uint32_t tmem;
};

// Tensor memory: state, scores (then P: for each 32 tokens 16 columns of the first parts and 16 of the second), outputs.
template <int D> struct PassColumns {
    static constexpr uint32_t state = 0, score = D, out = D + 128, all = D == 64 ? 256 : 512;
};

template <int D>
__global__ void __launch_bounds__(Shape<D>::threads, Shape<D>::per_sm)
    decay_tc_pass_kernel(const __grid_constant__ DecayCall c, const __grid_constant__ DecayPass p,
                         const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap my,
                         const __grid_constant__ CUtensorMap mz) {
    using F = Shape<D>;
    using C = PassColumns<D>;
    extern __shared__ __align__(1024) unsigned char raw[];
    PassSmem<D>& s = *reinterpret_cast<PassSmem<D>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const int h = blockIdx.x, index = blockIdx.y + 65535 * blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, part = warp >> 2, row = 32 * q + lane;
    const int block = part >> 1, c0 = (part & 1) * 4, col = 32 * part;      // this thread's 32 of D channels
    DecaySegment g;
    if (index >= c.segments || !decay_segment(c, index, g)) return;
    const DecayBase base = decay_base(c.log_decay[h]);
    const float* const enter = decay_entering(c, g, h, p.reverse, p.edge);
    const int chunks = (g.end - g.start + kC - 1) / kC;
    const bool reverse = p.reverse;
    auto token = [&](int it) { return g.start + (reverse ? chunks - 1 - it : it) * kC; };
    auto load_xy = [&](int it) {
        mbar_arrive_expect_tx(&s.full_xy, 2 * F::blocks * kTile);
        for (int b = 0; b < F::blocks; ++b) {
            tma_load_3d(s.x[b], &mx, 64 * b, h, token(it), &s.full_xy);
            tma_load_3d(s.y[b], &my, 64 * b, h, token(it), &s.full_xy);
        }
    };
    auto load_z = [&](int it) {
        mbar_arrive_expect_tx(&s.full_z, F::blocks * kTile);
        for (int b = 0; b < F::blocks; ++b) tma_load_3d(s.z[b], &mz, 64 * b, h, token(it), &s.full_z);
    };
    if (threadIdx.x == 0) {
        for (uint64_t* b : {&s.full_xy, &s.full_z, &s.mma_a, &s.mma_o, &s.mma_s, &s.mma_f, &s.drain, &s.never}) mbar_init(b, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&s.tmem, C::all);
        tmem_relinquish();
    }
    fill_powers(s.pw, base);
    if (threadIdx.x < 32) s.in_block[threadIdx.x] = decay_power(base, reverse ? threadIdx.x : 31 - threadIdx.x);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = s.tmem, lanes = tmem_addr(tm, 32 * q, 0);
    int xy_loads = 0, z_loads = 0;            // of thread 0
    if (threadIdx.x == 0) {
        load_xy(0);
        load_z(0);
        xy_loads = z_loads = 1;
    }
    if (enter) {
        // lanes are the state's rows; D = 64: rows 64 .. 127 hold the sums of the weighted y's second part
        uint32_t v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            float f = 0.f;
            if (row < p.ds && col + j < p.dz)
                f = enter[p.transposed ? (int64_t)(col + j) * p.ds + row : (int64_t)row * p.dz + col + j];
            v[j] = __float_as_uint(f);
        }
        tmem_st32(lanes + C::state + col, v);
        tmem_st_wait();
    }
    bool has = enter != nullptr, ok = true;   // whether there is a state
    if (g_force_wait_timeout) ok = mbar_wait(&s.never, 0, 1000000ull);

    for (int it = 0; it < chunks; ++it) {
        const int t0 = token(it), n = min(kC, g.end - t0), par = it & 1;
        const bool last = it + 1 == chunks;
        ok = ok && mbar_wait(&s.full_xy, par);
        const bool go = warp == 0 && __all_sync(0xffffffffu, ok);     // this warp issues the products
        if (go) {
            tc_fence_after();
            constexpr uint32_t id = idesc_bf16(128, 128, false, false);
            const uint64_t dx = sdesc_sw128(smem_u32(s.x), 16, 1024), dy = sdesc_sw128(smem_u32(s.y), 16, 1024);
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                const uint32_t at = (j >> 2) * kTile + 32 * (j & 3);
                mma_ss_w(tm + C::score, sdesc_add(dx, at), sdesc_add(dy, at), id, j > 0 ? 1u : 0u);
            }
            mma_commit_w(&s.mma_a);
        }
        if (has) {
            // the state as an operand, and decayed over this chunk
            if (it > 0) ok = ok && mbar_wait(&s.mma_s, (it - 1) & 1);
            tc_fence_after();
            uint32_t v[32];
            tmem_ld32(lanes + C::state + col, v);
            tmem_ld_wait();
            const bool rest = D == 64 && q >= 2;
            const int a = rest ? row - 64 : row;
            unsigned char* const hi = s.state[rest ? (D == 64 ? 2 : 0) : 0][block];
            unsigned char* const lo = s.state[1][block];
            const uint64_t keep = f32x2_splat(s.pw[n]);
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
                *reinterpret_cast<uint4*>(hi + sw128_chunk(a, c0 + j)) = make_uint4(oh[0], oh[1], oh[2], oh[3]);
                if (!rest) *reinterpret_cast<uint4*>(lo + sw128_chunk(a, c0 + j)) = make_uint4(ol[0], ol[1], ol[2], ol[3]);
            }
            if (!last) {
                tmem_st32(lanes + C::state + col, v);
                tmem_st_wait();
            }
        }
        if (!last) {
            const float w = row < n ? (reverse ? c.scale * s.pw[row + 1] : s.pw[n - 1 - row]) : 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t at = sw128_chunk(row, c0 + j);
                const uint4 v = *reinterpret_cast<const uint4*>(s.y[block] + at);
                const uint32_t in[4] = {v.x, v.y, v.z, v.w};
                uint32_t oh[4], ol[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint64_t f = f32x2_mul(pair_of(row < n ? in[i] : 0u), f32x2_splat(w));
                    oh[i] = split(f);
                    ol[i] = f32x2_to_bf16x2(f);
                }
                *reinterpret_cast<uint4*>(s.yw[0][block] + at) = make_uint4(oh[0], oh[1], oh[2], oh[3]);
                *reinterpret_cast<uint4*>(s.yw[1][block] + at) = make_uint4(ol[0], ol[1], ol[2], ol[3]);
            }
        }
        ok = ok && mbar_wait(&s.full_z, par);
        const bool found = inspect<F::blocks>(s.z[0], row, part, n);
        fence_async_smem();
        tc_fence_before();
        const bool strange = __syncthreads_or(found);
        if (go) {
            tc_fence_after();
            if (has) {
                constexpr uint32_t id = idesc_bf16(128, D, false, true);
                const uint64_t dx = sdesc_sw128(smem_u32(s.x), 16, 1024);
#pragma unroll
                for (int i = 0; i < (D == 64 ? 3 : 2); ++i) {
                    const uint64_t dst = sdesc_sw128(smem_u32(s.state[i]), D * 128, 1024);
#pragma unroll
                    for (int j = 0; j < D / 16; ++j)
                        mma_ss_w(tm + C::out, sdesc_add(dx, (j >> 2) * kTile + 32 * (j & 3)), sdesc_add(dst, 2048 * j), id,
                                 i > 0 || j > 0 ? 1u : 0u);
                }
            }
            mma_commit_w(&s.mma_o);
            if (!last) {
                constexpr uint32_t id = idesc_bf16(128, D, true, true);
                const uint64_t dz = sdesc_sw128(smem_u32(s.z), kTile, 1024);
#pragma unroll
                for (int i = 0; i < (D == 64 ? 1 : 2); ++i) {
                    const uint64_t dy = sdesc_sw128(smem_u32(s.yw[i]), kTile, 1024);
#pragma unroll
                    for (int j = 0; j < kC / 16; ++j)
                        mma_ss_w(tm + C::state, sdesc_add(dy, 2048 * j), sdesc_add(dz, 2048 * j), id,
                                 has || i > 0 || j > 0 ? 1u : 0u);
                }
                mma_commit_w(&s.mma_s);
            }
        }
        ok = ok && mbar_wait(&s.mma_a, par);
        tc_fence_after();
        // scores to P, 32 tokens at a time
#pragma unroll
        for (int b = 0; b < 4 / F::parts; ++b) {
            const int jb = part * (4 / F::parts) + b;
            uint32_t v[32];
            if (reverse ? jb < q : jb > q) {
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = 0;
            } else {
                tmem_ld32(lanes + C::score + 32 * jb, v);
                tmem_ld_wait();
                if (jb != q) {
                    // decay to the block's nearest token, times that inside the block
                    const uint64_t f = f32x2_splat(c.scale * s.pw[reverse ? 32 * jb - row : row - 32 * jb - 31]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float4 w = *reinterpret_cast<const float4*>(s.in_block + 4 * j);
                        const uint64_t a = f32x2_mul(f32x2_mul(f32x2_of(v[4 * j], v[4 * j + 1]), f),
                                                     f32x2_of(__float_as_uint(w.x), __float_as_uint(w.y)));
                        const uint64_t d = f32x2_mul(f32x2_mul(f32x2_of(v[4 * j + 2], v[4 * j + 3]), f),
                                                     f32x2_of(__float_as_uint(w.z), __float_as_uint(w.w)));
                        v[4 * j] = (uint32_t)a;
                        v[4 * j + 1] = (uint32_t)(a >> 32);
                        v[4 * j + 2] = (uint32_t)d;
                        v[4 * j + 3] = (uint32_t)(d >> 32);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const int apart = reverse ? j - lane : lane - j;
                        v[j] = apart >= 0 ? __float_as_uint(c.scale * s.pw[max(apart, 0)] * __uint_as_float(v[j])) : 0u;
                    }
                }
                if (reverse && 32 * jb + 32 > n) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (32 * jb + j >= n) v[j] = 0;
                }
                uint32_t o[32];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    uint64_t f = f32x2_of(v[2 * j], v[2 * j + 1]);
                    o[j] = split(f);
                    o[16 + j] = f32x2_to_bf16x2(f);
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = o[j];
            }
            tmem_st32(lanes + C::score + 32 * jb, v);
        }
        ok = ok && mbar_wait(&s.mma_o, par);
        if (has) {
            tc_fence_after();
            uint32_t v[32];
            tmem_ld32(lanes + C::out + col, v);
            tmem_ld_wait();
            const float f = reverse ? s.pw[max(n - 1 - row, 0)] : c.scale * s.pw[row + 1];
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(f * __uint_as_float(v[j]));
            tmem_st32(lanes + C::out + col, v);
        }
        if (threadIdx.x == 0 && ok && !last) {
            load_xy(it + 1);                  // the scores and x S are done, and every thread is past its y
            ++xy_loads;
        }
        __syncwarp();
        if (strange) {
            // the state has taken them (this wait is every thread's); now nothing else may meet them
            if (!last) ok = ok && mbar_wait(&s.mma_s, par);
            for (int i = threadIdx.x; i < D; i += F::threads) s.edge[i] = reverse ? -1 : kC;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint16_t* at = reinterpret_cast<uint16_t*>(s.z[block] + sw128_chunk(row, c0 + j));
                for (int i = 0; i < 8; ++i) {
                    if ((at[i] & 0x7f80u) != 0x7f80u) continue;
                    at[i] = 0;
                    if (reverse) atomicMax(&s.edge[col + 8 * j + i], row);
                    else atomicMin(&s.edge[col + 8 * j + i], row);
                }
            }
            fence_async_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        if (__syncthreads_or(!ok)) break;
        __syncwarp();
        if (warp == 0) {
            tc_fence_after();
            constexpr uint32_t id = idesc_bf16(128, D, false, true);
            const uint64_t dz = sdesc_sw128(smem_u32(s.z), kTile, 1024);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < kC / 16; ++j)
                    mma_ts_w(tm + C::out, tm + C::score + 32 * (j >> 1) + 16 * i + 8 * (j & 1), sdesc_add(dz, 2048 * j), id,
                             has || i > 0 || j > 0 ? 1u : 0u);
            mma_commit_w(&s.mma_f);
        }
        has = true;
        ok = ok && mbar_wait(&s.mma_f, par);
        tc_fence_after();
        if (threadIdx.x == 0 && ok && !last) {
            load_z(it + 1);
            ++z_loads;
        }
        __syncwarp();
        uint32_t v[32];
        tmem_ld32(lanes + C::out + col, v);
        tmem_ld_wait();
        if (strange) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (reverse ? row <= s.edge[col + j] : row >= s.edge[col + j]) v[j] = 0x7fc00000u;
        }
        // a warp's 32 rows of 32 channels by way of shared memory (where it alone puts its weighted y), 64 bytes a row
        unsigned char* const stage = s.yw[0][block];
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = pack_bf16x2(__uint_as_float(v[8 * j + 2 * i]), __uint_as_float(v[8 * j + 2 * i + 1]));
            *reinterpret_cast<uint4*>(stage + sw128_chunk(row, c0 + j)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = 32 * q + 8 * j + (lane >> 2), at = col + 8 * (lane & 3);
            const uint4 o = *reinterpret_cast<const uint4*>(stage + sw128_chunk(r, c0 + (lane & 3)));
            if (r < n && at < p.dz && ok)
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + ((int64_t)(t0 + r) * c.H + h) * p.dz + at) = o;
        }
        __syncwarp();
    }
    if (__syncthreads_or(!ok)) {
        // copies and products on their way end before the block does
        if (threadIdx.x == 0) {
            record_error(c.hdr, LA_DEVERR_WAIT_TIMEOUT);
            if (xy_loads) mbar_wait(&s.full_xy, (xy_loads - 1) & 1, kDrainNs);
            if (z_loads) mbar_wait(&s.full_z, (z_loads - 1) & 1, kDrainNs);
        }
        __syncwarp();
        if (warp == 0) {
            mma_commit_w(&s.drain);
            mbar_wait(&s.drain, 0, kDrainNs);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tm, C::all);
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

// [T][H][d] bf16 -> boxes of 128 tokens x 64 channels of one head, zeros behind the last channel and token.
bool rows_map(CUtensorMap* m, const void* base, const DecayCall& c, int d) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)c.H, (cuuint64_t)c.T};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)c.H * d * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)kC}, one[3] = {1, 1, 1};
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
cudaError_t states(const DecayCall& c, const DecayStates& p, bool final, cudaStream_t s) {
    CUtensorMap my{}, mz{};
    if (c.T > 0 && (!rows_map(&my, p.y, c, c.dk) || !rows_map(&mz, p.z, c, c.dv))) return cudaErrorInvalidValue;
    constexpr size_t smem = sizeof(StatesSmem<D>) + 1024;
    const cudaError_t e = opt_in(decay_tc_states_kernel<D>, smem);
    if (e != cudaSuccess) return e;
    decay_tc_states_kernel<D><<<grid_of(c.H, final ? c.nseq : c.segments), Shape<D>::threads, smem, s>>>(c, p, final, my, mz);
    return cudaGetLastError();
}

template <int D>
cudaError_t pass(const DecayCall& c, const DecayPass& p, cudaStream_t s) {
    CUtensorMap mx, my, mz;
    if (!rows_map(&mx, p.x, c, p.ds) || !rows_map(&my, p.y, c, p.ds) || !rows_map(&mz, p.z, c, p.dz)) return cudaErrorInvalidValue;
    constexpr size_t smem = sizeof(PassSmem<D>) + 1024;
    static_assert(smem <= 227 * 1024, "shared memory");
    const cudaError_t e = opt_in(decay_tc_pass_kernel<D>, smem);
    if (e != cudaSuccess) return e;
    decay_tc_pass_kernel<D><<<grid_of(c.H, c.segments), Shape<D>::threads, smem, s>>>(c, p, mx, my, mz);
    return cudaGetLastError();
}

}  // namespace

cudaError_t decay_force_wait_timeout(int enable) { return cudaMemcpyToSymbol(g_force_wait_timeout, &enable, sizeof(int)); }

bool decay_tc_fits(const DecayCall& c, int dtype) {
    return dtype == LA_BF16 && c.dk <= 128 && c.dv <= 128 && c.dk % 8 == 0 && c.dv % 8 == 0;
}

cudaError_t decay_tc_states(const DecayCall& c, const DecayStates& p, bool final, cudaStream_t s) {
    return c.dk <= 64 && c.dv <= 64 ? states<64>(c, p, final, s) : states<128>(c, p, final, s);
}

cudaError_t decay_tc_pass(const DecayCall& c, const DecayPass& p, cudaStream_t s) {
    return c.dk <= 64 && c.dv <= 64 ? pass<64>(c, p, s) : pass<128>(c, p, s);
}

}  // namespace la
