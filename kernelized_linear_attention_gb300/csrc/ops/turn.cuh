// Angles of rotary positions.  A position is an integer, so freq / 2 pi as a 64-bit fixed-point
// fraction of a turn times the position, modulo 2^64, is the angle modulo one
// turn.  The fraction is off by 2^-63 + 2^-106 |freq| turns at most, and the angle
// by |position| times that.  What is left of it beside whole quarters of a turn, pi / 4
// at most, is rounded to 2^-32 turns and to fp32, by pi 2^-27 in all, and goes through
// fp32 cos and sin.
#pragma once

#include "ops.h"

namespace la {

// freq / 2 pi modulo 1 in units of 2^-64, within two of them, or 2^-106 |freq|.  Below 4 a fixed-point product of the
// mantissa and 2^66 / (2 pi) (fp64 is slow here: with it for all, 65536 x 1 x 128 in bf16 took 25 us instead of 23);
// from there on two doubles, what a product rounds away and what the constant does, less their whole turns.
__device__ __forceinline__ unsigned long long turn_fraction(float freq) {
    const uint32_t bits = __float_as_uint(fabsf(freq)), exponent = bits >> 23;
    unsigned long long r;
    if (exponent <= 128) {
        // (numbers below the normal range, which have no leading one, are less than a unit like others above them)
        constexpr unsigned long long kTurn = 0xa2f9836e4e44152aull;
        const unsigned long long mantissa = (bits << 8) | 0x80000000u;
        const unsigned long long product = mantissa * (kTurn >> 32) + (mantissa * (kTurn & 0xffffffffu) >> 32);
        const uint32_t down = 128 - exponent;
        r = down < 64 ? product >> down : 0;
    } else {
        constexpr double kTurn = 0x1.45f306dc9c883p+61, kRest = -0x1.6b01ec5417056p+7;      // 2^64 / (2 pi)
        const double f = fabsf(freq);
        double turns = f * kTurn, rest = fma(f, kRest, fma(f, kTurn, -turns));
        turns = fma(rint(turns * 0x1p-64), -0x1p64, turns);
        rest = fma(rint(rest * 0x1p-64), -0x1p64, rest);
        r = (unsigned long long)__double2ll_rn(turns) + (unsigned long long)__double2ll_rn(rest);
    }
    return freq < 0.f ? 0 - r : r;
}

// What pair j turns by per position: the fraction is the same for all tokens (when all of it was fp64 work, which is slow
// here, 30000 x 3 x 201 with 100 pairs took 60 us with a fraction for every token; 42 now).
struct Turn {
    unsigned long long fraction;
    int axis;
    bool finite;
};
__device__ __forceinline__ Turn turn_of(const Turns& p, int j) {
    int axis = 0;
    while (axis + 1 < p.naxes && j >= p.first[axis + 1]) ++axis;
    const float f = p.freq[j];
    return {turn_fraction(f), axis, (bool)isfinite(f)};
}
// Token t's position on the pair's axis, and (cos, sin) there; sin negated for the inverse.
__device__ __forceinline__ int position_of(const Turns& p, const Turn& turn, int64_t t) {
    return p.positions[t * p.naxes + turn.axis];
}
__device__ __forceinline__ float2 cos_sin_at(const Turns& p, const Turn& turn, long long position) {
    const unsigned long long angle = turn.fraction * (unsigned long long)position;
    // the nearest quarter of a turn apart, so that fp32 rounds what is left: an eighth at most, in units of 2^-32
    const uint32_t turns = (uint32_t)(angle >> 32), quarter = (turns + (1u << 29)) >> 30;
    float s0, c0;
    sincospif((float)(int)(turns - (quarter << 30)) * 0x1p-31f, &s0, &c0);
    float s = __uint_as_float(__float_as_uint(quarter & 1 ? c0 : s0) ^ (quarter & 2) << 30);
    float c = __uint_as_float(__float_as_uint(quarter & 1 ? s0 : c0) ^ (quarter + 1 & 2) << 30);
    if (!turn.finite) s = c = __int_as_float(0x7fc00000);
    return make_float2(c, p.inverse ? -s : s);
}
__device__ __forceinline__ float2 cos_sin(const Turns& p, const Turn& turn, int64_t t) {
    return cos_sin_at(p, turn, position_of(p, turn, t));
}

}  // namespace la
