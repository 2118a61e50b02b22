// tk_select.h -- device pieces shared by the top-k gating (tk_topk.hip) and the
// routing (tk_route.hip): order-preserving keys of scores, the two best scores
// of a group of lanes, group ranks within 16-lane rows, and a lane's sort of
// eight scores.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace tk_select {

__device__ __forceinline__ uint32_t fbits(float f) { return __builtin_bit_cast(uint32_t, f); }
__device__ __forceinline__ float ffrom(uint32_t u) { return __builtin_bit_cast(float, u); }

// Order-preserving map of a (non-NaN) float to uint32; -0 and +0 map alike.
// Every non-NaN value maps above 0, which therefore marks "no candidate".
__device__ __forceinline__ uint32_t ordered(float f)
{
    const uint32_t b = fbits(f + 0.0f); // -0 + +0 = +0
    // negative: all bits flipped; otherwise only the sign bit set
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// The value of a key (a zero comes back as +0).
__device__ __forceinline__ float unordered(uint32_t h)
{
    return ffrom((h & 0x80000000u) ? (h & 0x7FFFFFFFu) : ~h);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t v)
{
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}

// +inf or -inf in a scalar register whose value the compiler does not see:
// a median against it stays one v_med3_f32 (against a known infinity the
// compiler turns it into an IEEE max or min, which first quiets each loaded
// operand with an instruction of its own)
__device__ __forceinline__ float opaque_inf(bool negative)
{
    uint32_t b;
    if (negative)
        asm volatile("s_mov_b32 %0, 0xff800000" : "=s"(b));
    else
        asm volatile("s_mov_b32 %0, 0x7f800000" : "=s"(b));
    return ffrom(b);
}

// max / min of two non-NaN floats, as a median against an infinity
__device__ __forceinline__ float fmax2(float a, float b, float pinf) { return __builtin_amdgcn_fmed3f(a, b, pinf); }
__device__ __forceinline__ float fmin2(float a, float b, float ninf) { return __builtin_amdgcn_fmed3f(a, b, ninf); }

// (a1, a2) <- the two largest of (a1, a2) and the pair CTRL brings from
// another lane, each pair ordered: the second is the median of the two
// firsts and the larger second
template <int CTRL>
__device__ __forceinline__ void merge_top2f(float& a1, float& a2, float pinf)
{
    const float b1 = ffrom((uint32_t)__builtin_amdgcn_update_dpp(0, (int)fbits(a1), CTRL, 0xF, 0xF, false));
    const float b2 = ffrom((uint32_t)__builtin_amdgcn_update_dpp(0, (int)fbits(a2), CTRL, 0xF, 0xF, false));
    a2 = __builtin_amdgcn_fmed3f(a1, b1, fmax2(a2, b2, pinf));
    a1 = fmax2(a1, b1, pinf);
}

// A lane's 8 raw scores (float bits, none NaN) sorted best first by (score,
// smaller slot), as sort_lane<8> sorts their keys, on 64-bit doubles: the
// high word is the score's own bits (-0 made +0), the low word the tie-break,
// 7 - slot for a non-negative score and slot for a negative one (a double's
// order runs backwards with its sign).  No NaN score makes a NaN or infinite
// double (that needs the top three mantissa bits set under an all-ones
// exponent), fp64 denormals are kept, and every word of a lane differs, so the
// 19 comparators are a max and a min each (v_max_f64 / v_min_f64, written out
// so that the compiler adds no canonicalising operation): 38 instructions
// instead of a 64-bit compare and four selects per comparator.  Returns the
// order-preserving keys and idx[j] = 7 - slot of entry j, as sort_lane does.
__device__ __forceinline__ double dmax(double a, double b)
{
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ double dmin(double a, double b)
{
    double r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ void sort_lane_raw8(uint32_t (&key)[8], uint32_t (&idx)[8])
{
    double x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t h = fbits(ffrom(key[j]) + 0.0f); // -0 + +0 = +0
        const uint32_t l = (uint32_t)(7 - j) ^ ((uint32_t)((int32_t)h >> 31) & 7u);
        x[j] = __builtin_bit_cast(double, ((uint64_t)h << 32) | l);
    }
    constexpr int net[19][2] = {{0, 2}, {1, 3}, {4, 6}, {5, 7}, {0, 4}, {1, 5}, {2, 6}, {3, 7}, {0, 1}, {2, 3},
                                {4, 5}, {6, 7}, {2, 4}, {3, 5}, {1, 4}, {3, 6}, {1, 2}, {3, 4}, {5, 6}};
#pragma unroll
    for (int c = 0; c < 19; ++c) {
        const double a = x[net[c][0]], b = x[net[c][1]];
        x[net[c][0]] = dmax(a, b);
        x[net[c][1]] = dmin(a, b);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint64_t u = __builtin_bit_cast(uint64_t, x[j]);
        const uint32_t h = (uint32_t)(u >> 32);
        const uint32_t s = (uint32_t)((int32_t)h >> 31);
        key[j] = h ^ (s | 0x80000000u);
        idx[j] = (uint32_t)u ^ (s & 7u);
    }
}

// The same for four scores: idx[j] = 7 - slot of entry j.
__device__ __forceinline__ void sort_lane_raw4(uint32_t (&key)[4], uint32_t (&idx)[4])
{
    double x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t h = fbits(ffrom(key[j]) + 0.0f); // -0 + +0 = +0
        const uint32_t l = (uint32_t)(7 - j) ^ ((uint32_t)((int32_t)h >> 31) & 7u);
        x[j] = __builtin_bit_cast(double, ((uint64_t)h << 32) | l);
    }
    constexpr int net[5][2] = {{0, 2}, {1, 3}, {0, 1}, {2, 3}, {1, 2}};
#pragma unroll
    for (int c = 0; c < 5; ++c) {
        const double a = x[net[c][0]], b = x[net[c][1]];
        x[net[c][0]] = dmax(a, b);
        x[net[c][1]] = dmin(a, b);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint64_t u = __builtin_bit_cast(uint64_t, x[j]);
        const uint32_t h = (uint32_t)(u >> 32);
        const uint32_t s = (uint32_t)((int32_t)h >> 31);
        key[j] = h ^ (s | 0x80000000u);
        idx[j] = (uint32_t)u ^ (s & 7u);
    }
}

// Group ranks within 16-lane rows (one token per row, 16 >> GL groups of
// 2^GL lanes): group H's sum, as an order-preserving key, reaches every lane
// of the row by row_newbcast from the group's first lane, and a lane counts
// the groups that beat its own ("a beats b": larger sum, or equal sums and the
// smaller group index): a group below its own by a key at least its own
// (above gkey_less = gkey - 1), one above it by a larger key.
template <int GL, int H = 0>
__device__ __forceinline__ void row_group_rank(uint32_t gkey, uint32_t gkey_less, uint32_t& rank)
{
    if constexpr ((H << GL) < 16) {
        const uint32_t gh = (uint32_t)__builtin_amdgcn_mov_dpp((int)gkey, 0x150 + (H << GL), 0xF, 0xF, false);
        // the lanes of groups above H, whose equal sums lose to group H (a
        // constant lane mask), count group H when its key is at least theirs
        constexpr uint64_t kAbove = (uint64_t)(0xFFFFu & ~((1u << ((H + 1) << GL)) - 1u)) * 0x0001000100010001ull;
        const uint32_t thr = __builtin_amdgcn_inverse_ballot_w64(kAbove) ? gkey_less : gkey;
        rank += gh > thr ? 1u : 0u;
        row_group_rank<GL, H + 1>(gkey, gkey_less, rank);
    }
}

} // namespace tk_select
