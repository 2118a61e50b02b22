// tk_swiglu.h -- device pieces shared by the fused SwiGLU + cast kernels
// (tk_swiglu_cast.hip) and the one that also leaves a checkpoint
// (tk_checkpoint.hip): the sigmoid by table and the activation of a step.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "tk.h"
#include "tk_quant.h"

namespace tk_detail {

// The current device's sigmoid table (set up on the first call) and CU count.
tk_status sigma_table(const float2*& table, int& cus);

// Sigmoid table: magnitudes m of bf16 bit patterns in [kLutFirst, kLutFirst+kLutSize),
// one (sigma(+g), sigma(-g)) pair per magnitude.  Below 2^-25 sigma rounds to
// 0.5 and at 127.5 and beyond it rounds to 1 (positive) or 0 (negative) in fp32,
// so clamping the magnitude into the table range is exact.
constexpr uint32_t kLutFirst = 0x3300u; // bf16 2^-25
constexpr uint32_t kLutLast = 0x42FFu;  // bf16 127.5
constexpr int kLutSize = 4096;
static_assert(kLutLast - kLutFirst + 1 == kLutSize, "table span");


// ---------------------------------------------------------------------------
// Correctly rounded fp32 sigmoid for table set-up and for the clamp limit.
// |g| < 2^-12: Taylor series 1/2 + g/4 - g^3/48 + g^5/480 (next term below
//   2^-96), summed as a double-double with Knuth's TwoSum; the double-double
//   is rounded to fp32 once, the low word deciding exact fp64 midpoints.
// otherwise: 1/(1+exp(-g)) in fp64.  Its error (a few fp64 ulps) is far below
//   the distance of any bf16 gate's sigmoid from an fp32 rounding midpoint
//   (at least 5.8e-5 fp32 ulps for |g| >= 2^-12); for other fp32 inputs it is
//   correct unless sigma lies within ~2^-50 of a midpoint.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void two_sum(double a, double b, double& s, double& e)
{
    s = a + b;
    const double bb = s - a;
    e = (a - (s - bb)) + (b - bb);
}

__device__ inline float round_dd_to_float(double hi, double lo)
{
    const float f = (float)hi;
    const double df = (double)f;
    if (df == hi || lo == 0.0)
        return f;
    const float f2 = nextafterf(f, hi > df ? INFINITY : -INFINITY);
    const double mid = 0.5 * (df + (double)f2); // exact
    if (mid != hi)
        return f; // hi is not a tie, so hi + lo rounds like hi
    // hi sits exactly on the midpoint between f and f2: lo decides.
    return ((lo > 0.0) == (hi > df)) ? f2 : f;
}

__device__ inline float sigmoid_rn(float gf)
{
    const double g = (double)gf;
    if (fabs(g) < 0x1p-12) {
        if (fabs(g) < 0x1p-40)
            return 0.5f; // |g/4| is far below half an ulp of 0.5
        double s, e;
        two_sum(0.5, 0.25 * g, s, e);
        const double g2 = g * g;
        const double c = g * g2 * (-1.0 / 48.0 + g2 * (1.0 / 480.0));
        double hi, lo;
        two_sum(s, e + c, hi, lo);
        return round_dd_to_float(hi, lo);
    }
    return (float)(1.0 / (1.0 + exp(-g)));
}

typedef float2 LutT;

// sigma(g) for a gate whose bf16 bits sit in bits [POS, POS+16) of `word`;
// gbits is the fp32 bit pattern of the same gate (its sign selects the entry).
template <int POS>
__device__ __forceinline__ float lut_sigma(const float2* lut, uint32_t word, uint32_t gbits)
{
    const uint32_t m = __builtin_amdgcn_ubfe(word, POS, 15);                 // |g| as bf16 bits
    const uint32_t c = min(max(m, kLutFirst), kLutLast) - kLutFirst;         // v_med3_u32
    const float2 pr = lut[c];
    return ((int32_t)gbits < 0) ? pr.y : pr.x;
}

// The 16 KiB form of the same lookup (g_sigma_lut16's layout).
template <int POS>
__device__ __forceinline__ float lut16_sigma(const uint32_t* lut, uint32_t word, uint32_t gbits)
{
    const uint32_t m = __builtin_amdgcn_ubfe(word, POS, 15);
    const uint32_t c = min(max(m, kLutFirst), kLutLast) - kLutFirst;
    const uint32_t e = lut[c];
    const float sn = as_float(e & 0x3FFFFFFFu);
    const float sp = as_float(as_uint(1.0f - sn) + (e >> 30) - 1u);
    return ((int32_t)gbits < 0) ? sn : sp;
}

// Clamp counters: a wave's count of gates above the limit.  WaveCount keeps
// the wave's total in scalar registers (a ballot and popcount per element);
// LaneCount keeps one count per lane (a VALU add per element) and sums the
// lanes once at the end.  Row-reduced units use WaveCount; per-block units use
// LaneCount, because there the compiler holds every element's compare mask in
// scalar registers until the step's group reductions are done and spills them
// to VGPR lanes (the per-block clamp launch of 32768 x 2048 took 65 us without
// the counter's atomics against 57 us unclamped; with LaneCount, 59.5 us).
struct WaveCount {
    unsigned long long n = 0;
    __device__ __forceinline__ void add(bool hit) { n += __builtin_popcountll(__ballot(hit)); }
    __device__ __forceinline__ unsigned long long total() const { return n; }
};
struct LaneCount {
    // a lane counts at most 32 gates per unit and ceil(units / waves) units,
    // with units < 2^31 and 8 waves per CU: below 2^32 on any device of more
    // than two CUs
    uint32_t n = 0;
    __device__ __forceinline__ void add(bool hit) { n += hit ? 1u : 0u; }
    // every lane of the wave must call this
    __device__ __forceinline__ unsigned long long total() const
    {
        unsigned long long t = n;
#pragma unroll
        for (int m = kWaveSize / 2; m >= 1; m >>= 1)
            t += __shfl_xor(t, m);
        return t;
    }
};

// One element: gate and up are the bf16 halves at bit POS of `gword` / `uword`.
// a = RN(g * sigma(g)) (or the clamped gate's activation), b = RN(a * u),
// y = RN(b * w); three fp32 products, never fused.  `counts` is false on lanes
// past the end of the row, whose gates must not enter the clamp count.
template <int POS, bool CLAMP, class CNT, bool T16 = false>
__device__ __forceinline__ float swiglu_elem(const LutT* lut, uint32_t gword, uint32_t uword, float w,
                                             float limit, float a_limit, CNT& clamped, bool counts = true)
{
    const uint32_t gbits = POS ? (gword & 0xFFFF0000u) : (gword << 16);
    float u = as_float(POS ? (uword & 0xFFFF0000u) : (uword << 16));
    const float g = as_float(gbits);
    float a = g * (T16 ? lut16_sigma<POS>(reinterpret_cast<const uint32_t*>(lut), gword, gbits)
                       : lut_sigma<POS>(lut, gword, gbits));
    if constexpr (CLAMP) {
        clamped.add(g > limit && counts);
        // The clamped gate's activation, RN(min(g, L) * sigma(min(g, L))), is
        // min(a, a_limit) with a_limit = RN(L * sigma(L)): L > 0, and
        // RN(g * sigma(g)) does not decrease with g > 0 and is <= -0 for g <= -0,
        // so a >= a_limit when g > L and a <= a_limit when g <= L.  The min is
        // taken on the bit patterns as signed integers, which order every
        // negative value (-0 included) below a_limit >= +0: a gate of -0 keeps
        // its -0 even when a_limit rounds to +0 (the smallest L).
        a = __builtin_bit_cast(float, min(__builtin_bit_cast(int32_t, a), __builtin_bit_cast(int32_t, a_limit)));
        u = __builtin_amdgcn_fmed3f(u, -limit, limit);
    }
    const float b = a * u;
    return b * w;
}

// One 8-column step of a loaded unit: ys = w * silu(gate) * up for the lane's
// columns; returns the lane's abs-max bits (0 for a lane past the row end).
template <bool CLAMP, bool PARTIAL, class CNT, bool T16 = false>
__device__ __forceinline__ uint32_t compute_step(const LutT* lut, uint4 g, uint4 u, float w, bool valid, float limit,
                                                 float a_limit, CNT& clamped, float (&ys)[8])
{
    const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
    const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        ys[2 * k] = swiglu_elem<0, CLAMP, CNT, T16>(lut, gw[k], uw[k], w, limit, a_limit, clamped, valid);
        ys[2 * k + 1] = swiglu_elem<16, CLAMP, CNT, T16>(lut, gw[k], uw[k], w, limit, a_limit, clamped, valid);
        m = fmaxf(m, fmaxf(fabsf(ys[2 * k]), fabsf(ys[2 * k + 1])));
    }
    if (PARTIAL && !valid)
        m = 0.0f;
    return as_uint(m);
}

} // namespace tk_detail
