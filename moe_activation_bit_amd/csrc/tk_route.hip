// tk_route.hip -- routing of tokens to experts from the router's logits and the
// gradient of its weights, behind tk_route and tk_route_backward in
// include/tk_layer.h.
//
// Scores are computed in 64 bits and rounded once, so that the order of two
// experts is that of their exact scores rounded to fp32 (plus the bias), and
// does not hang on how an fp32 exponential was built.  gfx950 runs fp64
// multiply-adds at the rate of fp32's (4.7 cycles a wave against 4.6), so the 22
// instructions of a sigmoid cost about 3 us at 16384 tokens x 256 experts.
//
// route_row_kernel (k <= 16, up to 16 groups): four tokens per wave, one per
// 16-lane row, a lane holding consecutive experts of a group as lists of eight
// sorted scores; k rounds take the largest list head of each row.  route_kernel takes what is left: one wave
// per token, the largest key searched anew each round.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "tk.h"
#include "tk_layer.h"
#include "tk_select.h"

namespace {

using namespace tk_select;

constexpr int kWave = 64;
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxExperts = 512;
constexpr int kMaxK = 64;
constexpr int64_t kMaxBlocks = 1 << 20; // a launch holds fewer than 2^32 work-items; tokens past the grid loop

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* base, size_t i)
{
    if constexpr (BF16)
        return ffrom((uint32_t)static_cast<const uint16_t*>(base)[i] << 16);
    else
        return static_cast<const float*>(base)[i];
}

__device__ __forceinline__ uint32_t wave_umax(uint32_t v)
{
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1)
        v = max(v, (uint32_t)__shfl_xor((int)v, m));
    return v;
}
__device__ __forceinline__ uint32_t wave_umin(uint32_t v)
{
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1)
        v = min(v, (uint32_t)__shfl_xor((int)v, m));
    return v;
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v)
{
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1)
        v += __shfl_xor(v, m);
    return v;
}

// e^x for a number x, |x| <= 1100, to about 2^-49: 2^n 2^f, n the nearest whole
// number to x log2(e) (taken by adding and subtracting 1.5 * 2^52, whose low
// word then holds n), 2^f by the polynomial that meets it at the 11 Chebyshev
// nodes of [-1/2, 1/2] (relative error 4.5e-16).
__device__ __forceinline__ double exp64(double x)
{
    constexpr double kLog2e = 0x1.71547652b82fep+0, kWhole = 0x1.8p+52;
    const double tn = __builtin_fma(x, kLog2e, kWhole);
    const double f = __builtin_fma(x, kLog2e, -(tn - kWhole));
    double r = 0x1.e60638d3aabfep-28;
    r = __builtin_fma(r, f, 0x1.b675bc9694c29p-24);
    r = __builtin_fma(r, f, 0x1.62bfd47c2b6d0p-20);
    r = __builtin_fma(r, f, 0x1.ffcb5406453b3p-17);
    r = __builtin_fma(r, f, 0x1.430913096ce36p-13);
    r = __builtin_fma(r, f, 0x1.5d87fe9d7a4ffp-10);
    r = __builtin_fma(r, f, 0x1.3b2ab6fba1df9p-7);
    r = __builtin_fma(r, f, 0x1.c6b08d703ce49p-5);
    r = __builtin_fma(r, f, 0x1.ebfbdff82c598p-3);
    r = __builtin_fma(r, f, 0x1.62e42fefa3a19p-1);
    r = __builtin_fma(r, f, 1.0);
    return __builtin_ldexp(r, (int)(uint32_t)__builtin_bit_cast(uint64_t, tn));
}
// ... for a number x <= 0 of any size: below -1100 it gives 0 as there
__device__ __forceinline__ double exp64_neg(double x) { return exp64(__builtin_fmax(x, -1100.0)); }
// ... and NaN gives NaN
__device__ __forceinline__ double exp64_nan(double x) { return exp64(x < -1100.0 ? -1100.0 : x); }

// 1/d for a normal d whose reciprocal is normal: the hardware's estimate and one Newton step
__device__ __forceinline__ double reciprocal64(double d)
{
    const double r = __builtin_amdgcn_rcp(d);
    return __builtin_fma(r, __builtin_fma(-d, r, 1.0), r);
}

// 1 / (1 + e^-l) of a number l without overflow: with t = e^-|l|, 1 / (1 + t) or t / (1 + t)
__device__ __forceinline__ double sigmoid64(float l)
{
    const double t = exp64_neg(-(double)fabsf(l)), r = reciprocal64(1.0 + t);
    return l >= 0.0f ? r : t * r;
}

// Two sigmoids rounded to fp32, with one reciprocal between them: 1/a = b/(ab).
// Logits past +-340 count as that, whose scores round to 0 and 1 too (e^340
// squared is still a double).
__device__ __forceinline__ void sigmoid_pair(float& l0, float& l1)
{
    const double a = 1.0 + exp64(-(double)__builtin_amdgcn_fmed3f(l0, -340.0f, 340.0f));
    const double b = 1.0 + exp64(-(double)__builtin_amdgcn_fmed3f(l1, -340.0f, 340.0f));
    const double r = reciprocal64(a * b);
    l0 = (float)(r * b);
    l1 = (float)(r * a);
}

struct RouteParams {
    const void* logits;
    const float* bias; // or null
    uint32_t tokens, experts, k, n_group, topk_group;
    uint32_t lane_experts; // route_row_kernel: experts a lane holds
    uint32_t gl_log2;      // ... and lanes a group, as a power of two
    uint32_t group_experts;
    int softmax, normalise;
    double scale;
    int32_t* idx;
    float* weight;
};

// One wave per token, lane l holding experts l, l + 64, ... (C of them).  Each
// of the k rounds takes the largest key over the wave and, among its holders,
// the smallest index.
template <bool BF16, int C>
__device__ __forceinline__ void route_token(const RouteParams& p, uint32_t t, uint32_t lane, float* s_key,
                                            float* s_group)
{
    const size_t row = (size_t)t * p.experts;
    float l[C];
    float top = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const uint32_t e = lane + kWave * j;
        l[j] = e < p.experts ? load_logit<BF16>(p.logits, row + e) : -INFINITY;
        bad |= l[j] != l[j];
        top = fmaxf(top, l[j]);
    }
    double inv_sum = 0.0;
    if (p.softmax) {
        top = unordered(wave_umax(ordered(top)));
        bad |= top == INFINITY;
        if (top == -INFINITY)
            top = 0.0f; // every expert masked: no exponential of inf - inf
        double sum = 0.0;
#pragma unroll
        for (int j = 0; j < C; ++j)
            sum += exp64_neg((double)l[j] - (double)top);
        sum = wave_sum(sum);
        inv_sum = sum > 0.0 ? 1.0 / sum : 0.0;
    }
    auto score = [&](float x) { return p.softmax ? exp64_neg((double)x - (double)top) * inv_sum : sigmoid64(x); };

    uint32_t key[C];
    const bool by_score = p.bias || p.n_group > 1;
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const uint32_t e = lane + kWave * j;
        float c = l[j];
        if (by_score && c > -INFINITY) {
            c = (float)score(c);
            if (p.bias)
                c += e < p.experts ? p.bias[e] : 0.0f;
        }
        bad |= c != c;
        key[j] = c > -INFINITY ? ordered(c) : 0u;
    }
    const bool poisoned = __builtin_amdgcn_ballot_w64(bad) != 0;

    if (p.n_group > 1) {
        const uint32_t per = p.experts / p.n_group;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const uint32_t e = lane + kWave * j;
            if (e < p.experts)
                s_key[e] = key[j] ? unordered(key[j]) : -INFINITY;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        for (uint32_t g = lane; g < p.n_group; g += kWave) {
            float a1 = -INFINITY, a2 = -INFINITY;
            for (uint32_t i = 0; i < per; ++i) {
                const float c = s_key[g * per + i];
                a2 = fmaxf(a2, fminf(a1, c));
                a1 = fmaxf(a1, c);
            }
            float v = a1 + (a2 > -INFINITY ? a2 : 0.0f);
            s_group[g] = v != v ? -INFINITY : v;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const uint32_t e = lane + kWave * j;
            if (e < p.experts) {
                const uint32_t g = e / per;
                const float mine = s_group[g];
                uint32_t rank = 0;
                for (uint32_t h = 0; h < p.n_group; ++h) {
                    const float o = s_group[h];
                    rank += o > mine || (o == mine && h < g) ? 1u : 0u;
                }
                if (rank >= p.topk_group)
                    key[j] = 0u;
            }
        }
    }

    int32_t pick = -1;
    for (uint32_t it = 0; it < p.k; ++it) {
        uint32_t head = key[0];
#pragma unroll
        for (int j = 1; j < C; ++j)
            head = max(head, key[j]);
        const uint32_t best = wave_umax(head);
        if (best == 0u)
            break; // no expert remains (wave-uniform)
        uint32_t e = 0xFFFFFFFFu;
#pragma unroll
        for (int j = C - 1; j >= 0; --j)
            e = key[j] == best ? lane + kWave * j : e;
        e = wave_umin(e);
#pragma unroll
        for (int j = 0; j < C; ++j)
            key[j] = lane + kWave * j == e ? 0u : key[j];
        pick = lane == it ? (int32_t)e : pick;
    }

    if (poisoned)
        pick = (int32_t)min(lane, p.experts - 1u);
    double s = 0.0;
    if (lane < p.k && pick >= 0)
        s = score(load_logit<BF16>(p.logits, row + (uint32_t)pick));
    if (p.normalise) {
        const double sum = wave_sum(s);
        if (sum != 0.0)
            s /= sum;
    }
    if (lane < p.k) {
        p.idx[(size_t)t * p.k + lane] = pick;
        p.weight[(size_t)t * p.k + lane] = poisoned ? ffrom(0x7FC00000u) : (float)(s * p.scale);
    }
}

template <bool BF16, int C>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteParams p)
{
    __shared__ float s_key[kWaves][kMaxExperts];
    __shared__ float s_group[kWaves][kMaxExperts / 2];
    const uint32_t lane = threadIdx.x & (kWave - 1), wv = threadIdx.x / kWave;
    for (uint32_t t = blockIdx.x * kWaves + wv; t < p.tokens; t += gridDim.x * kWaves)
        route_token<BF16, C>(p, t, lane, s_key[wv], s_group[wv]);
}

template <int CTRL>
__device__ __forceinline__ double dpp_add(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, false);
    return v + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// sum / maximum over each row of 16 lanes, or of 8, in every lane of it
template <int LANES = 16>
__device__ __forceinline__ double row_sum(double v)
{
    v = dpp_add<0xB1>(v);  // quad_perm [1,0,3,2]
    v = dpp_add<0x4E>(v);  // quad_perm [2,3,0,1]
    v = dpp_add<0x141>(v); // row_half_mirror
    return LANES == 16 ? dpp_add<0x140>(v) : v; // row_mirror
}
template <int LANES = 16>
__device__ __forceinline__ uint32_t row_umax(uint32_t v)
{
    v = dpp_umax<0xB1>(v);
    v = dpp_umax<0x4E>(v);
    v = dpp_umax<0x141>(v);
    return LANES == 16 ? dpp_umax<0x140>(v) : v;
}

// N consecutive logits as fp32.
template <bool BF16, int N>
__device__ __forceinline__ void load_logits(const void* base, size_t i, float* x)
{
    if constexpr (BF16) {
        static_assert(N % 2 == 0, "whole words");
        struct __attribute__((packed, aligned(2))) Words {
            uint32_t w[N / 2];
        };
        const Words v = *reinterpret_cast<const Words*>(static_cast<const uint16_t*>(base) + i);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            x[2 * j] = ffrom(v.w[j] << 16);
            x[2 * j + 1] = ffrom(v.w[j] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            x[j] = static_cast<const float*>(base)[i + j];
    }
}

constexpr uint32_t kMasked = 0x007FFFFFu; // ordered(-inf): the key of a masked or absent expert

// Four tokens per wave: lane q of row r holds experts q * C .. + C - 1 of token
// t0 + r (FC > 0: experts == 16 * C, groups of whole lanes) or, with C =
// p.lane_experts, up to C of group q >> p.gl_log2, in L lists of N (slots past
// the last expert hold -inf, as masked experts do; so does a group past the
// last, whose index is then the larger one).  The keys
// order as the gating's do: score, then the smaller index.
// RL = 8: eight tokens per wave in the same way, a row of 8 lanes each.
// MOVE (FC = 16, kept groups within 8 lanes): once the groups are ranked, each
// kept lane's halves go to two lanes of the row, in order, so that every lane
// sorts one list.
// Bound by its fp64 and selection arithmetic: 926 vector instructions a wave at
// 256 experts in 8 groups, top-8, some 7.4 us of the 9.7 to 10.9 us that 16384
// tokens take (1379 and 15.7 us before MOVE, the paired reciprocals and the masks
// looked for at once).
template <bool BF16, int L, int FC, bool K8, bool MOVE, int RL>
__global__ __launch_bounds__(kThreads, L <= 2 && FC > 0 ? 4 : 2) void route_row_kernel(RouteParams p)
{
    constexpr int N = FC == 4 ? 4 : 8;
    constexpr int M = N * L;
    constexpr int S = MOVE ? 1 : L; // lists to sort
    constexpr bool FULL = FC > 0;
    static_assert(!MOVE || (FC == 16 && L == 2), "two halves of eight");
    static_assert(RL == 16 || (FULL && !MOVE), "groups and other counts in rows of 16 lanes");
    constexpr uint32_t TW = kWave / RL; // tokens of a wave
    __shared__ uint2 s_pick[kWaves][kWave];                             // [row * 16 + round]: (expert, key)
    __shared__ float s_in[FULL ? 1 : kWaves][FULL ? 1 : 4][FULL ? 1 : 16 * M]; // the rows, to be read in lane order
    __shared__ uint4 s_move[MOVE ? kWaves : 1][2][MOVE ? kWave : 1];
    __shared__ uint32_t s_src[MOVE ? kWaves : 1][MOVE ? kWave : 1];
    const uint32_t lane = threadIdx.x & (kWave - 1), wv = threadIdx.x / kWave;
    const uint32_t q = lane & (RL - 1u), row = lane / RL;
    const uint32_t C = FULL ? (uint32_t)FC : p.lane_experts;
    // the lane's first expert, and how many it has
    uint32_t from = q * C, own = C;
    if constexpr (!FULL) {
        const uint32_t g = q >> p.gl_log2, sub = (q & ((1u << p.gl_log2) - 1u)) * C, per = p.group_experts;
        from = g * per + sub;
        own = g < p.n_group && sub < per ? min(C, per - sub) : 0u;
    }
    const bool by_score = p.bias || p.n_group > 1;
    const uint32_t first = TW * __builtin_amdgcn_readfirstlane(blockIdx.x * kWaves + wv);

    for (uint32_t t0 = first; t0 < p.tokens; t0 += gridDim.x * (TW * kWaves)) {
        // a wave past the last token repeats it in its other rows and stores nothing from them
        const uint32_t t = t0 + row;
        const size_t at = (size_t)min(t, p.tokens - 1u) * p.experts;
        float x[M];
        if constexpr (FULL) {
            load_logits<BF16, FULL ? FC : 2>(p.logits, at + q * FC, x);
#pragma unroll
            for (int j = FC; j < M; ++j)
                x[j] = -INFINITY;
        } else {
            for (uint32_t e = q; e < p.experts; e += 16u)
                s_in[wv][row][e] = load_logit<BF16>(p.logits, at + e);
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
            for (int j = 0; j < M; ++j) {
                x[j] = (uint32_t)j < own ? s_in[wv][row][min(from + j, 16u * M - 1u)] : -INFINITY;
            }
        }

        // ---- keys: the logits, or the scores (and the bias) with the masked at -inf
        auto held = [&](int j) { return FULL ? j < FC : (uint32_t)j < C; };
        bool bad = false;
#pragma unroll
        for (int j = 0; j < M; j += 2)
            bad |= __builtin_isunordered(x[j], x[j + 1]);
        double top = 0.0, inv_sum = 1.0; // softmax: the row's largest logit, and one over the sum
        if (p.softmax) {
            float m = -INFINITY;
#pragma unroll
            for (int j = 0; j < M; ++j)
                m = fmaxf(m, x[j]);
            m = unordered(row_umax<RL>(ordered(m)));
            bad |= m == INFINITY;
            top = m == -INFINITY ? 0.0 : (double)m; // every expert masked: no inf - inf
        }
        auto shifted = [&](float l) { return exp64_neg((double)l - top); };
        if (by_score) {
            uint32_t masked = 0; // looked for at once: most waves have none
            float least = x[0];
#pragma unroll
            for (int j = 1; j < M; ++j)
                least = held(j) ? fminf(least, x[j]) : least;
            if (__builtin_amdgcn_ballot_w64(least == -INFINITY) != 0) {
#pragma unroll
                for (int j = 0; j < M; ++j)
                    masked |= x[j] == -INFINITY ? 1u << j : 0u;
            }
            if (p.softmax) {
                double e[M], sum = 0.0;
#pragma unroll
                for (int j = 0; j < M; ++j) {
                    e[j] = 0.0;
                    if (held(j)) {
                        e[j] = shifted(x[j]);
                        sum += e[j];
                    }
                }
                sum = row_sum<RL>(sum);
                inv_sum = sum > 0.0 ? reciprocal64(sum) : 0.0; // at least 1
#pragma unroll
                for (int j = 0; j < M; ++j)
                    x[j] = held(j) ? (float)(e[j] * inv_sum) : x[j];
            } else {
#pragma unroll
                for (int j = 0; j < M; j += 2) {
                    if (held(j)) {
                        float s0 = x[j], s1 = x[j + 1];
                        sigmoid_pair(s0, s1);
                        x[j] = s0;
                        x[j + 1] = held(j + 1) ? s1 : x[j + 1];
                    }
                }
            }
            if (p.bias) {
                float b[M];
#pragma unroll
                for (int j = 0; j < M; ++j)
                    b[j] = held(j) ? p.bias[FULL ? q * FC + j : min(from + j, p.experts - 1u)] : 0.0f;
#pragma unroll
                for (int j = 0; j < M; ++j)
                    x[j] += b[j];
            }
            if (__builtin_amdgcn_ballot_w64(masked != 0) != 0) {
#pragma unroll
                for (int j = 0; j < M; ++j)
                    x[j] = (masked >> j) & 1u ? -INFINITY : x[j];
            }
            if (p.bias) {
#pragma unroll
                for (int j = 0; j < M; j += 2)
                    bad |= __builtin_isunordered(x[j], x[j + 1]);
            }
            if constexpr (!FULL) { // slots past the lane's last expert
#pragma unroll
                for (int j = 0; j < M; ++j)
                    x[j] = (uint32_t)j < own ? x[j] : -INFINITY;
            }
        } else if (p.softmax && !p.normalise) {
            double sum = 0.0;
#pragma unroll
            for (int j = 0; j < M; ++j)
                if (held(j))
                    sum += shifted(x[j]);
            sum = row_sum<RL>(sum);
            inv_sum = sum > 0.0 ? reciprocal64(sum) : 0.0; // at least 1
        }
        const uint64_t bad_lanes = __builtin_amdgcn_ballot_w64(bad);
        const bool poisoned = (uint32_t)(bad_lanes >> (row * RL)) & ((1u << RL) - 1u);
        if (bad_lanes != 0) { // a poisoned row still has to sort
#pragma unroll
            for (int j = 0; j < M; ++j)
                x[j] = x[j] == x[j] ? x[j] : -INFINITY;
        }

        // ---- groups: the lanes of those that are not among the best hold nothing any more
        uint32_t base0 = from; // the expert of the lane's first slot
        if (RL == 16 && p.n_group > 1) {
            const float pinf = opaque_inf(false);
            float a1 = fmax2(x[0], x[1], pinf), a2 = fmin2(x[0], x[1], opaque_inf(true));
#pragma unroll
            for (int j = 2; j < M; ++j) {
                a2 = __builtin_amdgcn_fmed3f(a1, a2, x[j]);
                a1 = fmax2(a1, x[j], pinf);
            }
            if (p.gl_log2 >= 1)
                merge_top2f<0xB1>(a1, a2, pinf); // quad_perm [1,0,3,2]
            if (p.gl_log2 >= 2)
                merge_top2f<0x4E>(a1, a2, pinf); // quad_perm [2,3,0,1]
            if (p.gl_log2 >= 3)
                merge_top2f<0x141>(a1, a2, pinf); // row_half_mirror
            const float value = a1 + (a2 > -INFINITY ? a2 : 0.0f); // one expert left counts alone
            const uint32_t gkey = ordered(value == value ? value : -INFINITY);
            uint32_t rank = 0;
            switch (p.gl_log2) {
            case 0: row_group_rank<0>(gkey, gkey - 1u, rank); break;
            case 1: row_group_rank<1>(gkey, gkey - 1u, rank); break;
            case 2: row_group_rank<2>(gkey, gkey - 1u, rank); break;
            default: row_group_rank<3>(gkey, gkey - 1u, rank); break;
            }
            const bool kept = rank < p.topk_group;
            if constexpr (MOVE) {
                // kept groups below this lane's own in its row, counted by their last lanes
                const uint32_t gmask = (1u << p.gl_log2) - 1u;
                const uint64_t last = __builtin_amdgcn_ballot_w64(kept && (q & gmask) == gmask);
                const uint32_t mine = (uint32_t)(last >> (lane & 48u)) & ((1u << q) - 1u);
                if (kept) {
                    const uint32_t d = (row << 4) + 2u * (((uint32_t)__builtin_popcount(mine) << p.gl_log2) | (q & gmask));
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int w = 0; w < 2; ++w)
                            s_move[wv][w][d + h] = make_uint4(fbits(x[8 * h + 4 * w]), fbits(x[8 * h + 4 * w + 1]),
                                                              fbits(x[8 * h + 4 * w + 2]), fbits(x[8 * h + 4 * w + 3]));
                        s_src[wv][d + h] = q * C + 8 * h;
                    }
                }
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
                const bool filled = q < 2u * (p.topk_group << p.gl_log2);
                const uint4 v0 = s_move[wv][0][lane], v1 = s_move[wv][1][lane];
                const uint32_t v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
                base0 = s_src[wv][lane];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[j] = filled ? ffrom(v[j]) : -INFINITY;
            } else {
#pragma unroll
                for (int j = 0; j < M; ++j)
                    x[j] = kept ? x[j] : -INFINITY;
            }
        }

        // ---- the lane's lists, best first, their slots 3 bits each with the head's lowest
        uint32_t key[S][N], slots[S];
#pragma unroll
        for (int l = 0; l < S; ++l) {
            uint32_t id[N];
#pragma unroll
            for (int j = 0; j < N; ++j)
                key[l][j] = fbits(x[N * l + j]);
            if constexpr (N == 4)
                sort_lane_raw4(key[l], id);
            else
                sort_lane_raw8(key[l], id);
            slots[l] = 0;
#pragma unroll
            for (int j = 0; j < N; ++j)
                slots[l] |= id[j] << (3 * j);
            slots[l] ^= 0xFFFFFFu;
        }

        // ---- k rounds, four tokens at once; depth: the picks left, this one included
        uint2* const pick_row = &s_pick[wv][row * RL];
        auto round = [&](uint32_t it, uint32_t depth) {
            uint32_t h = key[0][0];
#pragma unroll
            for (int l = 1; l < S; ++l)
                h = max(h, key[l][0]);
            const uint32_t m = row_umax<RL>(h);
            const uint64_t hit = __builtin_amdgcn_ballot_w64(h == m);
            // the lowest set bit of each row's bits (every row has one)
            const uint64_t win = hit & ~(hit - (RL == 16 ? 0x0001000100010001ull : 0x0101010101010101ull));
            const bool mine = __builtin_amdgcn_inverse_ballot_w64(win);
            if constexpr (S == 1) {
                if (mine) {
                    pick_row[it] = make_uint2(base0 + (slots[0] & 7u), h);
#pragma unroll
                    for (int j = 0; j + 1 < N; ++j)
                        if (j + 1u < depth)
                            key[0][j] = key[0][j + 1];
                    if (depth > (uint32_t)N)
                        key[0][N - 1] = 0u;
                    slots[0] >>= 3;
                }
                return;
            }
            bool taken = false;
            uint32_t pick = 0;
            bool pop[S];
#pragma unroll
            for (int l = 0; l < S; ++l) { // the first list that holds it: its experts have the smaller indices
                const bool here = !taken && key[l][0] == h;
                pick = here ? base0 + N * l + (slots[l] & 7u) : pick;
                taken = taken || here;
                pop[l] = mine && here;
            }
#pragma unroll
            for (int l = 0; l < S; ++l) {
#pragma unroll
                for (int j = 0; j + 1 < N; ++j)
                    if (j + 1u < depth)
                        key[l][j] = pop[l] ? key[l][j + 1] : key[l][j];
                if (depth > (uint32_t)N)
                    key[l][N - 1] = pop[l] ? 0u : key[l][N - 1];
                slots[l] = pop[l] ? slots[l] >> 3 : slots[l];
            }
            if (mine)
                pick_row[it] = make_uint2(pick, h);
        };
        if constexpr (K8) {
#pragma unroll
            for (uint32_t it = 0; it < 8; ++it)
                round(it, 8u - it);
        } else {
            for (uint32_t it = 0; it < p.k; ++it)
                round(it, 64u);
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");

        // ---- pick q of the row, its weight from its own logit again in 64 bits
        const uint2 got = s_pick[wv][lane];
        const bool out = q < p.k;
        const bool present = out && got.y > kMasked && !poisoned;
        double s = 0.0;
        if (present) {
            const float l = by_score ? load_logit<BF16>(p.logits, at + got.x) : unordered(got.y); // else the key itself
            s = p.softmax ? shifted(l) * inv_sum : sigmoid64(l);
        }
        if (p.normalise) {
            const double sum = row_sum<RL>(s);
            if (sum != 0.0)
                s /= sum;
        }
        if (out && t < p.tokens) {
            p.idx[(size_t)t * p.k + q] = poisoned ? (int32_t)q : present ? (int32_t)got.x : -1;
            p.weight[(size_t)t * p.k + q] = poisoned ? ffrom(0x7FC00000u) : (float)(s * p.scale);
        }
        __builtin_amdgcn_wave_barrier(); // the LDS is written again
    }
}

struct RouteBwdParams {
    const float* dweight;
    const int32_t* idx;
    const void* logits;
    uint32_t tokens, experts, k;
    int softmax, normalise;
    float scale;
    void* dlogits;
};

template <bool BF16>
__device__ __forceinline__ void store_grad(void* base, size_t i, float v)
{
    if constexpr (BF16) {
        const __bf16 b = (__bf16)v;
        static_cast<uint16_t*>(base)[i] = __builtin_bit_cast(uint16_t, b);
    } else {
        static_cast<float*>(base)[i] = v;
    }
}

// Sums, scores and differences in 64 bits here and below: d - dot is a small
// difference of large numbers where the gradients of a token's weights are
// nearly equal or one expert has nearly all of the weight (in 32 bits,
// gradients within 10^-3 of each other gave results off by 10^-4 of their
// size).  Softmax over all experts takes fp32 exponentials, the same ones in the
// sum and in the scores: what they are off by then scales the scores' shares and
// cancels nothing (64-bit ones: 8192 tokens x 512 experts in bf16 10.1 us instead
// of 8.6).
// One wave per token; lane j < k holds the token's slot j, and the row is put
// together in LDS before it is written.
template <bool BF16>
__device__ __forceinline__ void route_backward_token(const RouteBwdParams& p, uint32_t t, uint32_t lane,
                                                     float* s_row)
{
    const size_t row = (size_t)t * p.experts;
    int32_t e = -1;
    double d = 0.0;
    if (lane < p.k) {
        e = p.idx[(size_t)t * p.k + lane];
        d = (double)p.scale * (double)p.dweight[(size_t)t * p.k + lane];
    }
    bool live = (uint32_t)e < p.experts;
    for (uint32_t i = 0; i + 1 < p.k; ++i) {
        const int32_t o = __builtin_amdgcn_readlane(e, i);
        live = live && !(lane > i && o == e);
    }
    const float l = live ? load_logit<BF16>(p.logits, row + (uint32_t)e) : -INFINITY;

    const bool dense = p.softmax && !p.normalise;
    d = live ? d : 0.0;
    float grad;
    if (p.softmax) { // over the whole row, or, normalised, over the chosen experts alone
        float top = l;
        if (dense)
            for (uint32_t i = lane; i < p.experts; i += kWave)
                top = fmaxf(top, load_logit<BF16>(p.logits, row + i));
#pragma unroll
        for (int m = 1; m < kWave; m <<= 1)
            top = fmaxf(top, __shfl_xor(top, m));
        if (top == -INFINITY)
            top = 0.0f;
        const double own = !live ? 0.0 : dense ? (double)expf(l - top) : exp64_nan((double)l - (double)top);
        double sum = dense ? 0.0 : own;
        if (dense)
            for (uint32_t i = lane; i < p.experts; i += kWave)
                sum += (double)expf(load_logit<BF16>(p.logits, row + i) - top);
        sum = wave_sum(sum);
        const double inv_sum = sum == 0.0 ? 0.0 : reciprocal64(sum); // else at least 1, or NaN
        const double s = own * inv_sum, dot = wave_sum(d * s);
        const float rest = (float)-(inv_sum * dot);
        grad = (float)(s * (d - dot));
        for (uint32_t i = lane; i < p.experts; i += kWave)
            s_row[i] = dense ? expf(load_logit<BF16>(p.logits, row + i) - top) * rest : 0.0f;
    } else {
        double s = 0.0, slope = 0.0;
        if (live) {
            s = l == l ? sigmoid64(l) : (double)l;
            slope = sigmoid64(-l);
        }
        if (p.normalise) {
            // scores too small for 32 bits still share the weight between them
            const double total = wave_sum(s);
            if (total != 0.0) {
                s /= total;
                d -= wave_sum(d * s);
            }
        }
        grad = (float)(d * s * slope);
        for (uint32_t i = lane; i < p.experts; i += kWave)
            s_row[i] = 0.0f;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (live)
        s_row[e] = grad;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    for (uint32_t i = lane; i < p.experts; i += kWave)
        store_grad<BF16>(p.dlogits, row + i, s_row[i]);
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(RouteBwdParams p)
{
    __shared__ float s_row[kWaves][kMaxExperts];
    const uint32_t lane = threadIdx.x & (kWave - 1), wv = threadIdx.x / kWave;
    for (uint32_t t = blockIdx.x * kWaves + wv; t < p.tokens; t += gridDim.x * kWaves)
        route_backward_token<BF16>(p, t, lane, s_row[wv]);
}

// e of lane I of its 16-lane row, for I = 0 .. 14 while I < k - 1: whether an
// earlier lane names the same expert
template <int I = 0>
__device__ __forceinline__ bool named_before(int32_t e, uint32_t q, uint32_t k)
{
    if constexpr (I < 15) {
        if (I + 1u >= k)
            return false;
        const int32_t o = __builtin_amdgcn_mov_dpp(e, 0x150 + I, 0xF, 0xF, false); // row_newbcast
        const bool mine = q > (uint32_t)I && o == e;
        const bool later = named_before<I + 1>(e, q, k);
        return mine || later;
    } else {
        return false;
    }
}

// Four tokens per wave, one per 16-lane row (k <= 16): lane q < k of a row holds
// the token's slot q.  The four rows, consecutive in memory, are put together
// in LDS and written as one run; VEC: 16 bytes a lane (the rows' bytes and
// their addresses are multiples of 16).  DENSE: softmax over all experts, whose
// logits pass through the same LDS.
// Bound by the bytes written at large sizes.
template <bool BF16, bool DENSE, bool VEC>
__global__ __launch_bounds__(kThreads) void route_backward_row_kernel(RouteBwdParams p)
{
    constexpr uint32_t kPer = VEC ? (BF16 ? 8 : 4) : 1; // elements a lane moves at a time
    extern __shared__ float4 s_rows4[];
    const uint32_t lane = threadIdx.x & (kWave - 1), wv = threadIdx.x / kWave;
    const uint32_t q = lane & 15u, row = lane >> 4;
    float* const s_rows = reinterpret_cast<float*>(s_rows4) + (size_t)wv * 4u * p.experts;
    const uint32_t first = 4u * __builtin_amdgcn_readfirstlane(blockIdx.x * kWaves + wv);
    auto exchange = [] {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    };

    for (uint32_t t0 = first; t0 < p.tokens; t0 += gridDim.x * (4u * kWaves)) {
        const uint32_t t = min(t0 + row, p.tokens - 1u); // rows past the last token repeat it and are not written
        const uint32_t count = min(4u, p.tokens - t0) * p.experts;
        const size_t at = (size_t)t * p.experts, run = (size_t)t0 * p.experts;
        int32_t e = -1;
        double d = 0.0;
        if (q < p.k) {
            e = p.idx[(size_t)t * p.k + q];
            d = (double)p.scale * (double)p.dweight[(size_t)t * p.k + q];
        }
        const bool again = named_before(e, q, p.k);
        const bool live = (uint32_t)e < p.experts && !again;
        const float l = live ? load_logit<BF16>(p.logits, at + (uint32_t)e) : -INFINITY;
        d = live ? d : 0.0;

        // the rows before the chosen experts' gradients: zeros, or the logits
        if constexpr (DENSE) {
            for (uint32_t i = lane * kPer; i < count; i += kWave * kPer) {
                float x[kPer < 2 ? 2 : kPer];
                if constexpr (VEC)
                    load_logits<BF16, kPer < 2 ? 2 : kPer>(p.logits, run + i, x);
                else
                    x[0] = load_logit<BF16>(p.logits, run + i);
#pragma unroll
                for (uint32_t j = 0; j < kPer; ++j)
                    s_rows[i + j] = x[j];
            }
        } else {
            for (uint32_t i = lane * kPer; i < count; i += kWave * kPer) {
#pragma unroll
                for (uint32_t j = 0; j < kPer; ++j)
                    s_rows[i + j] = 0.0f;
            }
        }
        exchange();

        float grad;
        if (p.softmax) { // over the whole row, or, normalised, over the chosen experts alone
            float* const mine = s_rows + (DENSE ? (t - t0) * p.experts : 0u);
            float top = l;
            // (unrolled: 406 tokens x 512 experts 10.3 -> 6.9 us, 4096 x 160 5.6 -> 5.0)
            if constexpr (DENSE) {
#pragma unroll 8
                for (uint32_t i = q; i < p.experts; i += 16u)
                    top = fmaxf(top, mine[i]);
            }
            top = unordered(row_umax(ordered(top)));
            if (top == -INFINITY)
                top = 0.0f;
            const double own = !live ? 0.0 : DENSE ? (double)expf(l - top) : exp64_nan((double)l - (double)top);
            double sum = DENSE ? 0.0 : own;
            if constexpr (DENSE) {
#pragma unroll 8
                for (uint32_t i = q; i < p.experts; i += 16u) {
                    const float v = expf(mine[i] - top);
                    sum += (double)v;
                    if (t0 + row < p.tokens)
                        mine[i] = v;
                }
            }
            sum = row_sum(sum);
            const double inv_sum = sum == 0.0 ? 0.0 : reciprocal64(sum); // else at least 1, or NaN
            const double s = own * inv_sum, dot = row_sum(d * s);
            grad = (float)(s * (d - dot));
            if constexpr (DENSE) {
                const float rest = (float)-(inv_sum * dot);
                if (t0 + row < p.tokens) {
#pragma unroll 8
                    for (uint32_t i = q; i < p.experts; i += 16u)
                        mine[i] *= rest;
                }
            }
        } else {
            // s and 1 - s from one exponential, in 64 bits: scores too small for 32 still share the weight
            const double x = exp64_neg(-(double)fabsf(l)), one = reciprocal64(1.0 + x);
            double s = live ? (l >= 0.0f ? one : x * one) : 0.0;
            const double slope = l >= 0.0f ? x * one : one;
            if (l != l)
                s = (double)l;
            if (p.normalise) {
                const double total = row_sum(s);
                if (total != 0.0) {
                    s /= total;
                    d -= row_sum(d * s);
                }
            }
            grad = (float)(d * s * slope);
        }
        exchange();
        if (live && t0 + row < p.tokens)
            s_rows[row * p.experts + (uint32_t)e] = grad;
        exchange();
        for (uint32_t i = lane * kPer; i < count; i += kWave * kPer) {
            if constexpr (!VEC) {
                store_grad<BF16>(p.dlogits, run + i, s_rows[i]);
            } else if constexpr (BF16) { // past the caches: 16384 x 256 in fp32 5.7 us, through them 6.9
                typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
                bf16x8 v;
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j)
                    v[j] = (__bf16)s_rows[i + j];
                __builtin_nontemporal_store(
                    v, reinterpret_cast<bf16x8*>(static_cast<uint16_t*>(p.dlogits) + run + i));
            } else {
                typedef float f32x4 __attribute__((ext_vector_type(4)));
                __builtin_nontemporal_store(*reinterpret_cast<const f32x4*>(s_rows + i),
                                            reinterpret_cast<f32x4*>(static_cast<float*>(p.dlogits) + run + i));
            }
        }
        exchange(); // the LDS is written again
    }
}

bool overlaps(const void* a, size_t an, const void* b, size_t bn)
{
    if (!a || !b || an == 0 || bn == 0)
        return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + bn && b0 < a0 + an;
}

bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

template <bool BF16, int L, int FC, bool MOVE = false, int RL = 16>
void launch_route_k(const RouteParams& p, hipStream_t s)
{
    const uint32_t tokens = kWaves * (kWave / RL), blocks = (p.tokens + tokens - 1u) / tokens;
    const dim3 grid(blocks < kMaxBlocks ? blocks : (uint32_t)kMaxBlocks);
    if (p.k == 8)
        hipLaunchKernelGGL((route_row_kernel<BF16, L, FC, true, MOVE, RL>), grid, dim3(kThreads), 0, s, p);
    else
        hipLaunchKernelGGL((route_row_kernel<BF16, L, FC, false, MOVE, RL>), grid, dim3(kThreads), 0, s, p);
}

// by the lists of eight a lane needs, the usual expert counts with their count compiled in
template <bool BF16>
void launch_route_row(const RouteParams& p, hipStream_t s)
{
    switch ((p.n_group << p.gl_log2) == 16u && p.lane_experts * 16u == p.experts ? p.experts : 0u) {
    case 64: // 32768 tokens of bf16, softmax top-6: 6.1 us with eight tokens a wave, 7.3 with four (64 tokens 3.5 / 3.4)
        if (p.n_group == 1 && p.k <= 8)
            return launch_route_k<BF16, 1, 8, false, 8>(p, s);
        return launch_route_k<BF16, 1, 4>(p, s);
    case 128: return launch_route_k<BF16, 1, 8>(p, s);
    case 256:
        if (p.n_group > 1 && (p.topk_group << p.gl_log2) <= 8)
            return launch_route_k<BF16, 2, 16, true>(p, s);
        return launch_route_k<BF16, 2, 16>(p, s);
    case 160: return launch_route_k<BF16, 2, 10>(p, s);
    case 192: return launch_route_k<BF16, 2, 12>(p, s);
    case 384: return launch_route_k<BF16, 3, 24>(p, s);
    case 512: return launch_route_k<BF16, 4, 32>(p, s);
    }
    switch ((p.lane_experts + 7) / 8) {
    case 1: return launch_route_k<BF16, 1, 0>(p, s);
    case 2: return launch_route_k<BF16, 2, 0>(p, s);
    case 3: return launch_route_k<BF16, 3, 0>(p, s);
    default: return launch_route_k<BF16, 4, 0>(p, s);
    }
}

template <bool BF16>
void launch_backward_row(bool dense, bool vec, const RouteBwdParams& p, dim3 grid, hipStream_t s)
{
    const size_t lds = (size_t)kWaves * 4u * p.experts * 4u; // 32 KiB at 512 experts
    if (dense && vec)
        hipLaunchKernelGGL((route_backward_row_kernel<BF16, true, true>), grid, dim3(kThreads), lds, s, p);
    else if (dense)
        hipLaunchKernelGGL((route_backward_row_kernel<BF16, true, false>), grid, dim3(kThreads), lds, s, p);
    else if (vec)
        hipLaunchKernelGGL((route_backward_row_kernel<BF16, false, true>), grid, dim3(kThreads), lds, s, p);
    else
        hipLaunchKernelGGL((route_backward_row_kernel<BF16, false, false>), grid, dim3(kThreads), lds, s, p);
}

// what both directions check alike
bool route_sizes_ok(int in_dtype, int64_t tokens, int64_t experts, int64_t k, int scoring, int normalise, float scale)
{
    return (in_dtype == TK_DTYPE_BF16 || in_dtype == TK_DTYPE_FP32) && tokens >= 0 && tokens < (int64_t)INT_MAX &&
           experts > 0 && k > 0 && k <= experts && (scoring == TK_SCORE_SIGMOID || scoring == TK_SCORE_SOFTMAX) &&
           (normalise == 0 || normalise == 1) && std::isfinite(scale);
}

} // namespace

extern "C" {

tk_status tk_route(const void* logits, tk_dtype in_dtype, const float* bias, int64_t tokens, int64_t experts,
                   int64_t k, int64_t n_group, int64_t topk_group, tk_scoring scoring, int normalise, float scale,
                   int32_t* topk_idx, float* topk_weight, void* stream)
{
    if (!route_sizes_ok((int)in_dtype, tokens, experts, k, (int)scoring, normalise, scale))
        return TK_ERR_INVALID_ARG;
    if (n_group <= 0 || topk_group <= 0 || topk_group > n_group || experts % n_group != 0)
        return TK_ERR_INVALID_ARG;
    const int64_t per = experts / n_group;
    if ((n_group > 1 && per < 2) || k > topk_group * per)
        return TK_ERR_INVALID_ARG;
    if (tokens > 0 && (!logits || !topk_idx || !topk_weight))
        return TK_ERR_INVALID_ARG;
    const bool bf16 = (int)in_dtype == TK_DTYPE_BF16;
    if (misaligned(logits, bf16 ? 2 : 4) || misaligned(bias, 4) || misaligned(topk_idx, 4) ||
        misaligned(topk_weight, 4))
        return TK_ERR_INVALID_ARG;
    const size_t l_bytes = (size_t)tokens * (size_t)experts * (bf16 ? 2u : 4u);
    const size_t o_bytes = (size_t)tokens * (size_t)k * 4u, b_bytes = (size_t)experts * 4u;
    if (overlaps(topk_idx, o_bytes, logits, l_bytes) || overlaps(topk_weight, o_bytes, logits, l_bytes) ||
        overlaps(topk_idx, o_bytes, bias, b_bytes) || overlaps(topk_weight, o_bytes, bias, b_bytes) ||
        overlaps(topk_idx, o_bytes, topk_weight, o_bytes))
        return TK_ERR_INVALID_ARG;
    if (experts > kMaxExperts || k > kMaxK)
        return TK_ERR_UNSUPPORTED;
    if (tokens == 0)
        return TK_OK;
    RouteParams p{};
    p.logits = logits;
    p.bias = bias;
    p.tokens = (uint32_t)tokens;
    p.experts = (uint32_t)experts;
    p.k = (uint32_t)k;
    p.n_group = (uint32_t)n_group;
    p.topk_group = (uint32_t)topk_group;
    p.softmax = (int)scoring == TK_SCORE_SOFTMAX;
    p.normalise = normalise;
    p.scale = (double)scale;
    p.idx = topk_idx;
    p.weight = topk_weight;
    hipStream_t s = static_cast<hipStream_t>(stream);
    // four tokens per wave, a group to a power of two of a row's 16 lanes, 32 experts a lane at most
    p.gl_log2 = 4;
    while (p.gl_log2 > 0 && (n_group << p.gl_log2) > 16)
        --p.gl_log2;
    p.group_experts = (uint32_t)per;
    p.lane_experts = (uint32_t)((per + (1 << p.gl_log2) - 1) >> p.gl_log2);
    if (k <= 16 && n_group <= 16 && p.lane_experts <= 32) {
        if (bf16)
            launch_route_row<true>(p, s);
        else
            launch_route_row<false>(p, s);
        return hipGetLastError() == hipSuccess ? TK_OK : TK_ERR_HIP;
    }
    const int64_t blocks = (tokens + kWaves - 1) / kWaves;
    const dim3 grid((uint32_t)(blocks < kMaxBlocks ? blocks : kMaxBlocks));
#define TK_ROUTE(CC)                                                                        \
    case CC:                                                                                \
        if (bf16)                                                                           \
            hipLaunchKernelGGL((route_kernel<true, CC>), grid, dim3(kThreads), 0, s, p);    \
        else                                                                                \
            hipLaunchKernelGGL((route_kernel<false, CC>), grid, dim3(kThreads), 0, s, p);   \
        break;
    switch ((experts + kWave - 1) / kWave) {
        TK_ROUTE(1)
        TK_ROUTE(2)
        TK_ROUTE(3)
        TK_ROUTE(4)
        TK_ROUTE(5)
        TK_ROUTE(6)
        TK_ROUTE(7)
        TK_ROUTE(8)
    }
#undef TK_ROUTE
    return hipGetLastError() == hipSuccess ? TK_OK : TK_ERR_HIP;
}

tk_status tk_route_backward(const float* dweight, const int32_t* topk_idx, const void* logits, tk_dtype in_dtype,
                            int64_t tokens, int64_t experts, int64_t k, tk_scoring scoring, int normalise,
                            float scale, void* dlogits, void* stream)
{
    if (!route_sizes_ok((int)in_dtype, tokens, experts, k, (int)scoring, normalise, scale))
        return TK_ERR_INVALID_ARG;
    if (tokens > 0 && (!dweight || !topk_idx || !logits || !dlogits))
        return TK_ERR_INVALID_ARG;
    const bool bf16 = (int)in_dtype == TK_DTYPE_BF16;
    if (misaligned(logits, bf16 ? 2 : 4) || misaligned(dlogits, bf16 ? 2 : 4) || misaligned(topk_idx, 4) ||
        misaligned(dweight, 4))
        return TK_ERR_INVALID_ARG;
    const size_t l_bytes = (size_t)tokens * (size_t)experts * (bf16 ? 2u : 4u);
    const size_t o_bytes = (size_t)tokens * (size_t)k * 4u;
    if (overlaps(dlogits, l_bytes, logits, l_bytes) || overlaps(dlogits, l_bytes, topk_idx, o_bytes) ||
        overlaps(dlogits, l_bytes, dweight, o_bytes))
        return TK_ERR_INVALID_ARG;
    if (experts > kMaxExperts || k > kMaxK)
        return TK_ERR_UNSUPPORTED;
    if (tokens == 0)
        return TK_OK;
    RouteBwdParams p{};
    p.dweight = dweight;
    p.idx = topk_idx;
    p.logits = logits;
    p.tokens = (uint32_t)tokens;
    p.experts = (uint32_t)experts;
    p.k = (uint32_t)k;
    p.softmax = (int)scoring == TK_SCORE_SOFTMAX;
    p.normalise = normalise;
    p.scale = scale;
    p.dlogits = dlogits;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (k <= 16) { // four tokens per wave
        const size_t row_bytes = (size_t)experts * (bf16 ? 2u : 4u);
        const bool vec = row_bytes % 16 == 0 && !misaligned(dlogits, 16);
        const int64_t rblocks = (tokens + 4 * kWaves - 1) / (4 * kWaves);
        const dim3 rgrid((uint32_t)(rblocks < kMaxBlocks ? rblocks : kMaxBlocks));
        if (bf16)
            launch_backward_row<true>(p.softmax && !p.normalise, vec, p, rgrid, s);
        else
            launch_backward_row<false>(p.softmax && !p.normalise, vec, p, rgrid, s);
        return hipGetLastError() == hipSuccess ? TK_OK : TK_ERR_HIP;
    }
    const int64_t blocks = (tokens + kWaves - 1) / kWaves;
    const dim3 grid((uint32_t)(blocks < kMaxBlocks ? blocks : kMaxBlocks));
    if (bf16)
        hipLaunchKernelGGL((route_backward_kernel<true>), grid, dim3(kThreads), 0, s, p);
    else
        hipLaunchKernelGGL((route_backward_kernel<false>), grid, dim3(kThreads), 0, s, p);
    return hipGetLastError() == hipSuccess ? TK_OK : TK_ERR_HIP;
}

} // extern "C"
