// tk_route.hip -- routing of tokens to experts from the router's logits and the
// gradient of its weights, behind tk_route and tk_route_backward in
// include/tk_layer.h.
//
// Scores are computed in 64 bits and rounded once, so that the order of two
// experts is that of their exact scores rounded to fp32 (plus the bias), and
// does not hang on how an fp32 exponential was built.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "tk.h"
#include "tk_layer.h"

namespace {

constexpr int kWave = 64;
constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxExperts = 512;
constexpr int kMaxK = 64;
constexpr int64_t kMaxBlocks = 1 << 20; // a launch holds fewer than 2^32 work-items; tokens past the grid loop

__device__ __forceinline__ uint32_t fbits(float f) { return __builtin_bit_cast(uint32_t, f); }
__device__ __forceinline__ float ffrom(uint32_t u) { return __builtin_bit_cast(float, u); }

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* base, size_t i)
{
    if constexpr (BF16)
        return ffrom((uint32_t)static_cast<const uint16_t*>(base)[i] << 16);
    else
        return static_cast<const float*>(base)[i];
}

// Order-preserving map of a (non-NaN) float to uint32; -0 and +0 map alike, and
// 0 is below every value.
__device__ __forceinline__ uint32_t ordered(float f)
{
    const uint32_t b = fbits(f + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t h) { return ffrom((h & 0x80000000u) ? (h & 0x7FFFFFFFu) : ~h); }

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

__device__ __forceinline__ double sigmoid64(float l) { return 1.0 / (1.0 + exp(-(double)l)); }

struct RouteParams {
    const void* logits;
    const float* bias; // or null
    uint32_t tokens, experts, k, n_group, topk_group;
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
            sum += exp((double)l[j] - (double)top);
        sum = wave_sum(sum);
        inv_sum = sum > 0.0 ? 1.0 / sum : 0.0;
    }
    auto score = [&](float x) { return p.softmax ? exp((double)x - (double)top) * inv_sum : sigmoid64(x); };

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

// One wave per token; lane j < k holds the token's slot j, and the row is put
// together in LDS before it is written.
template <bool BF16>
__device__ __forceinline__ void route_backward_token(const RouteBwdParams& p, uint32_t t, uint32_t lane,
                                                     float* s_row)
{
    const size_t row = (size_t)t * p.experts;
    int32_t e = -1;
    float d = 0.0f;
    if (lane < p.k) {
        e = p.idx[(size_t)t * p.k + lane];
        d = p.scale * p.dweight[(size_t)t * p.k + lane];
    }
    bool live = (uint32_t)e < p.experts;
    for (uint32_t i = 0; i + 1 < p.k; ++i) {
        const int32_t o = __builtin_amdgcn_readlane(e, i);
        live = live && !(lane > i && o == e);
    }
    const float l = live ? load_logit<BF16>(p.logits, row + (uint32_t)e) : -INFINITY;

    const bool dense = p.softmax && !p.normalise;
    float s = 0.0f;               // the score of this lane's slot
    double s64 = 0.0;             // the same of a sigmoid, and 1 - s
    float slope = 0.0f;
    float top = 0.0f, inv_sum = 1.0f;
    if (p.softmax) {
        // over the whole row, or, normalised, over the chosen experts alone
        top = l;
        if (dense)
            for (uint32_t i = lane; i < p.experts; i += kWave)
                top = fmaxf(top, load_logit<BF16>(p.logits, row + i));
#pragma unroll
        for (int m = 1; m < kWave; m <<= 1)
            top = fmaxf(top, __shfl_xor(top, m));
        if (top == -INFINITY)
            top = 0.0f;
        float sum = 0.0f;
        if (dense) {
            for (uint32_t i = lane; i < p.experts; i += kWave)
                sum += expf(load_logit<BF16>(p.logits, row + i) - top);
        } else if (live) {
            sum = expf(l - top);
        }
        sum = wave_sum(sum);
        inv_sum = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
        s = live ? expf(l - top) * inv_sum : 0.0f;
    } else if (live) {
        s64 = sigmoid64(l);
        s = (float)s64;
        slope = (float)(1.0 / (1.0 + exp((double)l)));
    }
    float ds = live ? d : 0.0f;
    float grad;
    if (p.softmax) {
        const float dot = wave_sum(ds * s);
        grad = s * (ds - dot);
        for (uint32_t i = lane; i < p.experts; i += kWave)
            s_row[i] = dense ? -(expf(load_logit<BF16>(p.logits, row + i) - top) * inv_sum) * dot : 0.0f;
    } else {
        if (p.normalise) {
            // scores too small for 32 bits still share the weight between them
            const double total = wave_sum(s64);
            if (total != 0.0) {
                s = (float)(s64 / total);
                const float dot = wave_sum(ds * s);
                ds = live ? ds - dot : 0.0f;
            }
        }
        grad = ds * s * slope;
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

bool overlaps(const void* a, size_t an, const void* b, size_t bn)
{
    if (!a || !b || an == 0 || bn == 0)
        return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + bn && b0 < a0 + an;
}

bool misaligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

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
    const int64_t blocks = (tokens + kWaves - 1) / kWaves;
    const dim3 grid((uint32_t)(blocks < kMaxBlocks ? blocks : kMaxBlocks));
    if (bf16)
        hipLaunchKernelGGL((route_backward_kernel<true>), grid, dim3(kThreads), 0, s, p);
    else
        hipLaunchKernelGGL((route_backward_kernel<false>), grid, dim3(kThreads), 0, s, p);
    return hipGetLastError() == hipSuccess ? TK_OK : TK_ERR_HIP;
}

} // extern "C"
