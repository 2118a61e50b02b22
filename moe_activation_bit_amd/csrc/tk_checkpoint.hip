// tk_checkpoint.hip -- the SwiGLU step that leaves its input in FP8
// (tk_swiglu_checkpoint_fp8) and SwiGLU's gradient from that checkpoint
// (tk_swiglu_backward), behind include/tk_expert.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "tk.h"
#include "tk_expert.h"
#include "tk_quant.h"
#include "tk_swiglu.h"

namespace {

using namespace tk_detail;

// ---------------------------------------------------------------------------
// SwiGLU + cast, with the checkpoint
// ---------------------------------------------------------------------------

struct NoCount { // (the clamp's counter is tk_swiglu_cast_fp8's alone)
    __device__ __forceinline__ void add(bool) {}
};

// A wave takes SPU steps of 512 columns of a row: 16 bytes a lane of the gate and
// of the up half, once.  The activation is computed as in tk_swiglu_cast.hip (the
// same table, products and cast), and both halves are cast as they are, each
// group of 2^gl_log2 lanes by its own abs-max.  Bound by its bytes: 4 read and 3
// written for each column (two calls: 8 and 3).  32768 x 2048 in groups of 128: 87
// us, 5.4 TB/s; 349 x 7168 6.3, the table's copy into LDS and one trip to memory.
template <int SFMT, bool CLAMP, int SPU>
__global__ __launch_bounds__(kThreads) void swiglu_checkpoint_kernel(Params p, Params px, const float2* table)
{
    __shared__ float2 lut[kLutSize];
    const uint32_t lane = threadIdx.x & (kWaveSize - 1);
    {
        constexpr int kPer = kLutSize / 2 / kThreads; // 16-byte pieces a thread
        const uint4* const src = reinterpret_cast<const uint4*>(table);
        uint4 v[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            v[i] = src[i * kThreads + threadIdx.x];
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            reinterpret_cast<uint4*>(lut)[i * kThreads + threadIdx.x] = v[i];
        __syncthreads();
    }
    float limit = 0.0f, a_limit = 0.0f;
    if constexpr (CLAMP) {
        limit = p.clamp;
        a_limit = limit * sigmoid_rn(limit);
    }
    constexpr uint32_t kWaves = kThreads / kWaveSize;
    NoCount none;
    for (uint32_t u = blockIdx.x * kWaves + threadIdx.x / kWaveSize; u < p.units; u += gridDim.x * kWaves) {
        const uint32_t row = u / p.upr, step0 = (u - row * p.upr) * SPU;
        const uint4* const xg = p.x + (size_t)row * (2u * p.slots);
        uint4 g[SPU], up[SPU];
#pragma unroll
        for (int s = 0; s < SPU; ++s) { // lanes past the row's end read its last slot again
            const uint32_t slot = min((step0 + s) * kWaveSize + lane, p.slots - 1u);
            g[s] = load16(xg + slot);
            up[s] = load16(xg + p.slots + slot);
        }
        const float w = p.w ? p.w[row] : 1.0f;
        uint8_t* const codes = p.codes + (size_t)row * (p.slots * 8u);
        uint8_t* const x_codes = px.codes + (size_t)row * (p.slots * 16u);
#pragma unroll
        for (int s = 0; s < SPU; ++s) {
            const uint32_t slot = (step0 + s) * kWaveSize + lane;
            const bool valid = slot < p.slots;
            const bool first = (lane & ((1u << p.gl_log2) - 1u)) == 0;
            auto finish = [&](const Params& to, uint8_t* row_codes, uint32_t at, const float* v, uint32_t amax) {
                float s32 = 0.0f;
                uint32_t s8 = 0;
                const float inv = group_scale<8, SFMT>(group_umax(valid ? amax : 0u, p.gl_log2), s32, s8);
                if (valid) {
                    quantize_store<8>(row_codes, at, v, inv);
                    if (first)
                        store_scale<SFMT>(to, row, at >> p.gl_log2, s32, s8);
                }
            };
            float y[8];
            const uint32_t m = compute_step<CLAMP, true>(lut, g[s], up[s], w, valid, limit, a_limit, none, y);
            finish(p, codes, slot, y, m);
            auto as_is = [&](const uint4& v, uint32_t at) {
                const uint32_t word[4] = {v.x, v.y, v.z, v.w};
                float x[8], top = 0.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    x[2 * k] = as_float(word[k] << 16);
                    x[2 * k + 1] = as_float(word[k] & 0xFFFF0000u);
                    top = fmaxf(top, fmaxf(fabsf(x[2 * k]), fabsf(x[2 * k + 1]))); // (passes over NaN, as tk_cast_fp8)
                }
                finish(px, x_codes, at, x, as_uint(top));
            };
            as_is(g[s], slot);
            as_is(up[s], p.slots + slot);
        }
    }
}

template <int SFMT, bool CLAMP>
void launch_checkpoint(const Params& p, const Params& px, const float2* table, int spu, uint32_t blocks, hipStream_t s)
{
    if (spu == 4)
        hipLaunchKernelGGL((swiglu_checkpoint_kernel<SFMT, CLAMP, 4>), dim3(blocks), dim3(kThreads), 0, s, p, px, table);
    else
        hipLaunchKernelGGL((swiglu_checkpoint_kernel<SFMT, CLAMP, 1>), dim3(blocks), dim3(kThreads), 0, s, p, px, table);
}

// ---------------------------------------------------------------------------
// The gradient
// ---------------------------------------------------------------------------

struct BackwardParams {
    const uint4* dy;
    const void* h;
    const void* h_scales;
    const float* weight;
    uint4* dh;
    float* dweight;
    uint4* y;
    uint32_t n, slots; // hidden / 8
    uint32_t groups;   // scales a row of 2 * slots
    uint32_t magic;    // ceil(2^32 / slots a group), 0 for 1
    float clamp;
};

// sigma(g) = 1 / (1 + 2^(-g log2 e)) in fp32 to about two units in the last
// place: the exponent's product in two parts, since its rounding alone is up to
// 2^-24 |g| of the result; one Newton step on the reciprocal.  Beyond +-87, where
// e^|g| leaves fp32's range, the result at 87 stands (g sigma(g) is off by at
// most 1.4e-36 there).
__device__ __forceinline__ float sigmoid(float g)
{
    const float x = g < -87.0f ? -87.0f : g > 87.0f ? 87.0f : g;
    const float hi = x * -1.44269502f; // RN(log2 e)
    const float lo = __builtin_fmaf(x, -1.44269502f, -hi) + x * -1.92596303e-8f;
    const float e = __builtin_amdgcn_exp2f(hi), d = 1.0f + __builtin_fmaf(e, lo * 0.693147182f, e);
    const float r = __builtin_amdgcn_rcpf(d);
    return __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
}

__device__ __forceinline__ float e8m0_scale(uint32_t b)
{
    return b == 0u ? 0x1p-127f : as_float(b == 255u ? 0x7FC00000u : b << 23);
}

constexpr int kFromBf16 = 0, kFromF32 = 1, kFromE8 = 2; // h, or its codes' scales

// W waves of a workgroup share a row, 512 columns at a time in turn; the sum for
// dweight goes over a lane's columns, the lanes and the waves in an order that
// hidden alone fixes.  Bound by its bytes (2 of dy, 2 or 4 of h read, 4 of dh and 2
// of y written for each column): 32768 x 2048 from UE8M0 codes with y 109 us, 6.15
// TB/s.
template <int FROM, bool CLAMP, int W>
__global__ __launch_bounds__(kThreads) void swiglu_backward_kernel(BackwardParams p)
{
    constexpr uint32_t kRows = kThreads / kWaveSize / W;
    __shared__ float s_sum[2][kThreads / kWaveSize]; // of one pass and of the next
    const uint32_t lane = threadIdx.x & (kWaveSize - 1);
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveSize);
    auto gradient = [&](uint32_t row) { // the wave's part of a row; a lane's part of the sum for dweight
        float sum = 0.0f;
        const float w = p.weight ? p.weight[row] : 1.0f;
        const uint4* const dy = p.dy + (size_t)row * p.slots;
        const size_t line = (size_t)row * (2u * p.slots);
        auto divide = [&](uint32_t slot) { return p.magic ? __umulhi(slot, p.magic) : slot; };
        auto load = [&](uint32_t slot) -> uint4 { // 8 of h's columns
            if constexpr (FROM == kFromBf16)
                return load16(static_cast<const uint4*>(p.h) + line + slot);
            const v2u c = __builtin_nontemporal_load(static_cast<const v2u*>(p.h) + line + slot);
            const size_t at = (size_t)row * p.groups + divide(slot);
            if constexpr (FROM == kFromF32)
                return make_uint4(c.x, c.y, as_uint(static_cast<const float*>(p.h_scales)[at]), 0u);
            else
                return make_uint4(c.x, c.y, as_uint(e8m0_scale(static_cast<const uint8_t*>(p.h_scales)[at])), 0u);
        };
        auto widen = [](const uint4& v, float (&x)[8]) {
            if constexpr (FROM == kFromBf16) {
                const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    x[2 * k] = as_float(word[k] << 16);
                    x[2 * k + 1] = as_float(word[k] & 0xFFFF0000u);
                }
            } else {
                const float s = as_float(v.z);
                typedef float v2f __attribute__((ext_vector_type(2)));
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const v2f a = __builtin_amdgcn_cvt_pk_f32_fp8(k ? v.y : v.x, false);
                    const v2f b = __builtin_amdgcn_cvt_pk_f32_fp8(k ? v.y : v.x, true);
                    x[4 * k] = a.x * s;
                    x[4 * k + 1] = a.y * s;
                    x[4 * k + 2] = b.x * s;
                    x[4 * k + 3] = b.y * s;
                }
            }
        };
        auto pack = [](float a, float b) {
            typedef __bf16 v2b __attribute__((ext_vector_type(2)));
            return __builtin_bit_cast(uint32_t, v2b{(__bf16)a, (__bf16)b});
        };
        auto store = [](uint4* to, const uint32_t (&v)[4]) {
            __builtin_nontemporal_store(v4u{v[0], v[1], v[2], v[3]}, reinterpret_cast<v4u*>(to));
        };
        const uint32_t chunks = (p.slots + kWaveSize - 1) / kWaveSize;
        for (uint32_t c = wave % W; c < chunks; c += W) {
            const uint32_t slot = c * kWaveSize + lane;
            if (slot >= p.slots)
                break;
            const uint4 d = load16(dy + slot), g8 = load(slot), u8 = load(p.slots + slot);
            const uint32_t dw[4] = {d.x, d.y, d.z, d.w};
            float g[8], u[8];
            widen(g8, g);
            widen(u8, u);
            uint32_t dg2[4], du2[4], y2[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float dgate[2], dup[2], act[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 2 * k + e;
                    const float dv = as_float(e ? dw[k] & 0xFFFF0000u : dw[k] << 16);
                    float gv = g[i], uv = u[i];
                    bool gate_free = true, up_free = true;
                    if constexpr (CLAMP) {
                        gate_free = !(gv > p.clamp);
                        up_free = !(__builtin_fabsf(uv) > p.clamp);
                        gv = gate_free ? gv : p.clamp;
                        uv = up_free ? uv : __builtin_copysignf(p.clamp, uv);
                    }
                    const float s = sigmoid(gv), a = (gv < -87.0f ? -87.0f : gv) * s, t = dv * w;
                    dgate[e] = gate_free ? t * uv * __builtin_fmaf(a, 1.0f - s, s) : 0.0f;
                    dup[e] = up_free ? t * a : 0.0f;
                    act[e] = a * uv;
                    sum = __builtin_fmaf(dv, act[e], sum);
                    act[e] *= w;
                }
                dg2[k] = pack(dgate[0], dgate[1]);
                du2[k] = pack(dup[0], dup[1]);
                y2[k] = pack(act[0], act[1]);
            }
            store(p.dh + line + slot, dg2);
            store(p.dh + line + p.slots + slot, du2);
            if (p.y)
                store(p.y + (size_t)row * p.slots + slot, y2);
        }
        return sum;
    };
    uint32_t parity = 0;
    for (uint32_t row0 = blockIdx.x * kRows; row0 < p.n; row0 += gridDim.x * kRows, parity ^= 1u) {
        const uint32_t row = row0 + wave / W;
        float sum = row < p.n ? gradient(row) : 0.0f;
        if (!p.dweight) // the same for every thread, as row0 is
            continue;
#pragma unroll
        for (int m = kWaveSize / 2; m >= 1; m >>= 1)
            sum += __shfl_xor(sum, m);
        if constexpr (W > 1) {
            if (lane == 0)
                s_sum[parity][wave] = sum;
            __syncthreads();
            if (wave % W == 0)
#pragma unroll
                for (int i = 1; i < W; ++i)
                    sum += s_sum[parity][wave + i];
        }
        if (wave % W == 0 && lane == 0 && row < p.n)
            p.dweight[row] = sum;
    }
}

// Workgroups at most, each taking several rows from there on: a launch holds fewer than 2^32 work-items.
constexpr uint32_t kMaxBackwardBlocks = 1u << 20;

template <int FROM, bool CLAMP>
void launch_backward(const BackwardParams& p, hipStream_t s)
{
    // 32768 x 2048 115, 111 and 109 us with one, two and four waves a row, 1000 x 2048 8, 7 and 5, 16384 x 512 16, 17, 21
    auto blocks = [&](uint32_t rows) { return dim3(std::min((p.n + rows - 1u) / rows, kMaxBackwardBlocks)); };
    if (p.slots <= kWaveSize)
        hipLaunchKernelGGL((swiglu_backward_kernel<FROM, CLAMP, 1>), blocks(4), dim3(kThreads), 0, s, p);
    else if (p.slots <= 2 * kWaveSize)
        hipLaunchKernelGGL((swiglu_backward_kernel<FROM, CLAMP, 2>), blocks(2), dim3(kThreads), 0, s, p);
    else
        hipLaunchKernelGGL((swiglu_backward_kernel<FROM, CLAMP, 4>), blocks(1), dim3(kThreads), 0, s, p);
}

} // namespace

extern "C" tk_status tk_swiglu_checkpoint_fp8(const void* x, const float* topk_weight, int64_t n, int64_t hidden,
                                              int64_t group_size, float clamp_limit, tk_scale_fmt scale_fmt,
                                              void* codes, void* scales, void* x_codes, void* x_scales, void* stream)
{
    if (n < 0 || n >= (int64_t)INT_MAX || hidden <= 0 || hidden % kSlotCols != 0 || hidden > (int64_t)INT_MAX / 4 ||
        group_size < 0 || (group_size != 0 && (group_size % kSlotCols != 0 || hidden % group_size != 0)) ||
        std::isnan(clamp_limit) || clamp_limit <= 0.0f || (int)scale_fmt < TK_SCALE_FP32 ||
        (int)scale_fmt > TK_SCALE_UE8M0_PACKED)
        return TK_ERR_INVALID_ARG;
    const bool f32 = (int)scale_fmt == TK_SCALE_FP32;
    if (n > 0 && (!x || !codes || !scales || !x_codes || !x_scales))
        return TK_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(topk_weight, 4) || !aligned(codes, 8) || !aligned(x_codes, 8) ||
        (f32 && (!aligned(scales, 4) || !aligned(x_scales, 4))))
        return TK_ERR_INVALID_ARG;
    if ((int)scale_fmt > TK_SCALE_UE8M0 || group_size == 0 || group_size > 512 || (group_size & (group_size - 1)) != 0)
        return TK_ERR_UNSUPPORTED;
    const int64_t groups = hidden / group_size;
    const void* const out[4] = {codes, scales, x_codes, x_scales};
    const size_t rows = (size_t)n, width = f32 ? 4u : 1u;
    const size_t bytes[4] = {rows * (size_t)hidden, rows * (size_t)groups * width, rows * (size_t)hidden * 2u,
                             rows * (size_t)groups * 2u * width};
    for (int i = 0; i < 4; ++i) {
        if (overlaps(out[i], bytes[i], x, rows * (size_t)hidden * 4u) ||
            overlaps(out[i], bytes[i], topk_weight, rows * 4u))
            return TK_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i], bytes[i], out[j], bytes[j]))
                return TK_ERR_INVALID_ARG;
    }
    const uint32_t slots = (uint32_t)(hidden / kSlotCols), steps = (slots + kWaveSize - 1) / kWaveSize;
    // Four steps a wave where that leaves a wave of the card four units or more: 32768 x 2048 87 us (88 with one or two),
    // 1000 x 2048 8.0 (6.0 with one).
    const int spu = steps % 4 == 0 && (uint64_t)n * (steps / 4) >= 16384 ? 4 : 1;
    if ((uint64_t)n * (steps / spu) >= (uint64_t)INT_MAX)
        return TK_ERR_UNSUPPORTED;
    if (n == 0)
        return TK_OK;
    const float2* table = nullptr;
    int cus = 0;
    const tk_status rc = sigma_table(table, cus);
    if (rc != TK_OK)
        return rc;
    Params p{};
    p.x = static_cast<const uint4*>(x);
    p.w = topk_weight;
    p.codes = static_cast<uint8_t*>(codes);
    p.scales = scales;
    p.slots = slots;
    p.upr = steps / spu;
    p.units = (uint32_t)n * p.upr;
    p.gl_log2 = (uint32_t)__builtin_ctz((uint32_t)group_size / kSlotCols);
    p.groups_row = (uint32_t)groups;
    p.clamp = clamp_limit;
    p.scale_layout = kScaleRowMajor;
    Params px = p;
    px.codes = static_cast<uint8_t*>(x_codes);
    px.scales = x_scales;
    px.groups_row = 2u * p.groups_row;
    const uint32_t want = (p.units + kThreads / kWaveSize - 1) / (kThreads / kWaveSize), most = (uint32_t)cus * 4u;
    const uint32_t blocks = want < most ? want : most;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool clamp = !std::isinf(clamp_limit);
    if (f32)
        clamp ? launch_checkpoint<TK_SCALE_FP32, true>(p, px, table, spu, blocks, s)
              : launch_checkpoint<TK_SCALE_FP32, false>(p, px, table, spu, blocks, s);
    else
        clamp ? launch_checkpoint<TK_SCALE_UE8M0, true>(p, px, table, spu, blocks, s)
              : launch_checkpoint<TK_SCALE_UE8M0, false>(p, px, table, spu, blocks, s);
    return hipGetLastError() == hipSuccess ? TK_OK : TK_ERR_HIP;
}

extern "C" tk_status tk_swiglu_backward(const void* dy, const void* h, const void* h_scales, int h_dtype,
                                        tk_scale_fmt scale_fmt, int64_t group_size, const float* topk_weight,
                                        int64_t n, int64_t hidden, float clamp_limit, void* dh, float* dweight,
                                        void* y, void* stream)
{
    const bool fp8 = h_dtype == TK_DTYPE_FP8, f32 = (int)scale_fmt == TK_SCALE_FP32;
    if (n < 0 || n > (int64_t)INT_MAX || hidden <= 0 || hidden % 8 != 0 || hidden > 1 << 18 ||
        (!fp8 && h_dtype != TK_DTYPE_BF16) || std::isnan(clamp_limit) || clamp_limit <= 0.0f)
        return TK_ERR_INVALID_ARG;
    if (fp8 && ((int)scale_fmt < TK_SCALE_FP32 || (int)scale_fmt > TK_SCALE_UE8M0_PACKED || group_size < 0 ||
                (group_size && (group_size % 8 != 0 || 2 * hidden % group_size != 0))))
        return TK_ERR_INVALID_ARG;
    if (n > 0 && (!dy || !h || !dh || (fp8 && !h_scales)))
        return TK_ERR_INVALID_ARG;
    if (!aligned(dy, 16) || !aligned(h, 16) || !aligned(dh, 16) || !aligned(y, 16) || !aligned(topk_weight, 4) ||
        !aligned(dweight, 4) || (fp8 && f32 && !aligned(h_scales, 4)))
        return TK_ERR_INVALID_ARG;
    if (fp8 && (int)scale_fmt > TK_SCALE_UE8M0)
        return TK_ERR_UNSUPPORTED;
    const int64_t group = fp8 && group_size ? group_size : 2 * hidden;
    const size_t rows = (size_t)n, cols = (size_t)hidden;
    const size_t dy_bytes = rows * cols * 2u, h_bytes = rows * cols * (fp8 ? 2u : 4u);
    const size_t s_bytes = fp8 ? rows * (size_t)(2 * hidden / group) * (f32 ? 4u : 1u) : 0u;
    const void* const out[3] = {dh, dweight, y};
    const size_t bytes[3] = {rows * cols * 4u, dweight ? rows * 4u : 0u, y ? dy_bytes : 0u};
    for (int i = 0; i < 3; ++i) {
        // dh over h in bf16 and y over dy are element for element
        if ((!(i == 2 && y == dy) && overlaps(out[i], bytes[i], dy, dy_bytes)) ||
            (!(i == 0 && !fp8 && dh == h) && overlaps(out[i], bytes[i], h, h_bytes)) ||
            overlaps(out[i], bytes[i], h_scales, s_bytes) || overlaps(out[i], bytes[i], topk_weight, rows * 4u))
            return TK_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlaps(out[i], bytes[i], out[j], bytes[j]))
                return TK_ERR_INVALID_ARG;
    }
    if (n == 0)
        return TK_OK;
    BackwardParams p{};
    p.dy = static_cast<const uint4*>(dy);
    p.h = h;
    p.h_scales = h_scales;
    p.weight = topk_weight;
    p.dh = static_cast<uint4*>(dh);
    p.dweight = dweight;
    p.y = static_cast<uint4*>(y);
    p.n = (uint32_t)n;
    p.slots = (uint32_t)(hidden / 8);
    p.groups = (uint32_t)(2 * hidden / group);
    const uint32_t width = (uint32_t)(group / 8);
    p.magic = width == 1 ? 0u : 0xFFFFFFFFu / width + 1u; // exact, slots and widths being 2^16 at most
    p.clamp = clamp_limit;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool clamp = !std::isinf(clamp_limit);
    const int from = !fp8 ? kFromBf16 : f32 ? kFromF32 : kFromE8;
    switch (from * 2 + clamp) {
    case 0: launch_backward<kFromBf16, false>(p, s); break;
    case 1: launch_backward<kFromBf16, true>(p, s); break;
    case 2: launch_backward<kFromF32, false>(p, s); break;
    case 3: launch_backward<kFromF32, true>(p, s); break;
    case 4: launch_backward<kFromE8, false>(p, s); break;
    default: launch_backward<kFromE8, true>(p, s); break;
    }
    return hipGetLastError() == hipSuccess ? TK_OK : TK_ERR_HIP;
}
