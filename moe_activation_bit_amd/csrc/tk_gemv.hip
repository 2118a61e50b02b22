// tk_gemv.hip -- the experts' matrix-vector products with 4-bit weights, behind
// tk_expert_gemv_fp4 in include/tk_layer.h.
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>

#include "tk.h"
#include "tk_layer.h"
#include "tk_quant.h"

namespace {

using namespace tk_detail;

typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kXBf16 = 0, kXFp8F32 = 1, kXFp8E8 = 2; // how x is held

struct GemvParams {
    const void* x;
    const void* x_scales;
    const int32_t* idx;  // or null
    const uint8_t* codes;
    const void* scales;
    void* out;
    uint32_t rows;       // tokens * k
    uint32_t k;
    uint32_t x_div;      // out row r reads x row r / x_div
    uint32_t experts;
    uint32_t out_features;
    uint32_t in_features;
    uint32_t group, groups;     // weights: columns a scale, scales a row
    uint32_t x_group, x_groups;
    int x_kind, scale_u8, out_bf16;
};

// the value of a UE8M0 byte: 2^(b - 127), 255 NaN
__device__ __forceinline__ float e8m0(uint32_t b) { return b == 0u ? 0x1p-127f : b == 255u ? as_float(0x7FC00000u) : as_float(b << 23); }

// One wave per output value; a lane takes 32-column blocks 64 apart.
__global__ __launch_bounds__(kThreads) void gemv_fp4_simple_kernel(GemvParams p)
{
    const uint32_t lane = threadIdx.x & (kWaveSize - 1);
    const uint32_t o = blockIdx.x * (kThreads / kWaveSize) + threadIdx.x / kWaveSize;
    if (o >= p.out_features)
        return;
    for (uint32_t r = blockIdx.y; r < p.rows; r += gridDim.y) {
        const int32_t e = p.idx ? p.idx[r] : 0;
        float acc = 0.0f;
        if ((uint32_t)e < p.experts) {
            const size_t wrow = (size_t)(uint32_t)e * p.out_features + o;
            const size_t xrow = r / p.x_div;
            const uint4* wp = reinterpret_cast<const uint4*>(p.codes + wrow * (p.in_features / 2));
            for (uint32_t b = lane; b < p.in_features / 32; b += kWaveSize) {
                const size_t si = wrow * p.groups + b * 32 / p.group;
                const float sw = p.scale_u8 ? e8m0(static_cast<const uint8_t*>(p.scales)[si]) : static_cast<const float*>(p.scales)[si];
                float sx = 1.0f;
                if (p.x_kind != kXBf16) {
                    const size_t xi = xrow * p.x_groups + b * 32 / p.x_group;
                    sx = p.x_kind == kXFp8E8 ? e8m0(static_cast<const uint8_t*>(p.x_scales)[xi]) : static_cast<const float*>(p.x_scales)[xi];
                }
                const uint4 q = wp[b];
                const uint32_t w4[4] = {q.x, q.y, q.z, q.w};
                float part = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f32x2 w[4], x[4];
                    w[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w4[i], 1.0f, 0);
                    w[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w4[i], 1.0f, 1);
                    w[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w4[i], 1.0f, 2);
                    w[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w4[i], 1.0f, 3);
                    const size_t at = xrow * p.in_features + b * 32 + 8 * i;
                    if (p.x_kind == kXBf16) {
                        const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) + at);
                        const uint32_t v4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            x[j] = f32x2{as_float(v4[j] << 16), as_float(v4[j] & 0xFFFF0000u)};
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.x) + at);
                        x[0] = __builtin_amdgcn_cvt_pk_f32_fp8((int)v.x, false);
                        x[1] = __builtin_amdgcn_cvt_pk_f32_fp8((int)v.x, true);
                        x[2] = __builtin_amdgcn_cvt_pk_f32_fp8((int)v.y, false);
                        x[3] = __builtin_amdgcn_cvt_pk_f32_fp8((int)v.y, true);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        part = __builtin_fmaf(w[j].x, x[j].x, part);
                        part = __builtin_fmaf(w[j].y, x[j].y, part);
                    }
                }
                acc = __builtin_fmaf(part, sw * sx, acc);
            }
        }
#pragma unroll
        for (int m = 1; m < kWaveSize; m <<= 1)
            acc += __shfl_xor(acc, m);
        if (lane == 0) {
            const size_t at = (size_t)r * p.out_features + o;
            if (p.out_bf16)
                static_cast<__bf16*>(p.out)[at] = (__bf16)acc;
            else
                static_cast<float*>(p.out)[at] = acc;
        }
    }
}

// A group width's columns a scale; 0 when the kernels do not take it.
int64_t group_columns(int64_t group, int64_t in, bool u8)
{
    if (group == 0 || group == in)
        return in;
    return group % (u8 ? 32 : 128) == 0 ? group : 0;
}

} // namespace

extern "C" tk_status tk_expert_gemv_fp4(const void* x, const void* x_scales, int x_dtype, tk_scale_fmt x_scale_fmt,
                                        int64_t x_group, const int32_t* topk_idx, int64_t tokens, int64_t k,
                                        int x_slots, const void* codes, const void* scales, tk_scale_fmt scale_fmt,
                                        int64_t group_size, int64_t experts, int64_t out_features,
                                        int64_t in_features, tk_dtype out_dtype, void* out, void* stream)
{
    // ---- validation: no HIP call before every argument is checked ----
    const bool fp8 = x_dtype == TK_DTYPE_FP8;
    if (!fp8 && x_dtype != TK_DTYPE_BF16)
        return TK_ERR_INVALID_ARG;
    if ((int)out_dtype != TK_DTYPE_BF16 && (int)out_dtype != TK_DTYPE_FP32)
        return TK_ERR_INVALID_ARG;
    if ((int)scale_fmt < TK_SCALE_FP32 || (int)scale_fmt > TK_SCALE_UE8M0_PACKED ||
        (fp8 && ((int)x_scale_fmt < TK_SCALE_FP32 || (int)x_scale_fmt > TK_SCALE_UE8M0_PACKED)))
        return TK_ERR_INVALID_ARG;
    if (tokens < 0 || k <= 0 || tokens >= (int64_t)INT_MAX || k >= (int64_t)INT_MAX || tokens * k >= (int64_t)INT_MAX ||
        (x_slots != 0 && x_slots != 1) || (!topk_idx && k != 1))
        return TK_ERR_INVALID_ARG;
    if (experts <= 0 || experts > (1 << 20) || out_features <= 0 || out_features > (1 << 24) || in_features <= 0 ||
        in_features > (1 << 20) || in_features % 32 != 0)
        return TK_ERR_INVALID_ARG;
    if (group_size < 0 || (group_size != 0 && in_features % group_size != 0) ||
        (fp8 && (x_group < 0 || (x_group != 0 && in_features % x_group != 0))))
        return TK_ERR_INVALID_ARG;
    if (tokens > 0 && (!x || !codes || !scales || !out || (fp8 && !x_scales)))
        return TK_ERR_INVALID_ARG;
    const bool u8 = (int)scale_fmt == TK_SCALE_UE8M0, xu8 = (int)x_scale_fmt == TK_SCALE_UE8M0;
    const bool out_bf16 = (int)out_dtype == TK_DTYPE_BF16;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(topk_idx, 4) || !aligned(out, out_bf16 ? 2 : 4) ||
        (!u8 && !aligned(scales, 4)) || (fp8 && !xu8 && !aligned(x_scales, 4)))
        return TK_ERR_INVALID_ARG;
    if (((int)scale_fmt != TK_SCALE_FP32 && !u8) || (fp8 && (int)x_scale_fmt != TK_SCALE_FP32 && !xu8) || k > 64)
        return TK_ERR_UNSUPPORTED;
    const int64_t group = group_columns(group_size, in_features, u8);
    const int64_t xgroup = fp8 ? group_columns(x_group, in_features, xu8) : in_features;
    if (!group || !xgroup)
        return TK_ERR_UNSUPPORTED;
    const int64_t rows = tokens * k, x_rows = x_slots ? rows : tokens;
    const size_t w_rows = (size_t)experts * (size_t)out_features;
    const size_t o_bytes = (size_t)rows * (size_t)out_features * (out_bf16 ? 2u : 4u);
    if (overlaps(out, o_bytes, x, (size_t)x_rows * (size_t)in_features * (fp8 ? 1u : 2u)) ||
        overlaps(out, o_bytes, codes, w_rows * (size_t)(in_features / 2)) ||
        overlaps(out, o_bytes, scales, w_rows * (size_t)(in_features / group) * (u8 ? 1u : 4u)) ||
        overlaps(out, o_bytes, topk_idx, (size_t)rows * 4u) ||
        (fp8 && overlaps(out, o_bytes, x_scales, (size_t)x_rows * (size_t)(in_features / xgroup) * (xu8 ? 1u : 4u))))
        return TK_ERR_INVALID_ARG;
    if (tokens == 0)
        return TK_OK;

    GemvParams p{};
    p.x = x;
    p.x_scales = x_scales;
    p.idx = topk_idx;
    p.codes = static_cast<const uint8_t*>(codes);
    p.scales = scales;
    p.out = out;
    p.rows = (uint32_t)rows;
    p.k = (uint32_t)k;
    p.x_div = x_slots ? 1u : (uint32_t)k;
    p.experts = (uint32_t)experts;
    p.out_features = (uint32_t)out_features;
    p.in_features = (uint32_t)in_features;
    p.group = (uint32_t)group;
    p.groups = (uint32_t)(in_features / group);
    p.x_group = (uint32_t)xgroup;
    p.x_groups = (uint32_t)(in_features / xgroup);
    p.x_kind = fp8 ? (xu8 ? kXFp8E8 : kXFp8F32) : kXBf16;
    p.scale_u8 = u8;
    p.out_bf16 = out_bf16;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const uint32_t per = kThreads / kWaveSize;
    hipLaunchKernelGGL(gemv_fp4_simple_kernel,
                       dim3((p.out_features + per - 1) / per, p.rows < 65535u ? p.rows : 65535u), dim3(kThreads), 0, s, p);
    return hipGetLastError() == hipSuccess ? TK_OK : TK_ERR_HIP;
}
