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
    uint32_t group_magic, x_group_magic;       // of the groups' width in blocks of 32 columns
    uint32_t group_magic128, x_group_magic128; // ... in steps of 128
    uint32_t steps;      // of kBlock columns, the last part-filled when in_features is no multiple
    uint32_t steps_wave; // a wave's share of them
    uint32_t ks;         // waves that share a tile's columns: 1, 2 or 4
    uint32_t grid_y;     // rows, or experts and one more
    int by_row;
};

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));

// q / d by d's magic()
__device__ __forceinline__ uint32_t divide(uint32_t q, uint32_t magic) { return magic ? __umulhi(q, magic) : q; }

constexpr int kTile = 16;   // weight rows and x rows of a matrix instruction
constexpr int kBlock = 128; // columns of a step

// Matrix instructions on 16 weight rows at a time, for up to 16 * NT of the
// rows that chose the expert.  In a step of 128 columns lane (r, q) = (l & 15,
// l >> 4) holds weight row r's 32 codes of columns 32q.. (16 bytes, within one
// group) and x row r's same columns.  Codes and FP8 activations become bf16 in
// registers, with their UE8M0 scales on the way: both are exact (two and four
// significant bits), and the products and sums of the four 16x16x32 bf16
// instructions of a step are those of fp32.  (The E2M1 x E4M3 instruction would
// take the codes as they are, but drops what lies 2^-14 below the largest
// product of a step: random E4M3 bytes gave sums off by up to 7.7e-5 of their
// terms' magnitude, where the bf16 instructions were exact.)
// fp32 scales enter afterwards: one scale a row in the epilogue, one for 128
// columns or a multiple of that (PART) on each step's own result.
// A result's column n (x row) is lane & 15, its rows 4q .. 4q + 3.
//   WS 0: UE8M0, groups of 32, whole pairs of steps: a pair's eight scales of a
//     row are one load;  1: any group width;  2: a last step part-filled too.
template <bool FP8X, bool PART, int NT, int WS>
struct GemvWave {
    const GemvParams& p;
    uint32_t r, q;
    const uint8_t* w_row;  // this lane's weight row
    const uint8_t* s_row;  // its UE8M0 scales
    const char* x_row[NT]; // this lane's x rows
    const void* xs_row[NT];
    size_t tile_row;       // the tile's first row of weights, over all experts
    v4f acc[NT];

    __device__ __forceinline__ explicit GemvWave(const GemvParams& pp) : p(pp) {}

    __device__ __forceinline__ uint32_t w_scale(uint32_t b) const
    {
        if (!p.scale_u8)
            return 127u;
        const uint32_t g = min(4u * b + q, p.in_features / 32u - 1u);
        return s_row[divide(g, p.group_magic)];
    }
    __device__ __forceinline__ uint32_t x_scale(int nt, uint32_t b) const
    {
        if (p.x_kind != kXFp8E8)
            return 127u;
        const uint32_t g = min(4u * b + q, p.in_features / 32u - 1u);
        return static_cast<const uint8_t*>(xs_row[nt])[divide(g, p.x_group_magic)];
    }
    // the 16 bytes at column c of a row, zeros past its end
    __device__ __forceinline__ uint4 load(const char* row, uint32_t c, uint32_t bytes_num, uint32_t bytes_den) const
    {
        if (WS == 2 && c >= p.in_features)
            return make_uint4(0, 0, 0, 0);
        return *reinterpret_cast<const uint4*>(row + (size_t)c * bytes_num / bytes_den);
    }

    template <int U>
    __device__ __forceinline__ void steps(uint32_t b, uint32_t ntiles)
    {
        uint4 w[U];
        uint32_t ws[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            w[u] = load(reinterpret_cast<const char*>(w_row), (b + u) * kBlock + 32u * q, 1, 2);
        if constexpr (WS == 0) {
#pragma unroll
            for (int u = 0; u < U; u += 2) {
                const uint2 s = *reinterpret_cast<const uint2*>(s_row + 4u * (b + u));
                ws[u] = (s.x >> (8u * q)) & 255u;
                ws[U > 1 ? u + 1 : 0] = (s.y >> (8u * q)) & 255u;
            }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
                ws[u] = w_scale(b + u);
        }
        // fp32 scales of the weights by group, for the result's four rows
        float sw[PART ? U : 1][4];
        const bool w_part = PART && !p.scale_u8 && p.groups > 1;
        if constexpr (PART) {
            if (w_part) {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const size_t row = min(tile_row + 4u * q + i, (size_t)p.experts * p.out_features - 1u);
                        sw[u][i] = static_cast<const float*>(p.scales)[row * p.groups + divide(b + u, p.group_magic128)];
                    }
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (NT > 1 && (uint32_t)nt >= ntiles)
                break; // wave-uniform
#pragma unroll
            for (int u = 0; u < U; ++u) {
                v4f c = PART ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : acc[nt];
                const float s = as_float(ws[u] << 23); // only the exponent is looked at: 0 is 2^-127, 255 NaN
                const uint32_t w4[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
                const uint32_t col = (b + u) * kBlock + 32u * q;
                v8b B[4];
                if constexpr (FP8X) {
                    const uint4 x0 = load(x_row[nt], col, 1, 1), x1 = load(x_row[nt], col + 16u, 1, 1);
                    const uint32_t x8[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
                    const float sx = as_float(x_scale(nt, b + u) << 23);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const v2b a0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x8[2 * i], sx, false);
                        const v2b a1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x8[2 * i], sx, true);
                        const v2b a2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x8[2 * i + 1], sx, false);
                        const v2b a3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x8[2 * i + 1], sx, true);
                        B[i] = v8b{a0[0], a0[1], a1[0], a1[1], a2[0], a2[1], a3[0], a3[1]};
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        B[i] = __builtin_bit_cast(v8b, load(x_row[nt], col + 8u * i, 2, 1));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const v2b a0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w4[i], s, 0);
                    const v2b a1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w4[i], s, 1);
                    const v2b a2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w4[i], s, 2);
                    const v2b a3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w4[i], s, 3);
                    const v8b A = {a0[0], a0[1], a1[0], a1[1], a2[0], a2[1], a3[0], a3[1]};
                    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A, B[i], c, 0, 0, 0);
                }
                if constexpr (PART) {
                    const float sx = FP8X && p.x_kind == kXFp8F32 && p.x_groups > 1
                                         ? static_cast<const float*>(xs_row[nt])[divide(b + u, p.x_group_magic128)]
                                         : 1.0f;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[nt][i] = __builtin_fmaf(c[i], w_part ? sx * sw[u][i] : sx, acc[nt][i]);
                } else {
                    acc[nt] = c;
                }
            }
        }
    }
};

// One workgroup: KS waves along the columns of each of 4 / KS tiles of 16
// weight rows.  Its rows are those whose expert is e, in order, 16 * NT at a
// time.  by_row: blockIdx.y is a row, and the first row of an expert does the
// work of all of them; else blockIdx.y is an expert, and the one past the last
// writes the absent rows' zeros.
template <bool FP8X, bool PART, int NT, int WS>
__global__ __launch_bounds__(kThreads) void gemv_fp4_kernel(GemvParams p)
{
    constexpr uint32_t kWaves = kThreads / kWaveSize, kRows = kTile * NT;
    __shared__ uint32_t s_list[kWaves][kRows];
    __shared__ v4f s_acc[kWaves][NT][kWaveSize];
    const uint32_t lane = threadIdx.x & (kWaveSize - 1);
    const uint32_t wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveSize);
    const uint32_t ks = wv & (p.ks - 1u), rt = wv / p.ks;
    const uint32_t o0 = (blockIdx.x * (kWaves / p.ks) + rt) * kTile; // this wave's first weight row of the expert
    const uint64_t below = (1ull << lane) - 1u;

    for (uint32_t y = blockIdx.y; y < p.grid_y; y += gridDim.y) {
        uint32_t e = 0, next = 0;
        if (p.idx) {
            if (p.by_row) {
                next = y;
                e = (uint32_t)p.idx[y];
                bool earlier = false;
                for (uint32_t base = 0; base < y; base += kWaveSize)
                    earlier |= base + lane < y && (uint32_t)p.idx[base + lane] == e;
                if (e < p.experts && __builtin_amdgcn_ballot_w64(earlier) != 0)
                    continue; // an earlier row's workgroup does this one (the same for all its waves)
            } else {
                e = y;
            }
        }
        if (e >= p.experts) { // absent rows: this one, or all of them
            for (uint32_t row = p.by_row ? y : 0u; row < (p.by_row ? y + 1u : p.rows); ++row) {
                if ((uint32_t)p.idx[row] < p.experts)
                    continue;
                const uint32_t o = blockIdx.x * (kWaves / p.ks) * kTile + threadIdx.x;
                if (threadIdx.x < (kWaves / p.ks) * kTile && o < p.out_features) {
                    if (p.out_bf16)
                        static_cast<uint16_t*>(p.out)[(size_t)row * p.out_features + o] = 0;
                    else
                        static_cast<float*>(p.out)[(size_t)row * p.out_features + o] = 0.0f;
                }
            }
            continue;
        }
        while (true) {
            // ---- the next rows of this expert, at most kRows
            uint32_t n = 0;
            while (next < p.rows && n < kRows) {
                const uint32_t base = next & ~(uint32_t)(kWaveSize - 1), row = base + lane;
                const bool hit = row >= next && row < p.rows && (!p.idx || (uint32_t)p.idx[row] == e);
                const uint64_t mask = __builtin_amdgcn_ballot_w64(hit);
                const uint32_t rank = n + (uint32_t)__builtin_popcountll(mask & below);
                if (hit && rank < kRows)
                    s_list[wv][rank] = row;
                const uint64_t left = __builtin_amdgcn_ballot_w64(hit && rank >= kRows);
                next = left ? base + (uint32_t)__builtin_ctzll(left) : base + kWaveSize;
                n = left ? kRows : n + (uint32_t)__builtin_popcountll(mask);
            }
            if (n == 0)
                break; // the same for every wave of the workgroup
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();

            GemvWave<FP8X, PART, NT, WS> g(p);
            g.r = lane & 15u;
            g.q = lane >> 4;
            g.tile_row = (size_t)e * p.out_features + o0;
            const size_t w_row = (size_t)e * p.out_features + min(o0 + g.r, p.out_features - 1u);
            g.w_row = p.codes + w_row * (p.in_features / 2u);
            g.s_row = static_cast<const uint8_t*>(p.scales) + (p.scale_u8 ? w_row * p.groups : 0u);
            uint32_t row[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // columns past the last row repeat it and are not stored
                row[nt] = s_list[wv][min(nt * kTile + g.r, n - 1u)];
                const size_t xr = row[nt] / p.x_div;
                g.x_row[nt] = static_cast<const char*>(p.x) + xr * p.in_features * (FP8X ? 1u : 2u);
                g.xs_row[nt] = static_cast<const char*>(p.x_scales) + xr * p.x_groups * (p.x_kind == kXFp8F32 ? 4u : 1u);
                g.acc[nt] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            }
            const uint32_t ntiles = (n + kTile - 1) / kTile;
            if (o0 < p.out_features) {
                uint32_t b = ks * p.steps_wave;
                const uint32_t end = min(b + p.steps_wave, p.steps);
                for (; b + 4 <= end; b += 4)
                    g.template steps<4>(b, ntiles);
                if (b + 2 <= end) {
                    g.template steps<2>(b, ntiles);
                    b += 2;
                }
                if constexpr (WS != 0)
                    if (b < end)
                        g.template steps<1>(b, ntiles);
            }
            // ---- the waves' sums over the columns meet, in their order
            if (p.ks > 1) {
                __syncthreads();
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    s_acc[wv][nt][lane] = g.acc[nt];
                __syncthreads();
                if (ks != 0)
                    continue;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    for (uint32_t i = 1; i < p.ks; ++i) {
                        const v4f a = s_acc[wv + i][nt][lane];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            g.acc[nt][j] += a[j];
                    }
            }
            // ---- scales of whole rows, and the results
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (nt * kTile + g.r >= n)
                    continue;
                float sx = 1.0f;
                if (FP8X && p.x_kind == kXFp8F32 && p.x_groups == 1)
                    sx = *static_cast<const float*>(g.xs_row[nt]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t o = o0 + 4u * g.q + i;
                    if (o >= p.out_features)
                        continue;
                    float v = g.acc[nt][i] * sx;
                    if (!p.scale_u8 && p.groups == 1)
                        v *= static_cast<const float*>(p.scales)[g.tile_row + 4u * g.q + i];
                    const size_t at = (size_t)row[nt] * p.out_features + o;
                    if (p.out_bf16)
                        static_cast<__bf16*>(p.out)[at] = (__bf16)v;
                    else
                        static_cast<float*>(p.out)[at] = v;
                }
            }
        }
    }
}

template <bool FP8X, bool PART, int NT>
void launch_gemv(int ws, const GemvParams& p, dim3 grid, hipStream_t s)
{
    if (ws == 0)
        hipLaunchKernelGGL((gemv_fp4_kernel<FP8X, PART, NT, 0>), grid, dim3(kThreads), 0, s, p);
    else if (ws == 1)
        hipLaunchKernelGGL((gemv_fp4_kernel<FP8X, PART, NT, 1>), grid, dim3(kThreads), 0, s, p);
    else
        hipLaunchKernelGGL((gemv_fp4_kernel<FP8X, PART, NT, 2>), grid, dim3(kThreads), 0, s, p);
}

template <bool FP8X, bool PART>
void launch_gemv_nt(int nt, int ws, const GemvParams& p, dim3 grid, hipStream_t s)
{
    if (nt == 1)
        launch_gemv<FP8X, PART, 1>(ws, p, grid, s);
    else if (nt == 2)
        launch_gemv<FP8X, PART, 2>(ws, p, grid, s);
    else
        launch_gemv<FP8X, PART, 4>(ws, p, grid, s);
}

// ceil(2^32 / d), by which divide() is exact for q * d < 2^32; 0 stands for d = 1.
uint32_t magic(uint32_t d) { return d <= 1 ? 0u : (uint32_t)(((1ull << 32) + d - 1) / d); }

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
    p.group_magic = magic(p.group / 32u);
    p.x_group_magic = magic(p.x_group / 32u);
    p.group_magic128 = magic(p.group / kBlock);
    p.x_group_magic128 = magic(p.x_group / kBlock);
    p.steps = (p.in_features + kBlock - 1) / kBlock;
    // Columns are split over waves by the sizes alone, never by the number of
    // tokens, so that a row's sum has one order.
    const uint64_t waves = (uint64_t)p.k * ((p.out_features + kTile - 1) / kTile);
    p.ks = waves >= 4096 ? 1u : waves >= 2048 ? 2u : 4u;
    while (p.ks > 1 && p.steps < 2 * p.ks)
        p.ks >>= 1;
    p.steps_wave = (p.steps + p.ks - 1) / p.ks;
    p.steps_wave += p.steps_wave & 1u; // whole pairs
    p.by_row = topk_idx && rows <= experts;
    p.grid_y = !topk_idx ? 1u : p.by_row ? p.rows : p.experts + 1u;
    const bool part = (fp8 && !xu8 && p.x_groups > 1) || (!u8 && p.groups > 1);
    const int ws = p.in_features % kBlock != 0                                      ? 2
                   : u8 && group == 32 && in_features % 256 == 0 && aligned(scales, 8) ? 0
                                                                                     : 1;
    // x tiles of a pass by the rows an expert has on average
    const uint64_t load = topk_idx ? (uint64_t)rows / (uint64_t)experts : (uint64_t)rows;
    const int nt = tokens <= kTile || load <= 8 ? 1 : tokens <= 2 * kTile || load <= 24 ? 2 : 4;
    const uint32_t tiles_wg = kThreads / kWaveSize / p.ks;
    const dim3 grid((p.out_features + kTile * tiles_wg - 1) / (kTile * tiles_wg), p.grid_y < 65535u ? p.grid_y : 65535u);
    if (fp8)
        part ? launch_gemv_nt<true, true>(nt, ws, p, grid, s) : launch_gemv_nt<true, false>(nt, ws, p, grid, s);
    else
        part ? launch_gemv_nt<false, true>(nt, ws, p, grid, s) : launch_gemv_nt<false, false>(nt, ws, p, grid, s);
    return hipGetLastError() == hipSuccess ? TK_OK : TK_ERR_HIP;
}
