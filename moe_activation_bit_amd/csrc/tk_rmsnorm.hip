// tk_rmsnorm.hip -- residual addition + root-mean-square norm + FP8 cast and
// its gradient, behind tk_rmsnorm_cast_fp8 and tk_rmsnorm_backward in
// include/tk_layer.h.
//
// Forward, per row: h = x + residual (rounded to the stream's type), rstd =
// 1/sqrt(mean h^2 + eps), y = h * rstd * weight, then the abs-max -> scale ->
// code tail of the casts (tk_quant.h).  A row is held in registers between its
// sum and its cast, so every input is read and every output written once.
// Backward: dx = rstd * (g - a * mean(g*a)) + dresidual with g = dy * weight and
// a = rstd * h, and dweight = sum over the rows of dy * a: of many rows gathered
// by each workgroup over its own in registers, written as one partial row, and
// summed over the partial rows by a second kernel in their order; of few rows by
// workgroups of their own in the same launch.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "tk.h"
#include "tk_layer.h"
#include "tk_quant.h"

namespace {

using namespace tk_detail;

constexpr uint32_t kMaxBlocks = 1u << 20;
constexpr int64_t kMaxHidden = 32768; // 16 waves of 4 steps of 512 columns

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf16_lo(uint32_t w) { return as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return as_float(w & 0xFFFF0000u); }

// two floats rounded to bf16 (nearest even), the first in the low half
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// The lane slot's 8 columns as they lie in memory, and as fp32.
template <bool F32>
struct Slot {
    uint4 raw[F32 ? 2 : 1];

    __device__ __forceinline__ void load(const void* base, size_t slot)
    {
        const uint4* p = static_cast<const uint4*>(base) + (F32 ? 2 : 1) * slot;
        raw[0] = load16(p);
        if constexpr (F32)
            raw[F32 ? 1 : 0] = load16(p + 1);
    }
    __device__ __forceinline__ void load_cached(const void* base, size_t slot)
    {
        const uint4* p = static_cast<const uint4*>(base) + (F32 ? 2 : 1) * slot;
        raw[0] = *p;
        if constexpr (F32)
            raw[F32 ? 1 : 0] = p[1];
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        if constexpr (F32) {
            const uint4 a = raw[0], b = raw[F32 ? 1 : 0];
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = as_float(w[j]);
        } else {
            const uint32_t w[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = bf16_lo(w[j]);
                v[2 * j + 1] = bf16_hi(w[j]);
            }
        }
    }
};
__device__ __forceinline__ void load_weight(const float* weight, uint32_t slot, float (&w)[8])
{
    const float4* const p = reinterpret_cast<const float4*>(weight) + 2 * slot;
    const float4 a = p[0], b = p[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
}
template <bool F32>
__device__ __forceinline__ void load_slot(const void* base, size_t slot, float (&v)[8])
{
    Slot<F32> s;
    s.load(base, slot);
    s.get(v);
}

// ... and the 8 columns written, rounded to the type.
template <bool F32>
__device__ __forceinline__ void store_slot(void* base, size_t slot, const float (&v)[8])
{
    if constexpr (F32) {
        v4u* p = static_cast<v4u*>(base) + 2 * slot;
        const v4u a = {as_uint(v[0]), as_uint(v[1]), as_uint(v[2]), as_uint(v[3])};
        const v4u b = {as_uint(v[4]), as_uint(v[5]), as_uint(v[6]), as_uint(v[7])};
        __builtin_nontemporal_store(a, p);
        __builtin_nontemporal_store(b, p + 1);
    } else {
        const v4u a = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
        __builtin_nontemporal_store(a, static_cast<v4u*>(base) + slot);
    }
}

template <int CTRL>
__device__ __forceinline__ double dpp_add(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, false);
    return v + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v)
{
    return v + as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)as_uint(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ double read_lane(double v, int lane)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), lane);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ float read_lane(float v, int lane)
{
    return as_float(__builtin_amdgcn_readlane(as_uint(v), lane));
}

// sum over each row of 16 lanes, in every lane of it (every lane active), in a fixed order
template <typename T>
__device__ __forceinline__ T row_sum(T v)
{
    v = dpp_add<0xB1>(v);  // quad_perm [1,0,3,2]: lane ^ 1
    v = dpp_add<0x4E>(v);  // quad_perm [2,3,0,1]: lane ^ 2
    v = dpp_add<0x141>(v); // row_half_mirror
    return dpp_add<0x140>(v); // row_mirror
}
// ... over all 64 lanes
template <typename T>
__device__ __forceinline__ T wave_sum(T v)
{
    v = row_sum(v);
    return (read_lane(v, 0) + read_lane(v, 16)) + (read_lane(v, 32) + read_lane(v, 48));
}

// 1/sqrt(m) to within a few units of the 64-bit last place: the hardware's
// estimate refined twice by Newton's iteration.  0, infinity and NaN keep the
// estimate's own limit values.
__device__ __forceinline__ double rsqrt64(double m)
{
    const double r0 = __builtin_amdgcn_rsq(m);
    double r = r0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        r = r * __builtin_fma(-0.5 * m * r, r, 1.5);
    return (m > 0.0 && m < (double)INFINITY) ? r : r0;
}

struct NormParams {
    Params q;              // codes, scales and their layout
    const void* x;
    const void* residual;  // or null
    const float* weight;
    void* residual_out;    // or null
    void* y;               // or null
    float* rstd;           // or null
    uint32_t n;
    uint32_t waves;        // waves per row; 1: every wave of the workgroup has a row of its own
    double inv_hidden;
    double eps;
};

constexpr int kGroupRow = 0;   // one scale per row
constexpr int kGroupLanes = 1; // groups of 2^gl_log2 lanes of one step
constexpr int kGroupLds = 2;   // any other width: the slots' maxima meet in LDS

// One row per `waves` waves: step s of wave w of a row is slots
// (s * waves + w) * 64 .. + 63, a lane holding 8 columns of each of its S steps.
// Of rows of up to 16 steps each step's sum of squares is taken by itself, since
// there S goes by the number of rows too: squares of fp32 fill 48 bits, so that
// another order of their sum can show in 64.
template <bool F32, int S, int GM, int SFMT, int MAXT>
__global__ __launch_bounds__(MAXT) void rmsnorm_cast_kernel(NormParams p)
{
    constexpr int P = S <= 2 ? S : 1;
    __shared__ double part_sum[2][16]; // by the parity of the pass, so that one barrier a pass is enough
    __shared__ uint32_t part_max[2][16];
    extern __shared__ uint32_t dyn[]; // kGroupLds: each row's slot maxima, then its groups' multipliers
    const uint32_t lane = threadIdx.x & (kWaveSize - 1);
    const uint32_t wib = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveSize);
    const uint32_t rows = p.waves == 1 ? blockDim.x / kWaveSize : 1u; // rows of this workgroup
    const uint32_t part = p.waves == 1 ? 0u : wib;
    const uint32_t row_in = p.waves == 1 ? wib : 0u;
    const bool by_step = P > 1 && P * p.waves <= 16u; // else a wave's steps together
    const uint32_t parts = by_step ? P * p.waves : p.waves;
    uint32_t parity = 0;
    // rows past the grid (a launch holds fewer than 2^32 work-items) take further passes
    for (uint32_t first = blockIdx.x * rows; first < p.n; first += gridDim.x * rows, parity ^= 1u) {
        const uint32_t row = first + row_in;
        const bool valid = row < p.n; // wave-uniform; waves without a row still meet the barriers
        const uint32_t slots = p.q.slots;
        const size_t row_slot = (size_t)row * slots;

        float v[S][8], w[S][8];
        double sums[P] = {};
    #pragma unroll
        for (int s = 0; s < S; ++s) {
            double& sum = sums[s % P];
            const uint32_t slot = ((uint32_t)s * p.waves + part) * kWaveSize + lane;
    #pragma unroll
            for (int j = 0; j < 8; ++j)
                v[s][j] = 0.0f, w[s][j] = 0.0f;
            if (valid && slot < slots) {
                load_slot<F32>(p.x, row_slot + slot, v[s]);
                load_weight(p.weight, slot, w[s]);
                if (p.residual) {
                    float r[8];
                    load_slot<F32>(p.residual, row_slot + slot, r);
    #pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[s][j] += r[j];
                    if constexpr (!F32) { // the norm is of the stream as it is stored
    #pragma unroll
                        for (int j = 0; j < 8; j += 2) {
                            const uint32_t b2 = pack_bf16(v[s][j], v[s][j + 1]);
                            v[s][j] = bf16_lo(b2);
                            v[s][j + 1] = bf16_hi(b2);
                        }
                    }
                }
                if (p.residual_out)
                    store_slot<F32>(p.residual_out, row_slot + slot, v[s]);
    #pragma unroll
                for (int j = 0; j < 8; ++j)
                    sum = __builtin_fma((double)v[s][j], (double)v[s][j], sum);
            }
        }
        double sum = wave_sum(by_step ? sums[0] : sums[0] + (P > 1 ? sums[P - 1] : 0.0));
        if (p.waves > 1) {
            if (lane == 0)
                part_sum[parity][wib] = sum;
            if (by_step) {
                sum = wave_sum(sums[P - 1]);
                if (lane == 0)
                    part_sum[parity][p.waves + wib] = sum;
            }
            __syncthreads();
            const uint32_t i = lane & 15u;
            sum = row_sum(i < parts ? part_sum[parity][i] : 0.0); // steps past the row's end are zero, too
        }
        const float rstd = (float)rsqrt64(__builtin_fma(sum, p.inv_hidden, p.eps));
        if (valid && p.rstd && part == 0 && lane == 0)
            p.rstd[row] = rstd;

        uint32_t m[S];
    #pragma unroll
        for (int s = 0; s < S; ++s) {
            const uint32_t slot = ((uint32_t)s * p.waves + part) * kWaveSize + lane;
            m[s] = 0;
    #pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[s][j] = (v[s][j] * rstd) * w[s][j];
                m[s] = max(m[s], as_uint(v[s][j]) & 0x7FFFFFFFu);
            }
            if (!(valid && slot < slots))
                m[s] = 0;
            else if (p.y)
                store_slot<false>(p.y, row_slot + slot, v[s]);
        }
        if (!p.q.codes)
            continue; // the whole grid
        uint8_t* row_codes = p.q.codes + (size_t)row * slots * 8u;

        if constexpr (GM == kGroupRow) {
            uint32_t mb = wave_umax(lane_max<S>(m, S));
            if (p.waves > 1) {
                if (lane == 0)
                    part_max[parity][wib] = mb;
                __syncthreads();
                for (uint32_t i = 0; i < p.waves; ++i)
                    mb = max(mb, part_max[parity][i]);
            }
            float s32 = 0.0f;
            uint32_t s8 = 0;
            const float inv = group_scale<8, SFMT>(mb, s32, s8);
            if (valid && part == 0 && lane == 0)
                store_scale<SFMT>(p.q, row, 0, s32, s8);
    #pragma unroll
            for (int s = 0; s < S; ++s) {
                const uint32_t slot = ((uint32_t)s * p.waves + part) * kWaveSize + lane;
                if (valid && slot < slots)
                    quantize_store<8>(row_codes, slot, v[s], inv);
            }
        } else if constexpr (GM == kGroupLanes) {
    #pragma unroll
            for (int s = 0; s < S; ++s) {
                const uint32_t slot = ((uint32_t)s * p.waves + part) * kWaveSize + lane;
                float s32 = 0.0f;
                uint32_t s8 = 0;
                const float inv = group_scale<8, SFMT>(group_umax(m[s], p.q.gl_log2), s32, s8);
                if (valid && slot < slots) {
                    quantize_store<8>(row_codes, slot, v[s], inv);
                    if ((lane & ((1u << p.q.gl_log2) - 1u)) == 0)
                        store_scale<SFMT>(p.q, row, slot >> p.q.gl_log2, s32, s8);
                }
            }
        } else {
            const uint32_t gs = p.q.gslots, ngr = p.q.groups_row;
            uint32_t* buf = dyn + (size_t)row_in * (slots + ngr);
            float* invs = reinterpret_cast<float*>(buf + slots);
    #pragma unroll
            for (int s = 0; s < S; ++s) {
                const uint32_t slot = ((uint32_t)s * p.waves + part) * kWaveSize + lane;
                if (slot < slots)
                    buf[slot] = m[s];
            }
            __syncthreads();
            // 2^l_log2 lanes of one wave reduce a group, each a run of its slots
            const uint32_t lanes = p.waves * kWaveSize, at = part * kWaveSize + lane;
            uint32_t l_log2 = 0;
            while (l_log2 < 6 && (ngr << (l_log2 + 1)) <= lanes)
                ++l_log2;
            const uint32_t lpg = 1u << l_log2, chunk = (gs + lpg - 1u) >> l_log2;
            for (uint32_t base = 0; base < ngr; base += lanes >> l_log2) {
                const uint32_t k = base + (at >> l_log2), sub = at & (lpg - 1u);
                uint32_t mb = 0;
                if (k < ngr) {
                    const uint32_t e = min(k * gs + (sub + 1u) * chunk, (k + 1u) * gs);
                    for (uint32_t i = k * gs + sub * chunk; i < e; ++i)
                        mb = max(mb, buf[i]);
                }
                mb = group_umax(mb, l_log2);
                if (k < ngr && sub == 0) {
                    float s32 = 0.0f;
                    uint32_t s8 = 0;
                    invs[k] = group_scale<8, SFMT>(mb, s32, s8);
                    if (valid)
                        store_scale<SFMT>(p.q, row, k, s32, s8);
                }
            }
            __syncthreads();
    #pragma unroll
            for (int s = 0; s < S; ++s) {
                const uint32_t slot = ((uint32_t)s * p.waves + part) * kWaveSize + lane;
                if (valid && slot < slots)
                    quantize_store<8>(row_codes, slot, v[s], invs[__umulhi(slot, p.q.gmagic)]);
            }
        }
    }
}

struct NormBwdParams {
    const void* dy;
    const void* h;
    const float* weight;
    const float* rstd;
    const void* dresidual; // or null
    void* dx;
    float* partial;        // [gridDim.x][hidden], or null
    uint32_t n;
    uint32_t slots;
    float inv_hidden;
    // the short form's
    float* dweight;
    uint32_t column_blocks; // workgroups that sum dweight, before those of the rows
    uint32_t col_lanes_log2; // lanes that share a row's part in those, two columns each
    uint32_t waves;         // that share a row
    uint32_t rows;          // of a workgroup
    uint32_t first_row;     // of the launch
    int cached;             // the rows are read through the caches, as the columns are
};

// One row per pass of a workgroup, rows blockIdx.x, + gridDim.x, ...; the rows'
// dy * a sums stay in registers.  Rows of up to 16 steps (S = 1) keep the
// weight there too and have the next row's dy, h and dresidual on their way
// while the waves' parts of a row's dot meet; longer ones have no registers for
// either.  MANY: rows of up to four steps, p.rows of them a pass, so that a CU
// has waves enough (16384 x 512 in bf16 15.9 us instead of 28.0, x 1024 26.2
// instead of 34.8, x 2048 47.2 instead of 59.5).  Bound by the bytes of the
// rows: a workgroup a CU, since each writes a partial row (8192 x 4096 47.6 us
// with 256 of them, 51.8 with 512).
template <bool F32, int S, bool SKIP, bool MANY>
__global__ __launch_bounds__(MANY ? 512 : 1024) void rmsnorm_backward_kernel(NormBwdParams p)
{
    constexpr bool AHEAD = S == 1;
    __shared__ float part_dot[2][16];
    const uint32_t lane = threadIdx.x & (kWaveSize - 1);
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveSize);
    const uint32_t waves = p.waves, rows = MANY ? p.rows : 1u;
    const uint32_t local = MANY ? wave / waves : 0u, wib = wave - local * waves; // row of a pass, part of the row
    float w[AHEAD ? S : 1][8], dw[S][8];
    uint32_t slot[S]; // lanes past the row's end read its last slot and add nothing to the dot
#pragma unroll
    for (int s = 0; s < S; ++s) {
        slot[s] = ((uint32_t)s * waves + wib) * kWaveSize + lane;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            dw[s][j] = 0.0f;
        if constexpr (AHEAD)
            load_weight(p.weight, min(slot[s], p.slots - 1u), w[s]);
    }
    Slot<F32> dy[S], h[S], skip[SKIP ? S : 1];
    float rstd = 0.0f;
    auto fetch_skip = [&](uint32_t row) {
        if constexpr (SKIP) {
#pragma unroll
            for (int s = 0; s < S; ++s)
                skip[s].load(p.dresidual, (size_t)row * p.slots + min(slot[s], p.slots - 1u));
        }
    };
    auto fetch = [&](uint32_t row) {
        rstd = p.rstd[row];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const size_t at = (size_t)row * p.slots + min(slot[s], p.slots - 1u);
            dy[s].load(p.dy, at);
            h[s].load(p.h, at);
        }
        if constexpr (AHEAD)
            fetch_skip(row);
    };
    if constexpr (AHEAD)
        fetch(min(blockIdx.x * rows + local, p.n - 1u));
    uint32_t parity = 0;
    for (uint32_t base = blockIdx.x * rows; base < p.n; base += gridDim.x * rows, parity ^= 1u) {
        const uint32_t row = base + local;
        const bool valid = !MANY || row < p.n; // else the last row again, unused
        if constexpr (!AHEAD)
            fetch(row);
        const float r = rstd;
        float a[S][8], g[S][8], d[AHEAD && SKIP ? S : 1][8];
        float dot = 0.0f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            dy[s].get(g[s]);
            h[s].get(a[s]);
            if constexpr (AHEAD && SKIP)
                skip[s].get(d[s]);
            if constexpr (!AHEAD)
                load_weight(p.weight, min(slot[s], p.slots - 1u), w[0]);
            float part = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a[s][j] *= r;
                dw[s][j] = valid ? dw[s][j] + g[s][j] * a[s][j] : dw[s][j];
                g[s][j] *= w[AHEAD ? s : 0][j];
                part += g[s][j] * a[s][j];
            }
            dot += slot[s] < p.slots ? part : 0.0f;
        }
        if constexpr (AHEAD)
            fetch(min(row + gridDim.x * rows, p.n - 1u));
        else
            fetch_skip(row);
        dot = wave_sum(dot);
        if (waves > 1) {
            if (lane == 0)
                part_dot[parity][wave] = dot;
            __syncthreads();
            dot = 0.0f;
            for (uint32_t i = 0; i < waves; ++i)
                dot += part_dot[parity][wave - wib + i];
        }
        const float mean = dot * p.inv_hidden;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float e[8];
            if constexpr (!AHEAD && SKIP)
                skip[s].get(e);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                g[s][j] = r * (g[s][j] - a[s][j] * mean);
                if constexpr (SKIP)
                    g[s][j] += AHEAD ? d[AHEAD ? s : 0][j] : e[j];
            }
            if (valid && slot[s] < p.slots)
                store_slot<F32>(p.dx, (size_t)row * p.slots + slot[s], g[s]);
        }
    }
    if constexpr (MANY) { // the rows' sums meet in their order
        __shared__ float s_dw[8][kWaveSize * 8];
        if (p.partial) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s_dw[wave][j * kWaveSize + lane] = dw[0][j];
            __syncthreads();
            if (local != 0)
                return;
            for (uint32_t i = 1; i < rows; ++i) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    dw[0][j] += s_dw[i * waves + wib][j * kWaveSize + lane];
            }
        }
    }
    if (p.partial) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if (slot[s] < p.slots) {
                float4* o = reinterpret_cast<float4*>(p.partial + ((size_t)blockIdx.x * p.slots + slot[s]) * 8u);
                o[0] = make_float4(dw[s][0], dw[s][1], dw[s][2], dw[s][3]);
                o[1] = make_float4(dw[s][4], dw[s][5], dw[s][6], dw[s][7]);
            }
        }
    }
}

// dweight[c] = the partial rows' sum: 16 waves of a workgroup share 64 columns,
// wave w taking partial rows w, w + 16, ... (16 of them in flight), then their
// sums in wave order.  parts == 0 writes zeros.
__global__ __launch_bounds__(1024) void rmsnorm_dweight_kernel(const float* __restrict__ partial, uint32_t parts,
                                                              uint32_t hidden, float* __restrict__ dweight)
{
    constexpr uint32_t kBatch = 16;
    __shared__ float sums[16][kWaveSize];
    const uint32_t lane = threadIdx.x & (kWaveSize - 1), wv = threadIdx.x / kWaveSize;
    const uint32_t c = blockIdx.x * kWaveSize + lane;
    const float* const at = partial + min(c, hidden - 1u);
    float s = 0.0f;
    for (uint32_t i = wv; i < parts; i += 16 * kBatch) {
        float v[kBatch];
#pragma unroll
        for (uint32_t k = 0; k < kBatch; ++k)
            v[k] = at[(size_t)min(i + 16 * k, parts - 1u) * hidden];
#pragma unroll
        for (uint32_t k = 0; k < kBatch; ++k)
            s += i + 16 * k < parts ? v[k] : 0.0f;
    }
    sums[wv][lane] = s;
    __syncthreads();
    if (wv == 0 && c < hidden) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            s += sums[i][lane];
        dweight[c] = s;
    }
}

// Few rows, or very long ones: one launch for dx and dweight.  A partial row of
// dweight for each row or two would be more bytes than the rows themselves, so
// the first workgroups read dy and h again, from the caches, 32 or 64 columns
// each: every 16 or 32 lanes take a row at a time, eight rows in flight, and
// their sums meet in a fixed order.  The others take rows, as many as fit 16
// waves.  Bound by a launch and two trips to memory, later by the caches: 3 x
// 7168 in fp32 3.7 us (6.1 with partial rows and a second launch), 333 x 1024
// 4.4 (6.6), 356 x 8192 in bf16 9.4 (15.5).
template <bool F32, int S, bool SKIP>
__global__ __launch_bounds__(1024) void rmsnorm_backward_short_kernel(NormBwdParams p)
{
    __shared__ float sums[16][kWaveSize];
    const uint32_t lane = threadIdx.x & (kWaveSize - 1);
    const uint32_t wib = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveSize);
    if (blockIdx.x < p.column_blocks) {
        constexpr uint32_t kBatch = 8;
        const uint32_t hidden = p.slots * kSlotCols, lanes = 1u << p.col_lanes_log2;
        const uint32_t part = threadIdx.x >> p.col_lanes_log2, parts = 1024u >> p.col_lanes_log2;
        const uint32_t c = min(2u * (blockIdx.x * lanes + (lane & (lanes - 1u))), hidden - 2u);
        float s0 = 0.0f, s1 = 0.0f;
        for (uint32_t base = part; base < p.n; base += parts * kBatch) {
            float r[kBatch];
            uint2 dy[kBatch], h[kBatch]; // bf16: a word of each
#pragma unroll
            for (uint32_t k = 0; k < kBatch; ++k) {
                const uint32_t row = min(base + parts * k, p.n - 1u);
                const size_t at = (size_t)row * hidden + c;
                r[k] = p.rstd[row];
                if constexpr (F32) {
                    dy[k] = *reinterpret_cast<const uint2*>(static_cast<const float*>(p.dy) + at);
                    h[k] = *reinterpret_cast<const uint2*>(static_cast<const float*>(p.h) + at);
                } else {
                    dy[k].x = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.dy) + at);
                    h[k].x = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.h) + at);
                }
            }
            float b0 = 0.0f, b1 = 0.0f; // a batch's own sums first: long columns then lose less
#pragma unroll
            for (uint32_t k = 0; k < kBatch; ++k) {
                const bool in = base + parts * k < p.n;
                const float g0 = F32 ? as_float(dy[k].x) : bf16_lo(dy[k].x), a0 = F32 ? as_float(h[k].x) : bf16_lo(h[k].x);
                const float g1 = F32 ? as_float(dy[k].y) : bf16_hi(dy[k].x), a1 = F32 ? as_float(h[k].y) : bf16_hi(h[k].x);
                b0 = in ? b0 + g0 * (a0 * r[k]) : b0;
                b1 = in ? b1 + g1 * (a1 * r[k]) : b1;
            }
            s0 += b0;
            s1 += b1;
        }
        for (uint32_t x = lanes; x < kWaveSize; x <<= 1) {
            s0 += __shfl_xor(s0, x);
            s1 += __shfl_xor(s1, x);
        }
        if (lane < lanes) {
            sums[wib][2u * lane] = s0;
            sums[wib][2u * lane + 1u] = s1;
        }
        __syncthreads();
        const uint32_t o = 2u * blockIdx.x * lanes + lane;
        if (threadIdx.x < 2u * lanes && o < hidden) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                s += sums[i][lane];
            p.dweight[o] = s;
        }
        return;
    }
    const uint32_t local = wib / p.waves, part = wib - local * p.waves;
    const uint32_t mine = p.first_row + (blockIdx.x - p.column_blocks) * p.rows + local;
    const bool valid = local < p.rows && mine < p.n;
    const uint32_t row = min(mine, p.n - 1u);
    uint32_t slot[S];
    Slot<F32> dy[S], h[S], skip[SKIP ? S : 1];
    const float r = p.rstd[row];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        slot[s] = ((uint32_t)s * p.waves + part) * kWaveSize + lane;
        const size_t at = (size_t)row * p.slots + min(slot[s], p.slots - 1u);
        if (p.cached) {
            dy[s].load_cached(p.dy, at);
            h[s].load_cached(p.h, at);
        } else {
            dy[s].load(p.dy, at);
            h[s].load(p.h, at);
        }
        if constexpr (SKIP)
            skip[s].load(p.dresidual, at);
    }
    float a[S][8], g[S][8], dot = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        float w[8], sum = 0.0f;
        dy[s].get(g[s]);
        h[s].get(a[s]);
        load_weight(p.weight, min(slot[s], p.slots - 1u), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            a[s][j] *= r;
            g[s][j] *= w[j];
            sum += g[s][j] * a[s][j];
        }
        dot += slot[s] < p.slots ? sum : 0.0f;
    }
    dot = wave_sum(dot);
    if (p.waves > 1) {
        if (lane == 0)
            sums[0][wib] = dot;
        __syncthreads();
        dot = 0.0f;
        for (uint32_t i = 0; i < p.waves; ++i)
            dot += sums[0][min(local * p.waves + i, 15u)];
    }
    const float mean = dot * p.inv_hidden;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        float d[8];
        if constexpr (SKIP)
            skip[s].get(d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            g[s][j] = r * (g[s][j] - a[s][j] * mean);
            if constexpr (SKIP)
                g[s][j] += d[j];
        }
        if (valid && slot[s] < p.slots)
            store_slot<F32>(p.dx, (size_t)row * p.slots + slot[s], g[s]);
    }
}

template <bool F32, int S, int MAXT, int GM>
void launch_norm(int sfmt, const NormParams& p, dim3 grid, dim3 block, size_t lds, hipStream_t s)
{
    if (sfmt == TK_SCALE_FP32)
        hipLaunchKernelGGL((rmsnorm_cast_kernel<F32, S, GM, TK_SCALE_FP32, MAXT>), grid, block, lds, s, p);
    else
        hipLaunchKernelGGL((rmsnorm_cast_kernel<F32, S, GM, TK_SCALE_UE8M0, MAXT>), grid, block, lds, s, p);
}

template <bool F32, int S, int MAXT>
void launch_norm_gm(int gm, int sfmt, const NormParams& p, dim3 grid, dim3 block, size_t lds, hipStream_t s)
{
    if (gm == kGroupRow)
        launch_norm<F32, S, MAXT, kGroupRow>(sfmt, p, grid, block, 0, s);
    else if (gm == kGroupLanes)
        launch_norm<F32, S, MAXT, kGroupLanes>(sfmt, p, grid, block, 0, s);
    else
        launch_norm<F32, S, MAXT, kGroupLds>(sfmt, p, grid, block, lds, s);
}

template <bool F32, int S>
void launch_norm_backward(bool together, bool skip, const NormBwdParams& p, dim3 grid, dim3 block, hipStream_t s)
{
    if (together) {
        if (skip)
            hipLaunchKernelGGL((rmsnorm_backward_short_kernel<F32, S, true>), grid, block, 0, s, p);
        else
            hipLaunchKernelGGL((rmsnorm_backward_short_kernel<F32, S, false>), grid, block, 0, s, p);
        return;
    }
    if constexpr (S == 1) {
        if (p.rows > 1) {
            if (skip)
                hipLaunchKernelGGL((rmsnorm_backward_kernel<F32, S, true, true>), grid, block, 0, s, p);
            else
                hipLaunchKernelGGL((rmsnorm_backward_kernel<F32, S, false, true>), grid, block, 0, s, p);
            return;
        }
    }
    if constexpr (S <= 2) {
        if (skip)
            hipLaunchKernelGGL((rmsnorm_backward_kernel<F32, S, true, false>), grid, block, 0, s, p);
        else
            hipLaunchKernelGGL((rmsnorm_backward_kernel<F32, S, false, false>), grid, block, 0, s, p);
    }
}

// The steps a lane holds of a row of `steps` 512-column steps: `pref`, more
// where 16 waves would not cover the row.
uint32_t steps_per_wave(uint32_t steps, uint32_t pref)
{
    uint32_t S = pref;
    while ((steps + S - 1) / S > 16)
        S <<= 1;
    return S;
}

} // namespace

extern "C" {

tk_status tk_rmsnorm_cast_fp8(const void* x, const void* residual, tk_dtype in_dtype, const float* weight, int64_t n,
                              int64_t hidden, float eps, int64_t group_size, tk_scale_fmt scale_fmt,
                              void* residual_out, void* y, float* rstd, void* codes, void* scales, void* stream)
{
    // ---- validation: no HIP call before every argument is checked ----
    if (n < 0 || n >= (int64_t)INT_MAX || hidden <= 0 || hidden % kSlotCols != 0 || hidden > (int64_t)INT_MAX / 8)
        return TK_ERR_INVALID_ARG;
    if (group_size < 0 || (group_size != 0 && (group_size % kSlotCols != 0 || hidden % group_size != 0)))
        return TK_ERR_INVALID_ARG;
    if ((int)in_dtype != TK_DTYPE_BF16 && (int)in_dtype != TK_DTYPE_FP32)
        return TK_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !std::isfinite(eps))
        return TK_ERR_INVALID_ARG;
    const int64_t groups = hidden / (group_size ? group_size : hidden);
    ScaleSpec sp;
    if (!scale_spec((int)scale_fmt, n, groups, sp))
        return TK_ERR_INVALID_ARG;
    if (n > 0 && (!x || !weight || (!codes != !scales) || (!codes && !residual_out && !y && !rstd)))
        return TK_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(residual_out, 16) ||
        !aligned(y, 16) || !aligned(rstd, 4) || !aligned(codes, 8) || !aligned(scales, sp.align))
        return TK_ERR_INVALID_ARG;
    const bool f32 = (int)in_dtype == TK_DTYPE_FP32;
    const size_t elems = (size_t)n * (size_t)hidden, t_bytes = elems * (f32 ? 4u : 2u);
    if (n > 0) {
        struct Span {
            const void* p;
            size_t bytes;
        };
        const Span in[] = {{x, t_bytes}, {residual, t_bytes}, {weight, (size_t)hidden * 4u}};
        const Span out[] = {{residual_out, t_bytes}, {y, elems * 2u}, {rstd, (size_t)n * 4u}, {codes, elems},
                            {scales, sp.bytes}};
        for (int i = 0; i < 5; ++i) {
            for (int j = 0; j < 3; ++j) {
                if (i == 0 && j < 2 && out[i].p == in[j].p)
                    continue; // the stream updated in place
                if (overlaps(out[i].p, out[i].bytes, in[j].p, in[j].bytes))
                    return TK_ERR_INVALID_ARG;
            }
            for (int j = 0; j < i; ++j)
                if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
                    return TK_ERR_INVALID_ARG;
        }
    }
    if (hidden > kMaxHidden)
        return TK_ERR_UNSUPPORTED;
    if (n == 0)
        return TK_OK;

    NormParams p{};
    p.x = x;
    p.residual = residual;
    p.weight = weight;
    p.residual_out = residual_out;
    p.y = y;
    p.rstd = rstd;
    p.n = (uint32_t)n;
    p.inv_hidden = 1.0 / (double)hidden;
    p.eps = (double)eps;
    p.q.codes = static_cast<uint8_t*>(codes);
    p.q.scales = scales;
    p.q.scale_layout = sp.layout;
    p.q.scale_ld = sp.ld;
    p.q.slots = (uint32_t)(hidden / kSlotCols);
    p.q.groups_row = (uint32_t)groups;
    p.q.gslots = p.q.slots / p.q.groups_row;
    int gm = kGroupLds;
    if (groups == 1) {
        gm = kGroupRow;
    } else if ((p.q.gslots & (p.q.gslots - 1)) == 0 && p.q.gslots <= (uint32_t)kWaveSize) {
        gm = kGroupLanes;
        p.q.gl_log2 = (uint32_t)__builtin_ctz(p.q.gslots);
    } else {
        p.q.gmagic = (uint32_t)(((1ull << 32) + p.q.gslots - 1) / p.q.gslots);
    }
    const uint32_t steps = (p.q.slots + kWaveSize - 1) / kWaveSize;
    // One step a wave for rows of up to four and for launches too small to fill the chip, else two: in bf16 with every
    // output 16384 x 7168 200 / 191 / 191 us at 1 / 2 / 4 steps, 512 x 7168 8.2 / 8.0 / 9.8, 16384 x 4096 with the
    // stream and the codes 83.9 / 83.5 / 90.0, 57344 x 2048 178 / - / 181.
    const uint32_t S = steps_per_wave(steps, steps <= 4 || n < 512 ? 1u : 2u);
    p.waves = (steps + S - 1) / S;
    const uint32_t rows = p.waves == 1 ? 4u : 1u;
    const uint32_t blocks = (p.n + rows - 1) / rows;
    const dim3 grid(blocks < kMaxBlocks ? blocks : kMaxBlocks), block(rows * p.waves * kWaveSize);
    const size_t lds = (size_t)rows * (p.q.slots + p.q.groups_row) * 4u;
    hipStream_t s = static_cast<hipStream_t>(stream);
#define TK_NORM(SS, T)                                                          \
    f32 ? launch_norm_gm<true, SS, T>(gm, sp.kind, p, grid, block, lds, s)      \
        : launch_norm_gm<false, SS, T>(gm, sp.kind, p, grid, block, lds, s)
    if (S == 4) // more than 32 steps: nine waves or more
        TK_NORM(4, 1024);
    else if (S == 2)
        block.x <= 256 ? (TK_NORM(2, 256)) : (TK_NORM(2, 1024));
    else
        block.x <= 256 ? (TK_NORM(1, 256)) : (TK_NORM(1, 1024));
#undef TK_NORM
    return hipGetLastError() == hipSuccess ? TK_OK : TK_ERR_HIP;
}

tk_status tk_rmsnorm_backward(const void* dy, const void* h, tk_dtype in_dtype, const float* weight,
                              const float* rstd, const void* dresidual, int64_t n, int64_t hidden, void* dx,
                              float* dweight, float* workspace, void* stream)
{
    if (n < 0 || n >= (int64_t)INT_MAX || hidden <= 0 || hidden % kSlotCols != 0 || hidden > (int64_t)INT_MAX / 8)
        return TK_ERR_INVALID_ARG;
    if ((int)in_dtype != TK_DTYPE_BF16 && (int)in_dtype != TK_DTYPE_FP32)
        return TK_ERR_INVALID_ARG;
    if (n > 0 && (!dy || !h || !weight || !rstd || !dx || (dweight && !workspace)))
        return TK_ERR_INVALID_ARG;
    if (!aligned(dy, 16) || !aligned(h, 16) || !aligned(weight, 16) || !aligned(rstd, 4) || !aligned(dresidual, 16) ||
        !aligned(dx, 16) || !aligned(dweight, 16) || !aligned(workspace, 16))
        return TK_ERR_INVALID_ARG;
    const bool f32 = (int)in_dtype == TK_DTYPE_FP32;
    const size_t t_bytes = (size_t)n * (size_t)hidden * (f32 ? 4u : 2u), w_bytes = (size_t)hidden * 4u;
    uint32_t parts = (uint32_t)(n < TK_RMSNORM_PARTS ? n : TK_RMSNORM_PARTS);
    const size_t ws_bytes = dweight ? (size_t)parts * w_bytes : 0;
    {
        const void* in[] = {dy, h, dresidual, weight, rstd};
        const size_t in_bytes[] = {t_bytes, t_bytes, t_bytes, w_bytes, (size_t)n * 4u};
        const void* out[] = {dx, dweight, workspace};
        const size_t out_bytes[] = {t_bytes, w_bytes, ws_bytes};
        for (int i = 0; i < 3; ++i) {
            for (int j = 0; j < 5; ++j) {
                if (i == 0 && (j == 0 || j == 2) && out[i] == in[j])
                    continue; // a gradient replaced in place
                if (overlaps(out[i], out_bytes[i], in[j], in_bytes[j]))
                    return TK_ERR_INVALID_ARG;
            }
            for (int j = 0; j < i; ++j)
                if (overlaps(out[i], out_bytes[i], out[j], out_bytes[j]))
                    return TK_ERR_INVALID_ARG;
        }
    }
    if (hidden > kMaxHidden)
        return TK_ERR_UNSUPPORTED;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (n > 0) {
        NormBwdParams p{};
        p.dy = dy;
        p.h = h;
        p.weight = weight;
        p.rstd = rstd;
        p.dresidual = dresidual;
        p.dx = dx;
        p.partial = dweight ? workspace : nullptr;
        p.n = (uint32_t)n;
        p.slots = (uint32_t)(hidden / kSlotCols);
        p.inv_hidden = 1.0f / (float)hidden;
        const uint32_t steps = (p.slots + kWaveSize - 1) / kWaveSize;
        const uint32_t S = steps_per_wave(steps, 1u);
        p.waves = (steps + S - 1) / S;
        p.rows = p.waves <= 4 ? 8u / p.waves : 1u;
        const uint32_t passes = ((uint32_t)n + p.rows - 1u) / p.rows;
        parts = passes < TK_RMSNORM_PARTS ? passes : TK_RMSNORM_PARTS;
        dim3 grid(parts), block(p.rows * p.waves * kWaveSize);
        // Whether dweight is summed beside the rows: so and by partial rows, in bf16, 512 x 1024 3.7 / 6.1 us, 1024 x
        // 1024 4.4 / 6.6, 500 x 4096 8.2 / 9.7, 512 x 8192 10.4 / 14.8, 300 x 16384 15.2 / 19.4, 2048 x 1024 14.3 / 8.1;
        // in fp32 512 x 7168 16.3 / 21.6, 2048 x 1024 16.6 / 11.8.  Near the border the other form is up to 1.3 times as
        // fast: bf16 1024 x 2048 10.0 / 8.7, 700 x 7168 12.9 / 15.2, fp32 640 x 4096 12.3 / 16.2.  Beyond 16384
        // columns always: a wave has no registers left for their sums (2048 x 32768 133 us, with them spilled 326).
        const bool together = (dweight && n <= 1024 && n * hidden <= (n <= 512 ? 5 << 20 : 2 << 20)) || S == 4;
#define TK_NORM_BWD(SS)                                                      \
    case SS:                                                                 \
        f32 ? launch_norm_backward<true, SS>(together, dresidual != nullptr, p, grid, block, s)  \
            : launch_norm_backward<false, SS>(together, dresidual != nullptr, p, grid, block, s); \
        break;
        auto launch = [&] {
            switch (S) {
                TK_NORM_BWD(1)
                TK_NORM_BWD(2)
                TK_NORM_BWD(4)
            }
        };
        if (together) {
            p.partial = nullptr;
            p.dweight = dweight;
            // bf16 500 x 4096 8.5 us through the caches, past them 9.4, 1024 x 1536 8.1 / 11.0, fp32 512 x 5120 11.7 /
            // 15.1; bf16 1024 x 1024 7.0 / 4.9
            p.cached = n * hidden > 1 << 20;
            p.rows = 16u / p.waves;
            // 32 columns or 64: fp32 333 x 1024 4.5 / 6.5 us, 1024 x 4096 19.5 / 24.0, 320 x 7168 15.9 / 14.7;
            // bf16 1024 x 1024 4.9 / 6.4, 1024 x 4096 14.8 / 15.1, 320 x 7168 10.1 / 7.9
            p.col_lanes_log2 = hidden <= 4096 ? 4u : 5u;
            p.column_blocks = dweight ? (uint32_t)(hidden + (2 << p.col_lanes_log2) - 1) >> (p.col_lanes_log2 + 1) : 0u;
            block = dim3(1024);
            if (dweight && dx == dy) { // dweight first: it reads dy, which the rows write
                grid = dim3(p.column_blocks);
                launch();
                p.column_blocks = 0;
            }
            // a launch holds fewer than 2^32 work-items
            for (uint32_t row_blocks = ((uint32_t)n + p.rows - 1u) / p.rows; row_blocks;) {
                const uint32_t now = row_blocks < kMaxBlocks ? row_blocks : kMaxBlocks;
                grid = dim3(p.column_blocks + now);
                launch();
                p.column_blocks = 0;
                p.first_row += now * p.rows;
                row_blocks -= now;
            }
        } else {
            launch();
        }
#undef TK_NORM_BWD
        if (hipGetLastError() != hipSuccess)
            return TK_ERR_HIP;
        if (together)
            return TK_OK;
    }
    if (dweight) {
        hipLaunchKernelGGL(rmsnorm_dweight_kernel, dim3((uint32_t)((hidden + kWaveSize - 1) / kWaveSize)), dim3(1024),
                           0, s, workspace, parts, (uint32_t)hidden, dweight);
        if (hipGetLastError() != hipSuccess)
            return TK_ERR_HIP;
    }
    return TK_OK;
}

} // extern "C"
