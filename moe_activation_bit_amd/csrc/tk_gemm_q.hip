// tk_gemm_q.hip -- the experts' matrix products of FP8 rows with FP8 or FP4
// weights over ragged rows, and the entry point tk_expert_gemm of
// include/tk_expert.h.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "tk_gemm_host.h"
#include "tk_gemm_tile.h"

namespace {

using namespace tk_gemm;

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));

constexpr uint32_t kDepth = 128; // k of a step and of a matrix instruction

// How an operand is scaled: one scale a row (applied to the finished sum), power-of-two scales of groups of 32 k
// or a multiple (in the instruction), fp32 scales of groups of 128 k or a multiple (on each step's sum).
constexpr int kScaleRow = 0, kScaleMx = 1, kScaleStep = 2;

struct Scales {
    const void* at; // row-major
    uint32_t groups;
    uint32_t width; // kScaleMx: blocks of 32 k a group; kScaleStep: steps
    int kind;
    int u8;
    int words; // kScaleMx: bytes can be read four at a time
};

struct QuantParams {
    const char* w;
    const char* x;
    const int32_t* index;
    const int32_t* offsets;
    void* out;
    Scales ws, xs;
    uint32_t x_rows, n_rows, experts, cols, depth;
};

__device__ __forceinline__ float e8m0_value(uint32_t b)
{
    return b == 0u ? 0x1p-127f : as_float(b == 255u ? 0x7FC00000u : b << 23);
}

// A finished sum times one scale a row of x and one of the weights.  Of x's, what is below 1 comes before the weights'
// and what is above behind it: two scales at the ends of the range, whose product is an ordinary number, do not
// overflow on the way.  (Nor do powers of two lose bits: a sum is a multiple of 2^-18, and a multiple of 2^-145
// below 2^-121 is a fp32 number.)
struct RowScale {
    float before, after;
    __device__ __forceinline__ explicit RowScale(float r) : before(r < 1.0f ? r : 1.0f), after(r < 1.0f ? 1.0f : r) {}
    __device__ __forceinline__ float operator()(float sum, float c_scale) const { return sum * before * c_scale * after; }
};

// Groups of any width (a scale of one step, read in front of its products, may serve many steps or a part of one), and
// UE8M0 bytes at any address.  The layout and the pace of gemm_kernel (tk_gemm.hip) with 128 k a step and two steps in
// LDS; bound by reading the scales: FP4 weights with scales of 32 columns, one row of each of 64 experts 7168 -> 4096,
// 299 us where gemm_q_turn_kernel takes 227.
// W4: weights in FP4.  STEP: one operand has fp32 scales of groups (the other, or both, have power-of-two ones).
template <bool W4, bool STEP, int TC, int TR, int WC, int WR>
__global__ __launch_bounds__(64 * WC * WR) void gemm_q_kernel(QuantParams p)
{
    constexpr uint32_t kWaves = WC * WR, kThr = 64 * kWaves;
    constexpr int NC = TC / WC / 16, NR = TR / WR / 16;
    constexpr uint32_t kRowC = W4 ? 64 : 128; // bytes of a weight row's step
    constexpr uint32_t kBytesC = TC * kRowC, kBytesR = TR * 128;
    constexpr int kCopiesC = (kBytesC / 1024 + kWaves - 1) / kWaves, kCopiesR = (kBytesR / 1024 + kWaves - 1) / kWaves;
    constexpr bool kEvenC = kBytesC / 1024 % kWaves == 0, kEvenR = kBytesR / 1024 % kWaves == 0;
    constexpr int kOwn = (TC + TR + kThr - 1) / kThr; // rows whose scales a thread fetches
    __shared__ __attribute__((aligned(1024))) char s_c[2][kBytesC];
    __shared__ __attribute__((aligned(1024))) char s_r[2][kBytesR];
    __shared__ uint32_t s_mx[2][TC + TR];
    __shared__ __attribute__((aligned(16))) float s_step[STEP ? 2 : 1][STEP ? TC + TR : 1];

    const uint32_t lane = threadIdx.x & (kWaveSize - 1), r = lane & 15u, q = lane >> 4;
    const uint32_t wave = uniform(threadIdx.x / kWaveSize), wc = wave % WC, wr = wave / WC;

    // ---- this workgroup's tile
    const uint32_t col_tiles = (p.cols + TC - 1) / TC;
    Group g;
    uint32_t t = 0;
    if (!find_group(p.offsets, p.experts, p.n_rows, TR,
                    [&](uint32_t total) {
                        t = xcd_tile(blockIdx.x, total * col_tiles);
                        return t / col_tiles;
                    },
                    g))
        return;
    const uint2 tile = tile_in_group(t - g.first * col_tiles, g.tiles, col_tiles);
    const uint32_t row0 = g.row0 + tile.x * TR, rows = min((uint32_t)TR, g.rows - tile.x * TR);
    const uint32_t col0 = tile.y * TC, depth = p.depth;
    const size_t w_row0 = (size_t)g.expert * p.cols + col0;

    auto source = [&](uint32_t row) { // x's row for a row of the tile; x_rows or more: none
        const uint32_t at = row0 + min(row, rows - 1u);
        return p.index ? (uint32_t)p.index[at] : at;
    };

    // ---- where each lane's copies come from (the 16 bytes c of row i lie at c ^ (i & 7); of an FP4 row's 64 bytes
    // at c ^ (-(i / 4) & 3): the 16 rows of a fragment meet in no bank)
    const uint32_t ld_c = W4 ? depth / 2u : depth;
    const char* const base_c = p.w + w_row0 * ld_c;
    uint32_t offset_c[kCopiesC], piece_c[kCopiesC], piece_r[kCopiesR], bad = 0;
    const char* from_r[kCopiesR];
#pragma unroll
    for (int i = 0; i < kCopiesC; ++i) {
        const uint32_t no = i * kWaves + wave;
        const uint32_t row = no * (W4 ? 16u : 8u) + (W4 ? lane >> 2 : lane >> 3);
        const uint32_t c = W4 ? (lane & 3u) ^ (-(lane >> 4) & 3u) : (lane & 7u) ^ (lane >> 3);
        piece_c[i] = c * (W4 ? 32u : 16u); // its first k
        offset_c[i] = min(row, p.cols - 1u - col0) * ld_c + c * 16u;
    }
#pragma unroll
    for (int i = 0; i < kCopiesR; ++i) {
        const uint32_t row = (i * kWaves + wave) * 8u + (lane >> 3), c = (lane & 7u) ^ (lane >> 3);
        uint32_t at = source(row);
        if (at >= p.x_rows) {
            at = 0;
            bad |= 1u << i;
        }
        piece_r[i] = c * 16u;
        from_r[i] = p.x + (size_t)at * depth + c * 16u;
    }
    const bool any_bad = __builtin_amdgcn_ballot_w64(bad != 0) != 0;

    auto fetch = [&](uint32_t t, uint32_t buf) {
        const bool whole = (t + 1u) * kDepth <= depth && !any_bad; // wave-uniform
        const size_t step_c = (size_t)t * kRowC, step_r = (size_t)t * 128u;
        auto each = [&](auto&& copy_c, auto&& copy_r) {
#pragma unroll
            for (int i = 0; i < kCopiesC; ++i)
                if (kEvenC || i * kWaves + wave < kBytesC / 1024)
                    copy_c(i, s_c[buf] + (i * kWaves + wave) * 1024u);
#pragma unroll
            for (int i = 0; i < kCopiesR; ++i)
                if (kEvenR || i * kWaves + wave < kBytesR / 1024)
                    copy_r(i, s_r[buf] + (i * kWaves + wave) * 1024u);
        };
        if (whole)
            each([&](int i, char* to) { copy_to_lds(base_c + step_c, offset_c[i], to); },
                 [&](int i, char* to) { copy_to_lds(from_r[i] + step_r, to); });
        else
            each(
                [&](int i, char* to) {
                    copy_to_lds(t * kDepth + piece_c[i] < depth ? base_c + step_c + offset_c[i] : zeros(), to);
                },
                [&](int i, char* to) {
                    copy_to_lds(t * kDepth + piece_r[i] < depth && !(bad >> i & 1u) ? from_r[i] + step_r : zeros(), to);
                });
    };

    // ---- scales of the tile's rows (weights, then x): a thread fetches a row's of a step, and they meet in LDS
    uint32_t own_mx[kOwn];
    float own_step[kOwn];
    size_t own_row[kOwn]; // x: x_rows or more for none
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const uint32_t row = i * kThr + threadIdx.x;
        own_row[i] = row < TC ? w_row0 + min(row, p.cols - 1u - col0) : min(source(row - TC), p.x_rows);
    }
    auto fetch_scales = [&](uint32_t t) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const uint32_t row = i * kThr + threadIdx.x;
            const bool weights = row < TC; // the same for the whole wave
            const Scales& s = weights ? p.ws : p.xs;
            const bool none = row >= TC + TR || (!weights && own_row[i] >= p.x_rows);
            own_mx[i] = 0x7F7F7F7Fu;
            own_step[i] = 1.0f;
            if (none)
                continue;
            if (s.kind == kScaleMx) {
                const uint8_t* const at = static_cast<const uint8_t*>(s.at) + own_row[i] * s.groups;
                const uint32_t block = 4u * t, last = depth / 32u - 1u;
                if (s.words && s.width == 1)
                    own_mx[i] = *reinterpret_cast<const uint32_t*>(at + block);
                else if (s.width % 4u == 0)
                    own_mx[i] = at[t / (s.width / 4u)] * 0x01010101u;
                else {
                    uint32_t v = 0;
                    for (uint32_t b = 0; b < 4u; ++b)
                        v |= (block + b <= last ? (uint32_t)at[(block + b) / s.width] : 127u) << (8u * b);
                    own_mx[i] = v;
                }
            }
            if (STEP && s.kind == kScaleStep)
                own_step[i] = static_cast<const float*>(s.at)[own_row[i] * s.groups + t / s.width];
        }
    };
    auto put_scales = [&](uint32_t buf) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const uint32_t row = i * kThr + threadIdx.x;
            if (kOwn * kThr == TC + TR || row < TC + TR) {
                s_mx[buf][row] = own_mx[i];
                if constexpr (STEP)
                    s_step[buf][row] = own_step[i];
            }
        }
    };

    v4f acc[NC][NR];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < NR; ++j)
            acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    auto join = [](v4u lo, v4u hi) { return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w}; };
    auto multiply = [&](uint32_t buf) {
        v8i b[NR];
        int b_mx[NR];
        float b_step[NR];
        // FP8: a lane's k are 16q .. and 64 + 16q .., FP4: 32q ..; its scale is that of the 32 from 32q on
#pragma unroll
        for (int j = 0; j < NR; ++j) {
            const uint32_t row = 16u * (wr * NR + j) + r;
            const char* const at = s_r[buf] + row * 128u;
            b[j] = join(*reinterpret_cast<const v4u*>(at + (q ^ (r & 7u)) * 16u),
                        *reinterpret_cast<const v4u*>(at + ((q + 4u) ^ (r & 7u)) * 16u));
            b_mx[j] = reinterpret_cast<const uint8_t*>(s_mx[buf] + TC + row)[q];
            b_step[j] = STEP ? s_step[buf][TC + row] : 1.0f;
        }
        struct Weights {
            v8i v;
            int mx;
            v4f step;
        };
        auto weights = [&](int i) {
            const uint32_t row = 16u * (wc * NC + i) + r;
            Weights a;
            if constexpr (W4) {
                const v4u v = *reinterpret_cast<const v4u*>(s_c[buf] + row * 64u + (q ^ (-(r >> 2) & 3u)) * 16u);
                a.v = join(v, v4u{0, 0, 0, 0});
            } else {
                const char* const at = s_c[buf] + row * 128u;
                a.v = join(*reinterpret_cast<const v4u*>(at + (q ^ (r & 7u)) * 16u),
                           *reinterpret_cast<const v4u*>(at + ((q + 4u) ^ (r & 7u)) * 16u));
            }
            a.mx = reinterpret_cast<const uint8_t*>(s_mx[buf] + row)[q];
            a.step = STEP ? *reinterpret_cast<const v4f*>(s_step[buf] + 16u * (wc * NC + i) + 4u * q)
                          : v4f{1.0f, 1.0f, 1.0f, 1.0f};
            return a;
        };
        Weights ahead = weights(0);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const Weights a = ahead; // the next weights' reads under these products
            if (i + 1 < NC)
                ahead = weights(i + 1);
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                const v4f c = STEP ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : acc[i][j];
                const v4f d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b[j], c, W4 ? 4 : 0, 0, 0, a.mx, 0,
                                                                              b_mx[j]);
                if constexpr (STEP) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[i][j][e] = __builtin_fmaf(d[e], a.step[e] * b_step[j], acc[i][j][e]);
                } else {
                    acc[i][j] = d;
                }
            }
        }
    };

    // ---- the steps: one on its way while the one before it is multiplied
    const uint32_t steps = (depth + kDepth - 1) / kDepth;
    fetch(0, 0);
    fetch_scales(0);
    put_scales(0);
#pragma clang loop unroll(disable) // (nor peeled)
    for (uint32_t t = 0; t < steps; ++t) {
        copies_done<0>();
        __syncthreads(); // step t is there, and nobody reads step t - 1 any more
        const uint32_t buf = t & 1u;
        if (t + 1u < steps) {
            fetch(t + 1u, buf ^ 1u);
            fetch_scales(t + 1u);
        }
        multiply(buf);
        put_scales(buf ^ 1u); // (past the last step unused: a branch here would draw the products behind it)
    }

    // ---- whole rows' scales, and the results: a lane has four columns of a row
    auto row_scale = [](const Scales& s, size_t row) {
        return s.kind != kScaleRow ? 1.0f
               : s.u8              ? e8m0_value(static_cast<const uint8_t*>(s.at)[row])
                                   : static_cast<const float*>(s.at)[row];
    };
    float c_scale[NC][4];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e)
            c_scale[i][e] = row_scale(p.ws, w_row0 + min(16u * (wc * NC + i) + 4u * q + e, p.cols - 1u - col0));
#pragma unroll
    for (int j = 0; j < NR; ++j) {
        const uint32_t row = 16u * (wr * NR + j) + r;
        if (row >= rows)
            continue;
        const uint32_t at = source(row);
        const bool none = at >= p.x_rows;
        const RowScale scale(none ? 0.0f : row_scale(p.xs, at));
        const size_t line = (size_t)(row0 + row) * p.cols;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const uint32_t col = col0 + 16u * (wc * NC + i) + 4u * q;
            if (col >= p.cols)
                continue;
            v4b v;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = (__bf16)(none ? 0.0f : scale(acc[i][j][e], c_scale[i][e]));
            *reinterpret_cast<v4b*>(static_cast<__bf16*>(p.out) + line + col) = v;
        }
    }
}

// The same where the scales' groups are 32 or 128 columns (or there are none).  The
// weights' fragments of a step stay in registers, the rows' go by one ahead of
// their products.  Scales come four steps (a turn) at a time: a thread fetches
// those of one of the tile's rows, and they meet in LDS, power-of-two ones with a
// lane's four steps in one word, from which the instruction picks a byte.
//
// 8192 x 8192 x 8192 FP8 410 .. 450 us (2.4 .. 2.7 PFLOP/s) with one scale a row,
// the matrix units busy in 59% of cycles at 1.9 .. 2.0 GHz; 460 with UE8M0 scales
// of groups (50%, 2.1 GHz); FP8 x FP4 412 (54%); fp32 scales of groups, whose two
// vector operations for each result and 128 k take half of the cycles, 600 (39%).
// What is open beside them: a step's first fragments are read behind the meeting,
// and a tile's start (offsets, index, first copies) and its stores lie between
// sums.  These count for more where sums are short and experts' rows ragged: 4096
// tokens' top-8 of 64 experts 7168 -> 4096 FP8 x FP4 970 us (42%), 2048 -> 7168
// FP8 with fp32 scales of 128 columns 775 (25%).  Scales fetched step by step, in
// front of the products, took 1226 and 926.  Small tiles for few rows, bound by
// the weights' bytes: one row of each of 64 experts 7168 -> 4096 FP8 345 us (5.4
// TB/s), FP4 227.
struct NoScale {
    uint32_t mx;
    float one;
};
__device__ const NoScale g_no_scale = {0x7F7F7F7Fu, 1.0f};

template <bool W4, bool MX, bool STEP, int TC, int TR, int WC, int WR, int RING>
__global__ __launch_bounds__(64 * WC * WR) void gemm_q_turn_kernel(QuantParams p)
{
    constexpr uint32_t kWaves = WC * WR, kThr = 64 * kWaves;
    constexpr int kBlocks = TC / WC / 16, kRowBlocks = TR / WR / 16; // of 16 columns and of 16 rows a wave
    static_assert(TC + TR <= (int)kThr, "a thread for each row's scales");
    constexpr uint32_t kRowC = W4 ? 64 : 128, kBytesC = TC * kRowC, kBytesR = TR * 128;
    constexpr int kCopiesC = (kBytesC / 1024 + kWaves - 1) / kWaves, kCopies = (kBytesR / 1024 + kWaves - 1) / kWaves;
    // a copy's number; where there are fewer than waves, some make the same one, so that all count as many
    auto copy_no_c = [](int i, uint32_t wave) { return (i * kWaves + wave) % (kBytesC / 1024); };
    auto copy_no_r = [](int i, uint32_t wave) { return (i * kWaves + wave) % (kBytesR / 1024); };
    __shared__ __attribute__((aligned(1024))) char s_c[RING][kBytesC];
    __shared__ __attribute__((aligned(1024))) char s_r[RING][kBytesR];
    __shared__ __attribute__((aligned(16))) uint32_t s_mx[MX ? 2 : 1][MX ? kThr * 4 : 1];  // [row][q], four steps
    __shared__ __attribute__((aligned(16))) float s_step[STEP ? 2 : 1][4][STEP ? kThr : 1]; // [step][row]

    const uint32_t lane = threadIdx.x & (kWaveSize - 1), r = lane & 15u, q = lane >> 4;
    const uint32_t wave = uniform(threadIdx.x / kWaveSize), wc = wave % WC, wr = wave / WC;

    // ---- this workgroup's tile
    const uint32_t col_tiles = (p.cols + TC - 1) / TC;
    Group g;
    uint32_t t0 = 0;
    if (!find_group(p.offsets, p.experts, p.n_rows, TR,
                    [&](uint32_t total) {
                        t0 = xcd_tile(blockIdx.x, total * col_tiles);
                        return t0 / col_tiles;
                    },
                    g))
        return;
    const uint2 tile = tile_in_group(t0 - g.first * col_tiles, g.tiles, col_tiles);
    const uint32_t row0 = g.row0 + tile.x * TR, rows = min((uint32_t)TR, g.rows - tile.x * TR);
    const uint32_t col0 = tile.y * TC, depth = p.depth, steps = (depth + kDepth - 1) / kDepth;
    const size_t w_row0 = (size_t)g.expert * p.cols + col0;
    auto source = [&](uint32_t row) { // x's row for a row of the tile; x_rows or more: none
        const uint32_t at = row0 + min(row, rows - 1u);
        return p.index ? (uint32_t)p.index[at] : at;
    };

    // ---- where each lane's copies come from (layouts in LDS as in gemm_q_kernel)
    const uint32_t ld_c = W4 ? depth / 2u : depth;
    const char* const base_c = p.w + w_row0 * ld_c;
    const uint32_t lane_c = W4 ? (lane & 3u) ^ (-(lane >> 4) & 3u) : (lane & 7u) ^ (lane >> 3);
    const uint32_t lane_r = (lane & 7u) ^ (lane >> 3);
    const uint32_t k_c = lane_c * (W4 ? 32u : 16u), k_r = lane_r * 16u; // the lane's first k of a step
    uint32_t offset_c[kCopiesC], offset_r[kCopies], row_r[kCopies];
#pragma unroll
    for (int i = 0; i < kCopiesC; ++i) {
        const uint32_t row = copy_no_c(i, wave) * (W4 ? 16u : 8u) + (W4 ? lane >> 2 : lane >> 3);
        offset_c[i] = min(row, p.cols - 1u - col0) * ld_c + lane_c * 16u;
    }
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        const uint32_t at = source(copy_no_r(i, wave) * 8u + (lane >> 3));
        row_r[i] = at < p.x_rows ? at : 0u; // (a row that is none: any, and zeros as its result)
        offset_r[i] = row_r[i] * depth + k_r;
    }
    // FAST: whole steps whose offsets fit 32 bits; past the depth, else, zeros
    auto copy_c = [&](auto fast, uint32_t t, uint32_t buf, int i) {
        char* const to = s_c[buf] + copy_no_c(i, wave) * 1024u;
        if constexpr (decltype(fast)::value)
            copy_to_lds(base_c + (size_t)t * kRowC, offset_c[i], to);
        else
            copy_to_lds(t * kDepth + k_c < depth ? base_c + (size_t)t * kRowC + offset_c[i] : zeros(), to);
    };
    auto copy_r = [&](auto fast, uint32_t t, uint32_t buf, int i) {
        char* const to = s_r[buf] + copy_no_r(i, wave) * 1024u;
        if constexpr (decltype(fast)::value)
            copy_to_lds(p.x + (size_t)t * 128u, offset_r[i], to);
        else
            copy_to_lds(t * kDepth + k_r < depth ? p.x + (size_t)row_r[i] * depth + t * kDepth + k_r : zeros(), to);
    };

    // ---- scales: thread i has those of row i of the weights, or of row i - TC of x.  Every kind is read by the same
    // loads, those that there are not from a constant: a branch here would draw the products behind it.
    const bool weights = threadIdx.x < TC;
    const Scales& own = weights ? p.ws : p.xs;
    size_t own_row = 0;
    if constexpr (MX || STEP) {
        if (weights) {
            own_row = w_row0 + min(threadIdx.x, p.cols - 1u - col0);
        } else { // (threads past the last row: some row's, unused)
            const uint32_t at = source(threadIdx.x - TC);
            own_row = at < p.x_rows ? at : 0u;
        }
    }
    const bool is_mx = MX && own.kind == kScaleMx, by_block = is_mx && own.width == 1;
    const char* const own_mx = is_mx ? static_cast<const char*>(own.at) + own_row * own.groups
                                     : reinterpret_cast<const char*>(&g_no_scale.mx);
    const uint32_t mx_turn = by_block ? 16u : is_mx ? 4u : 0u, mx_last = is_mx ? own.groups - 4u : 0u;
    const bool is_step = STEP && own.kind == kScaleStep;
    const float* const own_step = is_step ? static_cast<const float*>(own.at) + own_row * own.groups : &g_no_scale.one;
    const uint32_t step_magic = is_step ? (1u << 31) / own.width : 0u;
    uint32_t turn_mx[4];
    float turn_step[4];
    auto fetch_scales = [&](uint32_t turn) { // of steps 4 turn ..
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            if constexpr (MX)
                turn_mx[i] = *reinterpret_cast<const uint32_t*>(own_mx + min(turn * mx_turn + (by_block ? 4u * i : 0u), mx_last));
            if constexpr (STEP) // (2 s + 1) floor(2^31 / width) / 2^32, rounded down, is s / width
                turn_step[i] = own_step[__umulhi(2u * min(4u * turn + i, steps - 1u) + 1u, step_magic)];
        }
    };
    auto put_scales = [&](uint32_t buf) {
        if constexpr (MX) {
            // a word a step with a byte for each q -> a word for each q with a byte a step
            const uint32_t a = __builtin_amdgcn_perm(turn_mx[1], turn_mx[0], 0x05010400u);
            const uint32_t b = __builtin_amdgcn_perm(turn_mx[3], turn_mx[2], 0x05010400u);
            const uint32_t c = __builtin_amdgcn_perm(turn_mx[1], turn_mx[0], 0x07030602u);
            const uint32_t d = __builtin_amdgcn_perm(turn_mx[3], turn_mx[2], 0x07030602u);
            const v4u v = {by_block ? __builtin_amdgcn_perm(b, a, 0x05040100u) : turn_mx[0],
                           by_block ? __builtin_amdgcn_perm(b, a, 0x07060302u) : turn_mx[0],
                           by_block ? __builtin_amdgcn_perm(d, c, 0x05040100u) : turn_mx[0],
                           by_block ? __builtin_amdgcn_perm(d, c, 0x07060302u) : turn_mx[0]};
            *reinterpret_cast<v4u*>(s_mx[buf] + threadIdx.x * 4u) = v;
        }
        if constexpr (STEP)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s_step[buf][i][threadIdx.x] = turn_step[i];
    };

    auto join = [](v4u lo, v4u hi) {
        return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };
    auto read_c = [&](uint32_t buf, int i) { // FP8: a lane's k are 16q .. and 64 + 16q .., FP4: 32q ..
        const uint32_t row = 16u * (wc * kBlocks + i) + r;
        if constexpr (W4) {
            const v4u v = *reinterpret_cast<const v4u*>(s_c[buf] + row * 64u + (q ^ (-(r >> 2) & 3u)) * 16u);
            return join(v, v4u{0, 0, 0, 0});
        } else {
            const char* const at = s_c[buf] + row * 128u;
            return join(*reinterpret_cast<const v4u*>(at + (q ^ (r & 7u)) * 16u),
                        *reinterpret_cast<const v4u*>(at + ((q + 4u) ^ (r & 7u)) * 16u));
        }
    };
    auto row_of = [&](int j) { return 16u * ((uint32_t)WR * j + wr); }; // every WR-th block: few rows are shared evenly
    auto read_r = [&](uint32_t buf, int j) {
        const char* const at = s_r[buf] + (row_of(j) + r) * 128u;
        return join(*reinterpret_cast<const v4u*>(at + (q ^ (r & 7u)) * 16u),
                    *reinterpret_cast<const v4u*>(at + ((q + 4u) ^ (r & 7u)) * 16u));
    };

    auto run = [&](auto n_blocks, auto fast) {
        constexpr int N = decltype(n_blocks)::value; // row blocks
        auto last_step = [&](uint32_t t) { return min(t, steps - 1u); }; // (past the last step that one again, unused)
        constexpr int kCopiesR = (int)(WR * N * 2 + kWaves - 1) / (int)kWaves;
        v4f acc[kBlocks][N];
#pragma unroll
        for (int i = 0; i < kBlocks; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j)
                acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        uint32_t a_mx[kBlocks], b_mx[N]; // four steps' scales of a lane
#pragma unroll
        for (uint32_t t = 0; t + 1u < (uint32_t)RING; ++t) {
            const uint32_t at = last_step(t);
#pragma unroll
            for (int n = 0; n < kCopiesC; ++n)
                copy_c(fast, at, t, n);
#pragma unroll
            for (int n = 0; n < kCopiesR; ++n)
                copy_r(fast, at, t, n);
        }
        fetch_scales(0);
        put_scales(0);
        uint32_t at_step = 0; // t % 3
        auto step = [&](auto number, uint32_t t) { // step t, number t % 4 of its turn
            constexpr int u = decltype(number)::value;
            const uint32_t turn = t / 4u, buf = RING == 3 ? at_step : u % RING;
            const uint32_t ahead = RING == 3 ? (at_step ? at_step - 1u : 2u) : (u + RING - 1) % RING;
            copies_done<(RING - 2) * (kCopiesC + kCopiesR)>();
            meet(); // step t is there, and nobody reads step t - 1 any more
            const uint32_t next = last_step(t + RING - 1u);
            if constexpr (MX) {
                if constexpr (u == 0) {
#pragma unroll
                    for (int i = 0; i < kBlocks; ++i)
                        a_mx[i] = s_mx[turn & 1u][(16u * (wc * kBlocks + i) + r) * 4u + q];
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        b_mx[j] = s_mx[turn & 1u][(TC + row_of(j) + r) * 4u + q];
                }
            }
            v8i a[kBlocks], b = read_r(buf, 0);
            v4f a_step[kBlocks];
            float b_step = STEP ? s_step[turn & 1u][u][TC + row_of(0) + r] : 1.0f;
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
                a[i] = read_c(buf, i);
                a_step[i] = STEP ? *reinterpret_cast<const v4f*>(&s_step[turn & 1u][u][16u * (wc * kBlocks + i) + 4u * q])
                                 : v4f{1.0f, 1.0f, 1.0f, 1.0f};
            }
            v4f before[kBlocks];
            float before_step = 0.0f;
            auto add_step = [&](int j, const v4f(&d)[kBlocks], float r_step) {
#pragma unroll
                for (int i = 0; i < kBlocks; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[i][j][e] = __builtin_fmaf(d[i][e], a_step[i][e] * r_step, acc[i][j][e]);
            };
#pragma unroll
            for (int j = 0; j < N; ++j) {
                __builtin_amdgcn_sched_barrier(0);
                const v8i now = b;
                const float now_step = b_step;
                if (j + 1 < N) {
                    b = read_r(buf, j + 1);
                    b_step = STEP ? s_step[turn & 1u][u][TC + row_of(j + 1) + r] : 1.0f;
                }
                v4f d[kBlocks];
#pragma unroll
                for (int i = 0; i < kBlocks; ++i) {
                    const v4f c = STEP ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : acc[i][j];
                    d[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[i], now, c, W4 ? 4 : 0, 0, MX ? u : 0,
                                                                            MX ? (int)a_mx[i] : 127, MX ? u : 0,
                                                                            MX ? (int)b_mx[j] : 127);
                    if constexpr (!STEP)
                        acc[i][j] = d[i];
                }
                if constexpr (STEP) { // the block before this one's, under this one's products
                    if (j > 0)
                        add_step(j - 1, before, before_step);
#pragma unroll
                    for (int i = 0; i < kBlocks; ++i)
                        before[i] = d[i];
                    before_step = now_step;
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int n = 0; n < kCopiesC + kCopiesR; ++n) // spread over the row blocks
                    if (n * N / (kCopiesC + kCopiesR) == j) {
                        if (n < kCopiesC)
                            copy_c(fast, next, ahead, n);
                        else
                            copy_r(fast, next, ahead, n - kCopiesC);
                    }
            }
            if constexpr (STEP) { // (the sums are done with here: left to the compiler, products move behind the branch)
                add_step(N - 1, before, before_step);
#pragma unroll
                for (int j = 0; j < N; ++j)
#pragma unroll
                    for (int i = 0; i < kBlocks; ++i)
                        asm volatile("" : "+v"(acc[i][j]));
            }
            // the next turn's scales, fetched during one step and put in place during the next
            if constexpr (u == 1)
                fetch_scales(turn + 1u);
            if constexpr (u == 2)
                put_scales((turn + 1u) & 1u);
            at_step = at_step < 2u ? at_step + 1u : 0u;
        };
        using std::integral_constant;
#pragma clang loop unroll(disable) // (nor peeled)
        for (uint32_t t = 0; t < steps; t += 4) {
            step(integral_constant<int, 0>{}, t);
            if (t + 1u < steps)
                step(integral_constant<int, 1>{}, t + 1u);
            if (t + 2u < steps)
                step(integral_constant<int, 2>{}, t + 2u);
            if (t + 3u < steps)
                step(integral_constant<int, 3>{}, t + 3u);
        }
        copies_done<0>(); // no copy outlives the workgroup's LDS

        // ---- whole rows' scales, and the results
        auto row_scale = [](const Scales& s, size_t row) {
            return s.kind != kScaleRow ? 1.0f
                   : s.u8              ? e8m0_value(static_cast<const uint8_t*>(s.at)[row])
                                       : static_cast<const float*>(s.at)[row];
        };
        float c_scale[kBlocks][4];
#pragma unroll
        for (int i = 0; i < kBlocks; ++i)
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e)
                c_scale[i][e] = row_scale(p.ws, w_row0 + min(16u * (wc * kBlocks + i) + 4u * q + e, p.cols - 1u - col0));
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint32_t row = row_of(j) + r, at = source(row);
            const bool none = at >= p.x_rows;
            const RowScale scale(none ? 0.0f : row_scale(p.xs, at));
            const size_t line = (size_t)(row0 + row) * p.cols;
#pragma unroll
            for (int i = 0; i < kBlocks; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[i][j][e] = none ? 0.0f : scale(acc[i][j][e], c_scale[i][e]);
            if constexpr (kBlocks % 2 == 0) {
#pragma unroll
                for (int i = 0; i < kBlocks; i += 2) {
                    const v4u pair = pair_columns(acc[i][j], acc[i + 1][j]);
                    const uint32_t col = col0 + 16u * (wc * kBlocks + i + (q & 1u)) + 8u * (q >> 1);
                    if (row < rows && col < p.cols)
                        *reinterpret_cast<v4u*>(static_cast<__bf16*>(p.out) + line + col) = pair;
                }
            } else {
                const uint32_t col = col0 + 16u * wc + 4u * q;
                const v4f v = acc[0][j];
                static_assert(kBlocks % 2 == 0 || kBlocks == 1, "blocks in pairs");
                if (row < rows && col < p.cols)
                    *reinterpret_cast<v4b*>(static_cast<__bf16*>(p.out) + line + col) =
                        v4b{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
            }
        }
    };
    using std::bool_constant;
    using std::integral_constant;
    auto run_blocks = [&](auto fast) {
        // Large tiles: no more blocks than there are rows, in even numbers (FP8 x FP4 964 us with odd ones too instead of
        // 976, FP8 785 and 782; they would double these kernels).
        if constexpr (kRowBlocks == 8) {
            const uint32_t blocks = uniform((rows + 16u * WR - 1u) / (16u * WR));
            if (blocks > 6)
                run(integral_constant<int, 8>{}, fast);
            else if (blocks > 4)
                run(integral_constant<int, 6>{}, fast);
            else if (blocks > 2)
                run(integral_constant<int, 4>{}, fast);
            else
                run(integral_constant<int, 2>{}, fast);
        } else {
            run(integral_constant<int, kRowBlocks>{}, fast);
        }
    };
    if (depth % kDepth == 0 && (uint64_t)p.x_rows * depth < (1ull << 32))
        run_blocks(bool_constant<true>{});
    else
        run_blocks(bool_constant<false>{});
}

// At most how many tiles of tr rows by tc columns there are, however the rows lie, in workgroups of whole turns over
// the XCDs.
uint64_t workgroups(const QuantParams& p, uint32_t tc, uint32_t tr)
{
    const uint64_t col_tiles = ((uint64_t)p.cols + tc - 1) / tc, most = p.n_rows < p.experts ? p.n_rows : p.experts;
    return ((p.n_rows / tr + most) * col_tiles + kXcds - 1) / kXcds * kXcds;
}

template <bool W4, bool MX, bool STEP, int TC, int TR, int WC, int WR, int RING>
tk_status launch_turn(const QuantParams& p, hipStream_t s)
{
    const uint64_t blocks = workgroups(p, TC, TR);
    if (!launchable(blocks, 64 * WC * WR))
        return TK_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((gemm_q_turn_kernel<W4, MX, STEP, TC, TR, WC, WR, RING>), dim3((uint32_t)blocks), dim3(64 * WC * WR), 0,
                       s, p);
    return hipGetLastError() == hipSuccess ? TK_OK : TK_ERR_HIP;
}

template <bool W4, bool STEP, int TC, int TR, int WC, int WR>
tk_status launch(const QuantParams& p, hipStream_t s)
{
    const uint64_t blocks = workgroups(p, TC, TR);
    if (!launchable(blocks, 64 * WC * WR))
        return TK_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((gemm_q_kernel<W4, STEP, TC, TR, WC, WR>), dim3((uint32_t)blocks), dim3(64 * WC * WR), 0, s,
                       p);
    return hipGetLastError() == hipSuccess ? TK_OK : TK_ERR_HIP;
}

template <bool W4, bool MX, bool STEP>
tk_status launch_size(const QuantParams& p, hipStream_t s)
{
    // as launch_forward; the large tiles for groups of 32 and of 128 columns (or none)
    const uint64_t load = average_rows(p.n_rows, p.experts);
    auto tiles = [&](uint32_t tr, uint32_t tc) { return tiles_of(load, p.experts, p.cols, tr, tc); };
    auto turns = [](const Scales& a) { return a.kind != kScaleMx || (a.words && (a.width == 1 || a.width == 4)); };
    const bool mid = load > 16 && tiles(64, 128) >= 128;
    if constexpr (MX)
        if (!turns(p.ws) || !turns(p.xs))
            return mid ? launch<W4, STEP, 128, 64, 2, 2>(p, s) : launch<W4, STEP, 64, 16, 4, 1>(p, s);
    if (load > 64 && tiles(256, 256) >= 128)
        return launch_turn<W4, MX, STEP, 256, 256, 4, 2, 2>(p, s);
    if (mid)
        return launch_turn<W4, MX, STEP, 128, 64, 2, 2, 3>(p, s);
    return launch_turn<W4, MX, STEP, 64, 16, 4, 1, 4>(p, s);
}

// The scales of rows of `depth` columns in groups of `group` (0: the row).  False: not taken.
bool scales_of(const void* at, int fmt, int64_t group, int64_t depth, Scales& s)
{
    s.at = at;
    s.u8 = fmt == TK_SCALE_UE8M0;
    s.kind = kScaleRow;
    s.groups = s.width = 1;
    s.words = 0;
    if (group == 0 || group == depth)
        return true;
    if (group % (s.u8 ? 32 : 128) != 0)
        return false;
    s.kind = s.u8 ? kScaleMx : kScaleStep;
    s.groups = (uint32_t)(depth / group);
    s.width = (uint32_t)(group / (s.u8 ? 32 : 128));
    s.words = s.u8 && s.groups % 4 == 0 && aligned(at, 4);
    return true;
}

} // namespace

extern "C" tk_status tk_expert_gemm(const void* x, const void* x_scales, int x_dtype, tk_scale_fmt x_scale_fmt,
                                    int64_t x_group, int64_t x_rows, const int32_t* row_index,
                                    const int32_t* expert_offsets, int64_t n_rows, const void* w, const void* w_scales,
                                    int w_dtype, tk_scale_fmt w_scale_fmt, int64_t w_group, int64_t experts,
                                    int64_t out_features, int64_t in_features, tk_dtype out_dtype, void* out,
                                    void* stream)
{
    const bool x8 = x_dtype == TK_DTYPE_FP8, w8 = w_dtype == TK_DTYPE_FP8, w4 = w_dtype == TK_DTYPE_FP4;
    const bool out_bf16 = (int)out_dtype == TK_DTYPE_BF16;
    if (!valid_rows({x_rows, row_index}, expert_offsets, n_rows, experts) ||
        !valid_shape(out_features, in_features, x8 || w8 || w4 ? 32 : 8) || (!x8 && x_dtype != TK_DTYPE_BF16) ||
        (!w8 && !w4 && w_dtype != TK_DTYPE_BF16) || (!out_bf16 && (int)out_dtype != TK_DTYPE_FP32))
        return TK_ERR_INVALID_ARG;
    auto bad_scales = [&](int fmt, int64_t group) {
        return fmt < TK_SCALE_FP32 || fmt > TK_SCALE_UE8M0_PACKED || group < 0 || (group && in_features % group != 0);
    };
    if ((x8 && bad_scales((int)x_scale_fmt, x_group)) || ((w8 || w4) && bad_scales((int)w_scale_fmt, w_group)))
        return TK_ERR_INVALID_ARG;
    if (n_rows > 0 && ((x_rows > 0 && (!x || (x8 && !x_scales))) || !w || !out || ((w8 || w4) && !w_scales)))
        return TK_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16) ||
        (x8 && (int)x_scale_fmt == TK_SCALE_FP32 && !aligned(x_scales, 4)) ||
        ((w8 || w4) && (int)w_scale_fmt == TK_SCALE_FP32 && !aligned(w_scales, 4)))
        return TK_ERR_INVALID_ARG;
    if (experts > kMaxExperts || x8 != (w8 || w4) || (x8 && !out_bf16))
        return TK_ERR_UNSUPPORTED;
    Scales xs{}, ws{};
    if (x8 && ((int)x_scale_fmt > TK_SCALE_UE8M0 || (int)w_scale_fmt > TK_SCALE_UE8M0 ||
               !scales_of(x_scales, x_scale_fmt, x_group, in_features, xs) ||
               !scales_of(w_scales, w_scale_fmt, w_group, in_features, ws)))
        return TK_ERR_UNSUPPORTED;
    const size_t o_bytes = (size_t)n_rows * (size_t)out_features * (out_bf16 ? 2u : 4u);
    const size_t w_rows = (size_t)experts * (size_t)out_features;
    if (overlaps(out, o_bytes, x, (size_t)x_rows * (size_t)in_features * (x8 ? 1u : 2u)) ||
        overlaps(out, o_bytes, w, w_rows * (size_t)in_features * 2u / (w4 ? 4u : w8 ? 2u : 1u)) ||
        overlaps_rows(out, o_bytes, row_index, expert_offsets, n_rows, experts) ||
        (x8 && (overlaps(out, o_bytes, x_scales, (size_t)x_rows * xs.groups * (xs.u8 ? 1u : 4u)) ||
                overlaps(out, o_bytes, w_scales, w_rows * ws.groups * (ws.u8 ? 1u : 4u)))))
        return TK_ERR_INVALID_ARG;
    if (n_rows == 0)
        return TK_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (!x8) {
        GemmParams p{};
        p.c = static_cast<const char*>(w);
        p.r = static_cast<const char*>(x_rows ? x : w); // (no row: what is read in its place is not used)
        p.r_index = row_index;
        p.r_rows = (uint32_t)x_rows;
        p.offsets = expert_offsets;
        p.n_rows = (uint32_t)n_rows;
        p.experts = (uint32_t)experts;
        p.cols = (uint32_t)out_features;
        p.depth = (uint32_t)in_features;
        p.out = out;
        p.out_bf16 = out_bf16;
        return launch_forward(p, s);
    }
    QuantParams p{};
    p.w = static_cast<const char*>(w);
    p.x = static_cast<const char*>(x_rows ? x : w); // (no row: what is read in its place is not used)
    p.index = row_index;
    p.offsets = expert_offsets;
    p.out = out;
    p.ws = ws;
    p.xs = xs;
    p.x_rows = (uint32_t)x_rows;
    p.n_rows = (uint32_t)n_rows;
    p.experts = (uint32_t)experts;
    p.cols = (uint32_t)out_features;
    p.depth = (uint32_t)in_features;
    if (x_rows == 0) // nor are there scales
        p.xs.kind = kScaleRow;
    const bool mx = xs.kind == kScaleMx || ws.kind == kScaleMx, step = xs.kind == kScaleStep || ws.kind == kScaleStep;
    if (w4)
        return mx ? (step ? launch_size<true, true, true>(p, s) : launch_size<true, true, false>(p, s))
                  : (step ? launch_size<true, false, true>(p, s) : launch_size<true, false, false>(p, s));
    return mx ? (step ? launch_size<false, true, true>(p, s) : launch_size<false, true, false>(p, s))
              : (step ? launch_size<false, false, true>(p, s) : launch_size<false, false, false>(p, s));
}
