// tk_gemm.hip -- the experts' matrix products in bf16 over ragged rows and
// their gradients, behind tk_expert_gemm (bf16 operands), tk_expert_gemm_dgrad
// and tk_expert_gemm_wgrad in include/tk_expert.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "tk_gemm_host.h"
#include "tk_gemm_tile.h"

namespace {

using namespace tk_gemm;

// The product that a launch computes, result[row][column] = sum over k:
//   kForward  rows r of x, columns o:       x[r][k] * w[o][k]
//   kDgrad    rows r of dy, columns c:      dy[r][k] * w[k][c]
//   kWgrad    rows o, columns c, k a row:   dy[k][o] * x[k][c]
constexpr int kForward = 0, kDgrad = 1, kWgrad = 2;

constexpr uint32_t kDepth = 64; // k of a step: 128 bytes of a row

// 8 values of a matrix instruction's lane from a tile kept [k][column]: two
// transposing reads of four rows each
__device__ __forceinline__ v8b read_transposed(const char* at, uint32_t pitch)
{
    typedef __attribute__((address_space(3))) v4s lds_v4s;
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(at));
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(at + 4u * pitch));
    return __builtin_bit_cast(v8b, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Four columns of a row, rounded once.
__device__ __forceinline__ void store_result(const GemmParams& p, size_t at, v4f v)
{
    if (p.out_bf16)
        *reinterpret_cast<v4b*>(static_cast<__bf16*>(p.out) + at) = v4b{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
    else
        *reinterpret_cast<v4f*>(static_cast<float*>(p.out) + at) = v;
}

// v[i] += the results in their places, from `at`(i); their loads are on their way together.
template <typename T4, typename T, int N, typename F>
__device__ __forceinline__ void add_result(const T* out, v4f* v, F&& at)
{
    T4 old[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        old[i] = *reinterpret_cast<const T4*>(out + at(i));
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] += __builtin_convertvector(old[i], v4f);
}

// A tile of TC columns x TR rows by WC x WR waves, 64 k a step; a column's and a row's fragments meet in the
// 16x16x32 instruction, so that a lane ends with four columns of a row.  The copies go straight into LDS and are
// waited for when their step comes up.  RING: steps in LDS, one of them being multiplied and the others on their way
// (wgrad: two).  For few rows, whose time is that of reading the weights: one row of each of 64 experts 7168 -> 4096
// 600 us (3.76 GB, 6.2 TB/s), 34 tokens' rows of a 512 -> 1024 layer 5.0 us (the launch, and one trip to memory for
// the indices and one for the first step).  More steps on their way are what few tiles need: 64 rows of 4096 -> 4096
// 39 us with two steps, 15 with three or four and smaller tiles; with weights kept [k][column], whose smallest tile has
// 128 columns, two (64 rows an expert) and three steps (16).
template <int KIND, int TC, int TR, int WC, int WR, bool X8, int RING>
__global__ __launch_bounds__(64 * WC * WR) void gemm_kernel(GemmParams p)
{
    constexpr uint32_t kWaves = WC * WR;
    constexpr bool kCT = KIND != kForward, kRT = KIND == kWgrad; // kept [k][..] in memory and in LDS
    constexpr int NC = TC / WC / 16, NR = TR / WR / 16;
    constexpr uint32_t kBytesC = TC * kDepth * 2, kBytesR = TR * kDepth * 2;
    constexpr int kCopiesC = (kBytesC / 1024 + kWaves - 1) / kWaves, kCopiesR = (kBytesR / 1024 + kWaves - 1) / kWaves;
    static_assert(KIND != kWgrad || RING == 2, "wgrad's sources are found a step ahead");
    // a copy's number; where there are fewer than waves, some make the same one, so that all count as many
    auto copy_no_c = [](int i, uint32_t wave) { return (i * kWaves + wave) % (kBytesC / 1024); };
    auto copy_no_r = [](int i, uint32_t wave) { return (i * kWaves + wave) % (kBytesR / 1024); };
    constexpr int kCodes = X8 ? TC * kDepth / 16 / (64 * kWaves) : 1; // 16-code pieces of x a thread
    __shared__ __attribute__((aligned(1024))) char s_c[RING][kBytesC];
    __shared__ __attribute__((aligned(1024))) char s_r[RING][kBytesR];

    const uint32_t lane = threadIdx.x & (kWaveSize - 1), r = lane & 15u, q = lane >> 4;
    const uint32_t wave = uniform(threadIdx.x / kWaveSize), wc = wave % WC, wr = wave / WC;

    // ---- this workgroup's tile
    const uint32_t col_tiles = (p.cols + TC - 1) / TC;
    uint32_t expert, row_base = 0, row0, rows, col0, depth; // result rows row0 .. row0 + rows - 1 (wgrad: of the weights)
    if constexpr (KIND == kWgrad) {
        const uint32_t row_tiles = (p.out_rows + TR - 1) / TR, per = row_tiles * col_tiles;
        const uint32_t t = xcd_tile(blockIdx.x, p.experts * per);
        if (t >= p.experts * per)
            return;
        expert = t / per;
        const uint32_t in = t - expert * per;
        row0 = in / col_tiles * TR;
        rows = min((uint32_t)TR, p.out_rows - row0);
        col0 = in % col_tiles * TC;
        expert_rows(p.offsets, expert, p.n_rows, row_base, depth);
        row_base = uniform(row_base);
        depth = uniform(depth);
        if (p.accumulate && depth == 0)
            return;
    } else {
        Group g;
        uint32_t t = 0;
        if (!find_group(p.offsets, p.experts, p.n_rows, TR,
                        [&](uint32_t total) {
                            t = xcd_tile(blockIdx.x, total * col_tiles);
                            return t / col_tiles;
                        },
                        g))
            return;
        expert = g.expert;
        const uint2 at = tile_in_group(t - g.first * col_tiles, g.tiles, col_tiles);
        row0 = g.row0 + at.x * TR;
        rows = min((uint32_t)TR, g.rows - at.x * TR);
        col0 = at.y * TC;
        depth = p.depth;
    }

    // ---- where each lane's copies come from
    // A tile kept [row][k] has 128 bytes a row; the 16 bytes c of row i lie at c ^ (i & 7), so that the 16 rows
    // of a fragment meet in no bank.  One kept [k][column] has its columns' 32 bytes c of row k at c ^ hash(k),
    // as the transposing reads take four rows k of 32 bytes from each of 16 lanes.
    auto hash = [](uint32_t k) { return (k & 3u) | ((k >> 1) & 4u); };
    const uint32_t ld_c = (KIND == kForward ? p.depth : p.cols) * (X8 ? 1u : 2u);
    const uint32_t ld_r = (KIND == kForward ? p.depth : KIND == kDgrad ? p.depth : p.out_rows) * 2u;
    const char* base_c = p.c; // forward and dgrad: the same for the whole wave; offset_c from there
    uint32_t offset_c[kCopiesC];
    const char* from_r[kCopiesR];
    uint32_t piece_c[kCopiesC], piece_r[kCopiesR]; // [row][k]: the first k; [k][column]: the row k
    if constexpr (KIND == kForward)
        base_c += ((size_t)expert * p.cols + col0) * ld_c;
    if constexpr (KIND == kDgrad)
        base_c += (size_t)expert * p.depth * ld_c;
    bool any_bad = false;
    uint32_t bad = 0; // rows of the forward's and dgrad's row operand whose index names none
#pragma unroll
    for (int i = 0; i < kCopiesC; ++i) {
        const uint32_t no = copy_no_c(i, wave);
        if constexpr (!kCT) {
            const uint32_t row = no * 8u + lane / 8u, k = ((lane & 7u) ^ (lane >> 3)) * 8u;
            piece_c[i] = k;
            offset_c[i] = min(row, p.cols - 1u - col0) * ld_c + k * 2u;
        } else {
            constexpr uint32_t kLanes = TC / 8; // lanes a row
            const uint32_t k = no * (64u / kLanes) + lane / kLanes, s = lane % kLanes;
            uint32_t col = col0 + (((s >> 1) ^ hash(k)) * 2u + (s & 1u)) * 8u;
            col = col < p.cols ? col : 0u; // not stored
            piece_c[i] = k;
            offset_c[i] = (KIND == kDgrad ? k * ld_c : 0u) + col * 2u;
        }
    }
#pragma unroll
    for (int i = 0; i < kCopiesR; ++i) {
        const uint32_t no = copy_no_r(i, wave);
        if constexpr (!kRT) {
            const uint32_t row = no * 8u + lane / 8u, k = ((lane & 7u) ^ (lane >> 3)) * 8u;
            uint32_t at = row0 + min(row, rows - 1u);
            if (p.r_index)
                at = (uint32_t)p.r_index[at];
            if (at >= p.r_rows) {
                at = 0;
                bad |= 1u << i;
            }
            piece_r[i] = k;
            from_r[i] = p.r + (size_t)at * ld_r + k * 2u;
        } else {
            constexpr uint32_t kLanes = TR / 8;
            const uint32_t k = no * (64u / kLanes) + lane / kLanes, s = lane % kLanes;
            uint32_t col = row0 + (((s >> 1) ^ hash(k)) * 2u + (s & 1u)) * 8u;
            col = col < p.out_rows ? col : 0u;
            piece_r[i] = k;
            from_r[i] = p.r + col * 2u;
        }
    }
    if constexpr (!kRT)
        any_bad = __builtin_amdgcn_ballot_w64(bad != 0) != 0;
    uint32_t result_row[NR]; // the operand's row of each of the lane's results (read here, long before its use)
#pragma unroll
    for (int j = 0; j < NR; ++j)
        result_row[j] = !kRT && p.r_index ? (uint32_t)p.r_index[row0 + min(16u * (wr * NR + j) + r, rows - 1u)] : 0u;

    // wgrad: the source row of the expert's row k, past whose last there are zeros
    auto source = [&](const int32_t* index, uint32_t k, uint32_t all) -> uint32_t {
        if (k >= depth)
            return ~0u;
        const uint32_t at = index ? (uint32_t)index[row_base + k] : row_base + k;
        return at < all ? at : ~0u;
    };
    uint32_t next_c[kCopiesC], next_r[kCopiesR], next_x[kCodes]; // the coming step's source rows
    auto find_sources = [&](uint32_t t) {
        if constexpr (KIND == kWgrad) {
            if constexpr (!X8) {
#pragma unroll
                for (int i = 0; i < kCopiesC; ++i)
                    next_c[i] = source(p.c_index, t * kDepth + piece_c[i], p.c_rows);
            } else {
#pragma unroll
                for (int i = 0; i < kCodes; ++i)
                    next_x[i] = source(p.c_index, t * kDepth + (i * 64u * kWaves + threadIdx.x) / (TC / 16u), p.c_rows);
            }
#pragma unroll
            for (int i = 0; i < kCopiesR; ++i)
                next_r[i] = source(p.r_index, t * kDepth + piece_r[i], p.r_rows);
        }
    };

    v4u codes[kCodes]; // X8: a step's codes and their scales on their way through registers
    uint32_t code_scale[kCodes];
    auto code_col = [&](int i) { return col0 + (i * 64u * kWaves + threadIdx.x) % (TC / 16u) * 16u; };

    // Step t of both operands on its way into LDS.  Past the depth, and for rows that are none, zeros.
    auto fetch = [&](uint32_t t, uint32_t buf) {
        const bool whole = (t + 1u) * kDepth <= depth && !any_bad; // wave-uniform
        if constexpr (KIND != kWgrad) {
            const size_t step_c = kCT ? (size_t)t * kDepth * ld_c : (size_t)t * (kDepth * 2u);
            const size_t step_r = (size_t)t * (kDepth * 2u);
            auto each = [&](auto&& copy_c, auto&& copy_r) {
#pragma unroll
                for (int i = 0; i < kCopiesC; ++i)
                        copy_c(i, s_c[buf] + copy_no_c(i, wave) * 1024u);
#pragma unroll
                for (int i = 0; i < kCopiesR; ++i)
                        copy_r(i, s_r[buf] + copy_no_r(i, wave) * 1024u);
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
                        copy_to_lds(t * kDepth + piece_r[i] < depth && !(bad >> i & 1u) ? from_r[i] + step_r : zeros(),
                                    to);
                    });
        } else {
            if constexpr (!X8) {
#pragma unroll
                for (int i = 0; i < kCopiesC; ++i)
                        copy_to_lds(next_c[i] != ~0u ? base_c + offset_c[i] + (size_t)next_c[i] * ld_c : zeros(),
                                    s_c[buf] + copy_no_c(i, wave) * 1024u);
            } else {
#pragma unroll
                for (int i = 0; i < kCodes; ++i) {
                    const uint32_t col = code_col(i) < p.cols ? code_col(i) : 0u;
                    const bool in = next_x[i] != ~0u;
                    const size_t row = in ? next_x[i] : 0u;
                    codes[i] = *reinterpret_cast<const v4u*>(in ? p.c + row * ld_c + col : zeros());
                    const uint8_t* const sc = p.c_scales + row * p.c_groups;
                    // two scales of 8 columns each, the same where a group is wider
                    code_scale[i] = in ? sc[col / p.c_group] | (uint32_t)sc[(col + 8u) / p.c_group] << 8 : 0u;
                }
            }
#pragma unroll
            for (int i = 0; i < kCopiesR; ++i)
                    copy_to_lds(next_r[i] != ~0u ? from_r[i] + (size_t)next_r[i] * ld_r : zeros(),
                                s_r[buf] + copy_no_r(i, wave) * 1024u);
            find_sources(t + 1u);
        }
    };
    // X8: the codes as bf16 numbers, with their power-of-two scales, into LDS
    auto put_codes = [&](uint32_t buf) {
        if constexpr (X8) {
#pragma unroll
            for (int i = 0; i < kCodes; ++i) {
                const uint32_t at = i * 64u * kWaves + threadIdx.x, k = at / (TC / 16u), s = at % (TC / 16u);
                const uint32_t word[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
                uint4 v[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float scale = as_float((code_scale[i] >> (8 * h) & 255u) << 23);
                    v[h] = make_uint4(fp8_to_bf16<false>(word[2 * h], scale), fp8_to_bf16<true>(word[2 * h], scale),
                                      fp8_to_bf16<false>(word[2 * h + 1], scale),
                                      fp8_to_bf16<true>(word[2 * h + 1], scale));
                }
                char* const to = s_c[buf] + k * (TC * 2u) + (s ^ hash(k)) * 32u;
                *reinterpret_cast<uint4*>(to) = v[0];
                *reinterpret_cast<uint4*>(to + 16) = v[1];
            }
        }
    };

    v4f acc[NC][NR];
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < NR; ++j)
            acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    auto multiply = [&](uint32_t buf) {
#pragma unroll
        for (int h = 0; h < (int)kDepth / 32; ++h) {
            v8b a[NC], b[NR];
            const uint32_t k = 32u * h + 8u * q + (r >> 2); // the transposing reads' row
            const uint32_t key = (r >> 2) | (q & 1u) << 2;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const uint32_t tile = wc * NC + i;
                if constexpr (!kCT)
                    a[i] = *reinterpret_cast<const v8b*>(s_c[buf] + (tile * 16u + r) * 128u +
                                                         ((4u * h + q) ^ (r & 7u)) * 16u);
                else
                    a[i] = read_transposed(s_c[buf] + k * (TC * 2u) + (tile ^ key) * 32u + (r & 3u) * 8u, TC * 2u);
            }
#pragma unroll
            for (int j = 0; j < NR; ++j) {
                const uint32_t tile = wr * NR + j;
                if constexpr (!kRT)
                    b[j] = *reinterpret_cast<const v8b*>(s_r[buf] + (tile * 16u + r) * 128u +
                                                         ((4u * h + q) ^ (r & 7u)) * 16u);
                else
                    b[j] = read_transposed(s_r[buf] + k * (TR * 2u) + (tile ^ key) * 32u + (r & 3u) * 8u, TR * 2u);
            }
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int j = 0; j < NR; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
        }
    };

    // ---- the steps: RING - 1 on their way while one is multiplied
    const uint32_t steps = (depth + kDepth - 1) / kDepth;
    constexpr int kStep = (X8 ? 0 : kCopiesC) + kCopiesR; // a wave's copies of a step
    if (steps) {
        find_sources(0);
#pragma unroll
        for (uint32_t t = 0; t + 1u < (uint32_t)RING; ++t) // (past the last step zeros, unused)
            fetch(t, t);
        put_codes(0);
    }
    uint32_t buf = 0, ahead = RING - 1u;
#pragma clang loop unroll(disable) // (nor peeled)
    for (uint32_t t = 0; t < steps; ++t) {
        copies_done<(RING - 2) * kStep>();
        meet(); // step t is there, and nobody reads step t - 1 any more
        fetch(t + RING - 1u, ahead);
        multiply(buf);
        buf = buf + 1u < (uint32_t)RING ? buf + 1u : 0u;
        ahead = ahead + 1u < (uint32_t)RING ? ahead + 1u : 0u;
        put_codes(buf); // (past the last step unused: a branch here would draw the products behind it)
    }
    copies_done<0>(); // no copy outlives the workgroup's LDS

    // ---- results: a lane has four columns of a row
    const size_t first = (KIND == kWgrad ? expert * (size_t)p.out_rows : 0u) + row0;
#pragma unroll
    for (int j = 0; j < NR; ++j) {
        const uint32_t row = 16u * (wr * NR + j) + r;
        if (row >= rows)
            continue;
        const size_t line = (first + row) * p.cols;
        const bool none = !kRT && p.r_index && result_row[j] >= p.r_rows;
        v4f v[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i)
            v[i] = none ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : acc[i][j];
        auto column = [&](int i) { return col0 + 16u * (wc * NC + i) + 4u * q; };
        if constexpr (KIND == kWgrad)
            if (p.accumulate) {
                auto at = [&](int i) { return line + min(column(i), p.cols - 4u); };
                if (p.out_bf16)
                    add_result<v4b, __bf16, NC>(static_cast<const __bf16*>(p.out), v, at);
                else
                    add_result<v4f, float, NC>(static_cast<const float*>(p.out), v, at);
            }
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (column(i) < p.cols)
                store_result(p, line + column(i), v[i]);
    }
}

// The same for tiles of 256 x 256 by eight waves, 64 columns x 128 rows each.  A
// step's 64 k are two halves.  While the first half is multiplied, the second's
// fragments are read; then the waves meet (every one has read all of this step,
// and the next one is in LDS); while the second half is multiplied, the next
// step's first fragments are read and the step after that is copied over this
// one.  The waves read each fragment of LDS two or four times, 192 KiB a step, in
// some 1500 of the 2048 cycles that its matrix instructions take: 128 x 128 by
// each of four waves reads a third less, but leaves a SIMD one wave (1359 us
// against 894, 8192 x 8192 x 8192), and four steps of 32 k in LDS are no faster
// (896 .. 910).
//
// Bound by the matrix units and the power that they and LDS take: 8192 x 8192 x
// 8192 870 us forward, 795 dgrad (790 a library's; MFMA busy 65% of cycles at 1.83
// GHz, at 1.98 without the copies and 2.2 without the reads), 840 .. 950 wgrad.
// 4096 tokens' top-8 of 64 experts 7168 -> 4096 1820 us (1.04 PFLOP/s).  wgrad of
// short sums by its stores too: 64 experts 4096 x 2048 from 502 rows each 992 us,
// 416 of them what storing 2.1 GB takes by itself.
// X8: x in FP8 (wgrad).  XI, DI: wgrad's rows of x and of dy are found by an index.
template <int KIND, bool X8, bool XI, bool DI>
__global__ __launch_bounds__(512) void gemm_big_kernel(GemmParams p)
{
    constexpr uint32_t TC = 256, TR = 256, kWaves = 8;
    constexpr bool kCT = KIND != kForward, kRT = KIND == kWgrad;
    constexpr int kBlocks = 4;           // of 16 columns a wave
    constexpr int kCopies = 4;           // 1 KiB pieces of an operand's step a wave
    constexpr uint32_t kBytes = TC * kDepth * 2;
    constexpr int kCodes = X8 ? 2 : 1;   // 16-code pieces of x a thread
    __shared__ __attribute__((aligned(1024))) char s_c[2][kBytes];
    __shared__ __attribute__((aligned(1024))) char s_r[2][kBytes];

    const uint32_t lane = threadIdx.x & (kWaveSize - 1), r = lane & 15u, q = lane >> 4;
    const uint32_t wave = uniform(threadIdx.x / kWaveSize), wc = wave & 3u, wr = wave >> 2;

    // ---- this workgroup's tile
    const uint32_t col_tiles = (p.cols + TC - 1) / TC;
    uint32_t expert, row_base = 0, row0, rows, col0, depth;
    if constexpr (KIND == kWgrad) {
        const uint32_t row_tiles = (p.out_rows + TR - 1) / TR, per = row_tiles * col_tiles;
        const uint32_t t = xcd_tile_in_turns(blockIdx.x, p.run);
        if (t >= p.experts * per)
            return;
        expert = t / per;
        const uint32_t in = t - expert * per;
        const uint2 at = tile_in_group<4>(in, row_tiles, col_tiles);
        row0 = at.x * TR;
        rows = min(TR, p.out_rows - row0);
        col0 = at.y * TC;
        expert_rows(p.offsets, expert, p.n_rows, row_base, depth);
        row_base = uniform(row_base);
        depth = uniform(depth);
        if (p.accumulate && depth == 0)
            return;
    } else {
        Group g;
        uint32_t t = 0;
        if (!find_group(p.offsets, p.experts, p.n_rows, TR,
                        [&](uint32_t total) {
                            t = xcd_tile_in_turns(blockIdx.x, p.run);
                            return t / col_tiles;
                        },
                        g))
            return;
        expert = g.expert;
        const uint2 at = tile_in_group(t - g.first * col_tiles, g.tiles, col_tiles);
        row0 = g.row0 + at.x * TR;
        rows = min(TR, g.rows - at.x * TR);
        col0 = at.y * TC;
        depth = p.depth;
    }
    const uint32_t steps = (depth + kDepth - 1) / kDepth;

    // ---- where each lane's copies come from (layouts in LDS as in gemm_kernel)
    auto hash = [](uint32_t k) { return (k & 3u) | ((k >> 1) & 4u); };
    const uint32_t ld_c = (KIND == kForward ? p.depth : p.cols) * (X8 ? 1u : 2u);
    const uint32_t ld_r = (kRT ? p.out_rows : p.depth) * 2u;
    const char* base_c = p.c;
    if constexpr (KIND == kForward)
        base_c += ((size_t)expert * p.cols + col0) * ld_c;
    if constexpr (KIND == kDgrad)
        base_c += (size_t)expert * p.depth * ld_c;
    const uint32_t row_k = ((lane & 7u) ^ (lane >> 3)) * 8u; // [row][k]: the lane's first k of a step
    auto k_of = [&](int i) { return (i * kWaves + wave) * 2u + (lane >> 5); }; // [k][column]: its row k of copy i
    auto col_of = [&](int i) {                                                // ... and its column
        const uint32_t s = lane & 31u;
        return (((s >> 1) ^ hash(k_of(i))) * 2u + (s & 1u)) * 8u;
    };
    auto wgrad_offset_r = [&](int i, uint32_t ln) {
        const uint32_t k = (i * kWaves + wave) * 2u + (ln >> 5), sl = ln & 31u;
        const uint32_t col = row0 + (((sl >> 1) ^ hash(k)) * 2u + (sl & 1u)) * 8u;
        return (DI ? 0u : k * ld_r) + (col < p.out_rows ? col : 0u) * 2u; // (columns past the last are not stored)
    };
    uint32_t offset_c[kCopies], offset_r[kCopies], row_r[kCopies];
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        const uint32_t row = (i * kWaves + wave) * 8u + lane / 8u;
        if constexpr (!kCT) {
            offset_c[i] = min(row, p.cols - 1u - col0) * ld_c + row_k * 2u;
        } else {
            uint32_t col = col0 + col_of(i);
            col = col < p.cols ? col : 0u; // not stored
            offset_c[i] = (KIND == kDgrad || !XI ? k_of(i) * ld_c : 0u) + col * 2u;
        }
        if constexpr (!kRT) {
            uint32_t at = row0 + min(row, rows - 1u);
            if (p.r_index)
                at = (uint32_t)p.r_index[at];
            row_r[i] = at < p.r_rows ? at : 0u; // (a row that is none: any, and zeros as its result)
            offset_r[i] = row_r[i] * ld_r + row_k * 2u;
        } else {
            offset_r[i] = wgrad_offset_r(i, lane);
        }
    }

    // wgrad: the row of x or dy for the expert's row k by its index, to be looked at only when it is used: until then
    // it may be on its way
    auto indexed = [&](const int32_t* index, uint32_t k) { return (uint32_t)index[row_base + min(k, depth - 1u)]; };
    uint32_t next_c[kCopies], next_r[kCopies], next_x[kCodes]; // of the coming copies
    auto find_rows = [&](uint32_t t) {
        if constexpr (KIND == kWgrad && (DI || (XI && !X8))) {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                if constexpr (XI && !X8)
                    next_c[i] = indexed(p.c_index, t * kDepth + k_of(i));
                if constexpr (DI)
                    next_r[i] = indexed(p.r_index, t * kDepth + k_of(i));
            }
        }
    };
    // X8: a thread takes the 16 codes s of the rows i * 32 + threadIdx / 16
    const uint32_t code_s = threadIdx.x & 15u, code_k = threadIdx.x >> 4;
    const uint32_t code_col = X8 && col0 + code_s * 16u < p.cols ? col0 + code_s * 16u : 0u;
    const uint32_t code_g = X8 ? code_col / p.c_group : 0u; // (a group is 16 columns or a multiple)
    v4u codes[kCodes];
    uint8_t code_scale[kCodes];
    uint32_t scale_there[kCodes];
    auto find_code_rows = [&](uint32_t t) {
        if constexpr (X8 && XI)
#pragma unroll
            for (int i = 0; i < kCodes; ++i)
                next_x[i] = indexed(p.c_index, t * kDepth + i * 32u + code_k);
    };
    bool code_in[kCodes];
    // what the loads above left in registers is there (after copies_done): the compiler, which does not count the
    // copies, would wait for them too at the first use behind some
    auto codes_there = [&] {
        if constexpr (X8)
#pragma unroll
            for (int i = 0; i < kCodes; ++i) {
                scale_there[i] = code_scale[i];
                asm volatile("" : "+v"(codes[i]), "+v"(scale_there[i]));
                if constexpr (XI)
                    asm volatile("" : "+v"(next_x[i]));
            }
    };
    auto load_codes = [&](uint32_t t) {
        if constexpr (X8)
#pragma unroll
            for (int i = 0; i < kCodes; ++i) {
                const uint32_t k = t * kDepth + i * 32u + code_k, at = XI ? next_x[i] : row_base + min(k, depth - 1u);
                code_in[i] = k < depth && at < p.c_rows;
                const size_t row = at < p.c_rows ? at : 0u;
                codes[i] = *reinterpret_cast<const v4u*>(p.c + row * ld_c + code_col);
                code_scale[i] = p.c_scales[row * p.c_groups + code_g];
            }
    };
    auto put_codes = [&](int i, uint32_t buf) { // as bf16 numbers, with their power-of-two scales
        if constexpr (X8) {
            const uint32_t k = i * 32u + code_k, keep = code_in[i] ? ~0u : 0u;
            const uint32_t word[4] = {codes[i].x & keep, codes[i].y & keep, codes[i].z & keep, codes[i].w & keep};
            char* const to = s_c[buf] + k * (TC * 2u) + (code_s ^ hash(k)) * 32u;
            const float scale = as_float((scale_there[i] & keep) << 23); // (255, a NaN, would make one of the zeros)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<uint4*>(to + 16 * h) =
                    make_uint4(fp8_to_bf16<false>(word[2 * h], scale), fp8_to_bf16<true>(word[2 * h], scale),
                               fp8_to_bf16<false>(word[2 * h + 1], scale), fp8_to_bf16<true>(word[2 * h + 1], scale));
        }
    };

    // Copy i of an operand's step t.  FAST: whole steps whose offsets fit 32 bits, from a base that is the same for
    // the whole wave (past the last step that one again, unused); else past the depth, and for rows that are none,
    // zeros.
    auto row_of_copy = [&](bool by_index, const char* base, uint32_t at, uint32_t all, uint32_t ld, uint32_t t, int i,
                           uint32_t offset) -> const char* { // wgrad; offset: of the column, and of the row in the step
        const uint32_t k = t * kDepth + k_of(i);
        if (by_index)
            return at < all && k < depth ? base + (size_t)at * ld + offset : zeros();
        return k < depth ? base + (size_t)(row_base + t * kDepth) * ld + here(offset) : zeros();
    };
    auto copy_c = [&](auto fast, uint32_t t, uint32_t buf, int i) {
        char* const to = s_c[buf] + (i * kWaves + wave) * 1024u;
        if constexpr (KIND == kWgrad) {
            if constexpr (!X8)
                copy_to_lds(row_of_copy(XI, p.c, next_c[i], p.c_rows, ld_c, t, i, offset_c[i]), to);
        } else {
            const uint32_t u = decltype(fast)::value ? min(t, steps - 1u) : t, k = t * kDepth + (kCT ? k_of(i) : row_k);
            const size_t step = kCT ? (size_t)u * kDepth * ld_c : (size_t)u * (kDepth * 2u);
            if constexpr (decltype(fast)::value)
                copy_to_lds(base_c + step, offset_c[i], to);
            else
                copy_to_lds(k < depth ? base_c + step + here(offset_c[i]) : zeros(), to);
        }
    };
    auto copy_r = [&](auto fast, uint32_t t, uint32_t buf, int i) {
        char* const to = s_r[buf] + (i * kWaves + wave) * 1024u;
        if constexpr (KIND == kWgrad) {
            // X8: computed again each time, its registers are full
            copy_to_lds(row_of_copy(DI, p.r, next_r[i], p.r_rows, ld_r, t, i,
                                    X8 ? wgrad_offset_r(i, here(lane)) : offset_r[i]),
                        to);
        } else if constexpr (decltype(fast)::value) {
            copy_to_lds(p.r + (size_t)min(t, steps - 1u) * (kDepth * 2u), offset_r[i], to);
        } else {
            copy_to_lds(t * kDepth + row_k < depth ? p.r + (size_t)here(row_r[i]) * ld_r + (t * kDepth + row_k) * 2u : zeros(),
                        to);
        }
    };

    // fragments of half h of a step; the wave's row blocks are every second one, so that a tile of few rows is
    // shared evenly
    const uint32_t key = (r >> 2) | (q & 1u) << 2;
    auto read_c = [&](uint32_t buf, int h, int i) -> v8b {
        const uint32_t tile = wc * kBlocks + i;
        if constexpr (!kCT)
            return *reinterpret_cast<const v8b*>(s_c[buf] + (tile * 16u + r) * 128u + ((4u * h + q) ^ (r & 7u)) * 16u);
        else
            return read_transposed(s_c[buf] + (32u * h + 8u * q + (r >> 2)) * (TC * 2u) + (tile ^ key) * 32u +
                                       (r & 3u) * 8u,
                                   TC * 2u);
    };
    auto read_r = [&](uint32_t buf, int h, int j) -> v8b {
        const uint32_t tile = 2u * j + wr;
        if constexpr (!kRT)
            return *reinterpret_cast<const v8b*>(s_r[buf] + (tile * 16u + r) * 128u + ((4u * h + q) ^ (r & 7u)) * 16u);
        else
            return read_transposed(s_r[buf] + (32u * h + 8u * q + (r >> 2)) * (TR * 2u) + (tile ^ key) * 32u +
                                       (r & 3u) * 8u,
                                   TR * 2u);
    };

    // ---- the steps, and the results, with N row blocks a wave
    auto run = [&](auto n_blocks, auto fast) {
        constexpr int N = decltype(n_blocks)::value;
        constexpr int kCopiesR = kRT ? kCopies : (N + 1) / 2; // [row][k]: the rows that the blocks have
        v4f acc[kBlocks][N];
#pragma unroll
        for (int i = 0; i < kBlocks; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j)
                acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        if (steps) {
            v8b a[2][kBlocks], b[2][N]; // of the half at hand and of the next
            // codes of steps 0 and 1 by way of registers, then the copies, then the codes of step 2
            if constexpr (X8)
#pragma unroll
                for (uint32_t t = 0; t < 2; ++t) {
                    find_code_rows(t);
                    load_codes(t);
                    codes_there();
#pragma unroll
                    for (int i = 0; i < kCodes; ++i)
                        put_codes(i, t);
                }
#pragma unroll
            for (uint32_t t = 0; t < 2; ++t) {
                find_rows(t);
#pragma unroll
                for (int i = 0; i < kCopies; ++i) {
                    copy_c(fast, t, t, i);
                    if (i < kCopiesR)
                        copy_r(fast, t, t, i);
                }
            }
            find_rows(2);
            find_code_rows(2);
            load_codes(2);
            find_code_rows(3);
            copies_done<0>();
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kBlocks; ++i)
                a[0][i] = read_c(0, 0, i);
#pragma unroll
            for (int j = 0; j < N; ++j)
                b[0][j] = read_r(0, 0, j);
            // Fragments of a half in the order that the products need them, some beside each row block's products and
            // none beside the last ones, under which they arrive; the copies behind the products.
            constexpr int kReadsEach = N >= 8 ? 2 : 3, kCopiesEach = (kCopies + kCopiesR + N - 1) / N;
            auto read_some = [&](int group, int set, uint32_t from, int half) {
#pragma unroll
                for (int n = group * kReadsEach; n < (group + 1) * kReadsEach; ++n) {
                    if (n == 1)
                        b[set][0] = read_r(from, half, 0);
                    else if (n <= kBlocks)
                        a[set][n ? n - 1 : 0] = read_c(from, half, n ? n - 1 : 0);
                    else if (n < kBlocks + N)
                        b[set][n - kBlocks] = read_r(from, half, n - kBlocks);
                }
            };
#pragma clang loop unroll(disable) // (nor peeled)
            for (uint32_t t = 0; t < steps; ++t) {
                const uint32_t buf = t & 1u;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    __builtin_amdgcn_sched_barrier(0);
                    read_some(j, 1, buf, 1);
#pragma unroll
                    for (int i = 0; i < kBlocks; ++i)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[0][i], b[0][j], acc[i][j], 0, 0, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
                copies_done<0>();
                codes_there();
                __syncthreads(); // step t + 1 is there, and every wave has read all of step t
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    __builtin_amdgcn_sched_barrier(0);
                    read_some(j, 0, buf ^ 1u, 0);
#pragma unroll
                    for (int i = 0; i < kBlocks; ++i)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[1][i], b[1][j], acc[i][j], 0, 0, 0);
                    __builtin_amdgcn_sched_barrier(0);
                    if (X8 && j < kCodes)
                        put_codes(j, buf);
                    if (X8 && j == kCodes)
                        load_codes(t + 3u);
                    if (X8 && j == kCodes + 1)
                        find_code_rows(t + 4u);
                    if (X8 && j < kCopiesR)
                        copy_r(fast, t + 2u, buf, j);
#pragma unroll
                    for (int n = X8 ? kCopies + kCopiesR : j * kCopiesEach; n < (j + 1) * kCopiesEach; ++n) {
                        if (n < kCopies)
                            copy_c(fast, t + 2u, buf, n);
                        else if (n < kCopies + kCopiesR)
                            copy_r(fast, t + 2u, buf, n - kCopies);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
                // what the next copies need, on its way until the waves meet again
                find_rows(t + 3u);
            }
            copies_done<0>(); // no copy outlives the workgroup's LDS
        }

        // ---- results: a lane has four columns of a row
        const size_t first = (KIND == kWgrad ? expert * (size_t)p.out_rows : 0u) + row0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint32_t row = 16u * (2u * j + wr) + r;
            const bool none = KIND != kWgrad && p.r_index && row < rows && (uint32_t)p.r_index[row0 + row] >= p.r_rows;
            const size_t line = (first + row) * p.cols;
            v4f v[kBlocks];
#pragma unroll
            for (int i = 0; i < kBlocks; ++i)
                v[i] = none ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : acc[i][j];
            if constexpr (KIND == kWgrad)
                if (p.accumulate) {
                    const size_t from = (first + min(row, rows - 1u)) * p.cols;
                    auto at = [&](int i) { return from + min(col0 + 16u * (wc * kBlocks + i) + 4u * q, p.cols - 4u); };
                    if (p.out_bf16)
                        add_result<v4b, __bf16, kBlocks>(static_cast<const __bf16*>(p.out), v, at);
                    else
                        add_result<v4f, float, kBlocks>(static_cast<const float*>(p.out), v, at);
                }
            if (p.out_bf16) { // the same for every thread
#pragma unroll
                for (int i = 0; i < kBlocks; i += 2) {
                    const v4u pair = pair_columns(v[i], v[i + 1]);
                    const uint32_t col = col0 + 16u * (wc * kBlocks + i + (q & 1u)) + 8u * (q >> 1);
                    if (row < rows && col < p.cols)
                        *reinterpret_cast<v4u*>(static_cast<__bf16*>(p.out) + line + col) = pair;
                }
                continue;
            }
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
                const uint32_t col = col0 + 16u * (wc * kBlocks + i) + 4u * q;
                if (row < rows && col < p.cols)
                    *reinterpret_cast<v4f*>(static_cast<float*>(p.out) + line + col) = v[i];
            }
        }
    };
    using std::integral_constant;
    using std::bool_constant;
    // As many row blocks as the tile's rows need: of 64 experts with some 500 rows each, products of whole tiles would
    // be a fifth more (1816 us; 1830 with even numbers of blocks only).
    auto run_blocks = [&](auto fast) {
        const uint32_t blocks = KIND == kWgrad ? 8u : uniform((rows + 31u) / 32u);
        if (blocks > 7)
            run(integral_constant<int, 8>{}, fast);
        if constexpr (KIND != kWgrad) {
            if (blocks == 7)
                run(integral_constant<int, 7>{}, fast);
            else if (blocks == 6)
                run(integral_constant<int, 6>{}, fast);
            else if (blocks == 5)
                run(integral_constant<int, 5>{}, fast);
            else if (blocks == 4)
                run(integral_constant<int, 4>{}, fast);
            else if (blocks == 3)
                run(integral_constant<int, 3>{}, fast);
            else if (blocks <= 2)
                run(integral_constant<int, 2>{}, fast);
        }
    };
    if (KIND != kWgrad && depth % kDepth == 0 && (uint64_t)p.r_rows * ld_r < (1ull << 32))
        run_blocks(bool_constant<true>{});
    else
        run_blocks(bool_constant<false>{});
}

// At most how many tiles of TR rows by TC columns there are, however the rows lie, in workgroups of whole turns
// over the XCDs, `run` tiles each.
template <int KIND>
uint64_t workgroups(const GemmParams& p, uint32_t tc, uint32_t tr, uint32_t run = 1)
{
    const uint64_t col_tiles = ((uint64_t)p.cols + tc - 1) / tc, most = p.n_rows < p.experts ? p.n_rows : p.experts;
    const uint64_t row_tiles =
        KIND == kWgrad ? (uint64_t)p.experts * (((uint64_t)p.out_rows + tr - 1) / tr) : p.n_rows / tr + most;
    return (row_tiles * col_tiles + kXcds * run - 1) / (kXcds * run) * (kXcds * run);
}

template <int KIND, int TC, int TR, int WC, int WR, int RING, bool X8 = false>
tk_status launch(const GemmParams& p, hipStream_t s)
{
    const uint64_t blocks = workgroups<KIND>(p, TC, TR);
    if (!launchable(blocks, 64 * WC * WR))
        return TK_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((gemm_kernel<KIND, TC, TR, WC, WR, X8, RING>), dim3((uint32_t)blocks), dim3(64 * WC * WR), 0, s, p);
    return hipGetLastError() == hipSuccess ? TK_OK : TK_ERR_HIP;
}

template <int KIND, bool X8 = false, bool XI = false, bool DI = false>
tk_status launch_big(GemmParams p, hipStream_t s)
{
    // Tiles that an XCD takes together.  wgrad's cost as much as their expert has rows: every XCD takes its part of each
    // expert.  64 experts 4096 x 2048 of unlike popularity (141 .. 1098 rows) 1149 us with an eighth of all tiles an XCD,
    // 981 .. 992 so; with 512 rows for each of 64, 7168 x 2048 1223 and 1130, 4096 x 7168 2332 and 2502.  Forward and
    // dgrad, 2.5 row tiles an expert, the last one shorter: dgrad 1134 and 1111, forward 1851 and 1833.
    const uint32_t per = ((p.out_rows + 255u) / 256u) * ((p.cols + 255u) / 256u);
    const uint64_t tiles = KIND == kWgrad ? per : tiles_of(average_rows(p.n_rows, p.experts), p.experts, p.cols, 256, 256);
    p.run = (uint32_t)std::min<uint64_t>((tiles + kXcds - 1u) / kXcds, KIND == kWgrad ? 64u : 32u);
    const uint64_t blocks = workgroups<KIND>(p, 256, 256, p.run);
    if (!launchable(blocks, 512))
        return TK_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((gemm_big_kernel<KIND, X8, XI, DI>), dim3((uint32_t)blocks), dim3(512), 0, s, p);
    return hipGetLastError() == hipSuccess ? TK_OK : TK_ERR_HIP;
}

} // namespace

namespace tk_gemm {

// Which tiles: the largest that the rows of an expert fill, of which there are enough for 256 CUs.  In us, 4096 ->
// 4096 for one expert: 64 rows 50 with 256 x 256 tiles, 29 with 128 columns x 64 rows, 19 with 64 x 64, 15 with 64 x
// 16; 256 rows 78, 30, 21, 35; 1024 rows 81, 45, 56, 133; 4096 rows 125, 200, 240, 494.  7168 -> 4096 for 64 experts:
// 24 rows each 772, 668, 697, 859; 64 each 787, 694, 794, 1324; 128 each 793 (256 x 256), 942 (128 x 64).  The rows of
// each expert are on the device; their average stands for them: 1000 rows of 4096 -> 4096 that all fall to one of 64
// experts take 138 us in 64 x 16 tiles (42 where that expert is the only one).
tk_status launch_forward(const GemmParams& p, hipStream_t s)
{
    const uint64_t load = average_rows(p.n_rows, p.experts);
    auto tiles = [&](uint32_t tr, uint32_t tc) { return tiles_of(load, p.experts, p.cols, tr, tc); };
    if (load > 64 && tiles(256, 256) >= 128)
        return launch_big<kForward>(p, s);
    if (load > 16 && tiles(64, 128) >= 384)
        return launch<kForward, 128, 64, 2, 2, 3>(p, s);
    if (load > 16 && tiles(64, 64) >= 128)
        return launch<kForward, 64, 64, 2, 2, 3>(p, s);
    return launch<kForward, 64, 16, 4, 1, 4>(p, s);
}

} // namespace tk_gemm

extern "C" tk_status tk_expert_gemm_dgrad(const void* dy, int64_t dy_rows, const int32_t* row_index,
                                          const int32_t* expert_offsets, int64_t n_rows, const void* w,
                                          int64_t experts, int64_t out_features, int64_t in_features,
                                          tk_dtype out_dtype, void* dx, void* stream)
{
    const bool out_bf16 = (int)out_dtype == TK_DTYPE_BF16;
    const RowsArgs rows = {dy_rows, row_index};
    if (!valid_rows(rows, expert_offsets, n_rows, experts) || !valid_shape(out_features, in_features, 8) ||
        (!out_bf16 && (int)out_dtype != TK_DTYPE_FP32))
        return TK_ERR_INVALID_ARG;
    if (n_rows > 0 && ((dy_rows > 0 && !dy) || !w || !dx))
        return TK_ERR_INVALID_ARG;
    if (!aligned(dy, 16) || !aligned(w, 16) || !aligned(dx, 16))
        return TK_ERR_INVALID_ARG;
    if (experts > kMaxExperts)
        return TK_ERR_UNSUPPORTED;
    const size_t o_bytes = (size_t)n_rows * (size_t)in_features * (out_bf16 ? 2u : 4u);
    if (overlaps(dx, o_bytes, dy, (size_t)dy_rows * (size_t)out_features * 2u) ||
        overlaps(dx, o_bytes, w, (size_t)experts * (size_t)out_features * (size_t)in_features * 2u) ||
        overlaps_rows(dx, o_bytes, row_index, expert_offsets, n_rows, experts))
        return TK_ERR_INVALID_ARG;
    if (n_rows == 0)
        return TK_OK;
    GemmParams p{};
    p.c = static_cast<const char*>(w);
    p.r = static_cast<const char*>(dy_rows ? dy : w); // (no row: what is read in its place is not used)
    p.r_index = row_index;
    p.r_rows = (uint32_t)dy_rows;
    p.offsets = expert_offsets;
    p.n_rows = (uint32_t)n_rows;
    p.experts = (uint32_t)experts;
    p.cols = (uint32_t)in_features;
    p.depth = (uint32_t)out_features;
    p.out = dx;
    p.out_bf16 = out_bf16;
    hipStream_t s = static_cast<hipStream_t>(stream);
    // as launch_forward; tiles kept [k][column] have 128 columns or more
    const uint64_t load = average_rows(p.n_rows, p.experts);
    auto tiles = [&](uint32_t tr, uint32_t tc) { return tiles_of(load, p.experts, p.cols, tr, tc); };
    if (load > 64 && tiles(256, 256) >= 128)
        return launch_big<kDgrad>(p, s);
    if (load > 16 && tiles(64, 128) >= 128)
        return launch<kDgrad, 128, 64, 2, 2, 2>(p, s);
    return launch<kDgrad, 128, 16, 4, 1, 3>(p, s);
}

extern "C" tk_status tk_expert_gemm_wgrad(const void* dy, int64_t dy_rows, const int32_t* dy_index, const void* x,
                                          const void* x_scales, int x_dtype, int64_t x_group, int64_t x_rows,
                                          const int32_t* x_index, const int32_t* expert_offsets, int64_t n_rows,
                                          int64_t experts, int64_t out_features, int64_t in_features, int accumulate,
                                          tk_dtype out_dtype, void* dw, void* stream)
{
    const bool out_bf16 = (int)out_dtype == TK_DTYPE_BF16, fp8 = x_dtype == TK_DTYPE_FP8;
    if (!valid_rows({dy_rows, dy_index}, expert_offsets, n_rows, experts) ||
        !valid_rows({x_rows, x_index}, expert_offsets, n_rows, experts) ||
        !valid_shape(out_features, in_features, fp8 ? 16 : 8) || (!fp8 && x_dtype != TK_DTYPE_BF16) ||
        (!out_bf16 && (int)out_dtype != TK_DTYPE_FP32) || (accumulate != 0 && accumulate != 1))
        return TK_ERR_INVALID_ARG;
    if (fp8 && (x_group < 0 || (x_group && in_features % x_group != 0)))
        return TK_ERR_INVALID_ARG;
    if (!dw || (n_rows > 0 && ((dy_rows > 0 && !dy) || (x_rows > 0 && (!x || (fp8 && !x_scales))))))
        return TK_ERR_INVALID_ARG;
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dw, 16))
        return TK_ERR_INVALID_ARG;
    if (experts > kMaxExperts || (fp8 && x_group % 8 != 0))
        return TK_ERR_UNSUPPORTED;
    const int64_t group = fp8 && x_group ? x_group : in_features;
    const size_t o_bytes = (size_t)experts * (size_t)out_features * (size_t)in_features * (out_bf16 ? 2u : 4u);
    if (overlaps(dw, o_bytes, dy, (size_t)dy_rows * (size_t)out_features * 2u) ||
        overlaps(dw, o_bytes, x, (size_t)x_rows * (size_t)in_features * (fp8 ? 1u : 2u)) ||
        (fp8 && overlaps(dw, o_bytes, x_scales, (size_t)x_rows * (size_t)(in_features / group))) ||
        overlaps_rows(dw, o_bytes, dy_index, expert_offsets, n_rows, experts) ||
        overlaps_rows(dw, o_bytes, x_index, nullptr, n_rows, experts))
        return TK_ERR_INVALID_ARG;
    if (dy_rows == 0 || x_rows == 0) // every row stands for zeros
        n_rows = 0;
    if (n_rows == 0 && accumulate)
        return TK_OK;
    GemmParams p{};
    p.c = static_cast<const char*>(x);
    p.c_scales = static_cast<const uint8_t*>(x_scales);
    p.c_group = (uint32_t)group;
    p.c_groups = (uint32_t)(in_features / group);
    p.c_index = x_index;
    p.c_rows = (uint32_t)x_rows;
    p.r = static_cast<const char*>(dy);
    p.r_index = dy_index;
    p.r_rows = (uint32_t)dy_rows;
    p.offsets = n_rows ? expert_offsets : nullptr;
    p.n_rows = (uint32_t)n_rows;
    p.experts = (uint32_t)experts;
    p.cols = (uint32_t)in_features;
    p.out_rows = (uint32_t)out_features;
    p.out = dw;
    p.out_bf16 = out_bf16;
    p.accumulate = accumulate;
    hipStream_t s = static_cast<hipStream_t>(stream);
    // The large tiles wherever a result is not much smaller than one, however few there are: a sum is one workgroup's.
    // 8192 rows of one expert 1024 x 1024 165 us (16 workgroups, 128 steps each), of eight experts 35.
    if (p.out_rows >= 192 && p.cols >= 192 && (!fp8 || group % 16 == 0)) {
        if (fp8)
            return x_index ? (dy_index ? launch_big<kWgrad, true, true, true>(p, s) : launch_big<kWgrad, true, true>(p, s))
                           : (dy_index ? launch_big<kWgrad, true, false, true>(p, s) : launch_big<kWgrad, true>(p, s));
        return x_index ? (dy_index ? launch_big<kWgrad, false, true, true>(p, s) : launch_big<kWgrad, false, true>(p, s))
                       : (dy_index ? launch_big<kWgrad, false, false, true>(p, s) : launch_big<kWgrad>(p, s));
    }
    if (fp8)
        return launch<kWgrad, 128, 128, 2, 2, 2, true>(p, s);
    return launch<kWgrad, 128, 128, 2, 2, 2>(p, s);
}
