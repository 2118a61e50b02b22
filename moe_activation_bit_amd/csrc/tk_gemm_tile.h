// tk_gemm_tile.h -- device pieces shared by the grouped matrix products
// (tk_gemm.hip, tk_gemm_q.hip): a workgroup's tile among the experts' ragged
// rows, the copies from memory straight into LDS, and the argument checks.
#pragma once

#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>

#include "tk.h"
#include "tk_expert.h"
#include "tk_quant.h"

namespace tk_gemm {

using namespace tk_detail;

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef __bf16 v4b __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));

constexpr uint32_t kXcds = 8;
constexpr uint32_t kMaxExperts = 512;

// 16 bytes of zeros: what a copy reads in the place of columns past a row's
// end, of rows past an expert's, and of rows whose index names none
__device__ __attribute__((aligned(16))) const uint4 g_zeros = {0, 0, 0, 0};

__device__ __forceinline__ const char* zeros() { return reinterpret_cast<const char*>(&g_zeros); }

// 16 bytes a lane from memory into LDS without a register in between: lane l's
// go to `to` + 16 l (`to` the same for the whole wave).  Written out, since the
// compiler, which cannot tell which half of a double buffer a copy fills, would
// wait for it before any later read of LDS; here copies_done() says when they are
// there.  (Its own counts of loads in flight are then too low, which only makes it
// wait for more.)  M0 is the LDS address (the compiler keeps nothing in it: it is reserved, and
// no other instruction of these kernels takes it); an instruction has to lie
// between its write and its use.
__device__ __forceinline__ uint32_t lds_address(const void* p)
{
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
__device__ __forceinline__ void copy_to_lds(const char* from, const char* to)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 :
                 : "v"(from), "s"(lds_address(to))
                 : "memory");
}
// ... from `base` (the same for the whole wave) + the lane's offset.  (A vector instruction that wrote the base,
// which the compiler would keep five instructions before a load that it can see, may come right before this.)
__device__ __forceinline__ void copy_to_lds(const char* base, uint32_t offset, const char* to)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(offset), "s"(base), "s"(lds_address(to))
                 : "memory");
}
// Waits until at most N of this wave's copies (and other loads) are in flight.
template <int N>
__device__ __forceinline__ void copies_done()
{
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// The waves of a workgroup meet: what each has read of LDS is read, what it has
// written there is written.  (The language's barrier would also wait for every
// copy.)
__device__ __forceinline__ void meet()
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// two of a word's four E4M3 codes, the lower or the upper ones, times a power of two
template <bool UPPER>
__device__ __forceinline__ uint32_t fp8_to_bf16(uint32_t codes, float scale)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, UPPER));
}

// Results of a row, x of block i and y of block i + 1, four columns a lane (4q ..)
// -> eight columns a lane in bf16: 8 (q / 2) .. of block i + (q & 1).  Lanes whose
// q differ in the lowest bit exchange a half, so that a row's 64 bytes are
// stored together.
__device__ __forceinline__ v4u pair_columns(v4f x, v4f y)
{
    typedef __bf16 v2b __attribute__((ext_vector_type(2)));
    auto pack = [](float a, float b) { return __builtin_bit_cast(uint32_t, v2b{(__bf16)a, (__bf16)b}); };
    const auto lo = __builtin_amdgcn_permlane16_swap(pack(x[0], x[1]), pack(y[0], y[1]), false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(pack(x[2], x[3]), pack(y[2], y[3]), false, false);
    return v4u{lo[0], hi[0], lo[1], hi[1]};
}

// x, opaque to the compiler: what is derived from it inside a loop stays there
// instead of being computed before the loop and held (or spilled) through it
__device__ __forceinline__ uint32_t here(uint32_t x)
{
    asm volatile("" : "+v"(x));
    return x;
}

// A number that is the same for the whole wave, in a scalar register
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __builtin_amdgcn_readfirstlane(x); }

struct Group {
    uint32_t expert;
    uint32_t row0, rows; // the expert's rows
    uint32_t tiles;      // its tiles of rows
    uint32_t first;      // number of the tiles before it
};

// The expert's rows by the offsets, kept inside 0 .. n whatever they hold.
__device__ __forceinline__ void expert_rows(const int32_t* off, uint32_t e, uint32_t n, uint32_t& row0, uint32_t& rows)
{
    if (!off) {
        row0 = 0;
        rows = n;
        return;
    }
    const int32_t lo = min(max(off[e], 0), (int32_t)n), hi = min(max(off[e + 1], lo), (int32_t)n);
    row0 = (uint32_t)lo;
    rows = (uint32_t)(hi - lo);
}

// The expert that row tile `u` belongs to, tiles of `height` rows numbered over
// the experts in order; `total` their number.  A wave by itself: each lane
// counts the tiles of up to eight consecutive experts, a scan over the lanes
// finds the lane, and the lane the expert.  False when u is past the last.
template <typename F>
__device__ __forceinline__ bool find_group(const int32_t* off, uint32_t experts, uint32_t n, uint32_t height,
                                           F&& tile_of_total, Group& g)
{
    const uint32_t lane = threadIdx.x & (kWaveSize - 1);
    if (!off) {
        g.expert = g.row0 = g.first = 0;
        g.rows = n;
        g.tiles = (n + height - 1) / height;
        const uint32_t u = tile_of_total(g.tiles);
        return u < g.tiles;
    }
    constexpr uint32_t kPer = kMaxExperts / kWaveSize;
    const uint32_t per = (experts + kWaveSize - 1) / kWaveSize, e0 = lane * per;
    int32_t at[kPer + 1];
#pragma unroll
    for (uint32_t i = 0; i <= kPer; ++i) // every load first
        at[i] = i <= per ? off[min(e0 + i, experts)] : 0;
    uint32_t mine = 0;
#pragma unroll
    for (uint32_t i = 0; i < kPer; ++i) {
        const int32_t lo = min(max(at[i], 0), (int32_t)n), hi = min(max(at[i + 1], lo), (int32_t)n);
        if (i < per && e0 + i < experts)
            mine += ((uint32_t)(hi - lo) + height - 1) / height;
    }
    uint32_t sum = mine;
#pragma unroll
    for (int d = 1; d < kWaveSize; d <<= 1) {
        const uint32_t other = (uint32_t)__shfl_up((int)sum, d);
        sum += lane >= (uint32_t)d ? other : 0u;
    }
    const uint32_t u = tile_of_total(uniform((uint32_t)__shfl((int)sum, kWaveSize - 1)));
    const uint64_t past = __builtin_amdgcn_ballot_w64(sum > u);
    if (past == 0)
        return false;
    uint32_t first = sum - mine, expert = 0, row0 = 0, rows = 0, tiles = 0;
    bool found = false;
#pragma unroll
    for (uint32_t i = 0; i < kPer; ++i) {
        const int32_t lo = min(max(at[i], 0), (int32_t)n), hi = min(max(at[i + 1], lo), (int32_t)n);
        const uint32_t t = ((uint32_t)(hi - lo) + height - 1) / height;
        if (i < per && e0 + i < experts && !found) {
            if (first + t > u) {
                found = true;
                expert = e0 + i;
                row0 = (uint32_t)lo;
                rows = (uint32_t)(hi - lo);
                tiles = t;
            } else {
                first += t;
            }
        }
    }
    const int who = __builtin_ctzll(past);
    g.expert = __builtin_amdgcn_readlane(expert, who);
    g.row0 = __builtin_amdgcn_readlane(row0, who);
    g.rows = __builtin_amdgcn_readlane(rows, who);
    g.tiles = __builtin_amdgcn_readlane(tiles, who);
    g.first = __builtin_amdgcn_readlane(first, who);
    return true;
}

// Workgroups go to the eight XCDs in turn; tile number for a workgroup so that
// each XCD takes a run of consecutive tiles, which share weights or rows in its
// L2.  `total` or more: none.
__device__ __forceinline__ uint32_t xcd_tile(uint32_t block, uint32_t total)
{
    const uint32_t run = (total + kXcds - 1) / kXcds, i = block / kXcds;
    return i < run ? (block % kXcds) * run + i : total;
}

// ... `run` of every 8 run tiles, so that experts with many rows do not all fall
// to one XCD.
__device__ __forceinline__ uint32_t xcd_tile_in_turns(uint32_t block, uint32_t run)
{
    const uint32_t i = block / kXcds;
    return (i / run * kXcds + block % kXcds) * run + i % run;
}

// (row tile, column tile) of an expert's tile: eight row tiles by all column
// tiles at a time, rows first, so that the 32 tiles which an XCD's CUs have at
// hand are about as many rows as columns and share them in its L2.
template <uint32_t kHeight = 8>
__device__ __forceinline__ uint2 tile_in_group(uint32_t tile, uint32_t row_tiles, uint32_t col_tiles)
{
    const uint32_t band = tile / (kHeight * col_tiles), in = tile - band * (kHeight * col_tiles);
    const uint32_t height = min(kHeight, row_tiles - band * kHeight);
    return make_uint2(band * kHeight + in % height, in / height);
}

// 64-bit number of a tile in bounds for a launch
inline bool launchable(uint64_t blocks, uint32_t threads) { return blocks * threads < (1ull << 32); }

} // namespace tk_gemm
