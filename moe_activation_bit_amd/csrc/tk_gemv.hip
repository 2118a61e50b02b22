// tk_gemv.hip -- the experts' matrix-vector products with 4-bit weights, behind
// tk_expert_gemv_fp4 in include/tk_layer.h.
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>
#include <type_traits>

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
    uint32_t x_div;      // out row r reads x row r / x_div
    uint32_t experts;
    uint32_t out_features;
    uint32_t in_features;
    uint32_t groups, x_groups; // scales a row
    int out_bf16;
    uint32_t group_magic, x_group_magic;       // of the groups' width in blocks of 32 columns
    uint32_t group_magic128, x_group_magic128; // ... in steps of 128
    uint32_t steps;      // of kStep columns, the last part-filled when in_features is no multiple
    uint32_t steps_wave; // a wave's share of them
    uint32_t steps_part; // ... summed in parts of so many, whose sums are then added in order
    uint32_t ks;         // waves that share a tile's columns: 1, 2 or 4
    uint32_t tiles;      // tiles of 16 weight rows a wave goes through
    uint32_t pass;       // x rows of a pass, at most
    uint32_t lds_x;      // bytes for staged rows
    int by_row;
};

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));

// ceil(2^32 / d), by which divide() is exact for q * d < 2^32; 0 stands for d = 1
__host__ __device__ __forceinline__ uint32_t magic(uint32_t d) { return d <= 1u ? 0u : 0xFFFFFFFFu / d + 1u; }
// q / d by d's magic()
__device__ __forceinline__ uint32_t divide(uint32_t q, uint32_t magic) { return magic ? __umulhi(q, magic) : q; }

// two of a word's four E4M3 codes, the lower or the upper ones, times a power of two
template <bool UPPER>
__device__ __forceinline__ uint32_t fp8_to_bf16(uint32_t codes, float scale)
{
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, UPPER));
}

// x, opaque to the compiler: what is derived from it inside a loop stays there
// instead of being computed before the loop and held (or spilled) through it
__device__ __forceinline__ uint32_t here(uint32_t x)
{
    asm volatile("" : "+v"(x));
    return x;
}

// LDS that only this wave's lanes exchange through: what was written before is
// read after, with no wait on the other waves
__device__ __forceinline__ void wave_exchange()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// 16 bytes of weights, past the caches when nothing reads them again
template <bool STREAM>
__device__ __forceinline__ v4u load_weights(const char* at)
{
    const v4u* const p = reinterpret_cast<const v4u*>(at);
    return STREAM ? __builtin_nontemporal_load(p) : *p;
}

// f(0), f(1), ... f(N - 1), each with its number as a constant
template <int N, int I = 0, typename F>
__device__ __forceinline__ void for_slots(F&& f)
{
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        for_slots<N, I + 1>(f);
    }
}

constexpr int kTile = 16;            // weight rows and x rows of a matrix instruction
constexpr int kStep = 256;           // columns of a step: 128 bytes, a cache line, of each weight row
constexpr int kAhead = 2;            // steps of weights in flight
constexpr uint32_t kMaxStage = 16;   // steps staged at a time at most
constexpr uint32_t kStepBytes = 512; // a staged x row's bytes a step
constexpr uint32_t kRowPad = 16;     // between staged x rows, which would else share their LDS banks
constexpr uint32_t kCus = 256, kCuLds = 160 * 1024;
constexpr uint32_t kScalePitch = 8 * kMaxStage + 8; // bytes of a weight row's staged scales

// LDS of a workgroup beside the staged x rows: the row lists, a step of weights and the scales of each wave
constexpr uint32_t kOwnLds = kThreads / kWaveSize * (kTile * 8 + kTile * 128 + kTile * kScalePitch);

// Matrix instructions on 16 weight rows at a time, for up to 16 of the rows that
// chose the expert.  Codes and FP8 activations become bf16 in
// registers, with their UE8M0 scales on the way: two and four significant bits,
// exact (but for activations below 2^-133, bf16's smallest step), and the
// products and sums of the 16x16x32 bf16 instructions are those of fp32.  (The E2M1 x E4M3 instruction would take the
// codes as they are, but drops what lies 2^-14 below the largest product of a
// step: random E4M3 bytes gave sums off by up to 7.7e-5 of their terms'
// magnitude, where the bf16 instructions were exact.)
//
// What bounds it is the weights' bytes (7168 -> 4096, top-8 of 8 experts for one
// token: 24.1 us, 5.2 TB/s, a bare read of as many bytes 19.4; 2048 -> 7168 for 16
// tokens' top-8 of 64: 80 us, 5.5 TB/s, a bare read 64; one row of a single
// expert, 7168 -> 4096: 8 us, a launch and the row's staging; scales of other
// groups than 32 columns, or in fp32, are read one by one: 7168 -> 4096 with one
// for 128 columns 29.5 us, in fp32 29.8), so everything else keeps out of their
// way.  For many rows of one expert it is the staging of the rows, once for every
// pass and workgroup (64 rows of 7168 -> 4096: 23 us in bf16, 25.5 in FP8).
// A wave reads a step's 16 x 128 bytes with two instructions of eight
// whole lines (lane l: row l / 8, 16 bytes l % 8), kAhead steps before their
// use, and passes them through 2 KiB of LDS of its own into the instruction's
// layout, lane (r, q) = (l & 15, l >> 4): weight row r, columns 32q.. of each
// half.  (Read in that layout, a line is asked for by two instructions and the
// lines in flight overfill the L1: 30.2 us instead of 25.8 for a bare stream of
// the 7168 -> 4096 top-8 weights.)  The x rows, as bf16, and the scales are
// staged in LDS, at most kMaxStage steps at a time (scales read step by step
// cost as many line requests as the weights: 25.8 instead of 24.7 us).
// fp32 scales enter afterwards: one scale a row in the epilogue, one for 128
// columns or a multiple of that on each half step's own result (PART 1: the
// activations' alone; 2: the weights' too).
// A result's column n (x row) is lane & 15, its rows 4q .. 4q + 3.
//   FAST: UE8M0 weight scales of 32 columns and whole steps; else any.
//   STREAM: weights past the caches.
template <int XK, int PART, bool FAST, bool STREAM>
__global__ __launch_bounds__(kThreads, PART == 2 ? 3 : 4) void gemv_fp4_kernel(GemvParams p)
{
    constexpr uint32_t kWaves = kThreads / kWaveSize;
    __shared__ uint2 s_list[kWaves][kTile]; // an output row and its x row
    __shared__ v4u s_w4[kWaves][kTile * 8];
    __shared__ uint2 s_ws2[kWaves][kTile * kScalePitch / 8];
    extern __shared__ uint4 s_x4[]; // the staged rows, then their fp32 scales
    char* const s_x = reinterpret_cast<char*>(s_x4);
    float* const s_sx = reinterpret_cast<float*>(s_x + p.lds_x);
    const uint32_t lane = threadIdx.x & (kWaveSize - 1);
    const uint32_t r = lane & 15u, q = lane >> 4;
    const uint32_t wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveSize);
    const uint32_t ks = wv & (p.ks - 1u), rt = wv / p.ks;
    // this wave's weight rows of an expert: tiles o_first, + o_next, ... of which it has p.tiles
    const uint32_t o_next = kWaves / p.ks * kTile;
    const uint32_t o_first = blockIdx.x * p.tiles * o_next + rt * kTile;
    // its steps of a row: `share` from b0 on (none from step 0 on when the waves before it have them all)
    const uint32_t share = ks * p.steps_wave < p.steps ? min(p.steps_wave, p.steps - ks * p.steps_wave) : 0u;
    const uint32_t b0 = share ? ks * p.steps_wave : 0u;
    const uint32_t last_step = share ? share - 1u : 0u;
    const uint64_t below = (1ull << lane) - 1u;
    const bool x_part = PART != 0 && XK == kXFp8F32 && p.x_groups > 1;
    // x rows of a pass: what leaves room for kAhead steps of each
    const uint32_t pass_rows = min(p.pass, p.lds_x / (p.ks * (kAhead * kStepBytes + kRowPad)));
    // LDS slots of this lane's weights: row r keeps columns 32p.. in slot p ^ (r / 2), so that neither the
    // writes nor the reads of 16 rows meet in a bank
    const uint32_t lrow = lane >> 3, lpiece = lane & 7u;
    v4u* const w_put = s_w4[wv] + lrow * 8u + (lpiece ^ (lrow >> 1));
    v4u* const w_put8 = s_w4[wv] + (lrow + 8u) * 8u + (lpiece ^ ((lrow + 8u) >> 1));
    const v4u* const w_get = s_w4[wv] + r * 8u + (q ^ (r >> 1));
    const v4u* const w_get4 = s_w4[wv] + r * 8u + ((q + 4u) ^ (r >> 1));
    char* const s_ws = reinterpret_cast<char*>(s_ws2[wv]);

    // One workgroup: ks waves along the columns of each of kWaves / ks tiles of
    // 16 weight rows.  Its rows are those whose expert is e, in order,
    // pass_rows at a time: z takes the passes z, z + gridDim.z, ...  by_row: y is
    // a row, and the first row of an expert does the work of all of them; else y
    // is an expert, and the one past the last writes the absent rows' zeros.  Every branch around a barrier is the
    // same for all waves.
    const uint32_t y = blockIdx.y;
    uint32_t e = 0, next = 0, seen = 0, first = blockIdx.z * pass_rows; // of the expert's rows
    if (p.idx) {
        if (p.by_row) {
            next = y;
            e = (uint32_t)p.idx[y];
            bool earlier = false;
            for (uint32_t base = 0; base < y; base += kWaveSize)
                earlier |= base + lane < y && (uint32_t)p.idx[base + lane] == e;
            if (e < p.experts && __builtin_amdgcn_ballot_w64(earlier) != 0)
                return; // an earlier row's workgroup does this one
        } else {
            e = y;
        }
    }
    auto zero_row = [&](uint32_t row) {
        for (uint32_t i = threadIdx.x; i < p.tiles * o_next; i += kThreads) {
            const uint32_t o = blockIdx.x * p.tiles * o_next + i;
            if (o >= p.out_features)
                break;
            if (p.out_bf16)
                static_cast<uint16_t*>(p.out)[(size_t)row * p.out_features + o] = 0;
            else
                static_cast<float*>(p.out)[(size_t)row * p.out_features + o] = 0.0f;
        }
    };
    if (e >= p.experts) { // absent rows: this one, or all of them
        if (blockIdx.z)
            return;
        for (uint32_t base = p.by_row ? y & ~(uint32_t)(kWaveSize - 1) : 0u; base < (p.by_row ? y + 1u : p.rows);
             base += kWaveSize) {
            const uint32_t mine = base + lane;
            const bool hit = p.by_row ? mine == y : mine < p.rows && (uint32_t)p.idx[mine] >= p.experts;
            for (uint64_t mask = __builtin_amdgcn_ballot_w64(hit); mask; mask &= mask - 1u)
                zero_row(base + (uint32_t)__builtin_ctzll(mask));
        }
        return;
    }

    const size_t e_row = (size_t)e * p.out_features;
    // The weights of the wave's steps go through kAhead slots of registers, over the tiles' ends: `cur` is the
    // tile that is computed, `nxt` the one after it.  Tile rows past the last weight row read that row, and
    // their results are not stored.
    struct Tile {
        const char* base;   // its first row (wave-uniform)
        uint32_t off, off8; // bytes from there to this lane's 16 of row lane / 8, and of row lane / 8 + 8
    };
    auto tile = [&](uint32_t j) {
        const uint32_t o = o_first + j * o_next, last = p.out_features - 1u, first = min(o, last);
        const uint32_t row_bytes = p.in_features / 2u, ln = here(lane), lrow = ln >> 3, lpiece = ln & 7u;
        return Tile{reinterpret_cast<const char*>(p.codes) + (e_row + first) * row_bytes,
                    (min(o + lrow, last) - first) * row_bytes + 16u * lpiece,
                    (min(o + lrow + 8u, last) - first) * row_bytes + 16u * lpiece};
    };
    v4u w0[kAhead], w1[kAhead];
    auto fetch = [&](auto slot, const Tile& from, uint32_t t) { // the wave's step t of a tile into a slot
        constexpr int u = decltype(slot)::value;
        const uint32_t b = b0 + t;
        if constexpr (FAST) {
            const char* const at = from.base + (size_t)b * (kStep / 2);
            w0[u] = load_weights<STREAM>(at + from.off);
            w1[u] = load_weights<STREAM>(at + from.off8);
        } else { // columns past the row's end: its first ones, made zero
            const bool in = b * kStep + 32u * lpiece < p.in_features;
            const uint32_t at = in ? b * (kStep / 2) : 0u - 16u * lpiece;
            const v4u v0 = load_weights<STREAM>(from.base + (from.off + at));
            const v4u v1 = load_weights<STREAM>(from.base + (from.off8 + at));
            const uint32_t keep = in ? ~0u : 0u;
            w0[u] = v0 & keep;
            w1[u] = v1 & keep;
        }
    };
    // The scales of a tile's rows, a byte for 32 columns, at the wave's steps t0 .. t0 + cnt - 1: lane l takes
    // row l / 4.  FAST: through registers, so that the next tile's can be on their way during this one.
    uint2 sreg[kMaxStage / 4];
    auto scale_row = [&](uint32_t j) {
        return (e_row + min(o_first + j * o_next + (lane >> 2), p.out_features - 1u)) * p.groups;
    };
    auto fetch_scales = [&](uint32_t j, uint32_t t0) {
        if constexpr (FAST) {
            const uint32_t o = o_first + j * o_next, last = p.out_features - 1u, first = min(o, last);
            const char* const base = static_cast<const char*>(p.scales) + (e_row + first) * p.groups;
            const uint32_t ln = here(lane), off = (min(o + (ln >> 2), last) - first) * p.groups;
#pragma unroll
            for (uint32_t i = 0; i < kMaxStage / 4; ++i)
                sreg[i] = *reinterpret_cast<const uint2*>(
                    base + (off + 8u * min(b0 + t0 + 4u * i + (ln & 3u), p.steps - 1u)));
        }
    };
    auto put_scales = [&](uint32_t j, uint32_t t0, uint32_t cnt) {
        const uint32_t ln = here(lane);
        char* const to = s_ws + (ln >> 2) * kScalePitch;
        if constexpr (FAST) {
#pragma unroll
            for (uint32_t i = 0; i < kMaxStage / 4; ++i)
                *reinterpret_cast<uint2*>(to + 8u * (4u * i + (ln & 3u))) = sreg[i];
        } else if constexpr (PART == 2) { // or an fp32 one for 128
            for (uint32_t h = ln & 3u; h < 2u * cnt; h += 4u)
                *reinterpret_cast<float*>(to + 4u * h) = static_cast<const float*>(
                    p.scales)[scale_row(j) +
                              divide(min(2u * (b0 + t0) + h, (p.in_features - 1u) / 128u), p.group_magic128)];
        } else {
            for (uint32_t i = ln & 3u; i < 8u * cnt; i += 4u)
                to[i] = (char)static_cast<const uint8_t*>(
                    p.scales)[scale_row(j) + divide(min(8u * (b0 + t0) + i, p.in_features / 32u - 1u), p.group_magic)];
        }
    };

    while (true) {
        // ---- this workgroup's next rows of the expert: those numbered first, first + 1, ..., at most pass_rows
        uint32_t n = 0;
        while (next < p.rows && n < pass_rows) {
            const uint32_t base = next & ~(uint32_t)(kWaveSize - 1), row = base + lane;
            const bool hit = row >= next && row < p.rows && (!p.idx || (uint32_t)p.idx[row] == e);
            const uint64_t mask = __builtin_amdgcn_ballot_w64(hit);
            const uint32_t rank = seen + (uint32_t)__builtin_popcountll(mask & below);
            if (hit && rank >= first && rank < first + pass_rows)
                s_list[wv][rank - first] = make_uint2(row, row / p.x_div);
            const uint64_t left = __builtin_amdgcn_ballot_w64(hit && rank >= first + pass_rows);
            next = left ? base + (uint32_t)__builtin_ctzll(left) : base + kWaveSize;
            seen = left ? first + pass_rows : seen + (uint32_t)__builtin_popcountll(mask);
            n = seen > first ? seen - first : 0u;
        }
        if (n == 0)
            break; // the same for every wave of the workgroup
        first += gridDim.z * pass_rows;
        Tile cur = tile(0);
        wave_exchange();

        // steps staged at a time: all of a wave's share when they fit, else a multiple of kAhead
        const uint32_t room = min(kMaxStage, (p.lds_x / (p.ks * n) - kRowPad) / kStepBytes) & ~(uint32_t)(kAhead - 1);
        const uint32_t cs = min(room, (p.steps_wave + kAhead - 1) & ~(uint32_t)(kAhead - 1));
        const uint32_t stride = cs * kStepBytes + kRowPad;
        // result columns past the last row repeat it and are not stored
        const uint32_t pr = ks * n + min(r, n - 1u), x_off = pr * stride + 64u * q;
        const uint2 mine = s_list[wv][min(r, n - 1u)];
        float x_scale = 1.0f;
        if (XK == kXFp8F32 && p.x_groups == 1) // one scale a row
            x_scale = static_cast<const float*>(p.x_scales)[mine.y];

        for (uint32_t j = 0; j < p.tiles; ++j) {
            const uint32_t o0 = o_first + j * o_next;
            const Tile nxt = tile(min(j + 1u, p.tiles - 1u));
            const uint32_t after = !FAST || j + 1u < p.tiles ? 0u : last_step; // (no register for it in the others)
            v4f acc = {0.0f, 0.0f, 0.0f, 0.0f}, total = acc; // of the part, and of the parts before it
            uint32_t part_end = p.steps_part;
            for (uint32_t c0 = 0; c0 < p.steps_wave; c0 += cs) {
                const uint32_t end = share > c0 ? min(cs, share - c0) : 0u; // the wave's steps of this part
                if (j == 0 || cs < p.steps_wave) { // the x rows stay when they all fit
                    __syncthreads(); // those before are done with
                    const uint32_t cols = min(cs, p.steps_wave - c0) * kStep;
                    const uint32_t pieces = cols / 8u; // of 8 columns, a row
                    const uint32_t per_piece = magic(pieces), per_n = magic(n);
                    // Pieces in flight a thread: one at a time, 64 tokens of one 7168 -> 4096 product took 93 us
                    // instead of 49, and of a top-8 of 64 experts 143 instead of 134 (147 with eight, of FP8).
                    constexpr int kBatch = XK == kXBf16 ? 8 : 4;
                    const uint32_t all = p.ks * n * pieces;
                    for (uint32_t i0 = here(threadIdx.x); i0 < all; i0 += kBatch * kThreads) {
                        uint4 v[kBatch]; // FP8: the codes' two words, then their scale's byte
                        uint32_t to[kBatch];
#pragma unroll
                        for (int m = 0; m < kBatch; ++m) { // every load first (past the end the last piece again)
                            const uint32_t i = min(i0 + m * kThreads, all - 1u);
                            const uint32_t pr = divide(i, per_piece), c = (i - pr * pieces) * 8u; // a wave's part of a row
                            const uint32_t pk = divide(pr, per_n), xr = s_list[wv][pr - pk * n].y;
                            const uint32_t col = (pk * p.steps_wave + c0) * kStep + c;
                            const bool in = col < p.in_features;
                            const size_t at = (size_t)xr * p.in_features + (in ? col : 0u);
                            to[m] = (pr * stride + 2u * c) | (in ? 1u : 0u);
                            if constexpr (XK != kXBf16) {
                                const uint2 x8 = *reinterpret_cast<const uint2*>(static_cast<const char*>(p.x) + at);
                                v[m] = make_uint4(x8.x, x8.y, 127u, 0u);
                                if constexpr (XK == kXFp8E8) {
                                    const uint32_t g = divide((in ? col : 0u) / 32u, p.x_group_magic);
                                    v[m].z = static_cast<const uint8_t*>(p.x_scales)[(size_t)xr * p.x_groups + g];
                                }
                            } else {
                                v[m] = *reinterpret_cast<const uint4*>(static_cast<const char*>(p.x) + 2u * at);
                            }
                        }
#pragma unroll
                        for (int m = 0; m < kBatch; ++m) {
                            if constexpr (XK != kXBf16) {
                                const float sx = as_float(v[m].z << 23);
                                v[m] = make_uint4(fp8_to_bf16<false>(v[m].x, sx), fp8_to_bf16<true>(v[m].x, sx),
                                                  fp8_to_bf16<false>(v[m].y, sx), fp8_to_bf16<true>(v[m].y, sx));
                            }
                            if (!(to[m] & 1u))
                                v[m] = make_uint4(0, 0, 0, 0);
                            if (i0 + m * kThreads < all)
                                *reinterpret_cast<uint4*>(s_x + (to[m] & ~1u)) = v[m];
                        }
                    }
                    if (x_part) {
                        for (uint32_t i = here(threadIdx.x); i < p.ks * n * (cols / 128u); i += kThreads) {
                            const uint32_t pr = i / (cols / 128u), h = i - pr * (cols / 128u);
                            const uint32_t pk = divide(pr, per_n), xr = s_list[wv][pr - pk * n].y;
                            const uint32_t first = (pk * p.steps_wave + c0) * (kStep / 128);
                            s_sx[pr * 2u * cs + h] = static_cast<const float*>(
                                p.x_scales)[(size_t)xr * p.x_groups +
                                            divide(min(first + h, (p.in_features - 1u) / 128u), p.x_group_magic128)];
                        }
                    }
                }
                if (j == 0 && c0 == 0) {
                    // Past a wave's share, here and below, its last step again, unused: a condition around the loads
                    // would leave the compiler unsure how many are in flight, and it would wait for all of them at
                    // every step.
                    for_slots<kAhead>([&](auto u) { fetch(u, cur, min((uint32_t)u.value, last_step)); });
                    fetch_scales(0, 0);
                }
                put_scales(j, c0, end); // read by this wave alone
                if (c0 + cs < p.steps_wave)
                    fetch_scales(j, c0 + cs);
                else
                    fetch_scales(min(j + 1u, p.tiles - 1u), 0);
                if (j == 0 || cs < p.steps_wave)
                    __syncthreads();
                else
                    wave_exchange();

                auto step = [&](auto slot, uint32_t t) { // step c0 + t, from slot u, whose next step is then fetched
                    constexpr int u = decltype(slot)::value;
                    if (c0 + t == part_end) { // wave-uniform
                        part_end += p.steps_part;
                        total += acc;
                        acc = v4f{0.0f, 0.0f, 0.0f, 0.0f};
                    }
                    // steps (and their halves) apart: interleaved, their operands would not fit 128 registers
                    __builtin_amdgcn_sched_barrier(0);
                    *w_put = w0[u];
                    *w_put8 = w1[u];
                    wave_exchange();
                    const bool in = c0 + t + kAhead < share;
                    const Tile from = {in ? cur.base : nxt.base, in ? cur.off : nxt.off, in ? cur.off8 : nxt.off8};
                    // (after the last tile that tile's last step, which is on its way or in the cache: its first ones,
                    // long evicted, were 13% more bytes with 14 steps a wave)
                    fetch(slot, from, in ? c0 + t + kAhead : max(min((uint32_t)u, last_step), after));
                    const uint2 sb2 = PART == 2 ? make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu)
                                                : *reinterpret_cast<const uint2*>(s_ws + r * kScalePitch + 8u * t);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h)
                            __builtin_amdgcn_sched_barrier(0);
                        // past the row's end there is no scale, and zero times an infinite one would be NaN (wave-uniform)
                        if (PART && !FAST && h && (b0 + c0 + t) * kStep + 128u >= p.in_features)
                            break;
                        // only the exponent is looked at: 0 is 2^-127, 255 NaN
                        const float s = as_float((((h ? sb2.y : sb2.x) >> (8u * q)) & 255u) << 23);
                        const v4u wh = h ? *w_get4 : *w_get;
                        const uint32_t w4[4] = {wh.x, wh.y, wh.z, wh.w};
                        v8b A[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const v2b a0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w4[i], s, 0);
                            const v2b a1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w4[i], s, 1);
                            const v2b a2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w4[i], s, 2);
                            const v2b a3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w4[i], s, 3);
                            A[i] = v8b{a0[0], a0[1], a1[0], a1[1], a2[0], a2[1], a3[0], a3[1]};
                        }
                        v4f c = PART ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : acc;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const v8b B = *reinterpret_cast<const v8b*>(s_x + x_off + t * kStepBytes + 256u * h +
                                                                        16u * i);
                            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[i], B, c, 0, 0, 0);
                        }
                        if constexpr (PART) {
                            const float sx = x_part ? s_sx[(pr * cs + t) * 2u + h] : 1.0f;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                float f = sx;
                                if constexpr (PART == 2)
                                    f *= *reinterpret_cast<const float*>(s_ws + (4u * q + i) * kScalePitch + 8u * t +
                                                                         4u * h);
                                acc[i] = __builtin_fmaf(c[i], f, acc[i]);
                            }
                        } else {
                            acc = c;
                        }
                    }
                };
                uint32_t t = 0;
                for (; t + kAhead <= end; t += kAhead)
                    for_slots<kAhead>([&](auto u) { step(u, t + u.value); });
                for_slots<kAhead>([&](auto u) {
                    if (t + u.value < end)
                        step(u, t + u.value);
                });
            }

            cur = nxt;
            // ---- the parts' sums meet, in their order, through the weights' LDS
            if (p.ks > 1) {
                s_w4[wv][lane] = __builtin_bit_cast(v4u, total);
                s_w4[wv][kWaveSize + lane] = __builtin_bit_cast(v4u, acc);
                __syncthreads();
            }
            acc = total + acc;
            if (p.ks > 1) {
                if (ks == 0)
                    for (uint32_t i = 1; i < p.ks; ++i) { // a wave has two parts at most when others share its tile
                        acc += __builtin_bit_cast(v4f, s_w4[wv + i][lane]);
                        acc += __builtin_bit_cast(v4f, s_w4[wv + i][kWaveSize + lane]);
                    }
                __syncthreads();
                if (ks != 0)
                    continue;
            }
            // ---- the activations' scales of whole rows, and the results
            if (r >= n)
                continue;
            const uint32_t o = o0 + 4u * (here(lane) >> 4);
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) {
                if (o + i >= p.out_features)
                    continue;
                const float v = acc[i] * x_scale;
                const size_t at = (size_t)mine.x * p.out_features + o + i;
                if (p.out_bf16)
                    static_cast<__bf16*>(p.out)[at] = (__bf16)v;
                else
                    static_cast<float*>(p.out)[at] = v;
            }
        }
    }
}

template <int XK, int PART, bool FAST>
void launch_gemv_stream(bool stream, const GemvParams& p, dim3 grid, hipStream_t s)
{
    const uint32_t lds = p.lds_x + p.lds_x / kStepBytes * 8u;
    if (stream)
        hipLaunchKernelGGL((gemv_fp4_kernel<XK, PART, FAST, true>), grid, dim3(kThreads), lds, s, p);
    else
        hipLaunchKernelGGL((gemv_fp4_kernel<XK, PART, FAST, false>), grid, dim3(kThreads), lds, s, p);
}

template <int XK, int PART>
void launch_gemv(bool fast, bool stream, const GemvParams& p, dim3 grid, hipStream_t s)
{
    if (PART != 2 && fast)
        launch_gemv_stream<XK, PART, PART != 2>(stream, p, grid, s);
    else
        launch_gemv_stream<XK, PART, false>(stream, p, grid, s);
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
    if (experts <= 0 || experts > 32768 || out_features <= 0 || out_features > (1 << 24) || in_features <= 0 ||
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
    p.x_div = x_slots ? 1u : (uint32_t)k;
    p.experts = (uint32_t)experts;
    p.out_features = (uint32_t)out_features;
    p.in_features = (uint32_t)in_features;
    p.groups = (uint32_t)(in_features / group);
    p.x_groups = (uint32_t)(in_features / xgroup);
    p.out_bf16 = out_bf16;
    hipStream_t s = static_cast<hipStream_t>(stream);
    p.group_magic = magic((uint32_t)group / 32u);
    p.x_group_magic = magic((uint32_t)xgroup / 32u);
    // (one scale a row may span a part of a step of 128)
    p.group_magic128 = magic(((uint32_t)group + 127u) / 128u);
    p.x_group_magic128 = magic(((uint32_t)xgroup + 127u) / 128u);
    p.steps = (p.in_features + kStep - 1) / kStep;
    const uint64_t tiles = (uint64_t)((p.out_features + kTile - 1) / kTile), waves = (uint64_t)k * tiles;
    const uint64_t active = topk_idx ? (uint64_t)(rows < experts ? rows : experts) : 1u;
    const uint64_t load = topk_idx ? (uint64_t)(rows / experts) : (uint64_t)rows; // an expert's rows on average
    // Workgroups side by side for an expert's passes of 16 rows, as many as an expert has on average (64 rows of
    // 7168 -> 4096: 54 us when one workgroup takes them all, 23 so; 512 rows of 4096 -> 4096 255 / 66; 64 tokens'
    // top-8 of 8 experts 7168 -> 2048 99 / 60).  Passes of 8 while those leave CUs with less than two (20 rows of 8032
    // -> 2048 in FP8 20.4 / 15.7 us, 15 of 4096 -> 1024 11.2 / 8.9; 32 of 7168 -> 4096 in bf16 18.3 / 19.1).
    auto passes_of = [&](uint64_t n) { return load <= n ? 1u : load < 256u * n ? (uint32_t)((load + n - 1) / n) : 256u; };
    p.pass = load > 8 && active * tiles * passes_of(kTile) < 2u * kCus ? 8u : (uint32_t)kTile;
    const uint32_t passes = passes_of(p.pass);
    // The columns' parts go by the sizes alone, never by the number of tokens, so that a row's sum has one order;
    // they are summed by as many waves (ks) as leave every CU the workgroups that its LDS has room for, with eight
    // steps of each x row staged.  (7168 -> 4096 bf16, one row: 15.3 us by one wave, 9.7 by two, 8.0 by four, 64 rows:
    // 23 by one, 57 by four; 7168 -> 2048 for 16 tokens' top-8 of 64 experts: 94, 110, 134.)
    const uint32_t pass = load < 1 ? 1u : load < p.pass ? (uint32_t)load : p.pass;
    uint32_t parts = waves >= 3072 ? 1u : waves >= 1536 ? 2u : 4u;
    while (parts > p.steps)
        parts >>= 1;
    p.steps_part = (p.steps + parts - 1) / parts;
    p.ks = parts;
    auto workgroups = [&] {
        return passes * active * ((tiles * p.ks + kThreads / kWaveSize - 1) / (kThreads / kWaveSize));
    };
    auto fit = [](uint32_t lds) { return lds > kCuLds / 2u ? 1u : lds > kCuLds / 4u ? kCuLds / lds : 4u; };
    while (p.ks > 1 && workgroups() > (p.pass < kTile ? 2u : 1u) * kCus * fit(kOwnLds + p.ks * pass * 8u * kStepBytes))
        p.ks >>= 1;
    p.steps_wave = p.ks == 1 ? p.steps : p.steps_part * (parts / p.ks);
    p.by_row = topk_idx && rows <= experts;
    const int part = !u8 ? 2 : fp8 && !xu8 && p.x_groups > 1 ? 1 : 0;
    // Weights that as a rule one pass reads, in whole lines, go past the caches: 2048 -> 7168 for 16 tokens' top-8 of
    // 64 experts 85.2 us, through them 94.0; 64 tokens 7168 -> 2048 122 / 129; but with several passes (64 tokens'
    // top-8 of 16 experts, 7168 -> 4096) 154 / 136 and with lines that two rows share (2016 -> 2048) 42.3 / 37.0.
    const bool once = passes == 1 && in_features % kStep == 0 && aligned(codes, 128);
    const bool fast = u8 && group == 32 && in_features % kStep == 0 && aligned(scales, 8);
    const uint32_t tiles_wg = kThreads / kWaveSize / p.ks;
    const uint64_t wgs = workgroups();
    // Staged x rows: what the LDS leaves beside a workgroup's own, with as many workgroups a CU as there are, up to
    // four; at most all the columns of a full pass, at least kAhead steps of a few rows more than an expert has on
    // average (a more crowded one takes further passes)
    const uint32_t want = p.ks * (topk_idx && 2 * load + 4 < p.pass ? (uint32_t)(2 * load + 4)
                                  : topk_idx || load >= p.pass      ? p.pass
                                                                    : (uint32_t)load);
    const uint32_t per_cu = wgs >= 4 * kCus ? 4u : (uint32_t)((wgs + kCus - 1) / kCus);
    const uint32_t room = (kCuLds / per_cu - kOwnLds) / 65u * 64u; // each 512 bytes with 8 of fp32 scales
    const uint32_t stage = p.steps_wave < kMaxStage ? p.steps_wave + kAhead : kMaxStage;
    const uint32_t all = want * (stage * kStepBytes + kRowPad), least = want * (kAhead * kStepBytes + kRowPad);
    p.lds_x = all < room ? all : room;
    p.lds_x = p.lds_x < least ? least : p.lds_x;
    p.lds_x = p.lds_x < 16448u ? 16448u : p.lds_x > 131072u ? 131072u : p.lds_x;
    p.lds_x &= ~15u;
    // Several tiles a wave where that leaves four workgroups a CU: the x rows are then staged once for all of them
    // and a tile's first weights are on their way during the one before (2048 -> 7168, 16 tokens top-8 of 64:
    // 90.6 us with one tile, 86.9 with two, 85.1 with four, 86.3 with eight).
    p.tiles = wgs >= 4096 ? 4u : wgs >= 2048 ? 2u : 1u;
    const uint32_t wg_rows = kTile * tiles_wg * p.tiles;
    const dim3 grid((p.out_features + wg_rows - 1) / wg_rows, !topk_idx ? 1u : p.by_row ? p.rows : p.experts + 1u, passes);
    if (!fp8)
        part == 2 ? launch_gemv<kXBf16, 2>(fast, once, p, grid, s) : launch_gemv<kXBf16, 0>(fast, once, p, grid, s);
    else if (xu8)
        part == 2 ? launch_gemv<kXFp8E8, 2>(fast, once, p, grid, s) : launch_gemv<kXFp8E8, 0>(fast, once, p, grid, s);
    else
        part == 2   ? launch_gemv<kXFp8F32, 2>(fast, once, p, grid, s)
        : part == 1 ? launch_gemv<kXFp8F32, 1>(fast, once, p, grid, s)
                    : launch_gemv<kXFp8F32, 0>(fast, once, p, grid, s);
    return hipGetLastError() == hipSuccess ? TK_OK : TK_ERR_HIP;
}
