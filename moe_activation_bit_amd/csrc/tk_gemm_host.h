// tk_gemm_host.h -- what the entry points of the grouped matrix products share:
// the launch parameters and the checks of their arguments.
#pragma once

#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>

#include "tk.h"
#include "tk_expert.h"
#include "tk_quant.h"

namespace tk_gemm {

using namespace tk_detail;

struct GemmParams {
    const char* c;          // the operand of the result's columns: w, or x of the weights' gradient
    const char* r;          // ... of its rows: x or dy
    const uint8_t* c_scales; // of x in FP8: [c_rows][c_groups], c_group columns each
    const int32_t* c_index; // the row of x for a row, or null
    const int32_t* r_index; // ... of r
    const int32_t* offsets; // [experts + 1], or null: one expert with all rows
    void* out;
    uint32_t c_rows, r_rows; // rows that there are for the indices
    uint32_t c_group, c_groups;
    uint32_t n_rows;
    uint32_t experts;
    uint32_t cols;          // of the result
    uint32_t out_rows;      // of the weights' gradient, for each expert
    uint32_t depth;         // of the sums (the weights' gradient: an expert's rows)
    uint32_t run;           // tiles that an XCD takes together
    int out_bf16;
    int accumulate;
};

struct RowsArgs {
    int64_t rows;
    const int32_t* index;
};

inline bool valid_rows(const RowsArgs& a, const int32_t* offsets, int64_t n_rows, int64_t experts)
{
    return n_rows >= 0 && n_rows <= (int64_t)INT_MAX && a.rows >= 0 && a.rows <= (int64_t)INT_MAX && experts >= 1 &&
           (offsets || experts == 1) && (a.index || a.rows >= n_rows) && aligned(a.index, 4) && aligned(offsets, 4);
}

inline bool valid_shape(int64_t out_features, int64_t in_features, int64_t step)
{
    return out_features > 0 && in_features > 0 && out_features % 8 == 0 && in_features % step == 0 &&
           out_features <= 1 << 20 && in_features <= 1 << 20;
}

inline bool overlaps_rows(const void* out, size_t bytes, const int32_t* index, const int32_t* offsets, int64_t n_rows,
                          int64_t experts)
{
    return overlaps(out, bytes, index, (size_t)n_rows * 4u) || overlaps(out, bytes, offsets, (size_t)(experts + 1) * 4u);
}

// An expert's rows on average, and how many tiles of tr rows by tc columns there are when all have as many.
inline uint64_t average_rows(uint32_t rows, uint32_t experts) { return (rows + experts - 1u) / experts; }
inline uint64_t tiles_of(uint64_t load, uint32_t experts, uint32_t cols, uint32_t tr, uint32_t tc)
{
    return experts * ((load + tr - 1u) / tr) * (((uint64_t)cols + tc - 1u) / tc);
}

// tk_expert_gemm with bf16 operands
tk_status launch_forward(const GemmParams& p, hipStream_t s);

} // namespace tk_gemm
