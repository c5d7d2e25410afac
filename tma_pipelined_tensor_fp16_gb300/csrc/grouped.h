// grouped.h -- the grouped product's parameter block and tile table, shared by
// its host side and its kernel.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "gemm_common.h"

namespace tg {

// Same values as the public gemm_grouped_op.
enum : int { GROUPED_FORWARD = 0, GROUPED_GRAD_INPUT = 1, GROUPED_GRAD_WEIGHT = 2 };

struct GroupedParams {
    int rows;         // rows of the sorted operands
    int out_rows;     // GRAD_WEIGHT: rows of one expert's output (N); else = rows
    int out_cols;     // columns of the output
    int depth;        // contraction length; GRAD_WEIGHT: taken from the offsets
    int experts;
    int tiles_n;
    int tiles_m;      // GRAD_WEIGHT: row tiles of one expert; else from the offsets
    int group_m;      // raster group height in row tiles
    int pipe_depth;
    const int* offsets;
    void* out;
    DevStatus* status;
    unsigned long long* counter;  // see grouped_take
    int epoch;
    unsigned long long budget_ns;
    int debug_stall;  // 1: the producer, 2: the epilogue first waits on a barrier nothing completes
};

struct GroupedSpec {
    int op;
    int block_n;
    bool pair;  // CTA pairs: tiles of 256 x 256
    bool f16out;
    int grid;
    unsigned smem_bytes;
    const CUtensorMap* tmA;  // the operand whose rows are output rows
    const CUtensorMap* tmS;  // the same with boxes of GROUPED_SMALL_ROWS rows (not GRAD_WEIGHT)
    const CUtensorMap* tmB;  // the operand whose rows (or columns) are output columns
    const CUtensorMap* tmC;
    GroupedParams p;
};

cudaError_t launch_grouped(const GroupedSpec& s, cudaStream_t stream);

constexpr int GROUPED_THREADS = 192;
constexpr int GROUPED_SMALL_ROWS = 32;
constexpr int GROUPED_MAX_EXPERTS = 1024;

// GRAD_WEIGHT sorts the experts by their rows up to this many of them (the sort
// compares each pair: at 128 experts 0.7 us of a launch).
constexpr int GROUPED_SORT_EXPERTS = 128;

// Shared memory behind the stage ring, the staging buffers and the barriers: first
// row and first row tile of every expert, of the rows that belong to none, and of
// the end; for GRAD_WEIGHT, where it sorts, the offsets and the order of experts.
TG_HD uint32_t grouped_table_bytes(int op, int experts)
{
    return op == GROUPED_GRAD_WEIGHT && experts > GROUPED_SORT_EXPERTS
               ? 0u
               : static_cast<uint32_t>(experts + 2) * 8u;
}

}  // namespace tg
