// mx_product.h -- launch interface of the block-scaled product kernels.
#pragma once

#include <cuda.h>

#include "gemm_common.h"
#include "launch.h"
#include "microscale.h"

namespace tg {

// Chunks (16 bytes of a row) and groups of scales per pipeline stage of single CTAs, ...
TG_HD constexpr int mx_stage_chunks(int format) { return format == MXFP4 ? 6 : 8; }
TG_HD constexpr int mx_stage_groups(int format)
{
    return mx_stage_chunks(format) * mx_chunk(format) / mx_group(format);
}
// ... and of pairs, whose MMAs take 96 values of either 4-bit format: two of them.  (Four:
// a ring of three stages instead of six, and 8192^3 mxfp4 in 164 us instead of 138.)
TG_HD constexpr int mx_pair_chunks(int format) { return format == MXFP8 ? 8 : 6; }
TG_HD constexpr int mx_pair_groups(int format)
{
    return mx_pair_chunks(format) * mx_chunk(format) / mx_group(format);
}

struct MxParams {
    int M, N;
    int steps;           // smallest MMAs of the whole contraction
    int stages;          // pipeline stages of the whole contraction
    int chunks, groups;  // of a row
    int tiles_m, tiles_n, group_m;
    int pipe_depth;
    int split;           // CTAs of a cluster that share a tile's length (single CTAs)
    const float* scale_a;
    const float* scale_b;
    void* C;
    DevStatus* status;
    int epoch;
    unsigned long long budget_ns;
    int debug_stall;
};

struct MxSpec {
    int format;
    bool f16out;
    bool pair;
    int cols;      // single CTAs: rows of the second operand in a tile, 16 .. 128
    bool swapped;  // single CTAs: B is the operand with 128 rows a tile
    int grid_x, grid_y;
    int staging;   // pair: output buffers of an epilogue warp, 1 or 2 (4-bit formats)
    unsigned smem_bytes;
    const CUtensorMap* codes_u;   // pair: A; single: the operand with 128 rows a tile
    const CUtensorMap* scales_u;
    const CUtensorMap* codes_v;
    const CUtensorMap* scales_v;
    const CUtensorMap* out;       // pair only
    MxParams p;
};

// Shared memory of a single CTA: `depth` stages of codes and scales of both operands, the
// barriers.  The sums of the tile (128 x cols fp32, padded) reuse the stages.
struct MxSingleLayout {
    uint32_t stage, v_codes, u_scales, v_scales;  // bytes of a stage, offsets in it
    uint32_t bars, total;
};

TG_HD uint32_t mx_partial_stride(int cols, bool swapped)
{
    return swapped ? 128u : static_cast<uint32_t>(cols) + 4u;
}

TG_HD MxSingleLayout mx_single_layout(int format, int cols, int depth, bool swapped)
{
    MxSingleLayout L;
    const uint32_t groups = static_cast<uint32_t>(mx_stage_groups(format));
    const uint32_t chunks = static_cast<uint32_t>(mx_stage_chunks(format));
    L.v_codes = chunks * MX_CHUNK_BYTES;
    L.u_scales = L.v_codes + chunks * static_cast<uint32_t>(cols) * 16u;
    L.v_scales = L.u_scales + groups * MX_GROUP_BYTES;
    L.stage = L.v_scales + groups * MX_GROUP_BYTES;
    L.stage = (L.stage + 1023u) / 1024u * 1024u;
    const uint32_t ring = L.stage * static_cast<uint32_t>(depth);
    const uint32_t sums = 4u * mx_partial_stride(cols, swapped) *
                          static_cast<uint32_t>(swapped ? cols : 128);
    L.bars = ring > sums ? ring : (sums + 1023u) / 1024u * 1024u;
    L.total = L.bars + BAR_AREA_BYTES + 1024;
    return L;
}

// Shared memory of a CTA of a pair: stages of 128 rows of each operand and the scales of
// 128 rows of A and 256 of B, the output staging (one buffer of 4 KB for each epilogue warp, or
// two: the second takes a stage's place, 8192^3 nvfp4 142 us instead of 134), the barriers.
struct MxPairLayout {
    uint32_t stage, b_codes, a_scales, b_scales;
    uint32_t staging, bars, total;
};

constexpr int MX_PAIR_MIN_STAGES = 6;  // they hold a whole tile of the output at the end

TG_HD MxPairLayout mx_pair_layout(int format, int depth, int staging)
{
    MxPairLayout L;
    const uint32_t groups = static_cast<uint32_t>(mx_pair_groups(format));
    L.b_codes = static_cast<uint32_t>(mx_pair_chunks(format)) * MX_CHUNK_BYTES;
    L.a_scales = 2 * L.b_codes;
    L.b_scales = L.a_scales + groups * MX_GROUP_BYTES;
    L.stage = (L.b_scales + 2 * groups * MX_GROUP_BYTES + 1023u) / 1024u * 1024u;
    L.staging = L.stage * static_cast<uint32_t>(depth);
    L.bars = L.staging + static_cast<uint32_t>(staging) * STAGING_BYTES;
    L.total = L.bars + BAR_AREA_BYTES + 1024;
    return L;
}

cudaError_t launch_mx_single(const MxSpec& s, cudaStream_t stream);
cudaError_t launch_mx_pair(const MxSpec& s, cudaStream_t stream);

}  // namespace tg
