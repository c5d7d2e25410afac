// microscale.h -- the block-scaled formats of include/tmamicro.h: their storage, and on
// the device the rounding of eight values at a time.
#pragma once

#include <cstdint>

#include "gemm_common.h"

namespace tg {

enum : int { MXFP8 = 0, MXFP4 = 1, NVFP4 = 2 };

constexpr int MX_ROWS = 128;          // rows of a storage block
constexpr int MX_CHUNK_BYTES = 2048;  // one chunk of each of its rows
constexpr int MX_GROUP_BYTES = 512;   // one group of four scales of each of its rows

TG_HD constexpr int mx_block(int format) { return format == NVFP4 ? 16 : 32; }
// Values of a chunk (16 bytes).
TG_HD constexpr int mx_chunk(int format) { return format == MXFP8 ? 16 : 32; }
// Blocks whose scales share a group of four bytes.  mxfp4: three, the scales of one MMA of
// 96 values (the fourth byte is not used); else a whole number of MMAs.
TG_HD constexpr int mx_group_blocks(int format) { return format == MXFP4 ? 3 : 4; }
TG_HD constexpr int mx_group(int format) { return mx_group_blocks(format) * mx_block(format); }
// Chunks and values of the smallest MMA; rows are filled up to whole ones.
TG_HD constexpr int mx_step_chunks(int format) { return format == MXFP4 ? 3 : 2; }
TG_HD constexpr int mx_step(int format) { return mx_step_chunks(format) * mx_chunk(format); }

TG_HD int64_t mx_chunks(int64_t K, int format)
{
    return (K + mx_step(format) - 1) / mx_step(format) * mx_step_chunks(format);
}
TG_HD int64_t mx_groups(int64_t K, int format)
{
    return (K + mx_group(format) - 1) / mx_group(format);
}
TG_HD int64_t mx_row_blocks(int64_t rows) { return (rows + MX_ROWS - 1) / MX_ROWS; }

// Byte offset of chunk `chunk` of row `row`, and of the four bytes of group `group`.
TG_HD int64_t mx_code_offset(int64_t row, int64_t chunk, int64_t chunks)
{
    return ((row / MX_ROWS) * chunks + chunk) * MX_CHUNK_BYTES + (row % MX_ROWS) * 16;
}
TG_HD int64_t mx_scale_offset(int64_t row, int64_t group, int64_t groups)
{
    const int r = static_cast<int>(row % MX_ROWS);
    return ((row / MX_ROWS) * groups + group) * MX_GROUP_BYTES + (r % 32) * 16 + r / 32 * 4;
}

}  // namespace tg
