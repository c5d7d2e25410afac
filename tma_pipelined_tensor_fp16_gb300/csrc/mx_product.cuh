// mx_product.cuh -- what the block-scaled product kernels share: descriptors, the MMA
// and the copy of scales into tensor memory.
//
// Operand storage (microscale.h) is the tensor core's own: a chunk's column of 16-byte
// pieces of consecutive rows is a stack of core matrices (8 rows x 16 bytes, 128 bytes
// each), so a stage is one box without a swizzle whatever the number of rows, and a step
// of the contraction is two chunks further on.  Scales go the same way: a group of four
// scales of 128 rows is the 32 x 16 bytes that one tcgen05.cp spreads over four columns
// of tensor memory.
#pragma once

#include "device_common.cuh"
#include "mx_product.h"
#include "ptx.cuh"

namespace tg {

// A value that is the same in the whole warp, made known as such.  The operands of tcgen05
// instructions are uniform registers: with the warp's number and the tensor-memory base
// known to be uniform an MMA warp issues them from there, and without each operand is
// moved first (a copy of scales took 20 cycles to issue, and 96 values of nvfp4 on a pair
// 125 ns instead of 74).
__device__ __forceinline__ uint32_t warp_uniform(uint32_t v)
{
    return __shfl_sync(0xffffffffu, v, 0);
}

// Shared-memory matrix descriptor of a K-major operand without a swizzle: core matrices of
// 8 rows x 16 bytes; `lead` bytes from one to the next along K, 128 along the rows.
//   [0,14) start >> 4   [16,30) leading offset >> 4   [32,46) stride offset >> 4
//   [46,49) 0b001       [61,64) swizzle mode (0 = none)
__device__ __forceinline__ uint64_t core_desc(uint32_t smem_addr, uint32_t lead)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(lead >> 4) << 16;
    d |= static_cast<uint64_t>(128 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    return d;
}

// Instruction descriptor of the block-scaled kinds:
//   [4,6) scale id of B   [7,10) type of A   [10,13) type of B   [17,23) N >> 3
//   [23] scale type (0 = ue4m3, 1 = ue8m0)   [24,29) M >> 4      [29,31) scale id of A
//   [31] K of the 4-bit kinds (0 = 64, 1 = 96: sm_103a)
// Types: kind::mxf8f6f4 e4m3 = 0; kind::mxf4 and mxf4nvf4 e2m1 = 1.
constexpr uint32_t MX_IDESC_K96 = 1u << 31;

template <int FORMAT>
__device__ __forceinline__ constexpr uint32_t mx_idesc(int M, int N, int scale_id)
{
    const uint32_t type = FORMAT == MXFP8 ? 0u : 1u;
    return (FORMAT == MXFP4 ? MX_IDESC_K96 : 0u) | static_cast<uint32_t>(scale_id) << 4 |
           type << 7 | type << 10 | static_cast<uint32_t>(N >> 3) << 17 | (FORMAT == NVFP4 ? 0u : 1u) << 23 |
           static_cast<uint32_t>(M >> 4) << 24 | static_cast<uint32_t>(scale_id) << 29;
}

// Bytes of the groups of scales per smallest MMA: mxfp8 one (32 values), mxfp4 a whole group
// of three scales (96), nvfp4 a whole group of four (64).
template <int FORMAT>
constexpr int mx_step_scales = FORMAT == MXFP8 ? 1 : 4;
// D (+)= A * B^T with scales from tensor memory, issued by the lane with `elected` set.
#define TG_MX_MMA(GROUP, KIND)                                                                  \
    asm volatile(                                                                               \
        "{\n\t"                                                                                 \
        ".reg .pred p, q;\n\t"                                                                  \
        "setp.ne.b32 p, %7, 0;\n\t"                                                             \
        "setp.ne.b32 q, %6, 0;\n\t"                                                             \
        "@p tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, [%4], [%5], q;\n\t" \
        "}\n" ::"r"(d_tmem),                                                                    \
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scales), "r"(b_scales), "r"(accumulate),    \
        "r"(elected)                                                                            \
        : "memory")

template <int FORMAT, bool PAIR>
__device__ __forceinline__ void mx_mma(uint32_t elected, uint32_t d_tmem, uint64_t a_desc,
                                       uint64_t b_desc, uint32_t idesc, uint32_t a_scales,
                                       uint32_t b_scales, uint32_t accumulate)
{
    if constexpr (FORMAT == MXFP8) {
        if constexpr (PAIR)
            TG_MX_MMA("2", "mxf8f6f4.block_scale.scale_vec::1X");
        else
            TG_MX_MMA("1", "mxf8f6f4.block_scale.scale_vec::1X");
    } else if constexpr (FORMAT == MXFP4) {
        if constexpr (PAIR)
            TG_MX_MMA("2", "mxf4.block_scale.block32");
        else
            TG_MX_MMA("1", "mxf4.block_scale.block32");
    } else {
        if constexpr (PAIR)
            TG_MX_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
        else
            TG_MX_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
    }
}

// The same over 96 values (three chunks) of nvfp4 on a pair; the instruction descriptor has
// MX_IDESC_K96.  Six scales: four of a group and two of the next, or (scale id 2) two and
// four.
__device__ __forceinline__ void mx_mma_k96_pair(uint32_t elected, uint32_t d_tmem, uint64_t a_desc,
                                                uint64_t b_desc, uint32_t idesc, uint32_t a_scales,
                                                uint32_t b_scales, uint32_t accumulate)
{
    TG_MX_MMA("2", "mxf4nvf4.block_scale.block16");
}
#undef TG_MX_MMA

// A group of scales of 128 rows (512 bytes of shared memory) to four columns of tensor
// memory, in each of the four quarters of its lanes.  Runs in order with the MMAs of
// the same thread.
template <bool PAIR>
__device__ __forceinline__ void copy_scales(uint32_t elected, uint32_t taddr, uint32_t smem_addr)
{
    const uint64_t desc = core_desc(smem_addr, 0);
    if constexpr (PAIR)
        asm volatile(
            "{\n\t"
            ".reg .pred p;\n\t"
            "setp.ne.b32 p, %2, 0;\n\t"
            "@p tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t"
            "}\n" ::"r"(taddr),
            "l"(desc), "r"(elected)
            : "memory");
    else
        asm volatile(
            "{\n\t"
            ".reg .pred p;\n\t"
            "setp.ne.b32 p, %2, 0;\n\t"
            "@p tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t"
            "}\n" ::"r"(taddr),
            "l"(desc), "r"(elected)
            : "memory");
}

// Product of the tensor scales (both NULL: 1).
__device__ __forceinline__ float mx_alpha(const MxParams& p)
{
    return (p.scale_a ? *p.scale_a : 1.0f) * (p.scale_b ? *p.scale_b : 1.0f);
}

__device__ __forceinline__ Watchdog mx_watchdog(const MxParams& p)
{
    Watchdog w;
    w.st = p.status;
    w.epoch = p.epoch;
    w.budget_ns = p.budget_ns;
    w.aborted = false;
    return w;
}

__device__ __forceinline__ void mx_commit(uint32_t elected, uint32_t bar)
{
    asm volatile(
        "{\n\t"
        ".reg .pred p;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t"
        "}\n" ::"r"(bar),
        "r"(elected)
        : "memory");
}

__device__ __forceinline__ void mx_commit_pair(uint32_t elected, uint32_t bar)
{
    asm volatile(
        "{\n\t"
        ".reg .pred p;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "@p tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
        ".b64 [%0], %2;\n\t"
        "}\n" ::"r"(bar),
        "r"(elected), "h"(static_cast<uint16_t>(3))
        : "memory");
}

}  // namespace tg
