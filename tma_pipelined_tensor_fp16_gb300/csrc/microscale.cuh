// microscale.cuh -- the arithmetic of quantisation on the device, shared by the
// quantisers and the norm.
//
// A scale is found once per block and each value costs a multiplication (by a power of
// two, exact) or three operations (nvfp4).  Rounding itself is the conversion
// instruction: to nearest, ties to even, beyond the largest value to the largest.
#pragma once

#include <cuda_fp16.h>

#include "microscale.h"

namespace tg {

// What a block's values are multiplied by, and the byte that is stored.
struct BlockScale {
    float divisor;  // nvfp4: s * t; the others: not used
    float factor;   // 1 / (s t): exact where s is a power of two
    uint32_t byte;
};

__device__ __forceinline__ float power_of_two(int e)  // e in [-126, 127]
{
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

__device__ __forceinline__ uint32_t e4m3_of(float x)  // x >= 0
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(x));
    return r & 0xffu;
}

__device__ __forceinline__ float float_of_e4m3(uint32_t byte)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(byte)));
    const __half2 v = *reinterpret_cast<__half2*>(&h);
    return __low2float(v);
}

// The power of two of an e8m0 byte (0: 2^-127, which fp32 holds without its leading
// bit; 255: NaN).
__device__ __forceinline__ float float_of_e8m0(uint32_t byte)
{
    const uint32_t bits = byte == 0 ? 0x00400000u : byte == 255u ? 0x7fc00000u : byte << 23;
    return __uint_as_float(bits);
}

// The scale of a block with the largest magnitude `most` (an infinity or a NaN where
// the block holds one); `t` and 1 / (6 t) are the tensor's (nvfp4).
template <int FORMAT>
__device__ __forceinline__ BlockScale block_scale(float most, float t, float sixth)
{
    BlockScale b;
    const bool finite = most < __uint_as_float(0x7f800000u);  // false for NaN
    if constexpr (FORMAT == NVFP4) {
        // a / (6 t) with the product instead of the quotient: a has 11 bits (24 in the
        // norm) and a border of e4m3 has 5, so for fp16 values the rounding error of
        // the product decides only where a / 6 lies on a border, which needs a = 6 m
        // with m of 5 bits: there the quotient is exact and the product is refined to it.
        // (With a given t that is no power of two, 6 t and s t are rounded to fp32 first: a
        // quotient within 2^-22 of a border may go either way.)
        float y = most * sixth;
        y = fmaf(fmaf(-y, 6.0f * t, most), sixth, y);
        uint32_t byte = max(e4m3_of(y), 1u);
        if (!finite) byte = 0x7fu;
        b.byte = byte;
        b.divisor = float_of_e4m3(byte) * t;
        // an approximation is enough: scaled() corrects with the exact remainder
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b.factor) : "f"(b.divisor));
    } else {
        // most = m * 2^k with 1 <= m < 2; the largest value is M * 2^K with the same
        // bounds: s = 2^(k - K), doubled where m > M
        constexpr uint32_t TOP = FORMAT == MXFP8 ? 0x600000u : 0x400000u;  // 1.75, 1.5
        constexpr int SHIFT = FORMAT == MXFP8 ? 8 : 2;
        const uint32_t bits = __float_as_uint(most);
        int byte = static_cast<int>(bits >> 23) - SHIFT + ((bits & 0x7fffffu) > TOP ? 1 : 0);
        byte = max(byte, 0);
        b.byte = finite ? static_cast<uint32_t>(byte) : 255u;
        // 2^-e; for the two ends of the exponent's range it is no normal number, but
        // there the block is not finite, or smaller than any fp16 value
        b.factor = power_of_two(min(127, 127 - byte));
        b.divisor = 0.0f;
    }
    if (!finite) b.divisor = b.factor = 0.0f;  // zeros (behind a row's end) stay codes of zero
    return b;
}

// x / s: for nvfp4 the rounded product and one correction, which gives the quotient
// wherever that decides a rounding (a border has 3 bits, so a quotient on it is exact).
template <int FORMAT>
__device__ __forceinline__ float scaled(float x, const BlockScale& b)
{
    if constexpr (FORMAT == NVFP4) {
        const float y = x * b.factor;
        return fmaf(-fmaf(y, b.divisor, -x), b.factor, y);  // in this form a zero keeps its sign
    } else {
        return x * b.factor;
    }
}

// Eight values to four bytes of e2m1 (the first in the lowest bits) or eight of e4m3.
__device__ __forceinline__ uint32_t pack_e2m1(const float (&v)[8])
{
    uint32_t r;
    asm("{\n\t"
        ".reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t"
        "}\n"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
}

// The codes of eight values: .x for the 4-bit formats, .x and .y for mxfp8.
template <int FORMAT>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], const BlockScale& b)
{
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = scaled<FORMAT>(x[i], b);
    uint2 r;
    if constexpr (FORMAT == MXFP8) {
        r.x = pack_e4m3(v[0], v[1], v[2], v[3]);
        r.y = pack_e4m3(v[4], v[5], v[6], v[7]);
    } else {
        r.x = pack_e2m1(v);
        r.y = 0;
    }
    return r;
}

// Eight halves (in four words) to mxfp8, scaled as pairs of halves: one multiplication for two
// values and no widening (5 % of a quantisation; the 4-bit conversion from halves is slower
// than from fp32).  That is exact where it decides a rounding: a
// product by a power of two is inexact only below 2^-14, the smallest normal half, and such
// values round to zero (the least border is 2^-10).  The factor 2^-e, e from -32 to 8 for fp16
// values, is applied in two steps that a half holds; beyond 2^30 (no value of the block
// above 2^-22) the words go through fp32.
__device__ __forceinline__ uint2 encode8_mxfp8(const uint4& v, const BlockScale& b)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const int e = 127 - static_cast<int>(b.byte);
    if (e > 30) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
        return encode8<MXFP8>(x, b);
    }
    const int e1 = min(e, 15);
    // a block that is not finite has the byte 255: factors of zero
    const bool finite = b.byte != 255u;
    const uint32_t f1 = finite ? static_cast<uint32_t>(e1 + 15) << 10 : 0u;
    const uint32_t f2 = static_cast<uint32_t>(finite ? e - e1 + 15 : 0) << 10;
    const uint32_t p1 = f1 | f1 << 16, p2 = f2 | f2 << 16;
    uint16_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 y = __hmul2(__hmul2(*reinterpret_cast<const __half2*>(&w[i]),
                                          *reinterpret_cast<const __half2*>(&p1)),
                                  *reinterpret_cast<const __half2*>(&p2));
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;"
            : "=h"(q[i])
            : "r"(*reinterpret_cast<const uint32_t*>(&y)));
    }
    return make_uint2(static_cast<uint32_t>(q[0]) | static_cast<uint32_t>(q[1]) << 16,
                      static_cast<uint32_t>(q[2]) | static_cast<uint32_t>(q[3]) << 16);
}

// Lanes that share a block when a lane holds eight consecutive values, and the largest
// magnitude over them.  A NaN counts as larger than everything (comparison of bits).
template <int FORMAT>
__device__ __forceinline__ float block_most(float most)
{
    uint32_t m = __float_as_uint(most);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    if constexpr (FORMAT != NVFP4) m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    return __uint_as_float(m);
}

__device__ __forceinline__ float most_of(const float (&x)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    return __uint_as_float(m);
}

// Quantise eight consecutive values per lane (`vec` counts them from the row's start; lane
// and lane + 1 hold neighbours, aligned so that a block's lanes are together) and store
// the codes and, by the first lane of each group (or block) of scales, the scales.  All lanes
// of the warp take part; those at or past the row's padded end store nothing.
template <int FORMAT>
__device__ __forceinline__ void quantize_store(const float (&x)[8], float t, float sixth,
                                               int vec, uint8_t* codes_row,
                                               uint8_t* scales_row, int chunks, int groups,
                                               bool row_valid)
{
    const BlockScale b = block_scale<FORMAT>(block_most<FORMAT>(most_of(x)), t, sixth);
    const uint2 q = encode8<FORMAT>(x, b);
    constexpr int PER_CHUNK = mx_chunk(FORMAT) / 8;
    const int chunk = vec / PER_CHUNK;
    const int part = vec % PER_CHUNK;
    if (row_valid && chunk < chunks) {
        uint8_t* to = codes_row + chunk * MX_CHUNK_BYTES;
        if constexpr (FORMAT == MXFP8)
            reinterpret_cast<uint2*>(to)[part] = q;
        else
            reinterpret_cast<uint32_t*>(to)[part] = q.x;
    }
    constexpr int LANES = mx_block(FORMAT) / 8;
    if constexpr (mx_group_blocks(FORMAT) == 4) {
        // the bytes of four blocks: lanes LANES apart
        uint32_t word = b.byte;
        word |= __shfl_down_sync(0xffffffffu, word, LANES) << 8;
        word |= __shfl_down_sync(0xffffffffu, word, 2 * LANES) << 16;
        const int group = vec / (4 * LANES);
        if (row_valid && vec % (4 * LANES) == 0 && group < groups)
            *reinterpret_cast<uint32_t*>(scales_row + group * MX_GROUP_BYTES) = word;
    } else {
        const int block = vec / LANES;
        const int group = block / mx_group_blocks(FORMAT);
        if (row_valid && vec % LANES == 0 && group < groups)
            scales_row[group * MX_GROUP_BYTES + block % mx_group_blocks(FORMAT)] =
                static_cast<uint8_t>(b.byte);
    }
}

// Magnitudes of eight fp16 values in four words: the largest, NaN above the infinity.
__device__ __forceinline__ float most_of_halves(const uint4& v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    __half2 m = __habs2(*reinterpret_cast<const __half2*>(&w[0]));
#pragma unroll
    for (int i = 1; i < 4; ++i)
        m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __half2*>(&w[i])));
    return __half2float(__hmax_nan(__low2half(m), __high2half(m)));
}

// Largest finite magnitude `bits` of a tensor -> the least power of two t with most <=
// 2688 t = 1.3125 * 2^11 t; 1 for zeros.
__device__ __forceinline__ float tensor_scale_of(uint32_t bits)
{
    if (bits == 0) return 1.0f;
    const int up = (bits & 0x7fffffu) > 0x280000u ? 1 : 0;
    const int e = static_cast<int>(bits >> 23) - 127 - 11 + up;
    return power_of_two(max(e, -126));
}

}  // namespace tg
