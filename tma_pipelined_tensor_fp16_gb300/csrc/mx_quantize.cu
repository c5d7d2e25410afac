// mx_quantize.cu -- fp16 matrices to the block-scaled formats of include/tmamicro.h and
// back.  On paper all are bound by memory: every value is read once (twice where the tensor
// scale has to be found first) and its codes and scales are written once.  Measured: 16384 x
// 4096 to mxfp8 31 us, 6.5 TB/s, mxfp4 28, nvfp4 33 (bound by issue slots, 5.2 TB/s); along
// columns 33, 30, 35; decoding 31, 27, 27 us, 6.3 to 6.6 TB/s.
#include <algorithm>
#include <type_traits>

#include "../../include/tmamicro.h"
#include "device_common.cuh"
#include "launch.h"
#include "microscale.cuh"
#include "runtime.h"

namespace tg {

namespace {

constexpr int AMAX_PARTS = GEMM_MX_WORKSPACE_BYTES / 4;

struct QuantizeParams {
    int64_t rows, K;  // of the quantised matrix
    int64_t chunks, groups;
    const __half* X;
    uint8_t* codes;
    uint8_t* scales;
    float* tensor_scale;
    const uint32_t* parts;  // largest magnitudes of parts of X, or nullptr
    int part_count;
};

// ------------------------------------------------------------ tensor scale

// Largest finite magnitude of each CTA's share of `vecs` vectors of eight values: 4096 of them
// at a time (64 KB).  Magnitudes of fp16 compare as their bits; infinities and NaN do not count.
// Two CTAs on an SM: there are few parts for every CTA of the quantiser to read.
constexpr int MOST_THREADS = 1024;

__global__ void __launch_bounds__(MOST_THREADS)
    k_mx_most(const uint4* X, int64_t vecs, uint32_t* parts)
{
    griddep_wait();
    griddep_launch_dependents();
    uint32_t most = 0;
    auto take = [&](uint32_t w) {
        const uint32_t a = w & 0x7fffu, b = (w >> 16) & 0x7fffu;
        if (a < 0x7c00u) most = max(most, a);
        if (b < 0x7c00u) most = max(most, b);
    };
    const int64_t turn = static_cast<int64_t>(gridDim.x) * 4 * MOST_THREADS;
    int64_t i = static_cast<int64_t>(blockIdx.x) * 4 * MOST_THREADS + threadIdx.x;
    for (; i + 3 * MOST_THREADS < vecs; i += turn) {
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = X[i + j * MOST_THREADS];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            take(v[j].x);
            take(v[j].y);
            take(v[j].z);
            take(v[j].w);
        }
    }
    for (; i < vecs; i += MOST_THREADS) {  // of the last 4096
        const uint4 v = X[i];
        take(v.x);
        take(v.y);
        take(v.z);
        take(v.w);
    }
    __shared__ uint32_t warps[MOST_THREADS / 32];
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane_id() == 0) warps[threadIdx.x / 32] = most;
    __syncthreads();
    if (threadIdx.x < 32) {
        most = __reduce_max_sync(0xffffffffu, warps[threadIdx.x]);
        if (threadIdx.x == 0) {
            const float f = __half2float(__ushort_as_half(static_cast<unsigned short>(most)));
            parts[blockIdx.x] = __float_as_uint(f);
        }
    }
}

// The tensor scale: from the parts, by every CTA for itself, as given, or none.
enum : int { SCALE_NONE, SCALE_GIVEN, SCALE_FOUND };

template <int SCALE>
__device__ __forceinline__ float find_tensor_scale(const QuantizeParams& p, uint32_t* shared)
{
    if constexpr (SCALE == SCALE_NONE) return 1.0f;
    if constexpr (SCALE == SCALE_GIVEN) {
        // Beyond 2^100 every fp16 value rounds to zero, and below 2^-100 every one but zero is cut
        // off, as at these borders: no quotient need leave fp32.  A negative number or a NaN
        // scales nothing: every block gets the scale NaN.
        const float t = *p.tensor_scale;
        return t >= 0.0f ? fminf(fmaxf(t, 0x1p-100f), 0x1p100f) : __uint_as_float(0x7fc00000u);
    }
    uint32_t most = 0;
    for (int i = static_cast<int>(threadIdx.x); i < p.part_count;
         i += 4 * static_cast<int>(blockDim.x)) {
        uint32_t v[4];  // on their way together
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = i + j * static_cast<int>(blockDim.x);
            v[j] = at < p.part_count ? p.parts[at] : 0u;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) most = max(most, v[j]);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane_id() == 0) shared[threadIdx.x / 32] = most;
    __syncthreads();
    most = 0;
    for (int i = 0; i < static_cast<int>(blockDim.x / 32); ++i) most = max(most, shared[i]);
    const float t = tensor_scale_of(most);
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.tensor_scale = t;
    return t;
}

// --------------------------------------------------------------- along rows
//
// A CTA takes 32 rows x 128 values (96 of mxfp4) through shared memory, and a thread 32 values
// of a row: a block (two of nvfp4), 16 or 32 bytes of codes.  So a scale is found once and
// without exchange between lanes (with four lanes a block, each finding it: 35, 33, 39 us), and
// a warp, whose lanes are consecutive rows, stores 512 contiguous bytes of a chunk's column.
TG_HD constexpr int row_spans(int format) { return format == MXFP4 ? 3 : 4; }
TG_HD constexpr int row_k(int format) { return 32 * row_spans(format); }

// Where the scale was found first, the tiles go from the last to the first: the L2 still holds
// what the search has read last (16384 x 4096 with the search 55 us, in the other order 61).
template <int SCALE>
__device__ __forceinline__ uint32_t tile_number()
{
    return SCALE == SCALE_FOUND ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
}

template <int FORMAT, int SCALE>
__global__ void __launch_bounds__(row_k(FORMAT))
    k_mx_quantize(const __grid_constant__ QuantizeParams p, uint32_t spans)
{
    constexpr int ROW_K = row_k(FORMAT), THREADS = ROW_K;
    constexpr int VECS = ROW_K / 8;               // of eight values in a row of the tile
    __shared__ uint32_t shared[THREADS / 32];
    __shared__ __align__(16) uint4 tile[32][VECS + 1];
    __shared__ __align__(4) uint8_t scale_bytes[32][8];
    const int tid = static_cast<int>(threadIdx.x);
    if (FORMAT == MXFP4 && tid < 32) scale_bytes[tid][3] = 0;
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t number = tile_number<SCALE>(), y = number / spans;
    const int64_t row0 = static_cast<int64_t>(y) * 32;
    const int64_t k0 = static_cast<int64_t>(number - y * spans) * ROW_K;
    const auto load = [&](int i) {
        const int at = i * THREADS + tid;
        const int64_t row = row0 + at / VECS, k = k0 + at % VECS * 8;
        return row < p.rows && k < p.K ? *reinterpret_cast<const uint4*>(p.X + row * p.K + k)
                                       : make_uint4(0, 0, 0, 0);
    };
    const auto place = [&](int i) -> uint4& {
        const int at = i * THREADS + tid;
        return tile[at / VECS][at % VECS];
    };
    constexpr int LOADS = 32 * VECS / THREADS;
    float t = 1.0f;
    if constexpr (FORMAT == NVFP4) {
        // the values are on their way while the tensor scale is found (1024 x 4096 with the search:
        // 0.9 us of 8)
        uint4 in[LOADS];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) in[i] = load(i);
        t = find_tensor_scale<SCALE>(p, shared);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) place(i) = in[i];
    } else {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) place(i) = load(i);
    }
    const float sixth = 1.0f / (6.0f * t);
    __syncthreads();
    const int line = tid % 32, part = tid / 32;  // 32 values of a row
    const int64_t row = row0 + line;
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = tile[line][part * 4 + j];
    constexpr int PER_BLOCK = mx_block(FORMAT) / 8;
    uint32_t out[8];
#pragma unroll
    for (int j = 0; j < 4; j += PER_BLOCK) {
        uint32_t most = 0;  // magnitudes compare as their bits, NaN above the infinity
#pragma unroll
        for (int i = 0; i < PER_BLOCK; ++i)
            most = max(most, __float_as_uint(most_of_halves(v[j + i])));
        const BlockScale b = block_scale<FORMAT>(__uint_as_float(most), t, sixth);
#pragma unroll
        for (int i = 0; i < PER_BLOCK; ++i) {
            if constexpr (FORMAT == MXFP8) {
                const uint2 q = encode8_mxfp8(v[j + i], b);
                out[2 * (j + i)] = q.x;
                out[2 * (j + i) + 1] = q.y;
            } else {
                float x[8];
                widen8(v[j + i], x);
                out[j + i] = encode8<FORMAT>(x, b).x;
            }
        }
        scale_bytes[line][(part * 4 + j) / PER_BLOCK] = static_cast<uint8_t>(b.byte);
    }
    if (row < p.rows) {
        constexpr int CHUNKS = 32 / mx_chunk(FORMAT);
        const int64_t chunk = (k0 + part * 32) / mx_chunk(FORMAT);
        uint8_t* to = p.codes + mx_code_offset(row, chunk, p.chunks);
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
            if (chunk + c < p.chunks)
                *reinterpret_cast<uint4*>(to + c * MX_CHUNK_BYTES) =
                    make_uint4(out[4 * c], out[4 * c + 1], out[4 * c + 2], out[4 * c + 3]);
    }
    __syncthreads();
    constexpr int GROUPS = ROW_K / mx_group(FORMAT);
    if (tid < 32 * GROUPS) {
        const int64_t to_row = row0 + tid % 32;
        const int64_t group = k0 / mx_group(FORMAT) + tid / 32;
        if (to_row < p.rows && group < p.groups)
            *reinterpret_cast<uint32_t*>(p.scales + mx_scale_offset(to_row, group, p.groups)) =
                *reinterpret_cast<const uint32_t*>(&scale_bytes[tid % 32][tid / 32 * 4]);
    }
}

// ------------------------------------------------------------ along columns
//
// X is K x rows; a CTA takes 128 of K (96 for mxfp4) x 64 columns through shared memory, and a
// thread two columns x 32 of K: a block (two of nvfp4) of each, 16 or 32 bytes of codes a column.
// The columns are rows of the result, so a warp stores 1 KB without gaps.
constexpr int COL_COLS = 64;
TG_HD constexpr int col_threads(int format) { return 32 * row_spans(format); }

template <int FORMAT, int SCALE>
__global__ void __launch_bounds__(col_threads(FORMAT))
    k_mx_quantize_columns(const __grid_constant__ QuantizeParams p, uint32_t col_tiles)
{
    constexpr int COL_K = row_k(FORMAT), COL_THREADS = col_threads(FORMAT);
    __shared__ uint32_t shared[COL_THREADS / 32];
    __shared__ __align__(16) uint32_t tile[COL_K][COL_COLS / 2];
    __shared__ __align__(4) uint8_t scale_bytes[COL_COLS][8];
    if (FORMAT == MXFP4 && threadIdx.x < COL_COLS) scale_bytes[threadIdx.x][3] = 0;
    griddep_wait();
    griddep_launch_dependents();
    const float t = find_tensor_scale<SCALE>(p, shared);
    const float sixth = 1.0f / (6.0f * t);
    const int tid = static_cast<int>(threadIdx.x);
    const uint32_t number = tile_number<SCALE>(), k_tile = number / col_tiles;
    const int64_t c0 = static_cast<int64_t>(number - k_tile * col_tiles) * COL_COLS;
    const int64_t k0 = static_cast<int64_t>(k_tile) * COL_K;
#pragma unroll
    for (int i = 0; i < COL_K * COL_COLS / 8 / COL_THREADS; ++i) {
        const int line = i * (COL_THREADS / 8) + tid / 8;
        const int64_t k = k0 + line, c = c0 + tid % 8 * 8;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (k < p.K && c < p.rows) v = *reinterpret_cast<const uint4*>(p.X + k * p.rows + c);
        *reinterpret_cast<uint4*>(&tile[line][tid % 8 * 4]) = v;
    }
    __syncthreads();
    const int pair = tid % 32, part = tid / 32;  // two columns, 32 of K
    uint32_t w[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i] = tile[part * 32 + i][pair];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t row = c0 + pair * 2 + h;  // of the result
        constexpr int BLOCK = mx_block(FORMAT);
        uint32_t out[8];
#pragma unroll
        for (int b0 = 0; b0 < 32; b0 += BLOCK) {
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < BLOCK; ++i) most = max(most, (w[b0 + i] >> (16 * h)) & 0x7fffu);
            // magnitudes of fp16 order as their bits, NaN above the infinity
            const BlockScale b = block_scale<FORMAT>(
                __half2float(__ushort_as_half(static_cast<unsigned short>(most))), t, sixth);
#pragma unroll
            for (int i0 = 0; i0 < BLOCK; i0 += 8) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    x[i] = __half2float(__ushort_as_half(
                        static_cast<unsigned short>(w[b0 + i0 + i] >> (16 * h))));
                const uint2 q = encode8<FORMAT>(x, b);
                if constexpr (FORMAT == MXFP8) {
                    out[(b0 + i0) / 4] = q.x;
                    out[(b0 + i0) / 4 + 1] = q.y;
                } else {
                    out[(b0 + i0) / 8] = q.x;
                }
            }
            scale_bytes[pair * 2 + h][(part * 32 + b0) / BLOCK] = static_cast<uint8_t>(b.byte);
        }
        if (row < p.rows) {
            constexpr int CHUNKS = 32 / mx_chunk(FORMAT);
            const int64_t chunk = (k0 + part * 32) / mx_chunk(FORMAT);
            uint8_t* to = p.codes + mx_code_offset(row, chunk, p.chunks);
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c)
                if (chunk + c < p.chunks)
                    *reinterpret_cast<uint4*>(to + c * MX_CHUNK_BYTES) =
                        make_uint4(out[4 * c], out[4 * c + 1], out[4 * c + 2], out[4 * c + 3]);
        }
    }
    __syncthreads();
    constexpr int GROUPS = COL_K / mx_group(FORMAT);
    for (int i = tid; i < COL_COLS * GROUPS; i += COL_THREADS) {
        const int64_t row = c0 + i % COL_COLS;
        const int64_t group = k0 / mx_group(FORMAT) + i / COL_COLS;
        if (row < p.rows && group < p.groups)
            *reinterpret_cast<uint32_t*>(p.scales + mx_scale_offset(row, group, p.groups)) =
                *reinterpret_cast<const uint32_t*>(&scale_bytes[i % COL_COLS][i / COL_COLS * 4]);
    }
}

// -------------------------------------------------------------------- values

constexpr int ROW_WARPS = 8;

// How a CTA's warps lie: 1 << k_log along a row, the others in the next rows.
struct RowTiling {
    uint32_t cta_spans;  // CTAs along a row
    int k_log;
    int64_t grid;
};

RowTiling row_tiling(int64_t rows, int64_t K, int format)
{
    const int64_t spans = (K + row_k(format) - 1) / row_k(format);
    RowTiling t;
    t.k_log = spans >= 8 ? 3 : spans >= 4 ? 2 : spans >= 2 ? 1 : 0;
    t.cta_spans = static_cast<uint32_t>((spans + (1 << t.k_log) - 1) >> t.k_log);
    const int64_t cta_rows = 8 * (ROW_WARPS >> t.k_log);
    t.grid = std::max<int64_t>(1, (rows + cta_rows - 1) / cta_rows) * t.cta_spans;
    return t;
}

// First row and first value of this warp's tile.
__device__ __forceinline__ void row_tile(uint32_t cta_spans, int k_log, int width, int64_t& row0,
                                         int64_t& k0)
{
    const uint32_t warp = threadIdx.x / 32;
    const uint32_t y = blockIdx.x / cta_spans, x = blockIdx.x - y * cta_spans;
    row0 = (static_cast<int64_t>(y) * (ROW_WARPS >> k_log) + (warp >> k_log)) * 8;
    k0 = (static_cast<int64_t>(x) * (1 << k_log) + (warp & ((1u << k_log) - 1u))) * width;
}

struct ValuesParams {
    int64_t rows, K, chunks, groups;
    const uint8_t* codes;
    const uint8_t* scales;
    const float* tensor_scale;
    void* values;
};

// Eight codes to fp16 pairs (exact).
template <int FORMAT>
__device__ __forceinline__ void decode8(uint2 q, __half2 (&v)[4])
{
    uint32_t h[4];
    if constexpr (FORMAT == MXFP8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = i < 2 ? q.x : q.y;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;"
                : "=r"(h[i])
                : "h"(static_cast<uint16_t>(w >> (16 * (i & 1)))));
        }
    } else {
        asm("{\n\t"
            ".reg .b8 a, b, c, d;\n\t"
            "mov.b32 {a, b, c, d}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
            "cvt.rn.f16x2.e2m1x2 %3, d;\n\t"
            "}\n"
            : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
            : "r"(q.x));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<__half2*>(&h[i]);
}

// The scale of a block in fp16, twice, where fp16 holds it: then one multiplication of halves
// rounds as a product in fp32 that is rounded to fp16 (both round the exact product once).
// False: the scale needs fp32.
template <int FORMAT>
__device__ __forceinline__ bool scale_of_halves(uint32_t byte, float t, uint32_t& scale)
{
    if constexpr (FORMAT == NVFP4) {
        // a multiple of 2^-9 up to 448 (or NaN), times a power of two from 2^-15 to 2^7
        const uint32_t bits = __float_as_uint(t);
        if ((bits & 0x7fffffu) || bits < (127u - 15u) << 23 || bits > (127u + 7u) << 23)
            return false;
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(byte * 0x101u)));
        const __half2 s = __hmul2(*reinterpret_cast<const __half2*>(&h), __float2half2_rn(t));
        scale = *reinterpret_cast<const uint32_t*>(&s);
    } else {
        const uint32_t e = byte - (127u - 15u);  // of a normal half
        if (e - 1u > 29u) return false;
        scale = e << 10 | e << 26;
    }
    return true;
}

template <int FORMAT>
__device__ __forceinline__ float scale_of(uint32_t byte)
{
    return FORMAT == NVFP4 ? float_of_e4m3(byte) : float_of_e8m0(byte);
}

// A value from its code and its block's scale, and the tensor's: q s is exact for nvfp4 (six
// bits) and rounded once by t, whose product with s alone may leave fp32 where q s t does not.
template <int FORMAT>
__device__ __forceinline__ float value_of(float q, float s, float t)
{
    return FORMAT == NVFP4 ? q * s * t : q * s;
}

__device__ __forceinline__ __half2 half2_of(uint32_t w)
{
    return *reinterpret_cast<const __half2*>(&w);
}

// The codes of eight values that start `skew` (0 to 7) before q's, of which `prev` are those in
// front.
template <int FORMAT>
__device__ __forceinline__ uint2 codes_before(uint2 prev, uint2 q, int skew)
{
    if constexpr (FORMAT == MXFP8) {
        const int n = 8 * (skew & 3);
        const bool far = skew >= 4;
        const uint32_t a = far ? prev.x : prev.y, b = far ? prev.y : q.x, c = far ? q.x : q.y;
        return make_uint2(__funnelshift_l(a, b, n), __funnelshift_l(b, c, n));
    } else {
        return make_uint2(__funnelshift_l(prev.x, q.x, 4 * skew), 0);
    }
}

// A lane decodes eight consecutive values; four lanes 32, eight rows a warp: a warp takes 8
// rows x 128 (96) values.  With ODD a row's length is no multiple of 8, so that rows start
// anywhere.  To fp32 the values then go through shared memory and leave as aligned words.  To
// fp16 a lane takes the eight values of an aligned vector of 16 bytes instead, which start up to
// seven in front of its own codes: it shifts its codes together with its neighbour's, and up to
// seven values have the scale of the block in front (5000 x 4001 nvfp4 11.4 us; through shared
// memory 13.8).
template <int FORMAT, bool F16OUT, bool ODD>
__global__ void __launch_bounds__(ROW_WARPS * 32)
    k_mx_values(const __grid_constant__ ValuesParams p, uint32_t cta_spans, int k_log)
{
    constexpr bool SHIFTED = ODD && F16OUT, STAGED = ODD && !F16OUT;
    int64_t row0, k0;
    row_tile(cta_spans, k_log, row_k(FORMAT), row0, k0);
    if (row0 >= p.rows || k0 >= p.K + (SHIFTED ? 7 : 0)) return;
    griddep_wait();
    griddep_launch_dependents();
    const int lane = static_cast<int>(lane_id());
    constexpr int SPANS = row_spans(FORMAT), ROW_K = row_k(FORMAT);
    __shared__ float staged[STAGED ? ROW_WARPS : 1][8][ROW_K + 2];
    float(*rows)[ROW_K + 2] = staged[STAGED ? threadIdx.x / 32 : 0];
    const int64_t row = row0 + lane / 4;
    if (!ODD && row >= p.rows) return;
    const bool valid = row < p.rows;
    const int part = lane % 4;
    const float t = p.tensor_scale ? *p.tensor_scale : 1.0f;
    constexpr int PER_CHUNK = mx_chunk(FORMAT) / 8;
    const uint8_t* codes = p.codes + mx_code_offset(row, k0 / mx_chunk(FORMAT), p.chunks);
    const uint8_t* scales = p.scales + mx_scale_offset(row, k0 / mx_group(FORMAT), p.groups);
    constexpr int GROUPS = ROW_K / mx_group(FORMAT);
    const auto codes_at = [](const uint8_t* chunk, int eight) {
        if constexpr (FORMAT == MXFP8)
            return reinterpret_cast<const uint2*>(chunk)[eight];
        else
            return make_uint2(reinterpret_cast<const uint32_t*>(chunk)[eight], 0);
    };
    uint32_t words[GROUPS];
#pragma unroll
    for (int g = 0; g < GROUPS; ++g)
        words[g] = valid && k0 / mx_group(FORMAT) + g < p.groups
                       ? *reinterpret_cast<const uint32_t*>(scales + g * MX_GROUP_BYTES)
                       : 0u;
    uint2 q[SPANS];
#pragma unroll
    for (int j = 0; j < SPANS; ++j) {
        const int64_t k = k0 + j * 32 + part * 8;
        const int chunk = (j * 4 + part) / PER_CHUNK;
        q[j] = make_uint2(0, 0);
        if (valid && k < p.K) q[j] = codes_at(codes + chunk * MX_CHUNK_BYTES, part % PER_CHUNK);
    }
    const auto byte_of = [&](int block) { return (words[block / 4] >> (8 * (block % 4))) & 0xffu; };
    const auto block_of = [&](int j) { return FORMAT == NVFP4 ? j * 2 + part / 2 : j; };
    if constexpr (SHIFTED) {
        __half* to = static_cast<__half*>(p.values) + row * p.K;
        const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(to) >> 1) & 7;
        uint2 front = make_uint2(0, 0);  // of the eight values in front of the tile
        uint32_t front_byte = byte_of(0);
        if (part == 0 && valid && k0 > 0) {
            constexpr int LAST = mx_group_blocks(FORMAT) - 1;
            front = codes_at(codes - MX_CHUNK_BYTES, PER_CHUNK - 1);
            front_byte = scales[LAST - MX_GROUP_BYTES];
        }
        // of a pair of values, which have the scale in front (the second word's)
        uint32_t pick[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            pick[i] = 2 * i + 1 < skew ? 0x7654u : 2 * i < skew ? 0x3254u : 0x3210u;
#pragma unroll
        for (int j = 0; j < SPANS; ++j) {
            // the codes of the lane in front; the row's first has them of the span in front
            const uint2 give = part == 3 && j > 0 ? q[j > 0 ? j - 1 : 0] : q[j];
            const int from = (lane & ~3) | ((lane + 3) & 3);
            uint2 prev;
            prev.x = __shfl_sync(0xffffffffu, give.x, from);
            prev.y = FORMAT == MXFP8 ? __shfl_sync(0xffffffffu, give.y, from) : 0u;
            if (j == 0 && part == 0) prev = front;
            const int block = block_of(j);
            const bool starts = (part * 8) % mx_block(FORMAT) == 0;  // a block
            const uint32_t byte = byte_of(block);
            const uint32_t before = !starts     ? byte
                                    : block > 0 ? byte_of(max(block - 1, 0))
                                                : front_byte;
            __half2 v[4];
            decode8<FORMAT>(codes_before<FORMAT>(prev, q[j], skew), v);
            uint32_t s = 0, s0 = 0;
            if (scale_of_halves<FORMAT>(byte, t, s) && scale_of_halves<FORMAT>(before, t, s0)) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = __hmul2(v[i], half2_of(__byte_perm(s, s0, pick[i])));
            } else {
                const float f = scale_of<FORMAT>(byte), f0 = scale_of<FORMAT>(before);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 x = __half22float2(v[i]);
                    v[i] = __floats2half2_rn(
                        value_of<FORMAT>(x.x, 2 * i < skew ? f0 : f, t),
                        value_of<FORMAT>(x.y, 2 * i + 1 < skew ? f0 : f, t));
                }
            }
            const int64_t at = k0 + j * 32 + part * 8 - skew;
            if (!valid) continue;
            if (at >= 0 && at + 8 <= p.K) {
                *reinterpret_cast<uint4*>(to + at) = *reinterpret_cast<const uint4*>(v);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (at + e >= 0 && at + e < p.K)
                        to[at + e] = e & 1 ? __high2half(v[e / 2]) : __low2half(v[e / 2]);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < SPANS; ++j) {
            const int64_t k = k0 + j * 32 + part * 8;
            if (k >= p.K) break;
            const uint32_t byte = byte_of(block_of(j));
            __half2 v[4];
            decode8<FORMAT>(q[j], v);
            if constexpr (F16OUT) {
                uint32_t s = 0;
                if (scale_of_halves<FORMAT>(byte, t, s)) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = __hmul2(v[i], half2_of(s));
                } else {
                    const float f = scale_of<FORMAT>(byte);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 x = __half22float2(v[i]);
                        v[i] = __floats2half2_rn(value_of<FORMAT>(x.x, f, t),
                                                 value_of<FORMAT>(x.y, f, t));
                    }
                }
                *reinterpret_cast<uint4*>(static_cast<__half*>(p.values) + row * p.K + k) =
                    *reinterpret_cast<const uint4*>(v);
            } else {
                const float f = scale_of<FORMAT>(byte);
                float2 x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = __half22float2(v[i]);
                    x[i].x = value_of<FORMAT>(x[i].x, f, t);
                    x[i].y = value_of<FORMAT>(x[i].y, f, t);
                }
                if constexpr (STAGED) {
                    float2* to = reinterpret_cast<float2*>(&rows[lane / 4][j * 32 + part * 8]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) to[i] = x[i];
                } else {
                    float* at = static_cast<float*>(p.values) + row * p.K + k;
                    float4* to = reinterpret_cast<float4*>(at);
                    to[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
                    to[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
                }
            }
        }
    }
    if constexpr (STAGED) {
        __syncwarp();
        const int n = static_cast<int>(min(p.K - k0, static_cast<int64_t>(ROW_K)));
        const int count = static_cast<int>(min(p.rows - row0, static_cast<int64_t>(8)));
        float* to = static_cast<float*>(p.values) + row0 * p.K + k0;
        for (int r = 0; r < count; ++r) {
            for (int e = lane; e < n; e += 32) to[e] = rows[r][e];
            to += p.K;
        }
    }
}

int check_mx(int64_t rows, int64_t K, int format)
{
    if (format < MXFP8 || format > NVFP4)
        return fail(GEMM_ERR_INVALID_ARG, "unknown gemm_mx_format");
    if (rows < 0 || rows > MAX_COORDINATE || K < 1 || K > MAX_COORDINATE)
        return fail(GEMM_ERR_INVALID_ARG, "rows must be in [0, 2^31-65536], K in [1, 2^31-65536]");
    if ((mx_row_blocks(rows) + 1) * mx_chunks(K, format) > MAX_COORDINATE)
        return fail(GEMM_ERR_UNSUPPORTED, "rows * K is too large");
    return GEMM_OK;
}

template <typename... P, typename... A>
cudaError_t launch_format(int format, void (*k8)(P...), void (*k4)(P...), void (*kn)(P...),
                          int64_t grid, int threads, cudaStream_t stream, A... args)
{
    auto kernel = format == MXFP8 ? k8 : format == MXFP4 ? k4 : kn;
    return launch_dependent(kernel, dim3(static_cast<unsigned>(grid)),
                            dim3(static_cast<unsigned>(threads)), 0, 1, stream, args...);
}

}  // namespace

}  // namespace tg

using namespace tg;

extern "C" {

int gemm_mx_sizes(int64_t rows, int64_t K, int format, int64_t* codes_bytes, int64_t* scales_bytes)
{
    return guarded([&] {
        const int r = check_mx(rows, K, format);
        if (r != GEMM_OK) return r;
        if (!codes_bytes || !scales_bytes)
            return fail(GEMM_ERR_INVALID_ARG, "codes_bytes and scales_bytes must be non-NULL");
        *codes_bytes = mx_row_blocks(rows) * mx_chunks(K, format) * MX_CHUNK_BYTES;
        *scales_bytes = mx_row_blocks(rows) * mx_groups(K, format) * MX_GROUP_BYTES;
        return ok();
    });
}

int gemm_mx_quantize(int64_t rows, int64_t K, int format, int transpose, const void* X, void* codes,
                     void* scales, float* tensor_scale, void* workspace, void* cuda_stream)
{
    return guarded([&] {
        int r = check_mx(rows, K, format);
        if (r != GEMM_OK) return r;
        if ((transpose ? rows : K) % 8 != 0)
            return fail(GEMM_ERR_UNSUPPORTED, "the rows of X must hold a multiple of 8 values");
        if ((format == NVFP4) != (tensor_scale != nullptr))
            return fail(GEMM_ERR_INVALID_ARG, "tensor_scale must be given exactly for GEMM_NVFP4");
        if (rows > 0 && (!X || !codes || !scales))
            return fail(GEMM_ERR_INVALID_ARG, "X, codes and scales must be non-NULL");
        if (!aligned16(X) || !aligned16(codes) || !aligned16(scales))
            return fail(GEMM_ERR_UNSUPPORTED, "X, codes and scales must be 16-byte aligned");
        if ((reinterpret_cast<uintptr_t>(tensor_scale) |
             reinterpret_cast<uintptr_t>(workspace)) & 3u)
            return fail(GEMM_ERR_UNSUPPORTED, "tensor_scale and workspace must be 4-byte aligned");
        int dev, sms;
        r = require_device(&dev, &sms, nullptr);
        if (r != GEMM_OK) return r;
        cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
        cudaError_t e = cudaSuccess;
        QuantizeParams p = {};
        p.rows = rows;
        p.K = K;
        p.chunks = mx_chunks(K, format);
        p.groups = mx_groups(K, format);
        p.X = static_cast<const __half*>(X);
        p.codes = static_cast<uint8_t*>(codes);
        p.scales = static_cast<uint8_t*>(scales);
        p.tensor_scale = tensor_scale;
        if (format == NVFP4 && workspace) {
            const int64_t vecs = rows * K / 8;
            const int64_t want =
                std::max<int64_t>(1, (vecs + 4 * MOST_THREADS - 1) / (4 * MOST_THREADS));
            p.part_count = static_cast<int>(std::min<int64_t>(want, std::min(2 * sms, AMAX_PARTS)));
            p.parts = static_cast<const uint32_t*>(workspace);
            e = launch_dependent(k_mx_most, dim3(static_cast<unsigned>(p.part_count)),
                                 dim3(MOST_THREADS), 0, 1, stream, static_cast<const uint4*>(X),
                                 vecs, static_cast<uint32_t*>(workspace));
            if (e != cudaSuccess) return cuda_fail("tensor scale launch", e);
        }
        if (rows == 0 && format != NVFP4) return ok();
        if (transpose) {
            const int64_t cols = std::max<int64_t>(1, (rows + COL_COLS - 1) / COL_COLS);
            const int64_t grid = cols * ((K + row_k(format) - 1) / row_k(format));
            if (grid > MAX_COORDINATE) return fail(GEMM_ERR_UNSUPPORTED, "rows * K is too large");
            e = launch_format(format, k_mx_quantize_columns<MXFP8, SCALE_NONE>,
                              k_mx_quantize_columns<MXFP4, SCALE_NONE>,
                              p.parts ? k_mx_quantize_columns<NVFP4, SCALE_FOUND>
                                      : k_mx_quantize_columns<NVFP4, SCALE_GIVEN>,
                              grid, col_threads(format), stream, p, static_cast<uint32_t>(cols));
        } else {
            const int64_t spans = (K + row_k(format) - 1) / row_k(format);
            const int64_t grid = std::max<int64_t>(1, (rows + 31) / 32) * spans;
            if (grid > MAX_COORDINATE) return fail(GEMM_ERR_UNSUPPORTED, "rows * K is too large");
            e = launch_format(format, k_mx_quantize<MXFP8, SCALE_NONE>,
                              k_mx_quantize<MXFP4, SCALE_NONE>,
                              p.parts ? k_mx_quantize<NVFP4, SCALE_FOUND>
                                      : k_mx_quantize<NVFP4, SCALE_GIVEN>,
                              grid, row_k(format), stream, p, static_cast<uint32_t>(spans));
        }
        return e == cudaSuccess ? ok() : cuda_fail("quantisation launch", e);
    });
}

int gemm_mx_values(int64_t rows, int64_t K, int format, const void* codes, const void* scales,
                   const float* tensor_scale, int dtype_out, void* values, void* cuda_stream)
{
    return guarded([&] {
        int r = check_mx(rows, K, format);
        if (r != GEMM_OK) return r;
        if (dtype_out != GEMM_OUT_F32 && dtype_out != GEMM_OUT_F16)
            return fail(GEMM_ERR_INVALID_ARG,
                        "dtype_out must be GEMM_OUT_F32 (0) or GEMM_OUT_F16 (1)");
        if (rows > 0 && (!codes || !scales || !values))
            return fail(GEMM_ERR_INVALID_ARG, "codes, scales and values must be non-NULL");
        if (!aligned16(codes) || !aligned16(scales) || !aligned16(values))
            return fail(GEMM_ERR_UNSUPPORTED, "codes, scales and values must be 16-byte aligned");
        if (tensor_scale && format != NVFP4)
            return fail(GEMM_ERR_INVALID_ARG, "only GEMM_NVFP4 has a tensor_scale");
        if (reinterpret_cast<uintptr_t>(tensor_scale) & 3u)
            return fail(GEMM_ERR_UNSUPPORTED, "tensor_scale must be 4-byte aligned");
        int dev;
        r = require_device(&dev, nullptr, nullptr);
        if (r != GEMM_OK) return r;
        if (rows == 0) return ok();
        ValuesParams p = {};
        p.rows = rows;
        p.K = K;
        p.chunks = mx_chunks(K, format);
        p.groups = mx_groups(K, format);
        p.codes = static_cast<const uint8_t*>(codes);
        p.scales = static_cast<const uint8_t*>(scales);
        p.tensor_scale = tensor_scale;
        p.values = values;
        const bool odd = K % 8 != 0;
        // shifted vectors reach up to seven values behind the row's end
        const RowTiling t =
            row_tiling(rows, odd && dtype_out == GEMM_OUT_F16 ? K + 7 : K, format);
        if (t.grid > MAX_COORDINATE) return fail(GEMM_ERR_UNSUPPORTED, "rows * K is too large");
        cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
        auto launch = [&](auto f16, auto odd) {
            constexpr bool F = decltype(f16)::value, O = decltype(odd)::value;
            return launch_format(format, k_mx_values<MXFP8, F, O>, k_mx_values<MXFP4, F, O>,
                                 k_mx_values<NVFP4, F, O>, t.grid, ROW_WARPS * 32, stream, p,
                                 t.cta_spans, t.k_log);
        };
        const std::true_type yes;
        const std::false_type no;
        const cudaError_t e = dtype_out == GEMM_OUT_F16 ? odd ? launch(yes, yes) : launch(yes, no)
                              : odd                     ? launch(no, yes)
                                                        : launch(no, no);
        return e == cudaSuccess ? ok() : cuda_fail("decoding launch", e);
    });
}

}  // extern "C"
