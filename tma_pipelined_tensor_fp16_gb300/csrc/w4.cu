// w4.cu -- products with 4-bit weights and group scales,
//
//     Y[m][n] = sum_g scale[n][g] * sum_{k in g} (q[n][k] - zero[n][g]) X[m][k],
//
// for a few rows of X (decoding), and the expansion of the weights to fp16 for
// many rows.
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdio>
#include <new>
#include <type_traits>

#include "../../include/tmaexperts.h"
#include "launch.h"
#include "ptx.cuh"
#include "runtime.h"

namespace tg {

namespace {

struct W4Params {
    int M, N, K;
    int experts;          // 0: one matrix
    int share;            // rows of Y per row of X
    const uint8_t* packed;
    const __half* scales;
    const uint8_t* zeros;  // nullptr: 8 everywhere
    const __half* X;
    const int32_t* ids;
    void* Y;
    int f16out;
};

// ---------------------------------------------------------------- few rows
//
// Both kernels below run the product on mma.sync m16n8k16 with the weights as
// the 16-row operand and rows of X as the 8-column one: a row of X needs one
// multiply-add per weight whatever the unit, and on the tensor cores that leaves
// the conversion of the codes as the only arithmetic.  (tcgen05.mma would need
// the converted weights written back to shared memory.)
//
// A 32-bit word holds the codes k..k+7.  Masking the word and its shift by 8
// with 0x000f000f and 0x00f000f0 and setting the exponent of 1024 gives half
// pairs (k, k+4), (k+1, k+5), (k+2, k+6), (k+3, k+7) of 1024 + q or 1024 + 16 q;
// one half2 add or fused multiply-add makes them q - zero, exact in fp16.  The
// pairs of X are permuted alike.  Each group is summed in fp32 by the tensor
// core and enters the row's sum times its scale, so no weight is rounded.
//
// Weights arrive as blocks of 256 codes a row (128 bytes), 16 rows x 128 bytes
// per warp and block, swizzled by 16-byte chunk, through asynchronous copies
// with W4_STAGES - 1 blocks in flight.  Scales are read a block ahead into
// registers and their lines brought into L2 with the weights' (a DRAM access
// one block ahead would be waited for in every block: 57 us instead of 32 for
// one row of 16384 x 16384, groups of 128).
constexpr int W4_WARPS = 8;
constexpr int W4_THREADS = W4_WARPS * 32;
constexpr int W4_ROWS = 16;
constexpr int W4_BLOCK = 256;  // weights of a row per block: 128 bytes
constexpr int W4_STAGES = 4;
constexpr int W4_FEW_STAGES = 3;
constexpr int W4_STAGE_BYTES = W4_ROWS * W4_BLOCK / 2;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool valid)
{
    const int bytes = valid ? 16 : 0;  // 0: fill with zeros, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void cp_async_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_m16n8k16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same onto zero: the first product of a group.
__device__ __forceinline__ void mma_m16n8k16_first(float (&d)[4], uint32_t a0, uint32_t a1,
                                                   uint32_t a2, uint32_t a3, uint32_t b0,
                                                   uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ __half2 as_half2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
__device__ __forceinline__ uint32_t as_u32(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }

// q - zero of the eight codes of `w` as four half pairs (k, k + 4), (k + 1,
// k + 5), (k + 2, k + 6), (k + 3, k + 7).  `z` is -(1024 + zero), twice.
__device__ __forceinline__ void decode8(uint32_t w, __half2 z, uint32_t (&e)[4])
{
    const __half2 sixteenth = as_half2(0x2c002c00u);               // 1/16
    const __half2 z64 = __hadd2(z, as_half2(0x63806380u));         // + 960: -(64 + zero)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        e[2 * h] = as_u32(__hadd2(as_half2((w & 0x000f000fu) | 0x64006400u), z));
        e[2 * h + 1] =
            as_u32(__hfma2(as_half2((w & 0x00f000f0u) | 0x64006400u), sixteenth, z64));
        w >>= 8;
    }
}

// One warp's ROWS = 16 * RT rows of the weights: the copies into its stage
// slots and the scales of a block, staged in shared memory as
// {scale, -(1024 + zero) twice}.
template <int GROUP, int RT>
struct W4Rows {
    static constexpr int ROWS = W4_ROWS * RT;
    static constexpr int GPS = W4_BLOCK / GROUP;  // groups per block and row
    static constexpr int SCALES = ROWS * GPS;
    static constexpr int EPL = SCALES / 32;       // scales a lane handles per block
    static constexpr int SLOT_BYTES = RT * W4_STAGE_BYTES;
    const uint8_t* packed;  // this lane's first chunk: row lane / 8, chunk lane % 8
    const __half* scales;   // this lane's first scale: row lane / GPS, group lane % GPS
    const uint8_t* zeros;   // alike, or nullptr
    int rows;               // rows that exist (0..ROWS)
    int half_k;             // bytes of a row
    int groups;             // groups of a row
    int whole;              // blocks below this need no check
    uint32_t lane;
    uint32_t dst[2];        // slot offset of the lane's even and odd chunks
    uint32_t ahead[EPL];    // scale bits | zero << 16

    __device__ __forceinline__ void init(const W4Params& p, int expert, int n0, uint32_t lane_)
    {
        lane = lane_;
        groups = p.K / GROUP;
        half_k = p.K / 2;
        rows = p.N - n0 < ROWS ? p.N - n0 : ROWS;
        if (rows < 0) rows = 0;
        whole = rows == ROWS ? p.K / W4_BLOCK : 0;
        const int64_t row = static_cast<int64_t>(expert) * p.N + (rows > 0 ? n0 : 0);
        const int r = static_cast<int>(lane >> 3), c = static_cast<int>(lane & 7u);
        packed = p.packed + (row + r) * half_k + c * 16;
        const int64_t at = (row + lane / GPS) * groups + lane % GPS;
        scales = p.scales + at;
        zeros = p.zeros ? p.zeros + at : nullptr;
        dst[0] = r * 128 + ((c ^ r) << 4);
        dst[1] = (r + 4) * 128 + ((c ^ (r + 4)) << 4);
    }

    __device__ __forceinline__ void copy_block(uint32_t slot, int kb) const
    {
        const uint8_t* src = packed + kb * (W4_BLOCK / 2);
        const int64_t next = static_cast<int64_t>(half_k) * 4;
        if (kb < whole) {
#pragma unroll
            for (int i = 0; i < SLOT_BYTES / 512; ++i) {
                cp_async16(slot + dst[i & 1] + (i / 2) * 1024, src);
                src += next;
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < SLOT_BYTES / 512; ++i) {
            const int row = static_cast<int>(lane >> 3) + 4 * i;
            const int byte = kb * (W4_BLOCK / 2) + static_cast<int>(lane & 7u) * 16;
            const bool ok = row < rows && byte < half_k;
            cp_async16_or_zero(slot + dst[i & 1] + (i / 2) * 1024, src + i * next, ok);
        }
    }

    // Whether the lane's i-th scale of block kb exists.
    __device__ __forceinline__ bool exists(int kb, int i) const
    {
        const int id = static_cast<int>(lane) + 32 * i;
        return kb < whole || (id / GPS < rows && kb * GPS + id % GPS < groups);
    }

    __device__ __forceinline__ int64_t index(int kb, int i) const
    {
        return static_cast<int64_t>(i) * (32 / GPS) * groups + kb * GPS;
    }

    // Into L2; one 32-byte sector holds 16 scales of a row.
    __device__ __forceinline__ void touch_scales(int kb) const
    {
        if (kb % (16 / GPS) != 0) return;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            if (!exists(kb, i)) continue;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(scales + index(kb, i)));
            if (zeros) asm volatile("prefetch.global.L2 [%0];" ::"l"(zeros + index(kb, i)));
        }
    }

    __device__ __forceinline__ void load_scales(int kb)
    {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            ahead[i] = 8u << 16;
            if (exists(kb, i)) {
                const int64_t at = index(kb, i);
                ahead[i] = __half_as_ushort(scales[at]);
                ahead[i] |= (zeros ? zeros[at] : 8u) << 16;
            }
        }
    }

    __device__ __forceinline__ void stage_scales(uint2* buf) const
    {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const float s =
                __half2float(__ushort_as_half(static_cast<unsigned short>(ahead[i] & 0xffffu)));
            const __half2 z = __float2half2_rn(-1024.0f - static_cast<float>(ahead[i] >> 16));
            buf[lane + 32 * i] = make_uint2(__float_as_uint(s), as_u32(z));
        }
    }
};

// The products of 16 rows with 32 codes each: e and f are decode8 of the words of
// rows g and g + 8, v the same positions of X in decode8's order.
__device__ __forceinline__ void mma_word(float (&d)[4], bool first, const uint32_t (&e)[4],
                                         const uint32_t (&f)[4], const uint4& v)
{
    if (first)
        mma_m16n8k16_first(d, e[0], f[0], e[2], f[2], v.x, v.y);
    else
        mma_m16n8k16(d, e[0], f[0], e[2], f[2], v.x, v.y);
    mma_m16n8k16(d, e[1], f[1], e[3], f[3], v.z, v.w);
}

// X[k..k+7] as decode8 orders the codes: pairs (k, k+4), (k+2, k+6), (k+1, k+5),
// (k+3, k+7).
__device__ __forceinline__ uint4 order_x(const uint4& v)
{
    return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.y, v.w, 0x5410),
                      __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x7632));
}

__device__ __forceinline__ void add_scaled(float (&acc)[4], const float (&part)[4], uint32_t s0,
                                           uint32_t s1)
{
    acc[0] = fmaf(__uint_as_float(s0), part[0], acc[0]);
    acc[1] = fmaf(__uint_as_float(s0), part[1], acc[1]);
    acc[2] = fmaf(__uint_as_float(s1), part[2], acc[2]);
    acc[3] = fmaf(__uint_as_float(s1), part[3], acc[3]);
}

__device__ __forceinline__ void store_y(const W4Params& p, int64_t row, int n, float v)
{
    const int64_t at = row * p.N + n;
    if (p.f16out)
        static_cast<__half*>(p.Y)[at] = __float2half_rn(v);
    else
        static_cast<float*>(p.Y)[at] = v;
}

__device__ __forceinline__ float ld_shared_rank(const float* local, uint32_t rank)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                 : "=f"(v)
                 : "r"(map_shared_rank(smem_u32(local), rank))
                 : "memory");
    return v;
}

// Up to eight rows of X (and, by expert, eight at a time).  Bound by reading the
// codes once.  A CTA owns 16 * RT rows of the weights and its eight warps take
// every eighth block of them, so that neighbouring warps read neighbouring
// 128-byte pieces of a row; no barrier joins the warps before the final sum.
// Where the rows alone leave SMs idle, the CTAs of a cluster share the rows'
// length and their sums meet through distributed shared memory, in rank order.
//
// By expert, grid.y is the row of Y: the first row of an expert does all of
// them, so an expert's weights are read once per eight rows, and nothing has to
// be sorted.
constexpr int W4_FEW = 8;
constexpr int W4_FEW_RT = 2;

template <int GROUP, int RT>
__host__ __device__ constexpr int w4_few_smem()
{
    return W4_WARPS * (W4_FEW_STAGES * RT * W4_STAGE_BYTES +
                       2 * RT * W4_ROWS * (W4_BLOCK / GROUP) * 8);
}

template <int GROUP, int RT>
__global__ void __launch_bounds__(W4_THREADS, 2)
    k_w4_few(const __grid_constant__ W4Params p)
{
    using Rows = W4Rows<GROUP, RT>;
    constexpr int STAGES = W4_FEW_STAGES;
    constexpr int WARP_BYTES = STAGES * Rows::SLOT_BYTES;
    extern __shared__ __align__(128) uint8_t w4_smem[];
    __shared__ int list[W4_FEW];
    __shared__ int list_count;
    const int tid = static_cast<int>(threadIdx.x);
    const int warp = tid >> 5;
    const uint32_t lane = lane_id();
    const int g = static_cast<int>(lane >> 2), t = static_cast<int>(lane & 3u);
    uint8_t* ring = w4_smem + warp * WARP_BYTES;
    uint2* scale_buf =
        reinterpret_cast<uint2*>(w4_smem + W4_WARPS * WARP_BYTES) + warp * 2 * Rows::SCALES;
    float* partial = reinterpret_cast<float*>(w4_smem);      // [warps][8][ROWS] after the loop
    float* sums = partial + W4_WARPS * W4_FEW * Rows::ROWS;  // [8][ROWS]
    const uint32_t csize = gridDim.z, crank = blockIdx.z;
    const int n0 = static_cast<int>(blockIdx.x) * Rows::ROWS;
    griddep_wait();
    griddep_launch_dependents();

    int expert = 0;
    if (p.experts > 0) {
        expert = p.ids[blockIdx.y];
        if (expert < 0 || expert >= p.experts) {  // a dropped row
            if (crank == 0 && tid < Rows::ROWS && n0 + tid < p.N)
                store_y(p, blockIdx.y, n0 + tid, 0.0f);
            return;
        }
        bool earlier = false;
        for (int r = tid; r < static_cast<int>(blockIdx.y); r += W4_THREADS)
            earlier |= p.ids[r] == expert;
        if (__syncthreads_or(earlier)) return;
    }
    Rows rows;
    rows.init(p, expert, n0, lane);
    const int blocks = (p.K + W4_BLOCK - 1) / W4_BLOCK;
    const int step = W4_WARPS * static_cast<int>(csize);
    const int kb0 = static_cast<int>(crank) * W4_WARPS + warp;

    int next_row = p.experts > 0 ? static_cast<int>(blockIdx.y) : 0;
    while (next_row < p.M) {
        // the rows of Y of this pass
        if (p.experts > 0) {
            if (warp == 0) {
                int found = 0;
                for (int r = next_row; r < p.M && found < W4_FEW; r += 32) {
                    const int i = r + static_cast<int>(lane);
                    const unsigned hit = __ballot_sync(0xffffffffu, i < p.M && p.ids[i] == expert);
                    const int slot = found + __popc(hit & ((1u << lane) - 1u));
                    if (((hit >> lane) & 1u) && slot < W4_FEW) list[slot] = i;
                    found += __popc(hit);
                }
                if (lane == 0) list_count = found < W4_FEW ? found : W4_FEW;
            }
            __syncthreads();
        }
        const int left = p.M - next_row;
        const int count = p.experts > 0 ? list_count : (left < W4_FEW ? left : W4_FEW);
        if (count == 0) break;
        // columns past the last row repeat the first one and are not stored
        const int column = g < count ? g : 0;
        const int xrow = p.experts > 0 ? list[column] : next_row + column;
        const __half* x = p.X + static_cast<int64_t>(xrow / p.share) * p.K + 8 * t;

        float acc[RT][4];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[rt][i] = 0.0f;

        // one block: FULL blocks lie inside K
        auto block = [&](auto full, int kb, const uint8_t* slot, const uint2* sc) {
            constexpr bool FULL = decltype(full)::value;
            constexpr int PER = GROUP / 32;
            const uint32_t* a = reinterpret_cast<const uint32_t*>(slot + g * 128) + t;
            float part[RT][4];
            uint2 s[RT][2];
#pragma unroll
            for (int j = 0; j < W4_BLOCK / 32; ++j) {
                const int k = kb * W4_BLOCK + j * 32;
                if (!FULL && k >= p.K) break;
                const uint4 v = order_x(*reinterpret_cast<const uint4*>(x + k));
                const int chunk = (g * 4) ^ (j * 4);
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    if (j % PER == 0) {
                        s[rt][0] = sc[(rt * 16 + g) * Rows::GPS + j / PER];
                        s[rt][1] = sc[(rt * 16 + g + 8) * Rows::GPS + j / PER];
                    }
                    uint32_t e[4], f[4];
                    decode8(a[rt * 512 + chunk], as_half2(s[rt][0].y), e);
                    decode8(a[rt * 512 + 256 + chunk], as_half2(s[rt][1].y), f);
                    mma_word(part[rt], j % PER == 0, e, f, v);
                    if (j % PER == PER - 1) add_scaled(acc[rt], part[rt], s[rt][0].x, s[rt][1].x);
                }
            }
        };

#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) {
            const int kb = kb0 + i * step;
            if (kb < blocks) {
                rows.copy_block(smem_u32(ring + i * Rows::SLOT_BYTES), kb);
                rows.touch_scales(kb);
            }
            cp_async_commit();
        }
        if (kb0 < blocks) rows.load_scales(kb0);
        int stage = 0, parity = 0;
        for (int kb = kb0; kb < blocks; kb += step) {
            const int far = kb + (STAGES - 1) * step;
            if (far < blocks) {
                const int slot = stage == 0 ? STAGES - 1 : stage - 1;
                rows.copy_block(smem_u32(ring + slot * Rows::SLOT_BYTES), far);
                rows.touch_scales(far);
            }
            cp_async_commit();
            uint2* sc = scale_buf + parity * Rows::SCALES;
            rows.stage_scales(sc);
            if (kb + step < blocks) rows.load_scales(kb + step);
            cp_async_wait<STAGES - 1>();
            __syncwarp();
            const uint8_t* slot = ring + stage * Rows::SLOT_BYTES;
            if ((kb + 1) * W4_BLOCK <= p.K)
                block(std::true_type(), kb, slot, sc);
            else
                block(std::false_type(), kb, slot, sc);
            __syncwarp();
            if (++stage == STAGES) stage = 0;
            parity ^= 1;
        }
        cp_async_wait<0>();
        __syncthreads();

        // sum over the warps, then over the CTAs that share the length, in order
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                partial[(warp * W4_FEW + 2 * t + (i & 1)) * Rows::ROWS + rt * 16 + g +
                        8 * (i >> 1)] = acc[rt][i];
        __syncthreads();
        float v = 0.0f;
        static_assert(W4_FEW * Rows::ROWS <= W4_THREADS, "one sum per thread");
        if (tid < W4_FEW * Rows::ROWS) {
#pragma unroll
            for (int w = 0; w < W4_WARPS; ++w) v += partial[w * W4_FEW * Rows::ROWS + tid];
            if (csize > 1) sums[tid] = v;
        }
        if (csize > 1) cluster_sync_all();
        const int c = tid / Rows::ROWS, n = n0 + tid % Rows::ROWS;
        if (crank == 0 && c < count && n < p.N) {
            for (uint32_t r = 1; r < csize; ++r) v += ld_shared_rank(sums + tid, r);
            store_y(p, p.experts > 0 ? list[c] : next_row + c, n, v);
        }
        const int last = p.experts > 0 ? list[count - 1] : next_row + count - 1;
        if (csize > 1)
            cluster_sync_all();  // rank 0 has read its peers' sums
        else
            __syncthreads();
        if (count < W4_FEW) break;
        next_row = last + 1;
    }
}

// 9 to 64 rows of X, COLS = 16, 32 or 64.  Every code now feeds COLS / 8 MMAs
// and X is read as often as the weights: a CTA owns 128 rows of the weights (16
// per warp) and keeps the block's part of X in shared memory for all of them, in
// decode8's order, read a block ahead through registers.  The CTAs of a cluster
// share the rows' length where the rows alone leave SMs idle; rank r then sums
// and stores columns r, r + size, ....
constexpr int W4_TILE = W4_WARPS * W4_ROWS;
// Bytes between rows of X in shared memory: 256 halves and 64 bytes more, so
// that the two rows a quarter of a warp reads at once lie in different banks.
constexpr int W4_X_PITCH = W4_BLOCK * 2 + 64;

template <int COLS, int GROUP>
__host__ __device__ constexpr int w4_tile_smem()
{
    return W4_WARPS * (W4_STAGES * W4_STAGE_BYTES + 2 * W4_ROWS * (W4_BLOCK / GROUP) * 8) +
           2 * COLS * W4_X_PITCH;
}

template <int COLS, int GROUP>
__global__ void __launch_bounds__(W4_THREADS, 1)
    k_w4_tile(const __grid_constant__ W4Params p)
{
    using Rows = W4Rows<GROUP, 1>;
    constexpr int NT = COLS / 8;
    constexpr int STAGES = W4_STAGES;
    constexpr int XPT = COLS * (W4_BLOCK / 8) / W4_THREADS;  // chunks of X per thread and block
    constexpr int SUM_PITCH = W4_TILE + 4;  // floats between columns of the sums
    constexpr int WARP_BYTES = STAGES * Rows::SLOT_BYTES;
    static_assert(COLS * SUM_PITCH * 4 <= W4_WARPS * WARP_BYTES, "sums fit the ring");
    extern __shared__ __align__(128) uint8_t w4_smem[];
    const int tid = static_cast<int>(threadIdx.x);
    const int warp = tid >> 5;
    const uint32_t lane = lane_id();
    const int g = static_cast<int>(lane >> 2), t = static_cast<int>(lane & 3u);
    uint8_t* ring = w4_smem + warp * WARP_BYTES;
    uint8_t* xbuf = w4_smem + W4_WARPS * WARP_BYTES;
    uint2* scale_buf =
        reinterpret_cast<uint2*>(xbuf + 2 * COLS * W4_X_PITCH) + warp * 2 * Rows::SCALES;
    float* sums = reinterpret_cast<float*>(w4_smem);  // [COLS][SUM_PITCH] after the loop
    const uint32_t csize = gridDim.z, crank = blockIdx.z;
    griddep_wait();
    griddep_launch_dependents();

    Rows rows;
    rows.init(p, 0, static_cast<int>(blockIdx.x) * W4_TILE + warp * W4_ROWS, lane);
    const int blocks = (p.K + W4_BLOCK - 1) / W4_BLOCK;
    const int step = static_cast<int>(csize);
    const int kb0 = static_cast<int>(crank);
    // rows past the last one repeat it and are not stored
    uint4 xa[XPT];
    auto load_x = [&](int kb) {
#pragma unroll
        for (int i = 0; i < XPT; ++i) {
            const int id = tid + W4_THREADS * i;
            int m = id / (W4_BLOCK / 8);
            if (m >= p.M) m = p.M - 1;
            const int k = kb * W4_BLOCK + id % (W4_BLOCK / 8) * 8;
            xa[i] = make_uint4(0, 0, 0, 0);
            if (k < p.K)
                xa[i] = *reinterpret_cast<const uint4*>(p.X + static_cast<int64_t>(m) * p.K + k);
        }
    };
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][i] = 0.0f;
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
        const int kb = kb0 + s * step;
        if (kb < blocks) {
            rows.copy_block(smem_u32(ring + s * Rows::SLOT_BYTES), kb);
            rows.touch_scales(kb);
        }
        cp_async_commit();
    }
    if (kb0 < blocks) {
        rows.load_scales(kb0);
        load_x(kb0);
    }
    int stage = 0, parity = 0;
    for (int kb = kb0; kb < blocks; kb += step) {
        const int far = kb + (STAGES - 1) * step;
        if (far < blocks) {
            const int slot = stage == 0 ? STAGES - 1 : stage - 1;
            rows.copy_block(smem_u32(ring + slot * Rows::SLOT_BYTES), far);
            rows.touch_scales(far);
        }
        cp_async_commit();
        uint2* sc = scale_buf + parity * Rows::SCALES;
        rows.stage_scales(sc);
        uint8_t* xs = xbuf + parity * COLS * W4_X_PITCH;
#pragma unroll
        for (int i = 0; i < XPT; ++i) {
            const int id = tid + W4_THREADS * i;
            *reinterpret_cast<uint4*>(xs + id / (W4_BLOCK / 8) * W4_X_PITCH +
                                      id % (W4_BLOCK / 8) * 16) = order_x(xa[i]);
        }
        if (kb + step < blocks) {
            rows.load_scales(kb + step);
            load_x(kb + step);
        }
        cp_async_wait<STAGES - 1>();
        // X and the scales of this block are staged; those of the block before
        // the last are used up, so their buffers may be written next time
        __syncthreads();
        const uint32_t* a = reinterpret_cast<const uint32_t*>(ring + stage * Rows::SLOT_BYTES +
                                                              g * 128) + t;
        const uint8_t* xg = xs + g * W4_X_PITCH + t * 16;
        constexpr int PER = GROUP / 32;
        float part[NT][4];
        uint2 s0, s1;
#pragma unroll
        for (int j = 0; j < W4_BLOCK / 32; ++j) {
            if (kb * W4_BLOCK + j * 32 >= p.K) break;
            if (j % PER == 0) {
                s0 = sc[g * Rows::GPS + j / PER];
                s1 = sc[(g + 8) * Rows::GPS + j / PER];
            }
            uint32_t e[4], f[4];
            const int chunk = (g * 4) ^ (j * 4);
            decode8(a[chunk], as_half2(s0.y), e);
            decode8(a[256 + chunk], as_half2(s1.y), f);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                mma_word(part[nt], j % PER == 0, e, f,
                         *reinterpret_cast<const uint4*>(xg + nt * 8 * W4_X_PITCH + j * 64));
            if (j % PER == PER - 1) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) add_scaled(acc[nt], part[nt], s0.x, s1.x);
            }
        }
        __syncwarp();
        if (++stage == STAGES) stage = 0;
        parity ^= 1;
    }
    cp_async_wait<0>();
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sums[(nt * 8 + 2 * t + (i & 1)) * SUM_PITCH + warp * W4_ROWS + g + 8 * (i >> 1)] =
                acc[nt][i];
    if (csize > 1)
        cluster_sync_all();
    else
        __syncthreads();
    for (int i = tid; i < COLS * W4_TILE; i += W4_THREADS) {
        const int m = i / W4_TILE, r = i % W4_TILE;
        const int n = static_cast<int>(blockIdx.x) * W4_TILE + r;
        if (m >= p.M || n >= p.N || static_cast<uint32_t>(m) % csize != crank) continue;
        const float* at = sums + m * SUM_PITCH + r;
        float v = 0.0f;
        if (csize == 1)
            v = *at;
        else
            for (uint32_t c = 0; c < csize; ++c) v += ld_shared_rank(at, c);
        store_y(p, m, n, v);
    }
    if (csize > 1) cluster_sync_all();  // nobody reads this CTA's sums any more
}

// ------------------------------------------------------------ many rows
//
// For many rows of X the product is bound by the tensor cores, which read fp16:
// the weights are written out once, scale * (q - zero) rounded to fp16 (nearest
// even), and the GEMM multiplies them.  The rounding is at most half a unit in
// the last place of each weight, the same as the output's.  A thread expands
// eight codes (4 bytes) to 16 bytes.
__global__ void __launch_bounds__(256)
    k_w4_expand(int64_t words, int words_per_row, int group_words, int groups,
                const uint32_t* packed, const __half* scales, const uint8_t* zeros, uint4* out)
{
    griddep_wait();
    griddep_launch_dependents();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < words;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t row = i / words_per_row;
        const int64_t at = row * groups + static_cast<int>(i - row * words_per_row) / group_words;
        const uint32_t w = packed[i];
        const float s = __half2float(scales[at]);
        const float z = zeros ? static_cast<float>(zeros[at]) : 8.0f;
        uint4 v;
        uint32_t* h = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __half2 q = __floats2half2_rn(s * (static_cast<float>((w >> (8 * j)) & 15u) - z),
                                                s * (static_cast<float>((w >> (8 * j + 4)) & 15u) - z));
            h[j] = *reinterpret_cast<const uint32_t*>(&q);
        }
        out[i] = v;
    }
}

// Clusters along z: the CTAs that share the rows' length.
cudaError_t launch_w4(void (*kernel)(W4Params), const W4Params& p, unsigned smem, dim3 grid,
                      cudaStream_t stream)
{
    cudaError_t e = ensure_smem_limit(kernel, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(W4_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = grid.z;
    cfg.attrs = attr;
    cfg.numAttrs = grid.z > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int GROUP>
cudaError_t launch_group(const W4Params& p, int cols, dim3 grid, cudaStream_t stream)
{
    switch (cols) {
    case 8:
        return launch_w4(k_w4_few<GROUP, W4_FEW_RT>, p, w4_few_smem<GROUP, W4_FEW_RT>(), grid,
                         stream);
    case 16: return launch_w4(k_w4_tile<16, GROUP>, p, w4_tile_smem<16, GROUP>(), grid, stream);
    case 32: return launch_w4(k_w4_tile<32, GROUP>, p, w4_tile_smem<32, GROUP>(), grid, stream);
    case 64: return launch_w4(k_w4_tile<64, GROUP>, p, w4_tile_smem<64, GROUP>(), grid, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

}  // namespace tg

using namespace tg;

struct gemm_w4_plan {
    int64_t M, N, K;
    int group, experts, share, dtype;
    int device, sms;
    int cols;        // rows of X per pass of the few-row kernel; 0: expand + GEMM
    int length_ctas; // CTAs that share a row's length
    void* d_weights; // N x K fp16
    gemm_plan* gemm;
    char desc[256];
};

namespace {
constexpr int W4_MAX_ROWS = 64;
}

extern "C" {

gemm_w4_plan* gemm_w4_create_plan(int64_t M, int64_t N, int64_t K, int group, int experts,
                                  int share, int dtype_out)
{
    gemm_w4_plan* plan = nullptr;
    guarded([&] {
        const int64_t LIM = (int64_t(1) << 31) - 1;
        if (M < 1 || N < 1 || K < 1 || M > LIM || N > LIM || K > LIM - 65536)
            return fail(GEMM_ERR_INVALID_ARG, "M, N, K must be in [1, 2^31-1]");
        if (group != 32 && group != 64 && group != 128)
            return fail(GEMM_ERR_INVALID_ARG, "group must be 32, 64 or 128");
        if (dtype_out != GEMM_OUT_F32 && dtype_out != GEMM_OUT_F16)
            return fail(GEMM_ERR_INVALID_ARG,
                        "dtype_out must be GEMM_OUT_F32 (0) or GEMM_OUT_F16 (1)");
        if (experts < 0 || share < 1 || (experts == 0 && share != 1))
            return fail(GEMM_ERR_INVALID_ARG,
                        "experts must be >= 0 and share >= 1 (1 without experts)");
        if (K % group != 0)
            return fail(GEMM_ERR_UNSUPPORTED, "K must be a multiple of group");
        const int elt = dtype_out == GEMM_OUT_F16 ? 2 : 4;
        if ((N * elt) % 16 != 0)
            return fail(GEMM_ERR_UNSUPPORTED,
                        "N * sizeof(output) must be a multiple of 16 bytes");
        if (experts > 0 && M > 1024)
            return fail(GEMM_ERR_UNSUPPORTED, "a plan with experts takes at most 1024 rows");
        gemm_w4_plan p = {};
        int r = require_device(&p.device, &p.sms, nullptr);
        if (r != GEMM_OK) return r;
        p.M = M;
        p.N = N;
        p.K = K;
        p.group = group;
        p.experts = experts;
        p.share = share;
        p.dtype = dtype_out;
        if (experts > 0 || M <= W4_MAX_ROWS) {
            p.cols = 8;
            while (experts == 0 && p.cols < M) p.cols *= 2;
            // CTAs of a cluster share a row's length where the rows alone leave
            // SMs idle: up to two CTAs per SM of the few-row kernel, each with
            // two blocks of 256 per warp at least; up to one of the tile kernel,
            // each with two blocks.
            const bool few = p.cols == W4_FEW;
            const int tile = few ? W4_ROWS * W4_FEW_RT : W4_TILE;
            const int64_t tiles =
                (N + tile - 1) / tile * (experts > 0 ? std::min<int64_t>(M, experts) : 1);
            const int64_t most = few ? 2 * p.sms : p.sms;
            const int64_t block = few ? W4_BLOCK * W4_WARPS : W4_BLOCK;
            p.length_ctas = 1;
            while (p.length_ctas < 8 && tiles * p.length_ctas * 2 <= most &&
                   K >= block * p.length_ctas * 4)
                p.length_ctas *= 2;
            std::snprintf(p.desc, sizeof(p.desc),
                          "w4 rows M=%lld N=%lld K=%lld group=%d experts=%d cols=%d "
                          "length_ctas=%d out=%s",
                          static_cast<long long>(M), static_cast<long long>(N),
                          static_cast<long long>(K), group, experts, p.cols, p.length_ctas,
                          elt == 2 ? "f16" : "f32");
        } else {
            p.gemm = gemm_create_plan(M, N, K, dtype_out);
            if (!p.gemm) return gemm_last_status();
            cudaError_t e = cudaMalloc(&p.d_weights, static_cast<size_t>(N) * K * 2);
            if (e != cudaSuccess) {
                gemm_destroy(p.gemm);
                return cuda_fail("allocating the expanded weights", e);
            }
            std::snprintf(p.desc, sizeof(p.desc), "w4 expand group=%d; %.180s", group,
                          gemm_plan_describe(p.gemm));
        }
        plan = new (std::nothrow) gemm_w4_plan(p);
        if (!plan) {
            if (p.gemm) gemm_destroy(p.gemm);
            if (p.d_weights) cudaFree(p.d_weights);
            return fail(GEMM_ERR_CUDA, "out of host memory");
        }
        return ok();
    });
    return plan;
}

int gemm_w4_run(gemm_w4_plan* plan, const void* X, const void* packed, const void* scales,
                const void* zeros, const int32_t* expert_ids, void* Y, void* cuda_stream)
{
    return guarded([&] {
        if (!plan) return fail(GEMM_ERR_INVALID_ARG, "plan is NULL");
        if (!X || !packed || !scales || !Y)
            return fail(GEMM_ERR_INVALID_ARG, "X, packed, scales and Y must be non-NULL");
        if ((plan->experts > 0) != (expert_ids != nullptr))
            return fail(GEMM_ERR_INVALID_ARG,
                        "expert_ids must be given exactly when the plan has experts");
        if (!aligned16(X) || !aligned16(packed) || !aligned16(Y) || !aligned16(scales))
            return fail(GEMM_ERR_UNSUPPORTED, "X, packed, scales and Y must be 16-byte aligned");
        int dev = -1;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return cuda_fail("cudaGetDevice", e);
        if (dev != plan->device)
            return fail(GEMM_ERR_INVALID_ARG, "plan was created on another device");
        cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
        if (plan->cols == 0) {
            const int64_t words = plan->N * (plan->K / 8);
            const int64_t blocks = std::min<int64_t>((words + 255) / 256, plan->sms * 32);
            e = launch_dependent(k_w4_expand, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, 1,
                                 stream, words, static_cast<int>(plan->K / 8), plan->group / 8,
                                 static_cast<int>(plan->K / plan->group),
                                 static_cast<const uint32_t*>(packed),
                                 static_cast<const __half*>(scales),
                                 static_cast<const uint8_t*>(zeros),
                                 static_cast<uint4*>(plan->d_weights));
            if (e != cudaSuccess) return cuda_fail("weight expansion launch", e);
            return gemm_run(plan->gemm, X, plan->d_weights, Y, cuda_stream);
        }
        W4Params p = {};
        p.M = static_cast<int>(plan->M);
        p.N = static_cast<int>(plan->N);
        p.K = static_cast<int>(plan->K);
        p.experts = plan->experts;
        p.share = plan->share;
        p.packed = static_cast<const uint8_t*>(packed);
        p.scales = static_cast<const __half*>(scales);
        p.zeros = static_cast<const uint8_t*>(zeros);
        p.X = static_cast<const __half*>(X);
        p.ids = expert_ids;
        p.Y = Y;
        p.f16out = plan->dtype == GEMM_OUT_F16;
        const int tile = plan->cols == W4_FEW ? W4_ROWS * W4_FEW_RT : W4_TILE;
        const dim3 grid(static_cast<unsigned>((plan->N + tile - 1) / tile),
                        plan->experts > 0 ? static_cast<unsigned>(plan->M) : 1u,
                        static_cast<unsigned>(plan->length_ctas));
        e = plan->group == 32   ? launch_group<32>(p, plan->cols, grid, stream)
            : plan->group == 64 ? launch_group<64>(p, plan->cols, grid, stream)
                                : launch_group<128>(p, plan->cols, grid, stream);
        return e == cudaSuccess ? ok() : cuda_fail("w4 product launch", e);
    });
}

int gemm_w4_get_device_status(gemm_w4_plan* plan)
{
    if (!plan) return fail(GEMM_ERR_INVALID_ARG, "plan is NULL");
    return plan->gemm ? gemm_get_device_status(plan->gemm) : ok();
}

void gemm_w4_destroy(gemm_w4_plan* plan)
{
    if (!plan) return;
    if (plan->gemm) gemm_destroy(plan->gemm);
    if (plan->d_weights) cudaFree(plan->d_weights);
    delete plan;
}

const char* gemm_w4_describe(const gemm_w4_plan* plan) { return plan ? plan->desc : "(null plan)"; }

}  // extern "C"
