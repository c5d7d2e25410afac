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
// Bound by reading the codes once.  A CTA owns 16 rows of the weights and its
// eight warps take every eighth block of 256 weights of those rows, so that
// neighbouring warps read neighbouring 128-byte pieces of a row.  Each warp
// keeps a ring of W4_STAGES blocks (16 rows x 128 bytes, swizzled by 16-byte
// chunk) in flight with 16-byte asynchronous copies of its own; no barrier
// joins the warps before the final sum.
//
// The product runs on mma.sync m16n8k16 with the weights as the 16-row operand
// and up to eight rows of X as the 8-column one: a single row of X needs one
// multiply-add per weight whatever the unit, and on the tensor cores that
// leaves the conversion of the codes as the only arithmetic.  (tcgen05.mma
// would need the converted weights written back to shared memory.)
//
// A 32-bit word holds the codes k..k+7.  Masking the word and its shift by 8
// with 0x000f000f and 0x00f000f0 and setting the exponent of 1024 gives
// half pairs (k, k+4), (k+1, k+5), (k+2, k+6), (k+3, k+7) of 1024 + q or
// 1024 + 16 q; one half2 add or fused multiply-add makes them q - zero, exact
// in fp16.  The pairs of X are permuted alike.  Each group is summed in fp32 by
// the tensor core and enters the row's sum times its scale, so no weight is
// rounded.
constexpr int W4_WARPS = 8;
constexpr int W4_ROWS = 16;
constexpr int W4_BLOCK = 256;  // weights of a row per stage: 128 bytes
constexpr int W4_STAGES = 4;
constexpr int W4_STAGE_BYTES = W4_ROWS * W4_BLOCK / 2;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid)
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

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void mma_m16n8k16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// q - zero of the eight codes of `w` as four half pairs (k, k + 4), (k + 1,
// k + 5), (k + 2, k + 6), (k + 3, k + 7).  zlow = -(1024 + zero), zhigh =
// -(64 + zero), twice each.
__device__ __forceinline__ void decode8(uint32_t w, __half2 zlow, __half2 zhigh, uint32_t (&e)[4])
{
    const __half2 sixteenth = __half2half2(__float2half_rn(0.0625f));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t lo = (w & 0x000f000fu) | 0x64006400u;
        uint32_t hi = (w & 0x00f000f0u) | 0x64006400u;
        const __half2 a = __hadd2(*reinterpret_cast<__half2*>(&lo), zlow);
        const __half2 b = __hfma2(*reinterpret_cast<__half2*>(&hi), sixteenth, zhigh);
        e[2 * h] = *reinterpret_cast<const uint32_t*>(&a);
        e[2 * h + 1] = *reinterpret_cast<const uint32_t*>(&b);
        w >>= 8;
    }
}

// A scale and a zero point as one word: the scale's fp16 bits below, the zero
// point (0..255) above.
__device__ __forceinline__ uint32_t load_scale(const W4Params& p, int64_t index)
{
    const uint32_t s = __half_as_ushort(p.scales[index]);
    const uint32_t z = p.zeros ? p.zeros[index] : 8u;
    return s | (z << 16);
}

template <int NT, int GROUP>
__global__ void __launch_bounds__(W4_WARPS * 32)
    k_w4_rows(const __grid_constant__ W4Params p)
{
    constexpr int COLS = NT * 8;                 // rows of X per pass
    constexpr int GPS = W4_BLOCK / GROUP;        // groups per stage and row
    constexpr int EPL = W4_ROWS * GPS / 32;      // scales a lane loads per stage
    constexpr int WARP_BYTES = W4_STAGES * W4_STAGE_BYTES;
    constexpr int SCALE_WORDS = W4_ROWS * GPS;
    extern __shared__ __align__(128) uint8_t w4_smem[];
    __shared__ int list[COLS];
    __shared__ int list_count;
    const int tid = static_cast<int>(threadIdx.x);
    const int warp = tid >> 5;
    const uint32_t lane = lane_id();
    const int g = static_cast<int>(lane >> 2), t = static_cast<int>(lane & 3u);
    const uint32_t ring = smem_u32(w4_smem) + warp * WARP_BYTES;
    uint32_t* scale_buf = reinterpret_cast<uint32_t*>(w4_smem + W4_WARPS * WARP_BYTES) +
                          warp * 2 * SCALE_WORDS;
    float* partial = reinterpret_cast<float*>(w4_smem);  // [warps][COLS][16] after the loop
    float* sums = reinterpret_cast<float*>(w4_smem + W4_WARPS * WARP_BYTES);  // [COLS][16]
    const uint32_t csize = gridDim.z, crank = blockIdx.z;  // CTAs that share the rows' length
    const int n0 = static_cast<int>(blockIdx.x) * W4_ROWS;
    griddep_wait();
    griddep_launch_dependents();

    int expert = 0;
    if (p.experts > 0) {
        expert = p.ids[blockIdx.y];
        if (expert < 0 || expert >= p.experts) {
            // a dropped row
            if (crank == 0 && tid < W4_ROWS && n0 + tid < p.N) {
                const int64_t at = static_cast<int64_t>(blockIdx.y) * p.N + n0 + tid;
                if (p.f16out)
                    static_cast<__half*>(p.Y)[at] = __float2half_rn(0.0f);
                else
                    static_cast<float*>(p.Y)[at] = 0.0f;
            }
            return;
        }
        // the first row of an expert does all of the expert's rows
        bool earlier = false;
        for (int r = tid; r < static_cast<int>(blockIdx.y); r += W4_WARPS * 32)
            earlier |= p.ids[r] == expert;
        if (__syncthreads_or(earlier)) return;
    }
    const uint8_t* packed = p.packed + static_cast<int64_t>(expert) * p.N * (p.K / 2);
    const int64_t groups = p.K / GROUP;
    const int64_t scale0 = static_cast<int64_t>(expert) * p.N * groups;
    const int blocks = (p.K + W4_BLOCK - 1) / W4_BLOCK;
    const int step = W4_WARPS * static_cast<int>(csize);
    const int kb0 = static_cast<int>(crank) * W4_WARPS + warp;

    int next_row = p.experts > 0 ? static_cast<int>(blockIdx.y) : 0;
    while (next_row < p.M) {
        // the rows of Y of this pass
        if (p.experts > 0) {
            if (warp == 0) {
                int found = 0, r = next_row;
                for (; r < p.M && found < COLS; r += 32) {
                    const int i = r + static_cast<int>(lane);
                    unsigned hit = __ballot_sync(0xffffffffu, i < p.M && p.ids[i] == expert);
                    const int slot = found + __popc(hit & ((1u << lane) - 1u));
                    if (((hit >> lane) & 1u) && slot < COLS) list[slot] = i;
                    found += __popc(hit);
                }
                if (lane == 0) list_count = found < COLS ? found : COLS;
            }
            __syncthreads();
        }
        const int count = p.experts > 0 ? list_count
                                        : (p.M - next_row < COLS ? p.M - next_row : COLS);
        if (count == 0) break;
        const __half* x[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int c = nt * 8 + g;
            x[nt] = nullptr;
            if (c < count) {
                const int row = p.experts > 0 ? list[c] : next_row + c;
                x[nt] = p.X + static_cast<int64_t>(row / p.share) * p.K;
            }
        }

        auto load_block = [&](int kb, int stage) {
            if (kb < blocks) {
#pragma unroll
                for (int i = 0; i < W4_STAGE_BYTES / 512; ++i) {
                    const int id = static_cast<int>(lane) + 32 * i;
                    const int row = id >> 3, c = id & 7;
                    const int byte = kb * (W4_BLOCK / 2) + c * 16;
                    const bool ok = n0 + row < p.N && byte < p.K / 2;
                    const uint8_t* src =
                        ok ? packed + static_cast<int64_t>(n0 + row) * (p.K / 2) + byte : packed;
                    cp_async16(ring + stage * W4_STAGE_BYTES + row * 128 + ((c ^ (row & 7)) << 4),
                               src, ok);
                }
            }
            cp_async_commit();
        };
        uint32_t ahead[EPL];
        auto load_scales = [&](int kb) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const int id = static_cast<int>(lane) + 32 * i;
                const int row = id / GPS, gi = kb * GPS + id % GPS;
                ahead[i] = 0;
                if (kb < blocks && n0 + row < p.N && gi < groups)
                    ahead[i] = load_scale(p, scale0 + (n0 + row) * groups + gi);
            }
        };
        float acc[NT][4], part[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[nt][i] = 0.0f;

#pragma unroll
        for (int s = 0; s < W4_STAGES - 1; ++s) load_block(kb0 + s * step, s);
        load_scales(kb0);
        int stage = 0, parity = 0;
        for (int kb = kb0; kb < blocks; kb += step) {
            load_block(kb + (W4_STAGES - 1) * step,
                       stage == 0 ? W4_STAGES - 1 : stage - 1);
            uint32_t* sc = scale_buf + parity * SCALE_WORDS;
#pragma unroll
            for (int i = 0; i < EPL; ++i) sc[lane + 32 * i] = ahead[i];
            load_scales(kb + step);
            cp_async_wait<W4_STAGES - 1>();
            __syncwarp();
            const uint32_t a = ring + stage * W4_STAGE_BYTES + g * 128 + t * 4;
            __half2 zlow[2], zhigh[2];
            float s[2];
#pragma unroll
            for (int j = 0; j < W4_BLOCK / 32; ++j) {
                const int k = kb * W4_BLOCK + j * 32;
                if (k >= p.K) break;
                if (j % (GROUP / 32) == 0) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t w = sc[(g + 8 * h) * GPS + j / (GROUP / 32)];
                        s[h] = __half2float(__ushort_as_half(static_cast<unsigned short>(w)));
                        const float z = static_cast<float>(w >> 16);
                        zlow[h] = __half2half2(__float2half_rn(-1024.0f - z));
                        zhigh[h] = __half2half2(__float2half_rn(-64.0f - z));
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) part[nt][i] = 0.0f;
                }
                uint32_t e[4], f[4];
                const uint32_t chunk = static_cast<uint32_t>(j ^ g) << 4;
                decode8(ld_shared_u32(a + chunk), zlow[0], zhigh[0], e);
                decode8(ld_shared_u32(a + 8 * 128 + chunk), zlow[1], zhigh[1], f);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (x[nt]) v = *reinterpret_cast<const uint4*>(x[nt] + k + 8 * t);
                    mma_m16n8k16(part[nt], e[0], f[0], e[2], f[2],
                                 __byte_perm(v.x, v.z, 0x5410), __byte_perm(v.y, v.w, 0x5410));
                    mma_m16n8k16(part[nt], e[1], f[1], e[3], f[3],
                                 __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x7632));
                }
                if (j % (GROUP / 32) == GROUP / 32 - 1) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[nt][i] = fmaf(s[i / 2], part[nt][i], acc[nt][i]);
                }
            }
            __syncwarp();
            if (++stage == W4_STAGES) stage = 0;
            parity ^= 1;
        }
        cp_async_wait<0>();
        __syncthreads();

        // sum over the warps, then over the CTAs that share the length, in order
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                partial[(warp * COLS + nt * 8 + 2 * t + (i & 1)) * W4_ROWS + g + 8 * (i >> 1)] =
                    acc[nt][i];
        __syncthreads();
        for (int i = tid; i < COLS * W4_ROWS; i += W4_WARPS * 32) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < W4_WARPS; ++w) v += partial[w * COLS * W4_ROWS + i];
            sums[i] = v;
        }
        if (csize > 1)
            cluster_sync_all();
        else
            __syncthreads();
        if (crank == 0) {
            for (int i = tid; i < COLS * W4_ROWS; i += W4_WARPS * 32) {
                const int c = i / W4_ROWS, n = n0 + i % W4_ROWS;
                if (c >= count || n >= p.N) continue;
                float v = sums[i];
                for (uint32_t r = 1; r < csize; ++r) {
                    float other;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                 : "=f"(other)
                                 : "r"(map_shared_rank(smem_u32(sums + i), r))
                                 : "memory");
                    v += other;
                }
                const int row = p.experts > 0 ? list[c] : next_row + c;
                const int64_t at = static_cast<int64_t>(row) * p.N + n;
                if (p.f16out)
                    static_cast<__half*>(p.Y)[at] = __float2half_rn(v);
                else
                    static_cast<float*>(p.Y)[at] = v;
            }
        }
        const int last = p.experts > 0 ? list[count - 1] : next_row + count - 1;
        if (csize > 1)
            cluster_sync_all();
        else
            __syncthreads();
        if (count < COLS) break;
        next_row = last + 1;
    }
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

template <int NT>
cudaError_t launch_rows(const W4Params& p, int group, dim3 grid, cudaStream_t stream)
{
    auto kernel = group == 32   ? k_w4_rows<NT, 32>
                  : group == 64 ? k_w4_rows<NT, 64>
                                : k_w4_rows<NT, 128>;
    const int scale_bytes = W4_WARPS * 2 * W4_ROWS * (W4_BLOCK / group) * 4;
    const int tail = std::max(scale_bytes, NT * 8 * W4_ROWS * 4);
    const unsigned smem = static_cast<unsigned>(W4_WARPS * W4_STAGES * W4_STAGE_BYTES + tail);
    cudaError_t e = ensure_smem_limit(kernel, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(W4_WARPS * 32);
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
            // CTAs of a cluster split a row's length where the rows alone leave
            // SMs idle, each with at least one block of 256 per warp.
            const int64_t tiles = (N + W4_ROWS - 1) / W4_ROWS * (experts > 0 ? std::min<int64_t>(M, experts) : 1);
            p.length_ctas = 1;
            while (p.length_ctas < 8 && tiles * p.length_ctas < 2 * p.sms &&
                   K >= static_cast<int64_t>(W4_BLOCK) * W4_WARPS * p.length_ctas * 2)
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
        const dim3 grid(static_cast<unsigned>((plan->N + W4_ROWS - 1) / W4_ROWS),
                        plan->experts > 0 ? static_cast<unsigned>(plan->M) : 1u,
                        static_cast<unsigned>(plan->length_ctas));
        e = plan->cols == 8    ? launch_rows<1>(p, plan->group, grid, stream)
            : plan->cols == 16 ? launch_rows<2>(p, plan->group, grid, stream)
            : plan->cols == 32 ? launch_rows<4>(p, plan->group, grid, stream)
                               : launch_rows<8>(p, plan->group, grid, stream);
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
