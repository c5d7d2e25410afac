// norm.cu -- root-mean-square norm with the residual's addition and quantised rows, and
// its gradient.  Bound by memory: every value is read once and written once per output.
// Measured on 67 M values, residual, fp16 and mxfp8 rows: 88 to 101 us for widths from 128 to
// 16384, 6.0 to 6.8 TB/s; nvfp4 rows alone 46 to 71; gradient with the residual's: 87 to 97 us for widths from 128 to 8192,
// 5.5 to 6.2 TB/s, 100 to 106 to 16384, 129 at 32768.  16 rows of 4096: 2.3 us.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "../../include/tmalayer.h"
#include "device_common.cuh"
#include "launch.h"
#include "microscale.cuh"
#include "runtime.h"

namespace tg {

namespace {

struct NormParams {
    int64_t tokens;
    int width;
    float eps, inv_width;
    const __half* X;
    const __half* residual;
    const __half* weight;
    __half* total;
    __half* Z;
    uint8_t* codes;
    uint8_t* scales;
    int64_t chunks, groups;
};

__device__ __forceinline__ void widen8(const uint4& v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ uint4 narrow8(const float (&x)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Sum over the LANES (16 or 32) lanes of a warp that share a row; rows of one warp may have
// left the loop they are in.
template <int LANES = 32>
__device__ __forceinline__ float warp_sum(float s)
{
    const uint32_t mask = LANES == 32 ? 0xffffffffu : 0xffffu << (lane_id() & 16u);
#pragma unroll
    for (int o = LANES / 2; o > 0; o /= 2) s += __shfl_xor_sync(mask, s, o);
    return s;
}

// Sum over the LANES lanes of a row: part of a warp, a warp, or the whole CTA.
template <int LANES>
__device__ __forceinline__ float row_sum(float s, float* shared)
{
    if constexpr (LANES <= 32) return warp_sum<LANES>(s);
    s = warp_sum(s);
    if (lane_id() == 0) shared[threadIdx.x / 32] = s;
    __syncthreads();
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < LANES / 32; ++i) s += shared[i];
    return s;
}

// A row by LANES lanes (half a warp, a warp, or all of the CTA), VEC vectors of eight values
// per lane, held in registers between the sum of squares and the outputs.
template <int FORMAT, int LANES, int VEC, int THREADS>
__global__ void __launch_bounds__(THREADS) k_rms_norm(const __grid_constant__ NormParams p)
{
    constexpr int ROWS = THREADS / LANES;  // per CTA
    __shared__ float shared[THREADS / 32];
    const int lane = static_cast<int>(threadIdx.x) % LANES;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / LANES;
    const bool valid = row < p.tokens;
    griddep_wait();
    griddep_launch_dependents();
    if (!__any_sync(0xffffffffu, valid)) return;  // a warp stays together for its shuffles
    float h[VEC][8];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const int k = (i * LANES + lane) * 8;
        uint4 x = make_uint4(0, 0, 0, 0), r = make_uint4(0, 0, 0, 0);
        if (valid && k < p.width) {
            x = *reinterpret_cast<const uint4*>(p.X + row * p.width + k);
            if (p.residual) r = *reinterpret_cast<const uint4*>(p.residual + row * p.width + k);
        }
        widen8(x, h[i]);
        if (p.residual) {
            float f[8];
            widen8(r, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] += f[j];
        }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(h[i][j], h[i][j], sum);
    sum = row_sum<LANES>(sum, shared);
    const float rstd = 1.0f / sqrtf(fmaf(sum, p.inv_width, p.eps));
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const int vec = i * LANES + lane;
        const int k = vec * 8;
        float z[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = 0.0f;
        if (valid && k < p.width) {
            if (p.total) *reinterpret_cast<uint4*>(p.total + row * p.width + k) = narrow8(h[i]);
            float w[8];
            widen8(__ldg(reinterpret_cast<const uint4*>(p.weight + k)), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] = h[i][j] * rstd * w[j];
            if (p.Z) *reinterpret_cast<uint4*>(p.Z + row * p.width + k) = narrow8(z);
        }
        if constexpr (FORMAT >= 0)
            quantize_store<FORMAT>(z, 1.0f, 1.0f / 6.0f, vec,
                                   p.codes + mx_code_offset(row, 0, p.chunks),
                                   p.scales + mx_scale_offset(row, 0, p.groups),
                                   static_cast<int>(p.chunks), static_cast<int>(p.groups), valid);
    }
}

template <int FORMAT>
cudaError_t launch_norm(const NormParams& p, cudaStream_t stream)
{
    // the row's vectors, up to the end of its codes and scales
    int64_t padded = p.width;
    if constexpr (FORMAT >= 0)
        padded = std::max<int64_t>(p.chunks * mx_chunk(FORMAT), p.groups * mx_group(FORMAT));
    const int64_t vecs = (padded + 7) / 8;
    auto go = [&](auto lanes, auto vec) {
        constexpr int LANES = decltype(lanes)::value;
        constexpr int THREADS = LANES <= 32 ? 256 : LANES;
        constexpr int ROWS = THREADS / LANES;
        const int64_t grid = (p.tokens + ROWS - 1) / ROWS;
        return launch_dependent(k_rms_norm<FORMAT, LANES, decltype(vec)::value, THREADS>,
                                dim3(static_cast<unsigned>(grid)), dim3(THREADS), 0, 1, stream, p);
    };
#define TG_NORM(lanes, vec) \
    go(std::integral_constant<int, lanes>{}, std::integral_constant<int, vec>{})
    // As long as the GPU (152 SMs) can hold a thread for every vector, a row is done soonest by
    // as many lanes (16 x 4096, fp16 and mxfp8: 512 lanes 2.6 us, 128 lanes 3.3; 16 x 1024: 128
    // lanes 2.05, 32 lanes 3.5).
    if (vecs <= 16) return TG_NORM(16, 1);
    if (p.tokens * vecs <= 152 * 2048) {
        if (vecs <= 32) return TG_NORM(32, 1);
        if (vecs <= 64) return TG_NORM(32, 2);
        if (vecs <= 128) return TG_NORM(128, 1);
        if (vecs <= 256) return TG_NORM(256, 1);
        if (vecs <= 512) return TG_NORM(512, 1);
        if (vecs <= 1024) return TG_NORM(1024, 1);
    }
    // Beyond, few lanes with four to six vectors each: fewer reductions, and hardly a lane
    // without values, whose codes would cost as much as another's (67 M values to nvfp4 alone, 1528
    // wide: 32 lanes of six 50 us, 256 of one 87; 5120 wide: 128 of five 46, 256 of four 68).
    if (vecs <= 32) return TG_NORM(16, 2);
    if (vecs <= 48) return TG_NORM(16, 3);
    if (vecs <= 64) return TG_NORM(16, 4);
    if (vecs <= 80) return TG_NORM(16, 5);
    if (vecs <= 96) return TG_NORM(32, 3);
    if (vecs <= 128) return TG_NORM(32, 4);
    if (vecs <= 160) return TG_NORM(32, 5);
    if (vecs <= 192) return TG_NORM(32, 6);
    if (vecs <= 256) return TG_NORM(64, 4);
    if (vecs <= 320) return TG_NORM(64, 5);
    if (vecs <= 384) return TG_NORM(64, 6);
    if (vecs <= 512) return TG_NORM(128, 4);
    if (vecs <= 640) return TG_NORM(128, 5);
    if (vecs <= 768) return TG_NORM(128, 6);
    if (vecs <= 1024) return TG_NORM(256, 4);
    if (vecs <= 1280) return TG_NORM(256, 5);
    if (vecs <= 1536) return TG_NORM(256, 6);
    if (vecs <= 2048) return TG_NORM(512, 4);
    if (vecs <= 2560) return TG_NORM(512, 5);
    return TG_NORM(1024, 4);
#undef TG_NORM
}

// ------------------------------------------------------------------ gradient

struct NormGradParams {
    int64_t tokens;
    int width;
    float eps, inv_width;
    const __half* dZ;
    const __half* H;
    const __half* weight;
    const __half* dH;
    __half* dX;
    float* parts;  // [part][width]
};


// CTAs on an SM, which the registers are held to.  Several of them cover each other's
// reductions better than one that reads a row ahead (16384 x 4096 with dH: four CTAs 87 us,
// three with a row ahead 96; 8192 x 8192: two 92, one 125).
constexpr int grad_resident(int lanes, int vec)
{
    return lanes <= 32   ? (vec == 1 ? 5 : 4)
           : lanes == 128 ? 10
           : lanes == 256 ? 6 - vec
           : lanes == 512 ? 2
                          : 1;
}

// 16 bytes to a thread's own place in shared memory, without a register on the way.
__device__ __forceinline__ void copy_ahead(uint4* to, const __half* from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(to))),
                 "l"(from)
                 : "memory");
}

// Rows as in k_rms_norm, each group of LANES lanes taking every stride-th row; a lane's
// columns stay the same, so their sums over its rows stay in registers and are written
// once as the group's part of dweight.
// STAGED: a row waits in shared memory instead of registers, every thread's vectors at places
// of its own, which the next row's take as soon as the last reading is over.  For rows whose
// registers would leave room for one CTA on an SM only (67 M values, 9472 wide: 104 us, in
// registers 146; 16384 wide 105, 111; 32768 wide 129, 170, with spills).  Shorter rows are faster
// in registers (4096 wide 87, staged 92; 8192 wide 92, 99).
template <int LANES, int VEC, int THREADS, bool STAGED = false>
__global__ void __launch_bounds__(THREADS, grad_resident(LANES, VEC))
    k_rms_norm_grad(const __grid_constant__ NormGradParams p)
{
    extern __shared__ uint4 staged[];  // STAGED: [VEC][h, dz, dh][THREADS]
    constexpr int ROWS = THREADS / LANES;
    __shared__ float2 shared[2][THREADS / 32];
    const int lane = static_cast<int>(threadIdx.x) % LANES;
    const int64_t group = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / LANES;
    const int64_t groups = static_cast<int64_t>(gridDim.x) * ROWS;
    griddep_wait();
    griddep_launch_dependents();
    float dw[VEC][8];
#pragma unroll
    for (int i = 0; i < VEC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
    const auto stage = [&](int i) { return staged + i * 3 * THREADS + threadIdx.x; };
    const auto fetch = [&](int64_t row, int i) {
        const int k = (i * LANES + lane) * 8;
        if (row >= p.tokens || k >= p.width) return;
        copy_ahead(stage(i), p.H + row * p.width + k);
        copy_ahead(stage(i) + THREADS, p.dZ + row * p.width + k);
        if (p.dH) copy_ahead(stage(i) + 2 * THREADS, p.dH + row * p.width + k);
    };
    if constexpr (STAGED)
#pragma unroll
        for (int i = 0; i < VEC; ++i) fetch(group, i);
    int turn = 0;
    for (int64_t row = group; row < p.tokens; row += groups) {
        constexpr int HELD = STAGED ? 1 : VEC;
        uint4 hv[HELD], dv[HELD], rv[HELD];
        if constexpr (STAGED) {
            asm volatile("cp.async.wait_all;" ::: "memory");  // a thread reads its own copies
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const int k = (i * LANES + lane) * 8;
                hv[i] = dv[i] = rv[i] = make_uint4(0, 0, 0, 0);
                if (k < p.width) {
                    hv[i] = *reinterpret_cast<const uint4*>(p.H + row * p.width + k);
                    dv[i] = *reinterpret_cast<const uint4*>(p.dZ + row * p.width + k);
                    if (p.dH) rv[i] = *reinterpret_cast<const uint4*>(p.dH + row * p.width + k);
                }
            }
        }
        float2 s = make_float2(0.0f, 0.0f);  // sum of h^2, of u h
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int k = (i * LANES + lane) * 8;
            if (k >= p.width) continue;
            float h[8], d[8], w[8];
            widen8(STAGED ? stage(i)[0] : hv[i % HELD], h);
            widen8(STAGED ? stage(i)[THREADS] : dv[i % HELD], d);
            widen8(__ldg(reinterpret_cast<const uint4*>(p.weight + k)), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s.x = fmaf(h[j], h[j], s.x);
                s.y = fmaf(d[j] * w[j], h[j], s.y);
            }
        }
        s.x = warp_sum<LANES < 32 ? LANES : 32>(s.x);
        s.y = warp_sum<LANES < 32 ? LANES : 32>(s.y);
        if constexpr (LANES > 32) {
            float2* slots = shared[turn & 1];
            ++turn;
            if (lane_id() == 0) slots[threadIdx.x / 32] = s;
            __syncthreads();
            s = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < LANES / 32; ++i) {
                s.x += slots[i].x;
                s.y += slots[i].y;
            }
        }
        const float rstd = 1.0f / sqrtf(fmaf(s.x, p.inv_width, p.eps));
        const float along = s.y * p.inv_width * rstd * rstd;  // mean(u n) * rstd
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int k = (i * LANES + lane) * 8;
            if (k >= p.width) continue;
            float h[8], d[8], w[8], x[8];
            widen8(STAGED ? stage(i)[0] : hv[i % HELD], h);
            widen8(STAGED ? stage(i)[THREADS] : dv[i % HELD], d);
            widen8(__ldg(reinterpret_cast<const uint4*>(p.weight + k)), w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dw[i][j] = fmaf(d[j], h[j] * rstd, dw[i][j]);
                x[j] = rstd * fmaf(-h[j], along, d[j] * w[j]);
            }
            if (p.dH) {
                float r[8];
                widen8(STAGED ? stage(i)[2 * THREADS] : rv[i % HELD], r);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] += r[j];
            }
            if constexpr (STAGED) fetch(row + groups, i);
            *reinterpret_cast<uint4*>(p.dX + row * p.width + k) = narrow8(x);
        }
    }
    // One part per CTA: the groups of a CTA add theirs up first (as parts of their own they kept
    // the second launch reading, 27608 x 312: 23 us).
    if constexpr (ROWS > 1) {
        __shared__ float sums[ROWS][LANES * VEC * 8];
        const int mine = static_cast<int>(threadIdx.x) / LANES;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            float4* to = reinterpret_cast<float4*>(&sums[mine][(i * LANES + lane) * 8]);
            to[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
            to[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        }
        __syncthreads();
        float* part = p.parts + static_cast<int64_t>(blockIdx.x) * p.width;
        for (int k = static_cast<int>(threadIdx.x); k < p.width; k += THREADS) {
            float sum = sums[0][k];
#pragma unroll
            for (int r = 1; r < ROWS; ++r) sum += sums[r][k];
            part[k] = sum;
        }
    } else {
        float* part = p.parts + group * p.width;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int k = (i * LANES + lane) * 8;
            if (k >= p.width) continue;
            reinterpret_cast<float4*>(part + k)[0] =
                make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
            reinterpret_cast<float4*>(part + k)[1] =
                make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        }
    }
}

// dweight = sum of the parts: a CTA takes 32 columns, its warps every 32nd part.
__global__ void __launch_bounds__(1024) k_rms_norm_weight(const float* parts, int64_t count,
                                                          int width, float* dweight)
{
    __shared__ float shared[32][33];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = static_cast<int>(lane_id()), warp = static_cast<int>(threadIdx.x) / 32;
    const int k = static_cast<int>(blockIdx.x) * 32 + lane;
    float s = 0.0f;
    if (k < width) {
#pragma unroll 8
        for (int64_t i = warp; i < count; i += 32) s += parts[i * width + k];
    }
    shared[warp][lane] = s;
    __syncthreads();
    const int column = static_cast<int>(blockIdx.x) * 32 + warp;
    s = warp_sum(shared[lane][warp]);
    if (lane == 0 && column < width) dweight[column] = s;
}

// How many parts dweight has: rows per CTA and CTAs, by the width.
struct GradShape {
    int config;
    int rows;  // per CTA
    int ctas;
};

// Independent of the device (GB300 has 152 SMs), so that the workspace is known without one.
constexpr int GRAD_SMS = 152;

GradShape grad_shape(int64_t tokens, int64_t width)
{
    const int64_t vecs = (width + 7) / 8;
    GradShape s;
    int resident;
    if (vecs <= 16) s = {0, 16, 0}, resident = grad_resident(16, 1);
    else if (vecs <= 32) s = {1, 8, 0}, resident = grad_resident(32, 1);
    else if (vecs <= 64) s = {2, 8, 0}, resident = grad_resident(32, 2);
    else if (vecs <= 128) s = {3, 1, 0}, resident = grad_resident(128, 1);
    else if (vecs <= 256) s = {4, 1, 0}, resident = grad_resident(256, 1);
    else if (vecs <= 512) s = {5, 1, 0}, resident = grad_resident(256, 2);
    else if (vecs <= 768) s = {6, 1, 0}, resident = grad_resident(256, 3);
    else if (vecs <= 1024) s = {7, 1, 0}, resident = grad_resident(512, 2);
    else if (vecs <= 1536) s = {8, 1, 0}, resident = grad_resident(512, 3);
    else if (vecs <= 2048) s = {9, 1, 0}, resident = grad_resident(512, 4);
    else s = {10, 1, 0}, resident = grad_resident(1024, 4);
    const int64_t want = (tokens + s.rows - 1) / s.rows;
    s.ctas = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, resident * GRAD_SMS)));
    return s;
}

cudaError_t launch_norm_grad(const NormGradParams& p, const GradShape& s, cudaStream_t stream)
{
    auto go = [&](auto kernel, int threads, unsigned smem = 0) {
        const cudaError_t e = smem ? ensure_smem_limit(kernel, smem) : cudaSuccess;
        if (e != cudaSuccess) return e;
        return launch_dependent(kernel, dim3(static_cast<unsigned>(s.ctas)),
                                dim3(static_cast<unsigned>(threads)), smem, 1, stream, p);
    };
    switch (s.config) {
    case 0: return go(k_rms_norm_grad<16, 1, 256>, 256);
    case 1: return go(k_rms_norm_grad<32, 1, 256>, 256);
    case 2: return go(k_rms_norm_grad<32, 2, 256>, 256);
    case 3: return go(k_rms_norm_grad<128, 1, 128>, 128);
    case 4: return go(k_rms_norm_grad<256, 1, 256>, 256);
    case 5: return go(k_rms_norm_grad<256, 2, 256>, 256);
    case 6: return go(k_rms_norm_grad<256, 3, 256>, 256);
    case 7: return go(k_rms_norm_grad<512, 2, 512>, 512);
    case 8: return go(k_rms_norm_grad<512, 3, 512, true>, 512, 3 * 3 * 512 * 16);
    case 9: return go(k_rms_norm_grad<512, 4, 512, true>, 512, 4 * 3 * 512 * 16);
    default: return go(k_rms_norm_grad<1024, 4, 1024, true>, 1024, 4 * 3 * 1024 * 16);
    }
}

int check_norm(int64_t tokens, int64_t width, float eps)
{
    if (tokens < 0 || tokens > MAX_COORDINATE)
        return fail(GEMM_ERR_INVALID_ARG, "tokens must be in [0, 2^31-65536]");
    if (width < 8 || width > 32768 || width % 8 != 0)
        return fail(GEMM_ERR_UNSUPPORTED, "width must be a multiple of 8 from 8 to 32768");
    if (!(eps >= 0.0f)) return fail(GEMM_ERR_INVALID_ARG, "eps must be >= 0");
    return GEMM_OK;
}

}  // namespace

}  // namespace tg

using namespace tg;

extern "C" {

int gemm_rms_norm(int64_t tokens, int64_t width, const void* X, const void* residual,
                  const void* weight, float eps, void* total, void* Z, int format, void* codes,
                  void* scales, void* cuda_stream)
{
    return guarded([&] {
        int r = check_norm(tokens, width, eps);
        if (r != GEMM_OK) return r;
        if ((codes != nullptr) != (scales != nullptr))
            return fail(GEMM_ERR_INVALID_ARG, "codes and scales must be given together");
        if (codes && (format < MXFP8 || format > NVFP4))
            return fail(GEMM_ERR_INVALID_ARG, "unknown gemm_mx_format");
        if (!weight || (tokens > 0 && !X))
            return fail(GEMM_ERR_INVALID_ARG, "X and weight must be non-NULL");
        if (tokens > 0 && !total && !Z && !codes)
            return fail(GEMM_ERR_INVALID_ARG, "no output is asked for");
        if (total && total == Z) return fail(GEMM_ERR_INVALID_ARG, "total and Z must differ");
        if (!aligned16(X) || !aligned16(residual) || !aligned16(weight) || !aligned16(total) ||
            !aligned16(Z) || !aligned16(codes) || !aligned16(scales))
            return fail(GEMM_ERR_UNSUPPORTED, "all tensors must be 16-byte aligned");
        int dev;
        r = require_device(&dev, nullptr, nullptr);
        if (r != GEMM_OK) return r;
        if (tokens == 0) return ok();
        NormParams p = {};
        p.tokens = tokens;
        p.width = static_cast<int>(width);
        p.eps = eps;
        p.inv_width = static_cast<float>(1.0 / static_cast<double>(width));
        p.X = static_cast<const __half*>(X);
        p.residual = static_cast<const __half*>(residual);
        p.weight = static_cast<const __half*>(weight);
        p.total = static_cast<__half*>(total);
        p.Z = static_cast<__half*>(Z);
        p.codes = static_cast<uint8_t*>(codes);
        p.scales = static_cast<uint8_t*>(scales);
        cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
        cudaError_t e;
        if (codes) {
            p.chunks = mx_chunks(width, format);
            p.groups = mx_groups(width, format);
            e = format == MXFP8   ? launch_norm<MXFP8>(p, stream)
                : format == MXFP4 ? launch_norm<MXFP4>(p, stream)
                                  : launch_norm<NVFP4>(p, stream);
        } else {
            e = launch_norm<-1>(p, stream);
        }
        return e == cudaSuccess ? ok() : cuda_fail("norm launch", e);
    });
}

int64_t gemm_rms_norm_grad_workspace(int64_t tokens, int64_t width)
{
    if (check_norm(tokens, width, 0.0f) != GEMM_OK) return -1;
    ok();
    const GradShape s = grad_shape(tokens, width);
    return static_cast<int64_t>(s.ctas) * width * 4;
}

int gemm_rms_norm_grad(int64_t tokens, int64_t width, const void* dZ, const void* H,
                       const void* weight, const void* dH, float eps, void* dX, float* dweight,
                       void* workspace, void* cuda_stream)
{
    return guarded([&] {
        int r = check_norm(tokens, width, eps);
        if (r != GEMM_OK) return r;
        if (!weight || !dweight || !workspace || (tokens > 0 && (!dZ || !H || !dX)))
            return fail(GEMM_ERR_INVALID_ARG,
                        "dZ, H, weight, dX, dweight and workspace must be non-NULL");
        if (!aligned16(dZ) || !aligned16(H) || !aligned16(weight) || !aligned16(dH) ||
            !aligned16(dX) || !aligned16(dweight) || !aligned16(workspace))
            return fail(GEMM_ERR_UNSUPPORTED, "all tensors must be 16-byte aligned");
        int dev;
        r = require_device(&dev, nullptr, nullptr);
        if (r != GEMM_OK) return r;
        NormGradParams p = {};
        p.tokens = tokens;
        p.width = static_cast<int>(width);
        p.eps = eps;
        p.inv_width = static_cast<float>(1.0 / static_cast<double>(width));
        p.dZ = static_cast<const __half*>(dZ);
        p.H = static_cast<const __half*>(H);
        p.weight = static_cast<const __half*>(weight);
        p.dH = static_cast<const __half*>(dH);
        p.dX = static_cast<__half*>(dX);
        p.parts = static_cast<float*>(workspace);
        cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
        const GradShape s = grad_shape(tokens, width);
        cudaError_t e = launch_norm_grad(p, s, stream);
        if (e == cudaSuccess)
            e = launch_dependent(k_rms_norm_weight, dim3(static_cast<unsigned>((width + 31) / 32)),
                                 dim3(1024), 0, 1, stream, static_cast<const float*>(p.parts),
                                 static_cast<int64_t>(s.ctas), p.width, dweight);
        return e == cudaSuccess ? ok() : cuda_fail("norm gradient launch", e);
    });
}

}  // extern "C"
