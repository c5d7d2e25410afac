// norm.cu -- root-mean-square norm with the residual's addition and quantised rows, and
// its gradient.  Bound by memory: every value is read once and written once per output.
// Measured on 67 M values, residual, fp16 and mxfp8 rows: 88 to 101 us for widths from 128 to
// 16384, 6.0 to 6.8 TB/s; nvfp4 rows alone 47 to 71; gradient with the residual's: 85 to 92 us
// for widths from 128 to 8192, 5.8 to 6.3 TB/s, 100 to 106 to 16384, 129 at 32768.
// 16 rows of 4096: 2.5 us.
#include <algorithm>
#include <cmath>
#include <type_traits>
#include <utility>

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

// The sum of a row's vectors, whose sums are `v` (vector i * LANES + lane), in an order that does
// not depend on LANES and VEC, so that a row's result does not depend on how many others there
// are: every 1024th vector in turn, and those 1024 sums in a tree from the highest bit of their
// number down.
template <int LANES, int VEC>
__device__ __forceinline__ float row_sum(const float (&v)[VEC], float* shared)
{
    constexpr int MINE = 1024 / LANES;  // of the 1024 sums, this lane's
    constexpr int LIVE = VEC < MINE ? VEC : MINE;
    float s[LIVE];
#pragma unroll
    for (int i = 0; i < LIVE; ++i) s[i] = v[i];
#pragma unroll
    for (int i = LIVE; i < VEC; ++i) s[i % MINE] += v[i];
#pragma unroll
    for (int n = MINE / 2; n > 0; n /= 2)
#pragma unroll
        for (int i = 0; i < n; ++i)
            if (i + n < LIVE) s[i] += s[i + n];
    if constexpr (LANES <= 32) {
        return warp_sum<LANES>(s[0]);
    } else {
        shared[threadIdx.x] = s[0];
        __syncthreads();
        float t[LANES / 32];
#pragma unroll
        for (int i = 0; i < LANES / 32; ++i) t[i] = shared[i * 32 + lane_id()];
#pragma unroll
        for (int n = LANES / 64; n > 0; n /= 2)
#pragma unroll
            for (int i = 0; i < n; ++i) t[i] += t[i + n];
        return warp_sum(t[0]);
    }
}

constexpr int64_t MAX_WIDTH = 32768;

// Rows of mxfp4 are filled up to whole steps of 96 values, those of the largest widths by up to
// 64 past MAX_WIDTH: past the vectors of the lanes that hold such a row.  The row's first warp
// writes them in a turn of its own.
template <int FORMAT, int LANES, int VEC>
constexpr bool fills_up_past =
    FORMAT == MXFP4 && static_cast<int64_t>(LANES) * VEC * 8 == MAX_WIDTH;
static_assert((MAX_WIDTH + 95) / 96 * 96 <= MAX_WIDTH + 32 * 8, "one turn of a warp");

// A row by LANES lanes (half a warp, a warp, or all of the CTA), VEC vectors of eight values
// per lane, held in registers between the sum of squares and the outputs.
template <int FORMAT, int LANES, int VEC, int THREADS>
__global__ void __launch_bounds__(THREADS) k_rms_norm(const __grid_constant__ NormParams p)
{
    constexpr int ROWS = THREADS / LANES;  // per CTA
    __shared__ float shared[LANES];
    const int lane = static_cast<int>(threadIdx.x) % LANES;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / LANES;
    const bool valid = row < p.tokens;
    griddep_wait();
    griddep_launch_dependents();
    if (!__any_sync(0xffffffffu, valid)) return;  // a warp stays together for its shuffles
    uint4 x[VEC], r[VEC];  // all on their way before the first is used
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const int k = (i * LANES + lane) * 8;
        x[i] = r[i] = make_uint4(0, 0, 0, 0);
        if (valid && k < p.width) {
            x[i] = *reinterpret_cast<const uint4*>(p.X + row * p.width + k);
            if (p.residual) r[i] = *reinterpret_cast<const uint4*>(p.residual + row * p.width + k);
        }
    }
    float h[VEC][8];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        widen8(x[i], h[i]);
        if (p.residual) {
            float f[8];
            widen8(r[i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] += f[j];
        }
    }
    float squares[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        squares[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) squares[i] = fmaf(h[i][j], h[i][j], squares[i]);
    }
    const float sum = row_sum<LANES, VEC>(squares, shared);
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
    if constexpr (fills_up_past<FORMAT, LANES, VEC>) {
        if (lane < 32) {
            const float zeros[8] = {};
            quantize_store<FORMAT>(zeros, 1.0f, 1.0f / 6.0f, VEC * LANES + lane,
                                   p.codes + mx_code_offset(row, 0, p.chunks),
                                   p.scales + mx_scale_offset(row, 0, p.groups),
                                   static_cast<int>(p.chunks), static_cast<int>(p.groups), valid);
        }
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
        constexpr int LANES = decltype(lanes)::value, VEC = decltype(vec)::value;
        constexpr int THREADS = LANES <= 32 ? 256 : LANES;
        constexpr int HELD = LANES * VEC + (fills_up_past<FORMAT, LANES, VEC> ? 32 : 0);
        if (vecs > HELD) return cudaErrorInvalidValue;
        constexpr int ROWS = THREADS / LANES;
        const int64_t grid = (p.tokens + ROWS - 1) / ROWS;
        return launch_dependent(k_rms_norm<FORMAT, LANES, VEC, THREADS>,
                                dim3(static_cast<unsigned>(grid)), dim3(THREADS), 0, 1, stream, p);
    };
#define TG_NORM(lanes, vec) \
    go(std::integral_constant<int, lanes>{}, std::integral_constant<int, vec>{})
    // As long as the GPU (152 SMs) can hold a thread for every vector, a row is done soonest by
    // about as many lanes (16 x 4096, fp16 and mxfp8: 512 lanes 2.6 us, 128 lanes 3.3; 16 x 1024:
    // 128 lanes 2.05, 32 lanes 3.5).
    if (vecs <= 16) return TG_NORM(16, 1);
    if (p.tokens * vecs <= 152 * 2048) {
        if (vecs <= 32) return TG_NORM(32, 1);
        if (vecs <= 64) return TG_NORM(32, 2);
        if (vecs <= 128) return TG_NORM(128, 1);
        if (vecs <= 256) return TG_NORM(256, 1);
        if (vecs <= 512) return TG_NORM(512, 1);
        if (vecs <= 1024) return TG_NORM(512, 2);
    }
    // Beyond, few lanes with four to six vectors each: fewer reductions, and hardly a lane
    // without values, whose codes would cost as much as another's (67 M values to nvfp4 alone, 1528
    // wide: 32 lanes of six 51 us, 256 of one 87; 5120 wide: 128 of five 47, 256 of four 68).
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

// How rows are held: by `lanes` lanes with `vec` vectors of eight values each; CTAs of `threads`
// threads, `resident` of them on an SM, which the registers are held to.  Several CTAs cover each
// other's reductions better than one that reads a row ahead (16384 x 4096 with dH: four 87 us,
// three with a row ahead 96).
//
// staged: a row waits in shared memory instead of registers, every thread's vectors at places
// of its own, which the next row's take as soon as the last reading is over.  For rows whose
// registers would leave room for one CTA on an SM only (67 M values, 9472 wide: 104 us, in
// registers 146; 16384 wide 105, 111; 32768 wide 129, 170, with spills).  Shorter rows are faster
// in registers (4096 wide 87, staged 92; 8192 wide 92, 99).
struct GradConfig {
    int lanes, vec, threads, resident;
    bool staged;
};

// A row takes the first that holds it, however many rows there are, so dX does not depend on
// the other rows (a vector a lane would be faster for few: 77 x 4096 5.1 us, 5.6): two to four
// vectors a lane, hardly a lane without any, and a few groups of lanes in a CTA, which write one
// part of dweight (640 wide: 32 lanes of three 90 us, 128 of one 119; 1528 wide: 64 of three 90,
// 256 of one 110; 1000 rows of 1024: 64 lanes of two, four groups a CTA, 6.4 us, 128 of one and
// a CTA for each 8.0).
constexpr GradConfig GRAD[] = {
    {16, 1, 256, 6, false},  {32, 1, 256, 5, false},  {16, 3, 256, 3, false},
    {32, 2, 256, 4, false},  {32, 3, 256, 3, false},  {64, 2, 256, 4, false},
    {64, 3, 256, 3, false},  {128, 2, 256, 4, false}, {160, 2, 160, 6, false},
    {128, 3, 128, 6, false}, {256, 2, 256, 4, false}, {160, 4, 160, 4, false},
    {256, 3, 256, 3, false}, {512, 2, 512, 2, false}, {512, 3, 512, 2, true},
    {512, 4, 512, 2, true},  {1024, 4, 1024, 1, true},
};
constexpr int GRAD_CONFIGS = static_cast<int>(sizeof(GRAD) / sizeof(GRAD[0]));

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
template <int LANES, int VEC, int THREADS, int RESIDENT, bool STAGED>
__global__ void __launch_bounds__(THREADS, RESIDENT)
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
            const int mine = static_cast<int>(threadIdx.x) / LANES;  // groups differ in their rows
            float2* slots = shared[turn & 1] + mine * (LANES / 32);
            ++turn;
            if (lane_id() == 0) slots[lane / 32] = s;
            if constexpr (LANES < THREADS)
                named_bar_sync(1 + mine, LANES);
            else
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

// Which configuration, and how many CTAs: each has a part of dweight.
struct GradShape {
    int config, ctas;
};

// Independent of the device (GB300 has 152 SMs), so that the workspace is known without one.
constexpr int GRAD_SMS = 152;

GradShape grad_shape(int64_t tokens, int64_t width)
{
    const int64_t vecs = (width + 7) / 8;
    GradShape s = {0, 0};
    while (GRAD[s.config].lanes * GRAD[s.config].vec < vecs) ++s.config;
    const GradConfig& c = GRAD[s.config];
    const int64_t rows = c.threads / c.lanes;
    s.ctas = static_cast<int>(std::max<int64_t>(
        1, std::min<int64_t>((tokens + rows - 1) / rows, c.resident * GRAD_SMS)));
    return s;
}

template <int I>
cudaError_t launch_grad_config(const NormGradParams& p, int ctas, cudaStream_t stream)
{
    constexpr GradConfig c = GRAD[I];
    constexpr unsigned smem = c.staged ? c.vec * 3 * c.threads * 16 : 0;
    auto kernel = k_rms_norm_grad<c.lanes, c.vec, c.threads, c.resident, c.staged>;
    const cudaError_t e = c.staged ? ensure_smem_limit(kernel, smem) : cudaSuccess;
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(static_cast<unsigned>(ctas)), dim3(c.threads), smem, 1,
                            stream, p);
}

template <int... I>
cudaError_t launch_norm_grad(const NormGradParams& p, const GradShape& s, cudaStream_t stream,
                             std::integer_sequence<int, I...>)
{
    cudaError_t e = cudaErrorInvalidValue;
    ((s.config == I ? void(e = launch_grad_config<I>(p, s.ctas, stream)) : void()), ...);
    return e;
}

cudaError_t launch_norm_grad(const NormGradParams& p, const GradShape& s, cudaStream_t stream)
{
    return launch_norm_grad(p, s, stream, std::make_integer_sequence<int, GRAD_CONFIGS>{});
}

int check_norm(int64_t tokens, int64_t width, float eps)
{
    if (tokens < 0 || tokens > MAX_COORDINATE)
        return fail(GEMM_ERR_INVALID_ARG, "tokens must be in [0, 2^31-65536]");
    if (width < 8 || width > MAX_WIDTH || width % 8 != 0)
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
    int64_t bytes = -1;
    guarded([&] {
        const int r = check_norm(tokens, width, 0.0f);
        if (r != GEMM_OK) return r;
        bytes = static_cast<int64_t>(grad_shape(tokens, width).ctas) * width * 4;
        return ok();
    });
    return bytes;
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
