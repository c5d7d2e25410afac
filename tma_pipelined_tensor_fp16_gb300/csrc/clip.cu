// clip.cu -- the global norm of many gradient tensors, and clipping to it.  Two launches:
// sums of squares, one per CTA, and then the scaled values, for which every CTA adds the
// sums up for itself in the same order.  Bound by memory: the gradients are read twice
// (the second time from the end, where the L2 still holds the last of them) and
// written once.  Measured: 1.07 GB of fp32 480 us, 6.7 TB/s over the three; the norm alone 152.
#include <algorithm>
#include <cmath>
#include <memory>
#include <new>
#include <vector>

#include "../../include/tmalayer.h"
#include "device_common.cuh"
#include "launch.h"
#include "runtime.h"

using namespace tg;

namespace {

constexpr int64_t CHUNK = 16384;  // values of a tensor that a CTA takes at a time
constexpr int CLIP_THREADS = 512;
constexpr int MAX_PARTS = GEMM_CLIP_WORKSPACE_BYTES / 8;

// A piece of a tensor.
struct Chunk {
    const void* src;
    void* dst;
    int count;
    int f16;
    int64_t pad;
};
static_assert(sizeof(Chunk) == 32, "two 16-byte loads");

}  // namespace

struct gemm_clip_plan {
    Chunk* d_chunks;
    int64_t chunks;
    int device, grid;
};

namespace {

__device__ __forceinline__ Chunk load_chunk(const Chunk* table, int64_t i)
{
    const int4* from = reinterpret_cast<const int4*>(table + i);
    int4 v[2] = {__ldg(from), __ldg(from + 1)};
    return *reinterpret_cast<Chunk*>(v);
}

// Squares are added up in fp32 over the 32 values that a thread takes of a chunk (in
// vectors of four or eight and those in a tree: each sum is off by at most 9 * 2^-24), and
// in fp64 from there: one fp64 addition for 32 values, as GB300 does few of them (with one
// for every four values 1.07 GB took 1.1 ms).  Sums that fp32 does not hold whole are
// formed again in fp64: those that overflow, and those below 2^-100, where squares may
// have vanished.
__device__ __forceinline__ bool holds(float s) { return s >= 0x1p-100f && s <= 0x1p126f; }

template <int N>
__device__ __forceinline__ float squares(const float (&x)[N])
{
    float s = x[0] * x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) s = fmaf(x[i], x[i], s);
    return s;
}

template <int N>
__device__ __noinline__ double squares_in_64(const float* x)
{
    float most = 0.0f;
    for (int i = 0; i < N; ++i) most = fmaxf(most, fabsf(x[i]));
    double d = 0.0;
    for (int i = 0; i < N; ++i) {
        if (most == 0.0f && x[i] == 0.0f) continue;  // zeros (NaN does not count as `most`)
        d = fma(static_cast<double>(x[i]), static_cast<double>(x[i]), d);
    }
    return d;
}

template <int N>
__device__ __forceinline__ double square_sum(const float (&x)[N])
{
    const float s = squares(x);
    return holds(s) ? static_cast<double>(s) : squares_in_64<N>(x);
}

__device__ __forceinline__ double warp_sum(double s)
{
#pragma unroll
    for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// The CTA's sum, in its first warp: which adds all up, as an fp64 addition keeps the SM's
// fp64 unit busy for 16 cycles whether a warp's lanes need it or not.
__device__ __forceinline__ double block_sum(double s, double (&shared)[CLIP_THREADS])
{
    shared[threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.x >= 32) return 0.0;
    s = 0.0;
#pragma unroll
    for (int i = 0; i < CLIP_THREADS / 32; ++i) s += shared[i * 32 + threadIdx.x];
    return warp_sum(s);
}

// Vectors of a whole chunk per thread.
constexpr int CHUNK_F32 = static_cast<int>(CHUNK / 4 / CLIP_THREADS);
constexpr int CHUNK_F16 = static_cast<int>(CHUNK / 8 / CLIP_THREADS);

__global__ void __launch_bounds__(CLIP_THREADS) k_grad_squares(const Chunk* table, int64_t chunks,
                                                               double* parts)
{
    __shared__ double shared[CLIP_THREADS];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = static_cast<int>(threadIdx.x);
    double sum = 0.0;
    for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const Chunk k = load_chunk(table, c);
        const bool vectors = (reinterpret_cast<uintptr_t>(k.src) & 15u) == 0;
        int done = 0;
        if (k.f16) {
            const __half* src = static_cast<const __half*>(k.src);
            const uint4* v = reinterpret_cast<const uint4*>(src);
            if (vectors && k.count == CHUNK) {
                uint4 w[CHUNK_F16];
#pragma unroll
                for (int i = 0; i < CHUNK_F16; ++i) w[i] = v[i * CLIP_THREADS + tid];
                float s = 0.0f;  // squares of fp16 values and their sums: fp32 holds them
#pragma unroll
                for (int i = 0; i < CHUNK_F16; ++i) {
                    float x[8];
                    widen8(w[i], x);
                    s += squares(x);
                }
                sum += static_cast<double>(s);
                continue;
            }
            if (vectors) {
                done = k.count & ~7;
                for (int i = tid; i < done / 8; i += CLIP_THREADS) {
                    float x[8];
                    widen8(v[i], x);
                    sum += static_cast<double>(squares(x));
                }
            }
            for (int i = done + tid; i < k.count; i += CLIP_THREADS) {
                const float x = __half2float(src[i]);
                sum += static_cast<double>(x * x);
            }
        } else {
            const float* src = static_cast<const float*>(k.src);
            const float4* v = reinterpret_cast<const float4*>(src);
            if (vectors && k.count == CHUNK) {
                float4 w[CHUNK_F32];
#pragma unroll
                for (int i = 0; i < CHUNK_F32; ++i) w[i] = v[i * CLIP_THREADS + tid];
                float s[CHUNK_F32];
#pragma unroll
                for (int i = 0; i < CHUNK_F32; ++i) {
                    const float x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                    s[i] = squares(x);
                }
#pragma unroll
                for (int n = CHUNK_F32 / 2; n > 0; n /= 2)
#pragma unroll
                    for (int i = 0; i < n; ++i) s[i] += s[i + n];
                if (holds(s[0])) {
                    sum += static_cast<double>(s[0]);
                } else {
                    for (int i = 0; i < CHUNK_F32; ++i) {
                        const float4 f = v[i * CLIP_THREADS + tid];
                        const float x[4] = {f.x, f.y, f.z, f.w};
                        sum += squares_in_64<4>(x);
                    }
                }
                continue;
            }
            if (vectors) {
                done = k.count & ~3;
                for (int i = tid; i < done / 4; i += CLIP_THREADS) {
                    const float4 f = v[i];
                    const float x[4] = {f.x, f.y, f.z, f.w};
                    sum += square_sum(x);
                }
            }
            for (int i = done + tid; i < k.count; i += CLIP_THREADS) {
                const float x[1] = {src[i]};
                sum += square_sum(x);
            }
        }
    }
    sum = block_sum(sum, shared);
    if (tid == 0) parts[blockIdx.x] = sum;
}

// Square root and reciprocal from fp32 ones and a Newton step in fp64 (2^-44 off at most),
// where fp32 holds them: the library's take several times the fp64 instructions.
__device__ __forceinline__ double square_root(double x)
{
    if (!(x >= 0x1p-100 && x <= 0x1p100)) return sqrt(x);
    const double y = static_cast<double>(rsqrtf(static_cast<float>(x)));
    const double root = x * y;  // root + (x - root^2) y / 2
    return fma(fma(-root, root, x), 0.5 * y, root);
}

__device__ __forceinline__ double reciprocal(double x)
{
    if (!(x >= 0x1p-100 && x <= 0x1p100)) return 1.0 / x;
    const double y = static_cast<double>(1.0f / static_cast<float>(x));
    return fma(fma(-x, y, 1.0), y, y);
}

__device__ __forceinline__ uint4 scaled8(const uint4& v, float first, float f)
{
    float x[8];
    widen8(v, x);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2 h = __floats2half2_rn(x[2 * j] * first * f, x[2 * j + 1] * first * f);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float4 scaled4(const float4& v, float first, float f)
{
    return make_float4(v.x * first * f, v.y * first * f, v.z * first * f, v.w * first * f);
}

__global__ void __launch_bounds__(CLIP_THREADS)
    k_grad_clip(const Chunk* table, int64_t chunks, const double* parts, int part_count,
                float max_norm, float eps, float* norm, int scale)
{
    __shared__ float factors[2];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = static_cast<int>(threadIdx.x);
    if (tid < 32) {
        // one warp adds the parts up, as fp64 instructions are slow
        double sum = 0.0;
        for (int i = tid; i < part_count; i += 32) sum += parts[i];
        sum = warp_sum(sum);
        if (tid == 0) {
            const double length = square_root(sum);
            if (blockIdx.x == 0) *norm = static_cast<float>(length);
            const double ratio =
                static_cast<double>(max_norm) * reciprocal(length + static_cast<double>(eps));
            // NaN stays NaN; no length, nothing to scale (and perhaps no quotient)
            const double factor = ratio >= 1.0 || length == 0.0 ? 1.0 : ratio;
            // in two steps, the first a power of two: fp32 does not hold the smallest
            // factors whole
            factors[0] = factor < 0x1p-100 ? 0x1p-64f : 1.0f;
            factors[1] = static_cast<float>(factor < 0x1p-100 ? factor * 0x1p64 : factor);
        }
    }
    if (!scale) return;
    __syncthreads();
    const float first = factors[0], f = factors[1];
    for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const Chunk k = load_chunk(table, chunks - 1 - c);
        const bool vectors =
            ((reinterpret_cast<uintptr_t>(k.src) | reinterpret_cast<uintptr_t>(k.dst)) & 15u) == 0;
        if (f == 1.0f && k.src == k.dst) continue;  // the values stay what they are
        int done = 0;
        if (k.f16) {
            const __half* src = static_cast<const __half*>(k.src);
            __half* dst = static_cast<__half*>(k.dst);
            if (vectors && k.count == CHUNK) {
                uint4 w[CHUNK_F16];
#pragma unroll
                for (int i = 0; i < CHUNK_F16; ++i)
                    w[i] = reinterpret_cast<const uint4*>(src)[i * CLIP_THREADS + tid];
#pragma unroll
                for (int i = 0; i < CHUNK_F16; ++i)
                    reinterpret_cast<uint4*>(dst)[i * CLIP_THREADS + tid] = scaled8(w[i], first, f);
                continue;
            }
            if (vectors) {
                done = k.count & ~7;
                for (int i = tid; i < done / 8; i += CLIP_THREADS)
                    reinterpret_cast<uint4*>(dst)[i] =
                        scaled8(reinterpret_cast<const uint4*>(src)[i], first, f);
            }
            for (int i = done + tid; i < k.count; i += CLIP_THREADS)
                dst[i] = __float2half_rn(__half2float(src[i]) * first * f);
        } else {
            const float* src = static_cast<const float*>(k.src);
            float* dst = static_cast<float*>(k.dst);
            if (vectors && k.count == CHUNK) {
                float4 w[CHUNK_F32];
#pragma unroll
                for (int i = 0; i < CHUNK_F32; ++i)
                    w[i] = reinterpret_cast<const float4*>(src)[i * CLIP_THREADS + tid];
#pragma unroll
                for (int i = 0; i < CHUNK_F32; ++i)
                    reinterpret_cast<float4*>(dst)[i * CLIP_THREADS + tid] =
                        scaled4(w[i], first, f);
                continue;
            }
            if (vectors) {
                done = k.count & ~3;
                for (int i = tid; i < done / 4; i += CLIP_THREADS)
                    reinterpret_cast<float4*>(dst)[i] =
                        scaled4(reinterpret_cast<const float4*>(src)[i], first, f);
            }
            for (int i = done + tid; i < k.count; i += CLIP_THREADS) dst[i] = src[i] * first * f;
        }
    }
}

// Whether no output shares memory with another output, or with a gradient other than the
// one at the same place (a sweep over the tensors by their addresses).
bool outputs_apart(int64_t count, const void* const* grads, void* const* outs,
                   const int64_t* sizes, const int* dtypes)
{
    struct Span {
        uintptr_t begin, end;
        bool out;
    };
    std::vector<Span> spans;
    for (int64_t i = 0; i < count; ++i) {
        if (sizes[i] == 0) continue;
        const uintptr_t bytes =
            static_cast<uintptr_t>(sizes[i]) * (dtypes[i] == GEMM_OUT_F16 ? 2 : 4);
        const uintptr_t to = reinterpret_cast<uintptr_t>(outs[i]);
        const uintptr_t from = reinterpret_cast<uintptr_t>(grads[i]);
        spans.push_back({to, to + bytes, true});
        if (from != to) spans.push_back({from, from + bytes, false});
    }
    std::sort(spans.begin(), spans.end(),
              [](const Span& a, const Span& b) { return a.begin < b.begin; });
    uintptr_t outs_end = 0, any_end = 0;
    for (const Span& s : spans) {
        if (s.begin < (s.out ? any_end : outs_end)) return false;
        any_end = std::max(any_end, s.end);
        if (s.out) outs_end = std::max(outs_end, s.end);
    }
    return true;
}

int run_clip(const gemm_clip_plan* plan, float max_norm, float eps, float* norm, void* workspace,
             void* cuda_stream, bool scale)
{
    if (!plan) return fail(GEMM_ERR_INVALID_ARG, "plan is NULL");
    if (!norm || !workspace)
        return fail(GEMM_ERR_INVALID_ARG, "norm and workspace must be non-NULL");
    if (reinterpret_cast<uintptr_t>(norm) & 3u || !aligned16(workspace))
        return fail(GEMM_ERR_UNSUPPORTED, "norm must be 4-byte and workspace 16-byte aligned");
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail("cudaGetDevice", e);
    if (dev != plan->device)
        return fail(GEMM_ERR_INVALID_ARG, "plan was created on another device");
    cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    const Chunk* table = plan->d_chunks;
    double* parts = static_cast<double*>(workspace);
    const dim3 grid(static_cast<unsigned>(plan->grid)), block(CLIP_THREADS);
    e = launch_dependent(k_grad_squares, grid, block, 0, 1, stream, table, plan->chunks, parts);
    if (e == cudaSuccess)
        e = launch_dependent(k_grad_clip, scale ? grid : dim3(1), block, 0, 1, stream, table,
                             plan->chunks, static_cast<const double*>(parts), plan->grid, max_norm,
                             eps, norm, scale ? 1 : 0);
    return e == cudaSuccess ? ok() : cuda_fail("clipping launch", e);
}

}  // namespace

extern "C" {

gemm_clip_plan* gemm_clip_create_plan(int64_t count, const void* const* grads, void* const* outs,
                                      const int64_t* sizes, const int* dtypes)
{
    gemm_clip_plan* made = nullptr;
    guarded([&] {
        if (count < 0 || (count > 0 && (!grads || !outs || !sizes || !dtypes)))
            return fail(GEMM_ERR_INVALID_ARG,
                        "grads, outs, sizes and dtypes must hold `count` entries");
        std::vector<Chunk> table;
        for (int64_t i = 0; i < count; ++i) {
            if (dtypes[i] != GEMM_OUT_F32 && dtypes[i] != GEMM_OUT_F16)
                return fail(GEMM_ERR_INVALID_ARG,
                            "dtypes must be GEMM_OUT_F32 (0) or GEMM_OUT_F16 (1)");
            if (sizes[i] < 0) return fail(GEMM_ERR_INVALID_ARG, "sizes must be >= 0");
            if (sizes[i] == 0) continue;
            const int elt = dtypes[i] == GEMM_OUT_F16 ? 2 : 4;
            const char* src = static_cast<const char*>(grads[i]);
            char* dst = static_cast<char*>(outs[i]);
            if (!src || !dst)
                return fail(GEMM_ERR_INVALID_ARG, "a tensor's address is NULL");
            if ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) % elt != 0)
                return fail(GEMM_ERR_UNSUPPORTED, "a tensor is not aligned to its values");
            for (int64_t at = 0; at < sizes[i]; at += CHUNK) {
                Chunk c = {};
                c.src = src + at * elt;
                c.dst = dst + at * elt;
                c.count = static_cast<int>(std::min(CHUNK, sizes[i] - at));
                c.f16 = elt == 2;
                table.push_back(c);
            }
        }
        if (!outputs_apart(count, grads, outs, sizes, dtypes))
            return fail(GEMM_ERR_INVALID_ARG,
                        "an output overlaps another one, or a gradient that is not its own");
        int dev, sms;
        const int r = require_device(&dev, &sms, nullptr);
        if (r != GEMM_OK) return r;
        std::unique_ptr<gemm_clip_plan> plan(new gemm_clip_plan{});
        plan->chunks = static_cast<int64_t>(table.size());
        plan->device = dev;
        plan->grid = static_cast<int>(std::max<int64_t>(
            1, std::min<int64_t>(plan->chunks, std::min(4 * sms, MAX_PARTS))));
        if (!table.empty()) {
            const size_t bytes = table.size() * sizeof(Chunk);
            cudaError_t e = cudaMalloc(&plan->d_chunks, bytes);
            if (e == cudaSuccess)
                e = fill_memory(plan->d_chunks, table.data(), bytes);
            if (e != cudaSuccess) {
                if (plan->d_chunks) cudaFree(plan->d_chunks);
                return cuda_fail("allocating the table of gradients", e);
            }
        }
        made = plan.release();
        return ok();
    });
    return made;
}

int gemm_clip_run(gemm_clip_plan* plan, float max_norm, float eps, float* norm, void* workspace,
                  void* cuda_stream)
{
    return guarded([&] {
        if (!(max_norm >= 0.0f) || !(eps >= 0.0f))
            return fail(GEMM_ERR_INVALID_ARG, "max_norm and eps must be >= 0");
        return run_clip(plan, max_norm, eps, norm, workspace, cuda_stream, true);
    });
}

int gemm_clip_norm(gemm_clip_plan* plan, float* norm, void* workspace, void* cuda_stream)
{
    return guarded(
        [&] { return run_clip(plan, 0.0f, 0.0f, norm, workspace, cuda_stream, false); });
}

void gemm_clip_destroy(gemm_clip_plan* plan)
{
    if (!plan) return;
    if (plan->d_chunks) cudaFree(plan->d_chunks);
    delete plan;
}

}  // extern "C"
