// expert_route.cu -- tokens sorted by expert and back: the stable counting
// sort of the routing slots, the copy of the tokens into sorted order, the
// weighted sum of the experts' rows per token, and the gradients of both.
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>
#include <vector>

#include "../../include/tmaexperts.h"
#include "launch.h"
#include "ptx.cuh"
#include "runtime.h"
#include "sort_shape.h"

namespace tg {

namespace {

// ------------------------------------------------------------------- sort
//
// Stable counting sort of S slots by key(s) = id, or E for a dropped slot:
//
//   position[s] = start[key] + |{s' < s : key(s') = key}|,
//   start[e] = |{s : key(s) < e}|.
//
// One cluster does it in one launch.  Every warp owns a contiguous run of
// slots and a histogram of its own in shared memory, so the count of equal
// keys before a slot is (keys in earlier CTAs) + (earlier warps) + (earlier in
// this warp), all taken in slot order: no result depends on timing.  The CTAs'
// totals are exchanged through distributed shared memory.
//
// Two passes over the ids, 12 bytes a slot in all: bound by latency, the launch, the
// cluster's barriers and the chains of shared-memory counts.  A cluster because its
// barrier costs less than a second launch; up to 16 CTAs of it, 1024 slots or more
// each (131072 slots of 128 experts: 11.0 us on 16 CTAs, 21.2 on 8; 128 slots: 2.6 us
// on one).
constexpr int SORT_MAX_EXPERTS = 1024;
// Slots per warp from which equal keys are found bit by bit.  The match
// instruction answers sooner (128 slots per warp in one CTA: 4.0 against 4.9 us)
// but few at a time (131072 slots of 128 experts: 13.4 against 10.7 us).
constexpr int SORT_BALLOT_RUN = 192;
constexpr int SORT_BATCH = 8;  // ids a lane loads at once

__device__ __forceinline__ uint32_t ld_shared_rank(uint32_t local, uint32_t rank)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_shared_rank(local, rank)));
    return v;
}

__global__ void __launch_bounds__(1024, 1)
    k_expert_sort(int slots, int experts, int run, const int32_t* ids, int32_t* offsets,
                  int32_t* order, int32_t* position)
{
    extern __shared__ uint32_t sort_smem[];
    const int keys = experts + 1;
    const int warps = static_cast<int>(blockDim.x) / 32;
    uint32_t* hist = sort_smem;             // [warps][keys]
    uint32_t* total = hist + warps * keys;  // [keys] of this CTA, read by its peers
    uint32_t* base = total + keys;          // [keys] first row of this CTA's slots of a key
    uint32_t* warp_sum = base + keys;       // [33]
    const int tid = static_cast<int>(threadIdx.x);
    const int warp = tid >> 5;
    const uint32_t lane = lane_id();
    const uint32_t rank = cluster_ctarank();
    const uint32_t ctas = gridDim.x;

    for (int i = tid; i < warps * keys; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();

    uint32_t* mine = hist + warp * keys;
    const int64_t first = (static_cast<int64_t>(rank) * warps + warp) * run;
    const int begin = static_cast<int>(first < slots ? first : slots);
    const int end = static_cast<int>(first + run < slots ? first + run : slots);
    auto load_keys = [&](int s0, int (&key)[SORT_BATCH]) {
#pragma unroll
        for (int b = 0; b < SORT_BATCH; ++b) {
            const int s = s0 + b * 32 + static_cast<int>(lane);
            int id = -1;
            if (s < end) id = ids[s];
            key[b] = static_cast<unsigned>(id) < static_cast<unsigned>(experts) ? id : experts;
        }
    };
    int key[SORT_BATCH];
    for (int s0 = begin; s0 < end; s0 += 32 * SORT_BATCH) {
        load_keys(s0, key);
#pragma unroll
        for (int b = 0; b < SORT_BATCH; ++b)
            if (s0 + b * 32 + static_cast<int>(lane) < end) atomicAdd(&mine[key[b]], 1u);
    }
    __syncthreads();

    // per key: exclusive sums over this CTA's warps, and the CTA's total
    for (int k = tid; k < keys; k += blockDim.x) {
        uint32_t acc = 0;
        for (int w = 0; w < warps; ++w) {
            const uint32_t v = hist[w * keys + k];
            hist[w * keys + k] = acc;
            acc += v;
        }
        total[k] = acc;
    }
    cluster_sync_all();

    // per key: rows of earlier CTAs, and of all; then the exclusive sum over
    // keys, a contiguous share of keys per thread
    const int share = (keys + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
    uint32_t sum = 0;
    for (int i = 0; i < share; ++i) {
        const int k = tid * share + i;
        if (k >= keys) break;
        uint32_t all = 0;
        for (uint32_t c = 0; c < ctas; ++c) all += ld_shared_rank(smem_u32(total + k), c);
        sum += all;
    }
    uint32_t scan = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= static_cast<uint32_t>(d)) scan += v;
    }
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    if (warp == 0) {
        uint32_t v = static_cast<int>(lane) < warps ? warp_sum[lane] : 0u;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= static_cast<uint32_t>(d)) v += u;
        }
        warp_sum[lane] = v;
    }
    __syncthreads();
    uint32_t row = scan - sum + (warp > 0 ? warp_sum[warp - 1] : 0u);
    for (int i = 0; i < share; ++i) {
        const int k = tid * share + i;
        if (k >= keys) break;
        uint32_t before = 0, all = 0;
        for (uint32_t c = 0; c < ctas; ++c) {
            const uint32_t v = ld_shared_rank(smem_u32(total + k), c);
            if (c < rank) before += v;
            all += v;
        }
        base[k] = row + before;
        if (rank == 0) offsets[k] = static_cast<int32_t>(row);
        row += all;
    }
    // peers have read this CTA's totals; base is complete
    cluster_sync_all();

    for (int s0 = begin; s0 < end; s0 += 32 * SORT_BATCH) {
        load_keys(s0, key);
#pragma unroll
        for (int b = 0; b < SORT_BATCH; ++b) {
            const int s = s0 + b * 32 + static_cast<int>(lane);
            const bool live = s < end;
            // lanes past the end share a key no slot has
            const int k = live ? key[b] : keys;
            unsigned same;
            if (run < SORT_BALLOT_RUN) {
                same = __match_any_sync(0xffffffffu, k);
            } else {
                same = 0xffffffffu;
                for (int bit = 0; (keys >> bit) != 0; ++bit) {
                    const unsigned ones = __ballot_sync(0xffffffffu, (k >> bit) & 1);
                    same &= ((k >> bit) & 1) ? ones : ~ones;
                }
            }
            const unsigned before = same & ((1u << lane) - 1u);
            uint32_t r = 0;
            if (live) r = mine[k] + __popc(before);
            __syncwarp();
            if (live && before == 0) mine[k] += __popc(same);
            __syncwarp();
            if (live) {
                r += base[k];
                position[s] = static_cast<int32_t>(r);
                // always true for ids that nobody changes meanwhile
                if (r < static_cast<uint32_t>(slots)) order[r] = s;
            }
        }
    }
}

// ----------------------------------------------------------- rows by chunk
//
// The three kernels below move rows of `width` halves as 16-byte chunks.  A
// thread owns one chunk column of one token, so a token's row is read once and
// used for all of its slots.  All are bound by memory: the slots' rows once, in or
// out, beside the tokens' (the gather of 16384 tokens x 8 slots of 2048: 90 us, 6.7
// TB/s).

struct RowMap {
    const int32_t* offsets;
    const int32_t* position;  // nullptr: slot order
    int experts;
    int64_t slots;
    const int32_t* ids;       // slot order: the slots' experts, or nullptr: none is dropped
};

// Rows that belong to an expert: [0, kept).
__device__ __forceinline__ uint32_t kept_rows(const RowMap& m)
{
    if (m.position == nullptr) return static_cast<uint32_t>(m.slots);
    const int32_t n = m.offsets[m.experts];
    return n < 0 ? 0u : (n > m.slots ? static_cast<uint32_t>(m.slots) : static_cast<uint32_t>(n));
}

__device__ __forceinline__ uint32_t row_of(const RowMap& m, int64_t slot)
{
    if (m.position != nullptr) return static_cast<uint32_t>(m.position[slot]);
    if (m.ids != nullptr && static_cast<unsigned>(m.ids[slot]) >= static_cast<unsigned>(m.experts))
        return 0xffffffffu;  // dropped
    return static_cast<uint32_t>(slot);
}

__global__ void __launch_bounds__(256)
    k_expert_gather(int64_t tokens, int topk, int chunks, RowMap map, const uint4* X, uint4* Xs)
{
    griddep_wait();
    griddep_launch_dependents();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const int c = static_cast<int>(blockIdx.y * blockDim.x + threadIdx.x);
    if (t >= tokens || c >= chunks) return;
    const uint32_t kept = kept_rows(map);
    const uint4 v = X[t * chunks + c];
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int j = 0; j < topk; ++j) {
        const uint32_t r = row_of(map, t * topk + j);
        if (r < map.slots) Xs[static_cast<int64_t>(r) * chunks + c] = r < kept ? v : zero;
    }
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8])
{
    const __half2* h = reinterpret_cast<const __half2*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = __half22float2(h[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    uint4 v;
    __half2* h = reinterpret_cast<__half2*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    return v;
}

// The sum of a token's rows.  Bound by reading Ys once.  BATCH is the number of
// slots whose rows a thread has in flight at once: registers for slots that a
// token does not have cost resident warps (32768 tokens x 2 slots of 1024: 84 us with 8, 42 with 4), and
// with many tokens four in flight and more warps beat eight (8192 tokens x 8 slots
// of 4096: 110 and 90 us, 6.7 TB/s); with few tokens the second batch is one more
// wait (3 tokens x 6 slots: 2.4 and 2.5 us).
template <bool F16OUT, int BATCH>
__global__ void __launch_bounds__(256, BATCH == 8 ? 3 : 6)
    k_expert_combine(int64_t tokens, int topk, int chunks, RowMap map, const uint4* Ys,
                     const float* weights, void* Y)
{
    griddep_wait();
    griddep_launch_dependents();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const int c = static_cast<int>(blockIdx.y * blockDim.x + threadIdx.x);
    if (t >= tokens || c >= chunks) return;
    const uint32_t kept = kept_rows(map);
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < topk; j0 += BATCH) {
        uint32_t row[BATCH];
        float w[BATCH];
        uint4 v[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            row[b] = 0xffffffffu;
            w[b] = 1.0f;
            if (j0 + b < topk) {
                row[b] = row_of(map, t * topk + j0 + b);
                if (weights) w[b] = weights[t * topk + j0 + b];
            }
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
            if (row[b] < kept) v[b] = Ys[static_cast<int64_t>(row[b]) * chunks + c];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            if (row[b] >= kept) continue;  // a dropped slot: its weight and row are not used
            float f[8];
            unpack8(v[b], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = fmaf(w[b], f[i], acc[i]);
        }
    }
    if constexpr (F16OUT) {
        static_cast<uint4*>(Y)[t * chunks + c] = pack8(acc);
    } else {
        float4* y = static_cast<float4*>(Y) + (t * chunks + c) * 2;
        y[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        y[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    }
}

// WPT warps share a token: each walks every WPT-th group of 32 chunks, and the
// dot products of the token's slots are summed over lanes by shuffles and over
// warps through shared memory, in a fixed order.  A thread reads a chunk of Ys
// before it writes the same chunk of dYs and no other thread touches it, so the
// two may be the same buffer.  BATCH as above (16384 tokens x 4 slots of 4096: 200
// us with 8, 178 with 4, 6.8 TB/s; 6 slots of 1000: 99 and 81 us; 3 tokens x 6
// slots: 4.0 and 5.2 us).
template <int WPT, int BATCH>
__global__ void __launch_bounds__(256, BATCH == 8 ? 2 : 4)
    k_expert_combine_grad(int64_t tokens, int topk, int chunks, RowMap map, const uint4* dY,
                          const uint4* Ys, const float* weights, uint4* dYs, float* dweights)
{
    __shared__ float part[8][BATCH];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = static_cast<int>(threadIdx.x) >> 5;
    const uint32_t lane = lane_id();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (8 / WPT) + warp / WPT;
    const bool live = t < tokens;
    const uint32_t kept = kept_rows(map);
    for (int j0 = 0; j0 < topk; j0 += BATCH) {
        uint32_t row[BATCH];
        float w[BATCH], dot[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            row[b] = 0xffffffffu;
            w[b] = 0.0f;
            dot[b] = 0.0f;
            if (live && j0 + b < topk) {
                row[b] = row_of(map, t * topk + j0 + b);
                if (row[b] < kept) w[b] = weights[t * topk + j0 + b];
            }
        }
        if (live) {
            for (int c = (warp % WPT) * 32 + static_cast<int>(lane); c < chunks; c += WPT * 32) {
                float g[8];
                unpack8(dY[t * chunks + c], g);
                uint4 v[BATCH];
#pragma unroll
                for (int b = 0; b < BATCH; ++b)
                    if (row[b] < kept) v[b] = Ys[static_cast<int64_t>(row[b]) * chunks + c];
#pragma unroll
                for (int b = 0; b < BATCH; ++b) {
                    if (row[b] >= map.slots) continue;  // past the last slot
                    uint4 out = make_uint4(0, 0, 0, 0);
                    if (row[b] < kept) {
                        float f[8], o[8];
                        unpack8(v[b], f);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            dot[b] = fmaf(g[i], f[i], dot[b]);
                            o[i] = w[b] * g[i];
                        }
                        out = pack8(o);
                    }
                    dYs[static_cast<int64_t>(row[b]) * chunks + c] = out;
                }
            }
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
#pragma unroll
            for (int d = 16; d > 0; d /= 2) dot[b] += __shfl_xor_sync(0xffffffffu, dot[b], d);
        }
        if (WPT == 1) {
            if (lane == 0 && live) {
#pragma unroll
                for (int b = 0; b < BATCH; ++b)
                    if (j0 + b < topk) dweights[t * topk + j0 + b] = dot[b];
            }
        } else {
            if (lane == 0) {
#pragma unroll
                for (int b = 0; b < BATCH; ++b) part[warp][b] = dot[b];
            }
            __syncthreads();
            if (warp % WPT == 0 && lane < BATCH && live && j0 + static_cast<int>(lane) < topk) {
                float s = 0.0f;
#pragma unroll
                for (int u = 0; u < WPT; ++u) s += part[warp + u][lane];
                dweights[t * topk + j0 + lane] = s;
            }
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------- host side

int check_slots(int64_t tokens, int topk, int experts)
{
    if (tokens < 0 || topk < 1 || topk > 256)
        return fail(GEMM_ERR_INVALID_ARG, "tokens must be >= 0 and topk in 1..256");
    if (experts < 1 || experts > SORT_MAX_EXPERTS)
        return fail(GEMM_ERR_INVALID_ARG, "experts must be in 1..1024");
    if (tokens > (int64_t(1) << 30) / topk)
        return fail(GEMM_ERR_UNSUPPORTED, "tokens * topk must be at most 2^30");
    return GEMM_OK;
}

int check_width(int64_t width)
{
    if (width < 1 || width >= (int64_t(1) << 31))
        return fail(GEMM_ERR_INVALID_ARG, "width must be in 1..2^31-1");
    if (width % 8 != 0)
        return fail(GEMM_ERR_UNSUPPORTED, "width must be a multiple of 8 (16-byte chunks of fp16)");
    return GEMM_OK;
}

template <int BATCH>
auto grad_kernel(int wpt)
{
    return wpt == 1   ? k_expert_combine_grad<1, BATCH>
           : wpt == 2 ? k_expert_combine_grad<2, BATCH>
           : wpt == 4 ? k_expert_combine_grad<4, BATCH>
                      : k_expert_combine_grad<8, BATCH>;
}

// Threads over the chunks of a row and, for narrow rows, over several tokens:
// 256 threads a block, 64 where that leaves fewer blocks than SMs.
struct RowGrid {
    dim3 grid, block;
};

// Slots in flight per thread (see k_expert_combine).
int slot_batch(int topk, bool few)
{
    if (topk <= 2) return 2;
    return topk <= 4 || !few ? 4 : 8;
}

RowGrid row_grid(int64_t tokens, int chunks, int sms)
{
    int threads = 256;
    while (threads > 64 && tokens * chunks / threads < sms) threads /= 2;
    int cx = 8;
    while (cx < threads && cx < chunks) cx *= 2;
    const int ty = threads / cx;
    RowGrid g;
    g.block = dim3(cx, ty);
    g.grid = dim3(static_cast<unsigned>((tokens + ty - 1) / ty),
                  static_cast<unsigned>((chunks + cx - 1) / cx));
    return g;
}

// Whether a cluster of SORT_CTAS fits the device (a GPC may have fewer SMs to spare than
// that, and with many experts each takes a CTA's worth of shared memory), asked of the
// runtime once for every size that earlier answers do not cover.
cudaError_t large_sort_cluster_fits(int dev, unsigned smem, bool* fits)
{
    struct Answer {
        unsigned fits, fails;  // the largest size that does, the smallest that does not
    };
    static std::mutex mutex;
    static std::vector<Answer> answers;
    std::lock_guard<std::mutex> lock(mutex);
    if (answers.size() <= static_cast<size_t>(dev)) answers.resize(dev + 1, Answer{0u, ~0u});
    Answer& a = answers[dev];
    if (smem > a.fits && smem < a.fails) {
        cudaError_t e =
            cudaFuncSetAttribute(k_expert_sort, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(SORT_CTAS);
        cfg.blockDim = dim3(1024);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = SORT_CTAS;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        e = cudaOccupancyMaxActiveClusters(&clusters, k_expert_sort, &cfg);
        if (e != cudaSuccess) return e;
        if (clusters > 0)
            a.fits = smem;
        else
            a.fails = smem;
    }
    *fits = smem <= a.fits;
    return cudaSuccess;
}

// Both forms of the combination: by `position`, or in slot order (position = nullptr)
// with the slots' expert ids or without.
int combine_rows(int64_t tokens, int topk, int experts, int64_t width, const void* Ys,
                 const int32_t* offsets, const int32_t* position, const int32_t* ids,
                 const float* weights, int dtype_out, void* Y, void* cuda_stream)
{
    return guarded([&] {
        int r = check_slots(tokens, topk, experts);
        if (r == GEMM_OK) r = check_width(width);
        if (r != GEMM_OK) return r;
        if (dtype_out != GEMM_OUT_F32 && dtype_out != GEMM_OUT_F16)
            return fail(GEMM_ERR_INVALID_ARG,
                        "dtype_out must be GEMM_OUT_F32 (0) or GEMM_OUT_F16 (1)");
        if (tokens == 0) return ok();
        if (!Ys || !Y || (position && !offsets)) return fail(GEMM_ERR_INVALID_ARG, "NULL pointer");
        if (!aligned16(Ys) || !aligned16(Y))
            return fail(GEMM_ERR_UNSUPPORTED, "Ys and Y must be 16-byte aligned");
        int dev, sms;
        r = require_device(&dev, &sms, nullptr);
        if (r != GEMM_OK) return r;
        const int chunks = static_cast<int>(width / 8);
        const RowGrid g = row_grid(tokens, chunks, sms);
        if (g.grid.y > 65535u) return fail(GEMM_ERR_UNSUPPORTED, "width is too large");
        const RowMap map = {offsets, position, experts, tokens * topk, ids};
        const bool f16 = dtype_out == GEMM_OUT_F16;
        const int64_t blocks = static_cast<int64_t>(g.grid.x) * g.grid.y;
        const int batch = slot_batch(topk, blocks <= 2 * sms);
        auto kernel = batch == 2   ? (f16 ? k_expert_combine<true, 2> : k_expert_combine<false, 2>)
                      : batch == 4 ? (f16 ? k_expert_combine<true, 4> : k_expert_combine<false, 4>)
                                   : (f16 ? k_expert_combine<true, 8> : k_expert_combine<false, 8>);
        cudaError_t e = launch_dependent(kernel, g.grid, g.block, 0, 1,
                                         static_cast<cudaStream_t>(cuda_stream), tokens, topk,
                                         chunks, map, static_cast<const uint4*>(Ys), weights, Y);
        return e == cudaSuccess ? ok() : cuda_fail("expert combine launch", e);
    });
}

}  // namespace

}  // namespace tg

using namespace tg;

extern "C" {

int gemm_expert_sort(int64_t tokens, int topk, int experts, const int32_t* expert_ids,
                     int32_t* offsets, int32_t* order, int32_t* position, void* cuda_stream)
{
    return guarded([&] {
        int r = check_slots(tokens, topk, experts);
        if (r != GEMM_OK) return r;
        const int64_t slots = tokens * topk;
        if (!offsets || (slots > 0 && (!expert_ids || !order || !position)))
            return fail(GEMM_ERR_INVALID_ARG, "NULL pointer");
        int dev, sms, smem_optin;
        r = require_device(&dev, &sms, &smem_optin);
        if (r != GEMM_OK) return r;
        SortShape s = sort_shape(slots, SORT_CTAS);
        cudaError_t e = ensure_smem_limit(k_expert_sort, s.smem_bytes(experts));
        if (e == cudaSuccess && s.ctas > SORT_PORTABLE_CTAS) {
            bool fits = false;
            e = large_sort_cluster_fits(dev, s.smem_bytes(experts), &fits);
            if (e == cudaSuccess && !fits) {
                s = sort_shape(slots, SORT_PORTABLE_CTAS);
                e = ensure_smem_limit(k_expert_sort, s.smem_bytes(experts));
            }
        }
        if (e == cudaSuccess)
            e = launch_dependent(k_expert_sort, dim3(s.ctas), dim3(s.warps * 32),
                                 s.smem_bytes(experts), s.ctas,
                                 static_cast<cudaStream_t>(cuda_stream), static_cast<int>(slots),
                                 experts, s.run, expert_ids, offsets, order, position);
        return e == cudaSuccess ? ok() : cuda_fail("expert sort launch", e);
    });
}

int gemm_expert_gather(int64_t tokens, int topk, int experts, int64_t width, const void* X,
                       const int32_t* offsets, const int32_t* position, void* Xs,
                       void* cuda_stream)
{
    return guarded([&] {
        int r = check_slots(tokens, topk, experts);
        if (r == GEMM_OK) r = check_width(width);
        if (r != GEMM_OK) return r;
        if (tokens == 0) return ok();
        if (!X || !offsets || !position || !Xs) return fail(GEMM_ERR_INVALID_ARG, "NULL pointer");
        if (!aligned16(X) || !aligned16(Xs))
            return fail(GEMM_ERR_UNSUPPORTED, "X and Xs must be 16-byte aligned");
        int dev, sms;
        r = require_device(&dev, &sms, nullptr);
        if (r != GEMM_OK) return r;
        const int chunks = static_cast<int>(width / 8);
        const RowGrid g = row_grid(tokens, chunks, sms);
        if (g.grid.y > 65535u) return fail(GEMM_ERR_UNSUPPORTED, "width is too large");
        const RowMap map = {offsets, position, experts, tokens * topk, nullptr};
        cudaError_t e = launch_dependent(k_expert_gather, g.grid, g.block, 0, 1,
                                         static_cast<cudaStream_t>(cuda_stream), tokens, topk,
                                         chunks, map, static_cast<const uint4*>(X),
                                         static_cast<uint4*>(Xs));
        return e == cudaSuccess ? ok() : cuda_fail("expert gather launch", e);
    });
}

int gemm_expert_combine(int64_t tokens, int topk, int experts, int64_t width, const void* Ys,
                        const int32_t* offsets, const int32_t* position, const float* weights,
                        int dtype_out, void* Y, void* cuda_stream)
{
    return combine_rows(tokens, topk, experts, width, Ys, offsets, position, nullptr, weights,
                        dtype_out, Y, cuda_stream);
}

int gemm_expert_combine_slots(int64_t tokens, int topk, int experts, int64_t width, const void* Ys,
                              const int32_t* expert_ids, const float* weights, int dtype_out,
                              void* Y, void* cuda_stream)
{
    return combine_rows(tokens, topk, experts, width, Ys, nullptr, nullptr, expert_ids, weights,
                        dtype_out, Y, cuda_stream);
}

int gemm_expert_combine_grad(int64_t tokens, int topk, int experts, int64_t width, const void* dY,
                             const void* Ys, const int32_t* offsets, const int32_t* position,
                             const float* weights, void* dYs, float* dweights, void* cuda_stream)
{
    return guarded([&] {
        int r = check_slots(tokens, topk, experts);
        if (r == GEMM_OK) r = check_width(width);
        if (r != GEMM_OK) return r;
        if (tokens == 0) return ok();
        if (!dY || !Ys || !offsets || !position || !weights || !dYs || !dweights)
            return fail(GEMM_ERR_INVALID_ARG, "NULL pointer");
        if (!aligned16(dY) || !aligned16(Ys) || !aligned16(dYs))
            return fail(GEMM_ERR_UNSUPPORTED, "dY, Ys and dYs must be 16-byte aligned");
        int dev, sms;
        r = require_device(&dev, &sms, nullptr);
        if (r != GEMM_OK) return r;
        const int chunks = static_cast<int>(width / 8);
        const RowMap map = {offsets, position, experts, tokens * topk, nullptr};
        int wpt = 1;
        while (wpt < 8 && chunks > 32 * wpt) wpt *= 2;
        const int64_t blocks = (tokens + 8 / wpt - 1) / (8 / wpt);
        const int batch = slot_batch(topk, blocks <= 2 * sms);
        cudaError_t e = launch_dependent(
            batch == 2 ? grad_kernel<2>(wpt) : batch == 4 ? grad_kernel<4>(wpt) : grad_kernel<8>(wpt),
            dim3(static_cast<unsigned>(blocks)), dim3(256), 0, 1,
            static_cast<cudaStream_t>(cuda_stream), tokens, topk, chunks, map,
            static_cast<const uint4*>(dY), static_cast<const uint4*>(Ys), weights,
            static_cast<uint4*>(dYs), dweights);
        return e == cudaSuccess ? ok() : cuda_fail("expert combine gradient launch", e);
    });
}

}  // extern "C"
