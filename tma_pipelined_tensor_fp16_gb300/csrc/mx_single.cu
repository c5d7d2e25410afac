// mx_single.cu -- block-scaled products on single CTAs: few rows (decoding), and
// products too small to fill the GPU with tiles of CTA pairs.
//
// Measured: one row of 16384 x 16384 nvfp4 25.8 us, 5.9 TB/s; 64 rows mxfp8 45 us, 6.2 TB/s (in
// both 2.5 to 4 us are the launch, the first loads and the cluster's sums); 4 rows of 4096 x
// 4096 nvfp4 4.5 us.
//
// One tile per CTA, or per cluster whose CTAs share its length: 128 rows of one operand
// (U, the MMA's M side) and COLS of the other (V, the N side).  With few rows of A, U is
// the weights B and a tile is stored transposed (`SWAPPED`); bound by reading the weights
// then, so that the CTAs in flight matter and not the MMA.
//
// Roles, joined by mbarriers: warp 0 copies stages (four boxes each), warp 1 copies the
// scales to tensor memory and issues the MMAs, warps 2..5 read the sums into shared memory
// (the stages' place), where the cluster adds them up in rank order, each CTA its share
// of the rows or columns.
#include "mx_product.cuh"
#include "runtime.h"

namespace tg {

namespace {

constexpr int MX_THREADS = 192;

__device__ __forceinline__ void tmem_load_16cols(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ constexpr uint32_t tmem_columns(int need)
{
    return need <= 32 ? 32u : need <= 64 ? 64u : need <= 128 ? 128u : need <= 256 ? 256u : 512u;
}

struct MxTile {
    const MxParams* p;
    uint32_t sums;  // shared address of this CTA's sums
    uint32_t rank;
    int u_tile, v0, tid, f16out;
};

// Add up the cluster's sums in rank order, this CTA's share of the tile, and store them.
// Sixteen (eight wide) loads are on their way at a time: one by one, the latency of
// distributed shared memory took 10 us of 64 rows with 16384 columns.
template <int COLS, bool SWAPPED, int SPLIT>
__device__ __forceinline__ void add_up(const MxTile& t)
{
    const MxParams& p = *t.p;
    const float alpha = mx_alpha(p);
    const int rank = static_cast<int>(t.rank);
    uint32_t from[SPLIT];
#pragma unroll
    for (int k = 0; k < SPLIT; ++k) from[k] = SPLIT > 1 ? map_shared_rank(t.sums, k) : t.sums;
    if constexpr (SWAPPED) {
        // C[v0 + c][u0 + r]; columns c = rank, rank + split, ...
        constexpr int G = 16 / SPLIT;
        const int64_t n = static_cast<int64_t>(t.u_tile) * MX_ROWS + t.tid;
        const int cols = min(COLS, p.M - t.v0);
        for (int c0 = rank; c0 < cols; c0 += G * SPLIT) {
            float x[G][SPLIT];
#pragma unroll
            for (int i = 0; i < G; ++i)
#pragma unroll
                for (int k = 0; k < SPLIT; ++k) {
                    const int c = c0 + i * SPLIT;
                    x[i][k] = c < cols ? ld_cluster_f32(from[k] + static_cast<uint32_t>(
                                                                      c * 128 + t.tid) * 4u)
                                       : 0.0f;
                }
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const int c = c0 + i * SPLIT;
                if (c >= cols || n >= p.N) continue;
                float sum = x[i][0];
#pragma unroll
                for (int k = 1; k < SPLIT; ++k) sum += x[i][k];
                const int64_t to = static_cast<int64_t>(t.v0 + c) * p.N + n;
                if (t.f16out)
                    static_cast<__half*>(p.C)[to] = __float2half_rn(sum * alpha);
                else
                    static_cast<float*>(p.C)[to] = sum * alpha;
            }
        }
    } else {
        // C[u0 + r][v0 + c], four columns a lane; rows by rank, then by warp
        constexpr int G = 8 / SPLIT;
        const int lane = t.tid % 32;
        const int n = t.v0 + lane * 4;
        const int64_t u0 = static_cast<int64_t>(t.u_tile) * MX_ROWS;
        const int rows = static_cast<int>(min(static_cast<int64_t>(MX_ROWS), p.M - u0));
        constexpr int STEP = 4 * SPLIT;
        for (int r0 = rank + t.tid / 32 * SPLIT; r0 < rows; r0 += G * STEP) {
            float4 x[G][SPLIT];
#pragma unroll
            for (int i = 0; i < G; ++i)
#pragma unroll
                for (int k = 0; k < SPLIT; ++k) {
                    const int r = r0 + i * STEP;
                    x[i][k] = r < rows ? ld_cluster_f32x4(from[k] + static_cast<uint32_t>(
                                             r * (COLS + 4) + lane * 4) * 4u)
                                       : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const int r = r0 + i * STEP;
                if (r >= rows || n >= p.N) continue;
                float4 sum = x[i][0];
#pragma unroll
                for (int k = 1; k < SPLIT; ++k) {
                    sum.x += x[i][k].x;
                    sum.y += x[i][k].y;
                    sum.z += x[i][k].z;
                    sum.w += x[i][k].w;
                }
                const int64_t to = (u0 + r) * p.N + n;
                if (t.f16out) {
                    const __half2 a = __floats2half2_rn(sum.x * alpha, sum.y * alpha);
                    const __half2 b = __floats2half2_rn(sum.z * alpha, sum.w * alpha);
                    *reinterpret_cast<uint2*>(static_cast<__half*>(p.C) + to) =
                        make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                   *reinterpret_cast<const uint32_t*>(&b));
                } else {
                    *reinterpret_cast<float4*>(static_cast<float*>(p.C) + to) = make_float4(
                        sum.x * alpha, sum.y * alpha, sum.z * alpha, sum.w * alpha);
                }
            }
        }
    }
}

}  // namespace

template <int FORMAT, int COLS, bool SWAPPED>
__global__ void __launch_bounds__(MX_THREADS)
    k_mx_single(const __grid_constant__ CUtensorMap tmUc, const __grid_constant__ CUtensorMap tmUs,
                const __grid_constant__ CUtensorMap tmVc, const __grid_constant__ CUtensorMap tmVs,
                const __grid_constant__ MxParams p, int f16out)
{
    constexpr int CHUNKS = mx_stage_chunks(FORMAT);
    constexpr int GROUPS = mx_stage_groups(FORMAT);
    constexpr int STEP_CHUNKS = mx_step_chunks(FORMAT);
    constexpr int STEPS = CHUNKS / STEP_CHUNKS;
    constexpr int SCALES = mx_step_scales<FORMAT>;
    constexpr uint32_t ACC_COLS = COLS < 32 ? 32 : COLS;
    constexpr uint32_t SET_COLS = GROUPS * 8;  // scales of one stage; two sets alternate
    constexpr uint32_t TMEM_COLS = tmem_columns(ACC_COLS + 2 * SET_COLS);
    constexpr uint32_t V_LEAD = COLS * 16;
    constexpr uint32_t TX = CHUNKS * (MX_CHUNK_BYTES + V_LEAD) + 2 * GROUPS * MX_GROUP_BYTES;
    extern __shared__ __align__(1024) uint8_t mx_smem[];
    const uint32_t raw = smem_u32(mx_smem);
    const uint32_t base = align1024(raw);
    uint8_t* gen = mx_smem + (base - raw);
    const int D = p.pipe_depth;
    const MxSingleLayout L = mx_single_layout(FORMAT, COLS, D, SWAPPED);
    const uint32_t bars = base + L.bars;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gen + L.bars + TMEM_SLOT_OFFSET);
    const int warp = static_cast<int>(warp_uniform(threadIdx.x >> 5));
    const uint32_t lane = lane_id();
    const uint32_t rank = p.split > 1 ? cluster_ctarank() : 0u;
    const int u_tile = static_cast<int>(blockIdx.x) / p.split;
    const int v0 = static_cast<int>(blockIdx.y) * COLS;
    const int s0 = static_cast<int>(static_cast<int64_t>(rank) * p.stages / p.split);
    const int s1 = static_cast<int>(static_cast<int64_t>(rank + 1) * p.stages / p.split);
    Watchdog wd = mx_watchdog(p);
    auto bar = [&](int slot) { return bars + static_cast<uint32_t>(slot) * 8u; };

    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmUc);
        prefetch_tensormap(&tmUs);
        prefetch_tensormap(&tmVc);
        prefetch_tensormap(&tmVs);
        for (int s = 0; s < D; ++s) {
            mbar_init(bar(BAR_FULL + s), 1);
            mbar_init(bar(BAR_EMPTY + s), 1);
        }
        mbar_init(bar(BAR_TMEM_FULL), 1);
        mbar_init(bar(BAR_DRAIN), 1);
        mbar_init(bar(BAR_STALL), 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish_alloc_permit();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t tmem_base = warp_uniform(*tmem_slot);

    if (warp == 0) {
        // ---------------------------------------------------- producer
        if (p.debug_stall == 1) wd.wait(bar(BAR_STALL), 0, WAIT_STALL, -1, -1);
        const int u_row = u_tile * p.chunks, u_group = u_tile * p.groups;
        const int v_block = v0 / MX_ROWS, v_x = v0 % MX_ROWS * 2;
        int stage = 0;
        uint32_t phase = 0;
        int armed = 0;
        for (int s = s0; s < s1; ++s) {
            const bool ok = wd.wait(bar(BAR_EMPTY + stage), phase ^ 1u, WAIT_EMPTY, u_tile, s);
            if (!__all_sync(0xffffffffu, ok)) break;
            if (lane == 0) {
                const uint32_t at = base + static_cast<uint32_t>(stage) * L.stage;
                const uint32_t full = bar(BAR_FULL + stage);
                mbar_arrive_expect_tx(full, TX);
                tma_load_2d(at, &tmUc, full, 0, u_row + s * CHUNKS);
                tma_load_2d(at + L.u_scales, &tmUs, full, 0, u_group + s * GROUPS);
                tma_load_2d(at + L.v_codes, &tmVc, full, v_x,
                            v_block * p.chunks + s * CHUNKS);
                tma_load_2d(at + L.v_scales, &tmVs, full, 0, v_block * p.groups + s * GROUPS);
            }
            ++armed;
            __syncwarp();
            if (++stage == D) {
                stage = 0;
                phase ^= 1u;
            }
        }
        // the copies in flight land before the CTA can exit
        if (lane == 0) {
            for (int i = 0; i < D && i < armed; ++i) {
                if (stage == 0) {
                    stage = D - 1;
                    phase ^= 1u;
                } else {
                    --stage;
                }
                wd.drain(bar(BAR_FULL + stage), phase);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // -------------------------------------------------- MMA issuer
        const uint32_t elected = lane == 0 ? 1u : 0u;
        int stage = 0;
        uint32_t phase = 0;
        for (int s = s0; s < s1; ++s) {
            const bool ok = wd.wait(bar(BAR_FULL + stage), phase, WAIT_FULL, u_tile, s);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after_sync();
            const uint32_t at = base + static_cast<uint32_t>(stage) * L.stage;
            const uint32_t u_sc = tmem_base + ACC_COLS + (s & 1) * SET_COLS;
            const uint32_t v_sc = u_sc + GROUPS * 4;
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                copy_scales<false>(elected, u_sc + g * 4, at + L.u_scales + g * MX_GROUP_BYTES);
                copy_scales<false>(elected, v_sc + g * 4, at + L.v_scales + g * MX_GROUP_BYTES);
            }
            const uint64_t u_desc = core_desc(at, MX_CHUNK_BYTES);
            const uint64_t v_desc = core_desc(at + L.v_codes, V_LEAD);
            const int left = p.steps - s * STEPS;
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                if (i >= left) break;  // uniform
                mx_mma<FORMAT, false>(elected, tmem_base,
                                      u_desc + i * (STEP_CHUNKS * MX_CHUNK_BYTES >> 4),
                                      v_desc + i * (STEP_CHUNKS * V_LEAD >> 4),
                                      mx_idesc<FORMAT>(128, COLS, i * SCALES % 4),
                                      u_sc + i * SCALES / 4 * 4, v_sc + i * SCALES / 4 * 4,
                                      s == s0 && i == 0 ? 0u : 1u);
            }
            mx_commit(elected, bar(BAR_EMPTY + stage));
            __syncwarp();
            if (++stage == D) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (__all_sync(0xffffffffu, !wd.aborted)) mx_commit(elected, bar(BAR_TMEM_FULL));
        if (lane == 0) {
            mma_commit(bar(BAR_DRAIN));
            wd.drain(bar(BAR_DRAIN), 0);
        }
        __syncwarp();
    } else {
        // ---------------------------------------- sums to shared memory
        if (p.debug_stall == 2) wd.wait(bar(BAR_STALL), 0, WAIT_STALL, -1, -1);
        const uint32_t q = static_cast<uint32_t>(warp & 3);
        const uint32_t row = q * 32u + lane;
        const bool ok = wd.wait(bar(BAR_TMEM_FULL), 0, WAIT_TMEM_FULL, u_tile, -1);
        tc_fence_after_sync();
        const uint32_t taddr = tmem_base + (q * 32u << 16);
        if (__all_sync(0xffffffffu, ok)) {
            float* sums = reinterpret_cast<float*>(gen);
            auto put = [&](const uint32_t* v, int c0, int n) {
                if constexpr (SWAPPED) {
                    for (int c = 0; c < n; ++c) sums[(c0 + c) * 128 + row] = __uint_as_float(v[c]);
                } else {
                    for (int c = 0; c < n; c += 4)
                        *reinterpret_cast<uint4*>(sums + row * (COLS + 4) + c0 + c) =
                            make_uint4(v[c], v[c + 1], v[c + 2], v[c + 3]);
                }
            };
            if constexpr (COLS == 16) {
                uint32_t v[16];
                tmem_load_16cols(taddr, v);
#pragma unroll
                for (int c = 0; c < 16; ++c) sums[c * 128 + row] = __uint_as_float(v[c]);
            } else {
#pragma unroll 1
                for (int j = 0; j < COLS / 32; ++j) {
                    uint32_t v[32];
                    tmem_load_32cols(taddr + j * 32, v);
                    put(v, j * 32, 32);
                }
            }
        }
        tc_fence_before_sync();
    }

    __syncwarp();
    if (p.split > 1)
        cluster_sync_all();
    else
        __syncthreads();

    if (warp >= 2 && !wd.aborted && !wd.peer_aborted()) {
        const int tid = static_cast<int>(threadIdx.x) - 64;
        const MxTile tile = {&p, base, rank, u_tile, v0, tid, f16out};
        switch (p.split) {
        case 1: add_up<COLS, SWAPPED, 1>(tile); break;
        case 2: add_up<COLS, SWAPPED, 2>(tile); break;
        case 4: add_up<COLS, SWAPPED, 4>(tile); break;
        default: add_up<COLS, SWAPPED, 8>(tile); break;
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    if (p.split > 1)
        cluster_sync_all();  // the others may still read these sums
    else
        __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

template <int FORMAT, int COLS, bool SWAPPED>
static cudaError_t launch_one(const MxSpec& s, cudaStream_t stream)
{
    auto kernel = k_mx_single<FORMAT, COLS, SWAPPED>;
    cudaError_t e = ensure_smem_limit(kernel, s.smem_bytes);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel,
                            dim3(static_cast<unsigned>(s.grid_x), static_cast<unsigned>(s.grid_y)),
                            dim3(MX_THREADS), s.smem_bytes, s.p.split, stream, *s.codes_u,
                            *s.scales_u, *s.codes_v, *s.scales_v, s.p, s.f16out ? 1 : 0);
}

template <int FORMAT>
static cudaError_t launch_format(const MxSpec& s, cudaStream_t stream)
{
    switch (s.cols) {
    case 16: return launch_one<FORMAT, 16, true>(s, stream);
    case 32: return launch_one<FORMAT, 32, true>(s, stream);
    case 64: return launch_one<FORMAT, 64, true>(s, stream);
    default: return launch_one<FORMAT, 128, false>(s, stream);
    }
}

cudaError_t launch_mx_single(const MxSpec& s, cudaStream_t stream)
{
    switch (s.format) {
    case MXFP8: return launch_format<MXFP8>(s, stream);
    case MXFP4: return launch_format<MXFP4>(s, stream);
    default: return launch_format<NVFP4>(s, stream);
    }
}

}  // namespace tg
