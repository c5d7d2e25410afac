// mx_pair.cu -- block-scaled products on CTA pairs: tiles of 256 x 256 with
// tcgen05.mma.cta_group::2, each CTA holding 128 rows of A, 128 of B, and the scales of
// its rows of A and of all of B's; clusters take tiles t, t + clusters, ... of the grouped
// raster.
//
// Measured: 8192 x 8192 x 8192 nvfp4 135 us, 8150 TFLOP/s, mxfp4 127, mxfp8 291 in a burst, at
// 1800, 1890 and 1690 MHz; held, under the power cap, 154, 142, 336 at 1500, 1575, 1425; 4000 x
// 3000 x 5000 mxfp4 with fp32 output 22 to 26; 2048 x 2048 x 2048 nvfp4 6.4.  Of 224,000 cycles
// of a pair's MMA warp (nvfp4, burst; held 215,500) 148,300 are its 13.5 tiles' MMAs at 128
// cycles each 96 values, 50,100 (41,400) waits for a stage, as its copies take about 2200 cycles
// to arrive and seven stages are all that fits, 6,500 waits for an accumulator (520 a tile's
// change), 2,200 the first stage, and the rest MMAs that take 143 cycles beside the copies.
//
// Tensor memory: two accumulators of 256 columns would leave no room for scales.  They
// lie at columns 0 and 192 and share 64; scales take columns 448 on.  The epilogue reads
// the shared columns first and gives them up, so the next tile's MMAs wait for a quarter
// of a tile's reading and not for its stores.
#include "mx_product.cuh"
#include "runtime.h"

namespace tg {

namespace {

constexpr int MX_THREADS = 192;
constexpr int TILE = 256;
constexpr uint32_t ACC_SHIFT = 192;   // second accumulator
constexpr uint32_t SCALE_COL = 448;
constexpr uint32_t TMEM_COLS = 512;

// 64 columns, one wait for both halves.
__device__ __forceinline__ void tmem_load_64cols(uint32_t taddr, uint32_t (&r)[64])
{
#define TG_LD32(base, col)                                                                       \
    asm volatile(                                                                                \
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "                                                \
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "                \
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];" \
        : "=r"(r[base + 0]), "=r"(r[base + 1]), "=r"(r[base + 2]), "=r"(r[base + 3]),            \
          "=r"(r[base + 4]), "=r"(r[base + 5]), "=r"(r[base + 6]), "=r"(r[base + 7]),            \
          "=r"(r[base + 8]), "=r"(r[base + 9]), "=r"(r[base + 10]), "=r"(r[base + 11]),          \
          "=r"(r[base + 12]), "=r"(r[base + 13]), "=r"(r[base + 14]), "=r"(r[base + 15]),        \
          "=r"(r[base + 16]), "=r"(r[base + 17]), "=r"(r[base + 18]), "=r"(r[base + 19]),        \
          "=r"(r[base + 20]), "=r"(r[base + 21]), "=r"(r[base + 22]), "=r"(r[base + 23]),        \
          "=r"(r[base + 24]), "=r"(r[base + 25]), "=r"(r[base + 26]), "=r"(r[base + 27]),        \
          "=r"(r[base + 28]), "=r"(r[base + 29]), "=r"(r[base + 30]), "=r"(r[base + 31])         \
        : "r"(taddr + (col))                                                                     \
        : "memory")
    TG_LD32(0, 0);
    TG_LD32(32, 32);
#undef TG_LD32
    // the registers are used as results of the wait, so that nothing reads them before it
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 64; ++i) asm volatile("" : "+r"(r[i])::"memory");
}

// As stage_and_store (device_common.cuh) from a buffer that the caller chooses; with `reused`
// it is written once the store from it has read it, STAGING calls before.  With two buffers every
// call is a group of stores, even one without any, as the wait counts them.
template <bool F16OUT, int STAGING>
__device__ __forceinline__ void stage_one(const uint32_t* v, uint32_t row, uint32_t staging,
                                          const CUtensorMap* tmap_c, int col0, int m0, int M,
                                          bool reused)
{
    const uint32_t quarter = row >> 5;
    const uint32_t r = row & 31u;
    const uint32_t buf = staging + quarter * WARP_STAGING_BYTES;
    if (reused) {
        if (r == 0) bulk_wait_group_read<STAGING - 1>();
        __syncwarp();
    }
    const uint32_t row_base = buf + r * 128u;
#pragma unroll
    for (uint32_t c = 0; c < 8; ++c) {
        const uint32_t dst = row_base + ((c ^ (r & 7u)) << 4);
        if constexpr (F16OUT)
            st_shared_v4(dst, pack_half2(v[8 * c + 0], v[8 * c + 1]),
                         pack_half2(v[8 * c + 2], v[8 * c + 3]),
                         pack_half2(v[8 * c + 4], v[8 * c + 5]),
                         pack_half2(v[8 * c + 6], v[8 * c + 7]));
        else
            st_shared_v4(dst, v[4 * c + 0], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    const int wm0 = m0 + static_cast<int>(quarter * 32u);
    if (r == 0 && (STAGING > 1 || wm0 < M)) {
        if (wm0 < M) tma_store_2d(tmap_c, buf, col0, wm0);
        bulk_commit_group();
    }
}

// Both blocks of B's scales in one box.
__device__ __forceinline__ void load_3d_pair(uint32_t dst, const CUtensorMap* map,
                                             uint32_t cluster_bar, int32_t x, int32_t y, int32_t z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(cluster_bar)
        : "memory");
}

// Whether the phase has completed, without waiting for it.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t"
        ".reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

}  // namespace

// STAGING: output buffers of an epilogue warp.
template <int FORMAT, bool F16OUT, int STAGING>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(MX_THREADS, 1)
    k_mx_pair(const __grid_constant__ CUtensorMap tmAc, const __grid_constant__ CUtensorMap tmAs,
              const __grid_constant__ CUtensorMap tmBc, const __grid_constant__ CUtensorMap tmBs,
              const __grid_constant__ CUtensorMap tmC, const __grid_constant__ MxParams p)
{
    constexpr int CHUNKS = mx_pair_chunks(FORMAT);
    constexpr int GROUPS = mx_pair_groups(FORMAT);
    constexpr int STEP_CHUNKS = mx_step_chunks(FORMAT);
    constexpr int STEPS = CHUNKS / STEP_CHUNKS;
    constexpr int SCALES = mx_step_scales<FORMAT>;
    constexpr uint32_t CTA_TX = 2 * CHUNKS * MX_CHUNK_BYTES + 3 * GROUPS * MX_GROUP_BYTES;
    static_assert(SCALE_COL + GROUPS * 12 <= TMEM_COLS, "scales fit");
    extern __shared__ __align__(1024) uint8_t mx_smem[];
    const uint32_t raw = smem_u32(mx_smem);
    const uint32_t base = align1024(raw);
    uint8_t* gen = mx_smem + (base - raw);
    const int D = p.pipe_depth;
    const MxPairLayout L = mx_pair_layout(FORMAT, D, STAGING);
    const uint32_t staging = base + L.staging;
    const uint32_t bars = base + L.bars;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gen + L.bars + TMEM_SLOT_OFFSET);
    const int warp = static_cast<int>(warp_uniform(threadIdx.x >> 5));
    const uint32_t lane = lane_id();
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int clusters = static_cast<int>(gridDim.x) / 2;
    const int first = static_cast<int>(blockIdx.x) / 2;
    const int tiles = p.tiles_m * p.tiles_n;
    Watchdog wd = mx_watchdog(p);
    auto bar = [&](int slot) { return bars + static_cast<uint32_t>(slot) * 8u; };

    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmAc);
        prefetch_tensormap(&tmAs);
        prefetch_tensormap(&tmBc);
        prefetch_tensormap(&tmBs);
        prefetch_tensormap(&tmC);
        for (int s = 0; s < D; ++s) {
            mbar_init(bar(BAR_FULL + s), 1);   // leader: its producer
            mbar_init(bar(BAR_EMPTY + s), 1);  // the leader's multicast commit
        }
        mbar_init(bar(BAR_TMEM_FULL), 1);      // the leader's multicast commit
        mbar_init(bar(BAR_TMEM_EMPTY), 8);     // leader: 4 epilogue warps x 2 CTAs
        mbar_init(bar(BAR_DRAIN), 1);
        mbar_init(bar(BAR_STALL), 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish_alloc_permit_pair();
    }
    tc_fence_before_sync();
    cluster_sync_all();
    tc_fence_after_sync();
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t tmem_base = warp_uniform(*tmem_slot);

    if (warp == 0) {
        // ---------------------------------------------------- producer
        if (p.debug_stall == 1) wd.wait(bar(BAR_STALL), 0, WAIT_STALL, -1, -1);
        int stage = 0;
        uint32_t phase = 0;
        int armed = 0;
        bool running = true;
        const uint32_t full0 = map_shared_rank(bar(BAR_FULL), 0);
        for (int t = first; t < tiles && running; t += clusters) {
            int mt, nt;
            raster_tile(t, p.tiles_m, p.tiles_n, p.group_m, mt, nt);
            const int a_block = mt * 2 + static_cast<int>(rank);
            const int b_block = nt * 2 + static_cast<int>(rank);
            for (int s = 0; s < p.stages; ++s) {
                const bool ok = wd.wait(bar(BAR_EMPTY + stage), phase ^ 1u, WAIT_EMPTY, t, s);
                running = __all_sync(0xffffffffu, ok);
                if (!running) break;
                if (lane == 0) {
                    const uint32_t at = base + static_cast<uint32_t>(stage) * L.stage;
                    if (leader) mbar_arrive_expect_tx(bar(BAR_FULL + stage), 2 * CTA_TX);
                    const uint32_t full = full0 + static_cast<uint32_t>(stage) * 8u;
                    const int c = s * CHUNKS, g = s * GROUPS;
                    tma_load_2d_pair(at, &tmAc, full, 0, a_block * p.chunks + c);
                    tma_load_2d_pair(at + L.b_codes, &tmBc, full, 0, b_block * p.chunks + c);
                    tma_load_2d_pair(at + L.a_scales, &tmAs, full, 0, a_block * p.groups + g);
                    load_3d_pair(at + L.b_scales, &tmBs, full, 0, g, nt * 2);
                }
                ++armed;
                __syncwarp();
                if (++stage == D) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        // The copies in flight land before the CTAs can exit: the leader drains the phases it
        // armed, which take in the peer's copies; a peer that gave up allows a grace
        // period too, as its leader may not have armed a phase for them.
        if (lane == 0) {
            if (leader) {
                for (int i = 0; i < D && i < armed; ++i) {
                    if (stage == 0) {
                        stage = D - 1;
                        phase ^= 1u;
                    } else {
                        --stage;
                    }
                    wd.drain(bar(BAR_FULL + stage), phase);
                }
            } else if (!running) {
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 200000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ----------------------------------------- MMA issuer (leader)
        if (leader) {
            // (Every branch is on a vote: with one that the lanes might take apart, operands
            // count as different per lane and each MMA of nvfp4 takes 203 ns.)
            const uint32_t elected = lane == 0 ? 1u : 0u;
            const uint32_t a_sc = tmem_base + SCALE_COL;
            const uint32_t b_sc = a_sc + GROUPS * 4;
            int stage = 0;
            uint32_t phase = 0;
            int j = 0;
            bool ready = false;  // the next stage has been seen to be full
            bool running = true;
            for (int t = first; t < tiles && running; t += clusters, ++j) {
                if (j > 0) {
                    const bool drained =
                        wd.wait(bar(BAR_TMEM_EMPTY), static_cast<uint32_t>(j - 1) & 1u,
                                WAIT_TMEM_EMPTY, t, -1);
                    running = __all_sync(0xffffffffu, drained);
                }
                const uint32_t d_tmem = tmem_base + (j & 1 ? ACC_SHIFT : 0u);
                for (int s = 0; s < p.stages && running; ++s) {
                    if (!ready) {
                        const bool full = wd.wait(bar(BAR_FULL + stage), phase, WAIT_FULL, t, s);
                        running = __all_sync(0xffffffffu, full);
                        if (!running) break;
                    }
                    tc_fence_after_sync();
                    const uint32_t at = base + static_cast<uint32_t>(stage) * L.stage;
                    const uint32_t empty = bar(BAR_EMPTY + stage);
                    if (++stage == D) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    const uint64_t a_desc = core_desc(at, MX_CHUNK_BYTES);
                    const uint64_t b_desc = core_desc(at + L.b_codes, MX_CHUNK_BYTES);
                    constexpr uint64_t CHUNK = MX_CHUNK_BYTES >> 4;
                    const int rest = p.steps - s * STEPS;  // steps from this stage on
                    const uint32_t more = s == 0 ? 0u : 1u;
#pragma unroll
                    for (int g = 0; g < GROUPS; ++g) {
                        const uint32_t off = g * MX_GROUP_BYTES;
                        copy_scales<true>(elected, a_sc + g * 4, at + L.a_scales + off);
                        copy_scales<true>(elected, b_sc + g * 8, at + L.b_scales + off);
                        copy_scales<true>(elected, b_sc + g * 8 + 4,
                                          at + L.b_scales + GROUPS * MX_GROUP_BYTES + off);
                    }
                    if (rest >= STEPS) {
                        if constexpr (FORMAT == NVFP4) {
                            // 192 values as two MMAs of 96
                            constexpr uint32_t idesc =
                                mx_idesc<FORMAT>(TILE, TILE, 0) | MX_IDESC_K96;
                            mx_mma_k96_pair(elected, d_tmem, a_desc, b_desc, idesc, a_sc, b_sc,
                                            more);
                            ready = __all_sync(0xffffffffu,
                                               mbar_test(bar(BAR_FULL + stage), phase));
                            mx_mma_k96_pair(elected, d_tmem, a_desc + 3 * CHUNK, b_desc + 3 * CHUNK,
                                            idesc | mx_idesc<FORMAT>(0, 0, 2), a_sc + 4, b_sc + 8,
                                            1u);
                        } else {
#pragma unroll
                            for (int i = 0; i < STEPS; ++i) {
                                // looked at before the stage's last MMA: those that are
                                // queued cover the look
                                if (i == STEPS - 1)
                                    ready = __all_sync(0xffffffffu,
                                                       mbar_test(bar(BAR_FULL + stage), phase));
                                mx_mma<FORMAT, true>(
                                    elected, d_tmem, a_desc + i * STEP_CHUNKS * CHUNK,
                                    b_desc + i * STEP_CHUNKS * CHUNK,
                                    mx_idesc<FORMAT>(TILE, TILE, i * SCALES % 4),
                                    a_sc + i * SCALES / 4 * 4, b_sc + i * SCALES / 4 * 8,
                                    i == 0 ? more : 1u);
                            }
                        }
                    } else {
                        ready = false;
#pragma unroll
                        for (int i = 0; i < STEPS - 1; ++i) {
                            if (i >= rest) break;  // uniform
                            mx_mma<FORMAT, true>(
                                elected, d_tmem, a_desc + i * STEP_CHUNKS * CHUNK,
                                b_desc + i * STEP_CHUNKS * CHUNK,
                                mx_idesc<FORMAT>(TILE, TILE, i * SCALES % 4),
                                a_sc + i * SCALES / 4 * 4, b_sc + i * SCALES / 4 * 8,
                                i == 0 ? more : 1u);
                        }
                    }
                    mx_commit_pair(elected, empty);
                }
                if (running) mx_commit_pair(elected, bar(BAR_TMEM_FULL));
            }
            if (lane == 0) {
                mma_commit_pair_multicast(bar(BAR_DRAIN), static_cast<uint16_t>(1u));
                wd.drain(bar(BAR_DRAIN), 0);
            }
            __syncwarp();
        }
    } else {
        // -------------------------------------------------------- epilogue
        if (p.debug_stall == 2) wd.wait(bar(BAR_STALL), 0, WAIT_STALL, -1, -1);
        constexpr int READ = 64;               // columns read at a time,
        constexpr int SUB = F16OUT ? 64 : 32;  // and stored: 128 bytes
        static_assert(TILE - static_cast<int>(ACC_SHIFT) == READ, "the shared columns");
        static_assert(TILE / SUB * STAGING_BYTES <=
                          MX_PAIR_MIN_STAGES * 2 * CHUNKS * MX_CHUNK_BYTES,
                      "the last tile's buffers");
        const uint32_t q = static_cast<uint32_t>(warp & 3);
        const uint32_t row = q * 32u + lane;
        const uint32_t to_leader = map_shared_rank(bar(BAR_TMEM_EMPTY), 0);
        const float alpha = mx_alpha(p);
        int j = 0;
        uint32_t turn = 0;  // which staging buffer's
        for (int t = first; t < tiles; t += clusters, ++j) {
            int mt, nt;
            raster_tile(t, p.tiles_m, p.tiles_n, p.group_m, mt, nt);
            const bool ok =
                wd.wait(bar(BAR_TMEM_FULL), static_cast<uint32_t>(j) & 1u, WAIT_TMEM_FULL, t, -1);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after_sync();
            const uint32_t taddr = tmem_base + (j & 1 ? ACC_SHIFT : 0u) + (q * 32u << 16);
            const int m0 = mt * TILE + static_cast<int>(rank) * MX_ROWS;
            // A cluster's last tile has the stages' memory to itself, a buffer for each store
            // (its MMAs are complete, and no copy follows): no store waits for another.
            const bool last = t + clusters >= tiles;
            // the columns that the next tile's accumulator shares come first
            const int start = j & 1 ? 0 : TILE - READ;
#pragma unroll 1
            for (int i = 0; i < TILE; i += READ) {
                const int col = (start + i) % TILE;
                uint32_t v[READ];
                tmem_load_64cols(taddr + col, v);
                if (i == 0) {
                    // Relaxed: what is handed over is that the 32 lanes have read.  The loads are
                    // the warp's (.sync.aligned), its wait::ld has completed them in every
                    // lane's registers, and instructions issue in order, so lane 0 arrives
                    // behind them; the next tile's MMAs, which write what was read, come behind
                    // the issuer's wait and its fence.  Nothing written is handed over, which a
                    // release would be for (with one the next tile waited another 1200 cycles).
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(to_leader);
                }
#pragma unroll
                for (int c = 0; c < READ; ++c)
                    v[c] = __float_as_uint(__uint_as_float(v[c]) * alpha);
#pragma unroll
                for (int c = 0; c < READ; c += SUB) {
                    const int col0 = nt * TILE + col + c;
                    if (col0 >= p.N) continue;  // uniform
                    stage_one<F16OUT, STAGING>(
                        v + c, row,
                        last ? base + static_cast<uint32_t>((i + c) / SUB) * STAGING_BYTES
                             : staging + turn * STAGING_BYTES,
                        &tmC, col0, m0, p.M, !last);
                    if constexpr (STAGING > 1) turn ^= 1u;
                }
            }
        }
        if (lane == 0) bulk_wait_group<0>();
        __syncwarp();
    }

    // nothing of either CTA is touched remotely after this point
    tc_fence_before_sync();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

template <int FORMAT, int STAGING>
static cudaError_t launch_format(const MxSpec& s, cudaStream_t stream)
{
    auto kernel = s.f16out ? k_mx_pair<FORMAT, true, STAGING> : k_mx_pair<FORMAT, false, STAGING>;
    cudaError_t e = ensure_smem_limit(kernel, s.smem_bytes);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(static_cast<unsigned>(s.grid_x)), dim3(MX_THREADS),
                            s.smem_bytes, 1, stream, *s.codes_u, *s.scales_u, *s.codes_v,
                            *s.scales_v, *s.out, s.p);
}

cudaError_t launch_mx_pair(const MxSpec& s, cudaStream_t stream)
{
    switch (s.format) {
    case MXFP8: return launch_format<MXFP8, 1>(s, stream);
    case MXFP4:
        return s.staging == 2 ? launch_format<MXFP4, 2>(s, stream)
                              : launch_format<MXFP4, 1>(s, stream);
    default:
        return s.staging == 2 ? launch_format<NVFP4, 2>(s, stream)
                              : launch_format<NVFP4, 1>(s, stream);
    }
}

}  // namespace tg
