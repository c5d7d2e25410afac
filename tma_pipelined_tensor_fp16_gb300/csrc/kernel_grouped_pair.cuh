// kernel_grouped_pair.cuh -- the grouped products on CTA pairs: tiles of 256 x 256
// computed with tcgen05.mma.cta_group::2, each CTA of the pair loading its own 128
// output rows' and 128 output columns' operands and storing its own 128 rows.
// Operand forms, tile table and epilogue are those of kernel_grouped.cuh; stages
// hold two K blocks of 64 (three stages of 64 KB a CTA), as the dense pair kernel's.
//
// Why pairs: a tile of 256 columns leaves a single CTA room for four stages of 64,
// and every operand byte from L2 feeds half as many MMAs (16 experts of 4096 x 4096
// with 1024 rows each: 1564 TFLOP/s on single CTAs, 1646 on pairs; one expert of 8192
// x 8192 with 8192 rows: 1582 and 1878).  A tile of 256 rows wastes more of an
// expert's last tile, so few rows per expert stay with single CTAs (the rule and its
// figures are in grouped.cu).
//
// Measured: 16384 uneven rows, 16 experts of 4096 x 4096, 355 us, 1548 TFLOP/s; what
// is lost are the last tiles of experts, part of whose rows are the next expert's, and
// the last wave.
//
// The leader's producer takes tiles from the counter and hands them to both CTAs.
// Contraction rows past an expert's last one (GRAD_WEIGHT) have to be zeroed in
// both CTAs' shared memory: the stage that holds them signals each CTA's own tail
// barrier instead of the leader's full barrier, warp 1 of each CTA zeroes its rows,
// and the peer tells the leader.
#pragma once

#include "kernel_grouped.cuh"

namespace tg {

namespace {

constexpr int PAIR_TILE_M = 2 * BLK_M;
constexpr int PAIR_TILE_N = 256;
constexpr int PAIR_KS = 2;                       // K blocks of 64 per stage
constexpr int PAIR_STAGE_K = PAIR_KS * BLK_K;
// Readers of every tile: the leader's MMA warp and epilogue, the peer's producer,
// warp 1 and epilogue.
constexpr int PAIR_READERS = 11;
// A stage's tail barriers, in the full and empty slots past the ring's (one pair per
// stage: a stage is reused only after its MMAs, so a wait by parity meets no later
// phase, however many short tiles are loaded ahead).
constexpr int PAIR_MAX_STAGES = 4;
enum : int { BAR_TAIL = BAR_FULL + PAIR_MAX_STAGES, BAR_TAIL_READY = BAR_EMPTY + PAIR_MAX_STAGES };
static_assert(2 * PAIR_MAX_STAGES <= MAX_STAGES, "slots for the tail barriers");

// Watchdog::wait with acquire semantics over the cluster: the phase is completed by
// the other CTA, whose writes are read afterwards.  (A fence after a plain wait
// would also wait for the tensor core's queued work: 3.7 us a tile against 2.5.)
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t"
        ".reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool wait_cluster(Watchdog& wd, uint32_t bar, uint32_t parity, int where,
                                             int tile, int kb)
{
    if (wd.aborted) return false;
    if (try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t polls = 1;; ++polls) {
        if (try_wait_cluster(bar, parity)) return true;
        if ((polls & 31u) == 0) {
            if (wd.peer_aborted()) {
                wd.aborted = true;
                return false;
            }
            if (globaltimer_ns() - t0 > wd.budget_ns) {
                wd.record(where, tile, kb);
                return false;
            }
        }
    }
}

// A reader warp's next tile (as grouped_read; the slot's empty barrier is the
// leader's).  Lane 0 reads and the shuffle uses the value, so the load has returned
// when the relaxed arrival issues (an arrival with release costs 2 %: 16 experts of 4096
// x 4096 with 1024 rows each 335 and 343 us).
__device__ __forceinline__ int pair_read(uint32_t bars, int use, Watchdog& wd, uint32_t lane)
{
    const int slot = use % GROUPED_SLOTS;
    const bool ok = wait_cluster(wd, bars + (BAR_CLC_FULL + slot) * 8u,
                                 static_cast<uint32_t>(use / GROUPED_SLOTS) & 1u, WAIT_CLC_FULL,
                                 -1, use);
    if (!__all_sync(0xffffffffu, ok)) return -1;  // the warp stays together
    int u = 0;
    if (lane == 0) u = ld_shared_int(bars + CLC_RESP_OFFSET + slot * 4u);
    u = __shfl_sync(0xffffffffu, u, 0);
    if (lane == 0)
        mbar_arrive_cluster_relaxed(map_shared_rank(bars + (BAR_CLC_EMPTY + slot) * 8u, 0));
    return u;
}

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map,
                                                 uint32_t cluster_bar, int32_t x, int32_t y,
                                                 int32_t z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(cluster_bar)
        : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T over the pair, issued by the lane with `elected`
// set, as mma_elected (8192 x 8192 x 8192 as one expert: 586 us, 619 behind `if (lane
// == 0)`).
__device__ __forceinline__ void mma_pair_elected(uint32_t elected, uint32_t d_tmem, uint64_t a_desc,
                                                 uint64_t b_desc, uint32_t idesc,
                                                 uint32_t accumulate)
{
    asm volatile(
        "{\n\t"
        ".reg .pred p, q;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "setp.ne.b32 q, %4, 0;\n\t"
        "@p tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, q;\n\t"
        "}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(elected)
        : "memory");
}

// An arrival in both CTAs once the lane's MMAs so far are complete.
__device__ __forceinline__ void commit_pair_elected(uint32_t elected, uint32_t bar)
{
    asm volatile(
        "{\n\t"
        ".reg .pred p;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "@p tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster"
        ".b64 [%0], %2;\n\t"
        "}\n" ::"r"(bar),
        "r"(elected), "h"(static_cast<uint16_t>(3))
        : "memory");
}

}  // namespace

template <int OP, bool F16OUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(GROUPED_THREADS, 1)
    k_grouped_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmC, const __grid_constant__ GroupedParams p)
{
    constexpr bool A_MN = OP == GROUPED_GRAD_WEIGHT;
    constexpr bool B_MN = OP != GROUPED_FORWARD;
    constexpr int HALF_N = PAIR_TILE_N / 2;
    constexpr uint32_t TMEM_COLS = 2 * PAIR_TILE_N;
    constexpr uint32_t B_BYTES = HALF_N * BLK_K * 2;
    extern __shared__ __align__(1024) uint8_t grouped_smem[];
    const uint32_t raw = smem_u32(grouped_smem);
    const uint32_t base = align1024(raw);
    uint8_t* gen = grouped_smem + (base - raw);
    const int D = p.pipe_depth;
    const SmemLayout L = smem_layout(D * PAIR_KS, HALF_N, NUM_STAGING);
    const uint32_t sA = base + L.a;
    const uint32_t sB = base + L.b;
    const uint32_t staging = base + L.staging;
    const uint32_t bars = base + L.bars;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gen + L.bars + TMEM_SLOT_OFFSET);
    int* row0 = reinterpret_cast<int*>(gen + L.bars + BAR_AREA_BYTES);
    int* tile0 = row0 + p.experts + 2;
    const int tid = static_cast<int>(threadIdx.x);
    const int warp = tid >> 5;
    const uint32_t lane = lane_id();
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int row_shift = static_cast<int>(rank) * BLK_M;   // this CTA's rows of a tile
    const int col_shift = static_cast<int>(rank) * HALF_N;  // its columns of the B operand
    Watchdog wd;
    wd.st = p.status;
    wd.epoch = p.epoch;
    wd.budget_ns = p.budget_ns;
    wd.aborted = false;
    auto bar = [&](int slot) { return bars + static_cast<uint32_t>(slot) * 8u; };

    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
        prefetch_tensormap(&tmC);
        for (int s = 0; s < D; ++s) {
            mbar_init(bar(BAR_FULL + s), 1);        // leader: its producer
            mbar_init(bar(BAR_EMPTY + s), 1);       // the leader's multicast commit
            mbar_init(bar(BAR_TAIL + s), 1);        // this CTA's producer
            mbar_init(bar(BAR_TAIL_READY + s), 1);  // leader: the peer's warp 1
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(bar(BAR_TMEM_FULL + a), 1);   // the leader's multicast commit
            mbar_init(bar(BAR_TMEM_EMPTY + a), 8);  // leader: 4 epilogue warps x 2 CTAs
        }
        for (int j = 0; j < GROUPED_SLOTS; ++j) {
            mbar_init(bar(BAR_CLC_FULL + j), 1);
            mbar_init(bar(BAR_CLC_EMPTY + j), PAIR_READERS);
        }
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
    const uint32_t tmem_base = *tmem_slot;

    GroupedTiles<OP, PAIR_TILE_M, PAIR_TILE_N> tiles0;
    tiles0.p = &p;
    tiles0.row0 = row0;
    tiles0.tile0 = tile0;
    if constexpr (OP == GROUPED_GRAD_WEIGHT) {
        grouped_order(p, row0, tile0, tid);
        tiles0.total = p.experts * p.tiles_m * p.tiles_n;
    } else {
        grouped_table<PAIR_TILE_M>(p, row0, tile0,
                                   reinterpret_cast<int*>(gen + L.bars + CLC_RESP_OFFSET + 32),
                                   tid, lane);
        tiles0.total = tile0[p.experts + 1] * p.tiles_n;
    }
    // contraction rows of the last stage that belong to the next expert
    auto dirty_of = [&](const GroupedUnit& w) {
        return OP == GROUPED_GRAD_WEIGHT && w.klen % MMA_K != 0;
    };

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        constexpr uint32_t cta_tx = (A_TILE_BYTES + B_BYTES) * PAIR_KS;
        if (p.debug_stall == 1) wd.wait(bar(BAR_STALL), 0, WAIT_STALL, -1, -1);
        int stage = 0;
        uint32_t phase = 0;
        int armed = 0;
        uint32_t tail_bits = 0;  // phase of each stage's tail barrier
        uint32_t tails = 0;      // the stages that have had a tail
        int end_stage = 0;
        uint32_t end_phase = 0;
        GroupedUnit w;
        // The leader hands the tile after the one whose loads are being issued to
        // both CTAs before them, and has the one after that on its way from the
        // counter.
        auto take = [&] {
            return leader && lane == 0
                       ? static_cast<int>(gridDim.x / 2) + grouped_take(p.counter)
                       : 0;
        };
        auto hand_out = [&](int use, int tile) {
            const int slot = use % GROUPED_SLOTS;
            const bool free = wd.wait(bar(BAR_CLC_EMPTY + slot),
                                      (static_cast<uint32_t>(use / GROUPED_SLOTS) & 1u) ^ 1u,
                                      WAIT_CLC_EMPTY, -1, use);
            if (lane < 2 && free) {  // lane r tells the CTA of rank r
                const uint32_t to = map_shared_rank(bars + CLC_RESP_OFFSET + slot * 4u, lane);
                asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(to), "r"(tile) : "memory");
                mbar_arrive_cluster(map_shared_rank(bar(BAR_CLC_FULL + slot), lane));
            }
            __syncwarp();
        };
        int u = static_cast<int>(blockIdx.x) / 2;
        int after = take();
        if (leader)
            hand_out(0, u);
        else
            u = pair_read(bars, 0, wd, lane);
        for (int use = 1; tiles0.at(u, w); ++use) {
            const int next = __shfl_sync(0xffffffffu, after, 0);
            if (leader) {
                hand_out(use, next);  // also the first one past the end
                after = take();
            }
            if (__any_sync(0xffffffffu, wd.aborted)) break;
            const int stages = (w.klen + PAIR_STAGE_K - 1) / PAIR_STAGE_K;
            for (int ki = 0; ki < stages; ++ki) {
                const bool tail = ki == stages - 1 && dirty_of(w);
                const bool ok = wd.wait(bar(BAR_EMPTY + stage), phase ^ 1u, WAIT_EMPTY, w.n0, ki);
                if (lane == 0 && ok) {
                    uint32_t to_bar;
                    if (tail) {
                        // own bytes to the own tail barrier; the full barrier's
                        // phase passes at once
                        mbar_arrive_expect_tx(bar(BAR_TAIL + stage), cta_tx);
                        to_bar = map_shared_rank(bar(BAR_TAIL + stage), rank);
                        if (leader) mbar_arrive(bar(BAR_FULL + stage));
                        tail_bits ^= 1u << stage;
                        tails |= 1u << stage;
                    } else {
                        if (leader) mbar_arrive_expect_tx(bar(BAR_FULL + stage), 2 * cta_tx);
                        to_bar = map_shared_rank(bar(BAR_FULL + stage), 0);
                    }
                    ++armed;
#pragma unroll
                    for (int s = 0; s < PAIR_KS; ++s) {
                        const uint32_t dA = sA + (stage * PAIR_KS + s) * A_TILE_BYTES;
                        const uint32_t dB = sB + (stage * PAIR_KS + s) * B_BYTES;
                        const int k = w.k0 + ki * PAIR_STAGE_K + s * BLK_K;
                        const int m = w.m0 + row_shift, n = w.n0 + col_shift;
                        if constexpr (A_MN) {
#pragma unroll
                            for (int b = 0; b < BLK_M / 64; ++b)
                                tma_load_2d_pair(dA + b * MN_BOX_BYTES, &tmA, to_bar, m + b * 64, k);
                        } else {
                            tma_load_2d_pair(dA, &tmA, to_bar, k, m);
                        }
                        if constexpr (OP == GROUPED_FORWARD) {
                            tma_load_3d_pair(dB, &tmB, to_bar, k, n, w.expert);
                        } else {
#pragma unroll
                            for (int b = 0; b < HALF_N / 64; ++b) {
                                if constexpr (OP == GROUPED_GRAD_INPUT)
                                    tma_load_3d_pair(dB + b * MN_BOX_BYTES, &tmB, to_bar,
                                                     n + b * 64, k, w.expert);
                                else
                                    tma_load_2d_pair(dB + b * MN_BOX_BYTES, &tmB, to_bar,
                                                     n + b * 64, k);
                            }
                        }
                    }
                }
                __syncwarp();
                if (++stage == D) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (!wd.aborted) {
                    end_stage = stage;
                    end_phase = phase;
                }
            }
            u = leader ? next : pair_read(bars, use, wd, lane);
        }
        if (leader && lane == 0) grouped_finish(p.counter, gridDim.x / 2);
        // The copies in flight land before the CTAs can exit, whichever role may have
        // given up without waiting for them: the leader drains the phases it armed, which
        // take in the peer's copies, each CTA those of its tails; a peer that gave up
        // allows a grace period too, as its leader may not have armed a phase for them.
        if (lane == 0) {
            if (leader) {
                int st = end_stage;
                uint32_t ph = end_phase;
                for (int i = 0; i < D && i < armed; ++i) {
                    if (st == 0) {
                        st = D - 1;
                        ph ^= 1u;
                    } else {
                        --st;
                    }
                    wd.drain(bar(BAR_FULL + st), ph);
                }
            }
            for (int st = 0; st < D; ++st)
                if ((tails >> st) & 1u) wd.drain(bar(BAR_TAIL + st), ((tail_bits >> st) & 1u) ^ 1u);
            if (!leader && wd.aborted) {
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 200000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------- MMA issuer (leader), tail rows (both CTAs)
        constexpr uint32_t idesc = idesc_f16_f32(PAIR_TILE_M, PAIR_TILE_N) |
                                   (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
        int stage = 0;
        uint32_t phase = 0;
        constexpr uint64_t A_STEP = A_MN ? KSTEP_MNMAJOR : KSTEP_KMAJOR;
        constexpr uint64_t B_STEP = B_MN ? KSTEP_MNMAJOR : KSTEP_KMAJOR;
        const uint32_t elected = lane == 0 ? 1u : 0u;
        int acc = 0;
        uint32_t acc_phase = 0;
        uint32_t tail_bits = 0;
        GroupedUnit w;
        for (int use = 0; tiles0.at(pair_read(bars, use, wd, lane), w); ++use) {
            const int stages = (w.klen + PAIR_STAGE_K - 1) / PAIR_STAGE_K;
            if (stages == 0) continue;  // a tile of zeros has no accumulator
            const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * PAIR_TILE_N);
            if (leader) {
                wd.wait(bar(BAR_TMEM_EMPTY + acc), acc_phase ^ 1u, WAIT_TMEM_EMPTY, w.n0, -1);
                tc_fence_after_sync();
            }
            for (int ki = 0; ki < stages; ++ki) {
                const int left = w.klen - ki * PAIR_STAGE_K;  // contraction from this stage on
                const bool tail = ki == stages - 1 && dirty_of(w);
                bool ok = !wd.aborted;
                if (leader) ok = wd.wait(bar(BAR_FULL + stage), phase, WAIT_FULL, w.n0, ki);
                if (tail) {
                    const uint32_t tail_phase = (tail_bits >> stage) & 1u;
                    ok = wd.wait(bar(BAR_TAIL + stage), tail_phase, WAIT_FULL, w.n0, ki);
                    if (ok) {
                        // lines left .. of the last slice, in every box of this CTA
                        constexpr int BOXES = (BLK_M + HALF_N) / 64;
                        const int s = left > BLK_K ? 1 : 0;
                        const int first = left - s * BLK_K;
                        const int dirty = (MMA_K - first % MMA_K) % MMA_K;
                        const uint32_t a = sA + (stage * PAIR_KS + s) * A_TILE_BYTES;
                        const uint32_t b = sB + (stage * PAIR_KS + s) * B_BYTES;
                        for (int i = static_cast<int>(lane); i < dirty * BOXES * 8; i += 32) {
                            const int box = i / (dirty * 8);
                            const int line = first + (i / 8) % dirty;
                            const uint32_t to = (box < BLK_M / 64
                                                     ? a + box * MN_BOX_BYTES
                                                     : b + (box - BLK_M / 64) * MN_BOX_BYTES) +
                                                line * 128u + (i % 8) * 16u;
                            st_shared_v4(to, 0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (leader)
                        ok = wait_cluster(wd, bar(BAR_TAIL_READY + stage), tail_phase, WAIT_FULL,
                                          w.n0, ki);
                    else if (lane == 0 && ok)
                        mbar_arrive_cluster(map_shared_rank(bar(BAR_TAIL_READY + stage), 0));
                    tail_bits ^= 1u << stage;
                }
                if (leader && __all_sync(0xffffffffu, ok)) {
                    tc_fence_after_sync();
                    const uint32_t a = sA + stage * PAIR_KS * A_TILE_BYTES;
                    const uint32_t b = sB + stage * PAIR_KS * B_BYTES;
                    auto issue = [&](int i) {  // slice i of the stage
                        const int s = i / (BLK_K / MMA_K), kk = i % (BLK_K / MMA_K);
                        const uint32_t as = a + s * A_TILE_BYTES, bs = b + s * B_BYTES;
                        mma_pair_elected(
                            elected, d_tmem,
                            (A_MN ? sw128_mnmajor_desc(as) : sw128_kmajor_desc(as)) + kk * A_STEP,
                            (B_MN ? sw128_mnmajor_desc(bs) : sw128_kmajor_desc(bs)) + kk * B_STEP,
                            idesc, i == 0 && ki == 0 ? 0u : 1u);
                    };
                    if (left >= PAIR_STAGE_K) {
#pragma unroll
                        for (int i = 0; i < PAIR_STAGE_K / MMA_K; ++i) issue(i);
                    } else {
                        for (int i = 0; i * MMA_K < left; ++i) issue(i);
                    }
                    commit_pair_elected(elected, bar(BAR_EMPTY + stage));
                }
                __syncwarp();
                if (++stage == D) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (leader && __all_sync(0xffffffffu, !wd.aborted))
                commit_pair_elected(elected, bar(BAR_TMEM_FULL + acc));
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
        if (leader && lane == 0) {
            mma_commit_pair_multicast(bar(BAR_DRAIN), static_cast<uint16_t>(1u));
            wd.drain(bar(BAR_DRAIN), 0);
        }
        __syncwarp();
    } else {
        // -------------------------------------------------------- epilogue
        if (p.debug_stall == 2) wd.wait(bar(BAR_STALL), 0, WAIT_STALL, -1, -1);
        const int q = warp & 3;
        int acc = 0;
        uint32_t acc_phase = 0;
        uint32_t sub_count = 0;
        GroupedUnit w;
        for (int use = 0; tiles0.at(pair_read(bars, use, wd, lane), w); ++use) {
            const bool zero = w.klen == 0;
            if (!zero) {
                wd.wait(bar(BAR_TMEM_FULL + acc), acc_phase, WAIT_TMEM_FULL, w.n0, -1);
                tc_fence_after_sync();
            }
            w.m0 += row_shift;
            store_tile<OP, PAIR_TILE_N, F16OUT>(
                tmem_base + static_cast<uint32_t>(acc * PAIR_TILE_N), zero, q, lane, staging, &tmC,
                p, w, sub_count, !wd.aborted);
            if (!zero) {
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster(map_shared_rank(bar(BAR_TMEM_EMPTY + acc), 0));
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
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

template <int OP>
cudaError_t launch_grouped_pair(const GroupedSpec& s, cudaStream_t stream)
{
    auto kernel = s.f16out ? k_grouped_pair<OP, true> : k_grouped_pair<OP, false>;
    cudaError_t e = ensure_smem_limit(kernel, s.smem_bytes);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(static_cast<unsigned>(s.grid)), dim3(GROUPED_THREADS),
                            s.smem_bytes, 1, stream, *s.tmA, *s.tmB, *s.tmC, s.p);
}

extern template cudaError_t launch_grouped_pair<GROUPED_FORWARD>(const GroupedSpec&, cudaStream_t);
extern template cudaError_t launch_grouped_pair<GROUPED_GRAD_INPUT>(const GroupedSpec&,
                                                                   cudaStream_t);
extern template cudaError_t launch_grouped_pair<GROUPED_GRAD_WEIGHT>(const GroupedSpec&,
                                                                    cudaStream_t);

}  // namespace tg
