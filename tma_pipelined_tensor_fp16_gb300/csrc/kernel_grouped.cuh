// kernel_grouped.cuh -- the experts' grouped products, one kernel in three
// forms.  Rows of A and C are sorted by expert; expert e owns rows
// [offsets[e], offsets[e+1]) and a weight B[e] of N x K:
//
//   FORWARD      C[r]  = A[r] . B[e]^T     contraction over K
//   GRAD_INPUT   dA[r] = dC[r] . B[e]      contraction over N
//   GRAD_WEIGHT  dB[e] = dC_e^T . A_e      contraction over the expert's rows
//
// Each is D = P . Q^T on tiles of 128 x BN with one tcgen05.mma chain per tile.
// The tensor core reads an operand either with the contraction index running
// along its rows' memory ("K-major") or across it ("MN-major"), so no operand
// is transposed in memory: FORWARD reads both K-major, GRAD_INPUT reads B[e]
// MN-major, GRAD_WEIGHT reads both MN-major.  A K-major tile of one stage is
// rows x 64 halves, one 128-byte swizzled line per row.  An MN-major tile is a
// row of boxes, each 64 contraction rows x 64 columns (128-byte lines again).
//
// The split of the rows over the experts is data: it is read from `offsets` on
// the device.  Every CTA builds the prefix sum of the experts' row tiles in
// shared memory, so no host copy of the counts and no padding of the rows is
// needed.  A tile's cost depends on its expert (GRAD_WEIGHT contracts over the
// expert's rows), so tiles are handed out while the kernel runs: a CTA starts on
// tile blockIdx.x and takes the next ones from a counter, which the last CTA to
// finish sets back to zero.  Which CTA computes a tile varies, its sum does not.
//   * A row tile that reaches past its expert's last row multiplies the next
//     expert's rows too, or what was there before, and does not store them.
//   * Rows from offsets[experts] on form a last group without products: its
//     tiles store zeros.  So do GRAD_WEIGHT's tiles of an expert without rows.
//   * GRAD_WEIGHT's last stage of an expert may hold rows of the next one: the
//     MMA warp overwrites them with zeros in both operands (an infinity there
//     must not meet a zero) and skips the MMAs past the last row.
//
// Roles per CTA (192 threads) as in the persistent GEMM: warp 0 TMA producer,
// warp 1 MMA issuer, warps 2..5 epilogue; two TMEM accumulators, so a tile's
// epilogue overlaps the next tile's main loop.
#pragma once

#include "device_common.cuh"
#include "grouped.h"
#include "launch.h"
#include "runtime.h"

namespace tg {

namespace {

// Box (64 x rows x 1) of a 3-D tensor map, completing on `bar`.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t x, int32_t y, int32_t z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int32_t x,
                                             int32_t y, int32_t z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::
            "l"(reinterpret_cast<uint64_t>(map)),
        "r"(x), "r"(y), "r"(z), "r"(src)
        : "memory");
}

// Shared-memory descriptor of an MN-major operand stored as boxes of 64
// contraction rows x 64 columns with the 128-byte swizzle: the next 64 columns
// (leading dimension) start one box (8 KB) on, the next 8 contraction rows
// (stride dimension) 1 KB on.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>((64 * 128) >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

constexpr uint32_t MN_BOX_BYTES = 64 * 128;
// Descriptor steps (16-byte units) from one MMA_K slice to the next.
constexpr uint64_t KSTEP_KMAJOR = MMA_K * 2 / 16;
constexpr uint64_t KSTEP_MNMAJOR = MMA_K * 128 / 16;

struct GroupedUnit {
    int expert;   // = experts for the rows that belong to none
    int m0;       // first output row (global row; GRAD_WEIGHT: row within dB[e])
    int row_end;  // output rows at or past this are not stored
    int n0;       // first output column
    int k0;       // GRAD_WEIGHT: first contraction row
    int klen;     // contraction length; 0: the tile is zero
};

__device__ __forceinline__ int clamp_row(int r, int rows) { return r < 0 ? 0 : (r > rows ? rows : r); }

// Tiles handed from the producer warp to the others through a ring in shared
// memory: GROUPED_SLOTS words, each with a full and an empty barrier.
constexpr int GROUPED_SLOTS = 4;
constexpr int GROUPED_READERS = 5;  // the MMA warp and the four epilogue warps

__device__ __forceinline__ int ld_shared_int(uint32_t addr)
{
    int v;
    asm volatile("ld.shared.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void st_shared_int(uint32_t addr, int v)
{
    asm volatile("st.shared.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// A reader warp's next tile, or -1 when there is none (or the run is abandoned).
__device__ __forceinline__ int grouped_read(uint32_t bars, int use, Watchdog& wd, uint32_t lane)
{
    const int slot = use % GROUPED_SLOTS;
    const bool ok = wd.wait(bars + (BAR_CLC_FULL + slot) * 8u,
                            static_cast<uint32_t>(use / GROUPED_SLOTS) & 1u, WAIT_CLC_FULL, -1, use);
    if (!__all_sync(0xffffffffu, ok)) return -1;  // the warp stays together
    const int u = ld_shared_int(bars + CLC_RESP_OFFSET + slot * 4u);
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + (BAR_CLC_EMPTY + slot) * 8u);
    return u;
}

// Decoding of a tile number.
template <int OP, int BM, int BN>
struct GroupedTiles {
    const GroupedParams* p;
    const int* row0;   // [experts + 2] first row of a group; the end
    const int* tile0;  // [experts + 2] first row tile of a group; the end
                       // (GRAD_WEIGHT: the experts in the order of their turns)
    int total;         // tiles

    __device__ __forceinline__ bool at(int u, GroupedUnit& w) const
    {
        if (u < 0 || u >= total) return false;
        int l, tm;
        if constexpr (OP == GROUPED_GRAD_WEIGHT) {
            const int per = p->tiles_m * p->tiles_n;
            const int turn = u / per;
            w.expert = p->experts <= GROUPED_SORT_EXPERTS ? tile0[turn] : turn;
            l = u - turn * per;
            tm = p->tiles_m;
        } else {
            // last group whose first unit is at or before u (empty groups in
            // between start at the same unit and are passed over)
            int lo = 0, hi = p->experts + 1;
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (tile0[mid] * p->tiles_n <= u)
                    lo = mid;
                else
                    hi = mid;
            }
            w.expert = lo;
            l = u - tile0[lo] * p->tiles_n;
            tm = tile0[lo + 1] - tile0[lo];
        }
        int mt, nt;
        raster_tile(l, tm, p->tiles_n, p->group_m, mt, nt);
        w.n0 = nt * BN;
        if constexpr (OP == GROUPED_GRAD_WEIGHT) {
            w.m0 = mt * BM;
            w.row_end = p->out_rows;
            const int* from = p->experts <= GROUPED_SORT_EXPERTS ? row0 : p->offsets;
            w.k0 = clamp_row(from[w.expert], p->rows);
            w.klen = clamp_row(from[w.expert + 1], p->rows) - w.k0;
            if (w.klen < 0) w.klen = 0;
        } else {
            w.m0 = row0[w.expert] + mt * BM;
            w.row_end = row0[w.expert + 1];
            w.k0 = 0;
            w.klen = w.expert < p->experts ? p->depth : 0;
        }
        return true;
    }
};

// The run's counter: tiles taken beyond each worker's first one in the lower half,
// workers that have finished in the upper half.  Both halves are one word on
// purpose: a worker's operations on one address take effect in program order, on
// two they need not, and a tile counted after the last worker has set the counter
// back would be missing from the next run.
__device__ __forceinline__ int grouped_take(unsigned long long* counter)
{
    return static_cast<int>(static_cast<unsigned>(atomicAdd(counter, 1ull)));
}

// A worker takes no more; the last one sets the counter back.
__device__ __forceinline__ void grouped_finish(unsigned long long* counter, unsigned workers)
{
    if (atomicAdd(counter, 1ull << 32) >> 32 == workers - 1) atomicExch(counter, 0ull);
}

// GRAD_WEIGHT: the experts with the most rows, whose tiles take longest, come
// first, so that the last tiles of a launch are short ones.
__device__ __forceinline__ void grouped_order(const GroupedParams& p, int* row0, int* order, int tid)
{
    if (p.experts > GROUPED_SORT_EXPERTS) return;
    for (int e = tid; e <= p.experts; e += GROUPED_THREADS) row0[e] = clamp_row(p.offsets[e], p.rows);
    __syncthreads();
    for (int e = tid; e < p.experts; e += GROUPED_THREADS) {
        const int n = row0[e + 1] - row0[e];
        int rank = 0;
        for (int o = 0; o < p.experts; ++o) {
            const int m = row0[o + 1] - row0[o];
            rank += m > n || (m == n && o < e) ? 1 : 0;
        }
        order[rank] = e;
    }
    __syncthreads();
}

// First row and first tile of BM rows of the experts and of the rest, by all
// threads of the CTA: each sums a contiguous share of the groups, the shares are
// scanned.  `warp_tiles` is scratch for one word per warp.  The experts of a table that
// descends could overlap, and their tiles together pass what the plan has counted on
// (and 32 bits), so such a table gives every row to none.
template <int BM>
__device__ __forceinline__ void grouped_table(const GroupedParams& p, int* row0, int* tile0,
                                              int* warp_tiles, int tid, uint32_t lane)
{
    const int warp = tid >> 5;
    const int groups = p.experts + 1;
    const int share = (groups + GROUPED_THREADS - 1) / GROUPED_THREADS;
    const int g0 = tid * share;
    auto start = [&](int g) { return g <= p.experts ? clamp_row(p.offsets[g], p.rows) : p.rows; };
    int sum = 0;
    bool descends = false;
    for (int i = 0; i < share && g0 + i < groups; ++i) {
        const int a = start(g0 + i), b = start(g0 + i + 1);
        sum += b > a ? (b - a + BM - 1) / BM : 0;
        descends |= b < a;
    }
    descends = __syncthreads_or(descends);
    int scan = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= static_cast<uint32_t>(d)) scan += v;
    }
    if (lane == 31) warp_tiles[warp] = scan;
    __syncthreads();
    int at = scan - sum;
    for (int w = 0; w < warp; ++w) at += warp_tiles[w];
    for (int i = 0; i < share && g0 + i < groups; ++i) {
        const int a = start(g0 + i), b = start(g0 + i + 1);
        row0[g0 + i] = descends ? 0 : a;
        tile0[g0 + i] = descends ? 0 : at;
        at += b > a ? (b - a + BM - 1) / BM : 0;
        if (g0 + i == groups - 1) {
            row0[groups] = p.rows;
            tile0[groups] = descends ? (p.rows + BM - 1) / BM : at;
        }
    }
    __syncthreads();
}

// One 128-byte-wide sub-tile of the output: each warp stages its 32 rows
// (swizzled) and stores them with one bulk tensor store, or, where only the
// first `valid` of them belong to the tile's expert, row by row.  Every call
// commits one bulk group (possibly empty), which keeps the count of groups in
// step with the two staging buffers.
template <int OP, bool F16OUT>
__device__ __forceinline__ void store_sub_tile(const uint32_t* v, int q, uint32_t lane,
                                               uint32_t staging, const CUtensorMap* tmC,
                                               const GroupedParams& p, const GroupedUnit& w,
                                               int col0, uint32_t& sub_count, bool do_store)
{
    const uint32_t buf = staging + static_cast<uint32_t>(q) * (2u * WARP_STAGING_BYTES) +
                         (sub_count & 1u) * WARP_STAGING_BYTES;
    if (sub_count >= 2) {
        if (lane == 0) bulk_wait_group_read<1>();
        __syncwarp();
    }
    const uint32_t row_base = buf + lane * 128u;
#pragma unroll
    for (uint32_t c = 0; c < 8; ++c) {
        const uint32_t dst = row_base + ((c ^ (lane & 7u)) << 4);
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
    const int wm0 = w.m0 + q * 32;
    const int valid = w.row_end - wm0;
    const bool whole = OP == GROUPED_GRAD_WEIGHT ? valid > 0 : valid >= 32;
    if (do_store && whole) {
        if (lane == 0) {
            if constexpr (OP == GROUPED_GRAD_WEIGHT)
                tma_store_3d(tmC, buf, col0, wm0, w.expert);  // clipped at the expert's last row
            else
                tma_store_2d(tmC, buf, col0, wm0);
        }
    } else if (do_store && valid > 0) {
        constexpr int ELT = F16OUT ? 2 : 4;
        const int chunk = static_cast<int>(lane & 7u);
        const int col = col0 + chunk * (16 / ELT);
        char* out = static_cast<char*>(p.out);
        for (int r = static_cast<int>(lane >> 3); r < valid; r += 4) {
            uint32_t a, b, c, d;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
                         : "r"(buf + r * 128u + ((chunk ^ (r & 7)) << 4))
                         : "memory");
            if (col < p.out_cols)
                *reinterpret_cast<uint4*>(
                    out + (static_cast<size_t>(wm0 + r) * p.out_cols + col) * ELT) =
                    make_uint4(a, b, c, d);
        }
        __syncwarp();
    }
    if (lane == 0) bulk_commit_group();
    ++sub_count;
}

// A 128 x BN accumulator (or zeros) to the output, sub-tile by sub-tile.
template <int OP, int BN, bool F16OUT>
__device__ __forceinline__ void store_tile(uint32_t tmem_acc, bool zero, int q, uint32_t lane,
                                           uint32_t staging, const CUtensorMap* tmC,
                                           const GroupedParams& p, const GroupedUnit& w,
                                           uint32_t& sub_count, bool do_store)
{
    constexpr int SUB_COLS = F16OUT ? 64 : 32;
    const uint32_t taddr = tmem_acc + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
    for (int j = 0; j < BN / SUB_COLS; ++j) {
        const int col0 = w.n0 + j * SUB_COLS;
        if (col0 >= p.out_cols) break;
        uint32_t v[SUB_COLS];
        if (zero) {
#pragma unroll
            for (int i = 0; i < SUB_COLS; ++i) v[i] = 0u;
        } else if constexpr (F16OUT) {
            tmem_load_32cols(taddr + j * 64, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
            tmem_load_32cols(taddr + j * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
        } else {
            tmem_load_32cols(taddr + j * 32, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
        }
        store_sub_tile<OP, F16OUT>(v, q, lane, staging, tmC, p, w, col0, sub_count, do_store);
    }
}

// D[tmem] (+)= A[smem] * B[smem]^T, issued by the lane with `elected` set.  The whole
// warp executes the statement: without a branch around it the operands stay in
// uniform registers (16 experts of 4096 x 4096 with 1024 rows each: 460 us on tiles of
// 128 x 128 and 348 on 128 x 256; 628 and 362 behind `if (lane == 0)`).
__device__ __forceinline__ void mma_elected(uint32_t elected, uint32_t d_tmem, uint64_t a_desc,
                                            uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t"
        ".reg .pred p, q;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "setp.ne.b32 q, %4, 0;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, q;\n\t"
        "}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(elected)
        : "memory");
}

__device__ __forceinline__ void commit_elected(uint32_t elected, uint32_t bar)
{
    asm volatile(
        "{\n\t"
        ".reg .pred p;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t"
        "}\n" ::"r"(bar),
        "r"(elected)
        : "memory");
}

}  // namespace

template <int OP, int BN, bool F16OUT>
__global__ void __launch_bounds__(GROUPED_THREADS, 1)
    k_grouped(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmS,
              const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmC,
              const __grid_constant__ GroupedParams p)
{
    constexpr bool A_MN = OP == GROUPED_GRAD_WEIGHT;
    constexpr bool B_MN = OP != GROUPED_FORWARD;
    constexpr uint32_t TMEM_COLS = 2 * BN;
    constexpr uint32_t B_BYTES = BN * BLK_K * 2;
    extern __shared__ __align__(1024) uint8_t grouped_smem[];
    const uint32_t raw = smem_u32(grouped_smem);
    const uint32_t base = align1024(raw);
    uint8_t* gen = grouped_smem + (base - raw);
    const int D = p.pipe_depth;
    const SmemLayout L = smem_layout(D, BN, NUM_STAGING);
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
    Watchdog wd;
    wd.st = p.status;
    wd.epoch = p.epoch;
    wd.budget_ns = p.budget_ns;
    wd.aborted = false;
    auto bar = [&](int slot) { return bars + static_cast<uint32_t>(slot) * 8u; };

    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmA);
        if (OP != GROUPED_GRAD_WEIGHT) prefetch_tensormap(&tmS);
        prefetch_tensormap(&tmB);
        prefetch_tensormap(&tmC);
        for (int s = 0; s < D; ++s) {
            mbar_init(bar(BAR_FULL + s), 1);
            mbar_init(bar(BAR_EMPTY + s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(bar(BAR_TMEM_FULL + a), 1);
            mbar_init(bar(BAR_TMEM_EMPTY + a), 128);
        }
        for (int j = 0; j < GROUPED_SLOTS; ++j) {
            mbar_init(bar(BAR_CLC_FULL + j), 1);
            mbar_init(bar(BAR_CLC_EMPTY + j), GROUPED_READERS);
        }
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
    const uint32_t tmem_base = *tmem_slot;

    GroupedTiles<OP, BLK_M, BN> tiles0;
    tiles0.p = &p;
    tiles0.row0 = row0;
    tiles0.tile0 = tile0;
    if constexpr (OP == GROUPED_GRAD_WEIGHT) {
        grouped_order(p, row0, tile0, tid);
        tiles0.total = p.experts * p.tiles_m * p.tiles_n;
    } else {
        grouped_table<BLK_M>(p, row0, tile0,
                             reinterpret_cast<int*>(gen + L.bars + CLC_RESP_OFFSET + 32), tid,
                             lane);
        tiles0.total = tile0[p.experts + 1] * p.tiles_n;
    }

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        constexpr uint32_t SMALL_BYTES = GROUPED_SMALL_ROWS * 128;
        if (p.debug_stall == 1) wd.wait(bar(BAR_STALL), 0, WAIT_STALL, -1, -1);
        int stage = 0;
        uint32_t phase = 0;
        int issued = 0;
        int end_stage = 0;
        uint32_t end_phase = 0;
        GroupedUnit w;
        // The tile after the one whose loads are being issued is handed out
        // before them, and the one after that is on its way from the counter.
        auto take = [&] {
            return lane == 0 ? static_cast<int>(gridDim.x) + grouped_take(p.counter) : 0;
        };
        auto hand_out = [&](int use, int u) {
            const int slot = use % GROUPED_SLOTS;
            const bool free = wd.wait(bar(BAR_CLC_EMPTY + slot),
                                      (static_cast<uint32_t>(use / GROUPED_SLOTS) & 1u) ^ 1u,
                                      WAIT_CLC_EMPTY, -1, use);
            if (lane == 0 && free) {
                st_shared_int(bars + CLC_RESP_OFFSET + slot * 4u, u);
                mbar_arrive(bar(BAR_CLC_FULL + slot));
            }
            __syncwarp();
        };
        int u = static_cast<int>(blockIdx.x);
        int after = take();
        hand_out(0, u);
        for (int use = 1; tiles0.at(u, w); ++use) {
            const int next = __shfl_sync(0xffffffffu, after, 0);
            hand_out(use, next);  // also the first one past the end
            if (__any_sync(0xffffffffu, wd.aborted)) break;
            after = take();
            const int kb_count = (w.klen + BLK_K - 1) / BLK_K;
            // Small boxes for the tile's rows where they do not fill it; the rest of the
            // A tile keeps what it had, in rows that are not stored.  (40 experts with 19
            // rows on average, rows off 128-byte lines, where each costs L2 two requests:
            // 48.2 us, 51.8 with whole boxes; on lines 45.8 both.)
            constexpr int WHOLE = BLK_M / GROUPED_SMALL_ROWS;
            int small = WHOLE;
            if (OP != GROUPED_GRAD_WEIGHT && w.row_end - w.m0 < BLK_M)
                small = (w.row_end - w.m0 + GROUPED_SMALL_ROWS - 1) / GROUPED_SMALL_ROWS;
            const uint32_t tx =
                B_BYTES + static_cast<uint32_t>(small) * SMALL_BYTES;
            for (int kb = 0; kb < kb_count; ++kb) {
                const bool ok = wd.wait(bar(BAR_EMPTY + stage), phase ^ 1u, WAIT_EMPTY, w.n0, kb);
                if (lane == 0 && ok) {
                    const uint32_t fb = bar(BAR_FULL + stage);
                    mbar_arrive_expect_tx(fb, tx);
                    const uint32_t dA = sA + stage * A_TILE_BYTES;
                    const uint32_t dB = sB + stage * B_BYTES;
                    const int k = w.k0 + kb * BLK_K;
                    if constexpr (A_MN) {
#pragma unroll
                        for (int b = 0; b < BLK_M / 64; ++b)
                            tma_load_2d(dA + b * MN_BOX_BYTES, &tmA, fb, w.m0 + b * 64, k);
                    } else if (small < WHOLE) {
                        for (int b = 0; b < small; ++b)
                            tma_load_2d(dA + b * SMALL_BYTES, &tmS, fb, k,
                                        w.m0 + b * GROUPED_SMALL_ROWS);
                    } else {
                        tma_load_2d(dA, &tmA, fb, k, w.m0);
                    }
                    if constexpr (OP == GROUPED_FORWARD) {
                        tma_load_3d(dB, &tmB, fb, k, w.n0, w.expert);
                    } else {
#pragma unroll
                        for (int b = 0; b < BN / 64; ++b) {
                            if constexpr (OP == GROUPED_GRAD_INPUT)
                                tma_load_3d(dB + b * MN_BOX_BYTES, &tmB, fb, w.n0 + b * 64, k,
                                            w.expert);
                            else
                                tma_load_2d(dB + b * MN_BOX_BYTES, &tmB, fb, w.n0 + b * 64, k);
                        }
                    }
                    ++issued;
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
            u = next;
        }
        if (lane == 0) grouped_finish(p.counter, gridDim.x);
        // the last min(D, issued) loads land before the CTA exits, whichever role may have
        // given up without waiting for them
        if (lane == 0) {
            int st = end_stage;
            uint32_t ph = end_phase;
            for (int i = 0; i < D && i < issued; ++i) {
                if (st == 0) {
                    st = D - 1;
                    ph ^= 1u;
                } else {
                    --st;
                }
                wd.drain(bar(BAR_FULL + st), ph);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------- MMA issuer
        constexpr uint32_t idesc = idesc_f16_f32(BLK_M, BN) | (A_MN ? 1u << 15 : 0u) |
                                   (B_MN ? 1u << 16 : 0u);
        const uint32_t elected = lane == 0 ? 1u : 0u;
        int stage = 0;
        uint32_t phase = 0;
        int acc = 0;
        uint32_t acc_phase = 0;
        GroupedUnit w;
        for (int use = 0; tiles0.at(grouped_read(bars, use, wd, lane), w); ++use) {
            const int kb_count = (w.klen + BLK_K - 1) / BLK_K;
            if (kb_count == 0) continue;  // a tile of zeros has no accumulator
            wd.wait(bar(BAR_TMEM_EMPTY + acc), acc_phase ^ 1u, WAIT_TMEM_EMPTY, w.n0, -1);
            tc_fence_after_sync();
            const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
            for (int kb = 0; kb < kb_count; ++kb) {
                const bool ok = wd.wait(bar(BAR_FULL + stage), phase, WAIT_FULL, w.n0, kb);
                const int left = w.klen - kb * BLK_K;
                const int slices = left >= BLK_K ? BLK_K / MMA_K : (left + MMA_K - 1) / MMA_K;
                const uint32_t a = sA + stage * A_TILE_BYTES;
                const uint32_t b = sB + stage * B_BYTES;
                if constexpr (OP == GROUPED_GRAD_WEIGHT) {
                    // contraction rows past the expert's last one, up to the
                    // end of the last slice: one 128-byte line per row and box
                    const int dirty = slices * MMA_K - left;
                    if (ok && dirty > 0) {
                        constexpr int BOXES = (BLK_M + BN) / 64;
                        for (int i = static_cast<int>(lane); i < dirty * BOXES * 8; i += 32) {
                            const int box = i / (dirty * 8);
                            const int line = left + (i / 8) % dirty;
                            const uint32_t to = (box < BLK_M / 64
                                                     ? a + box * MN_BOX_BYTES
                                                     : b + (box - BLK_M / 64) * MN_BOX_BYTES) +
                                                line * 128u + (i % 8) * 16u;
                            st_shared_v4(to, 0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
                if (__all_sync(0xffffffffu, ok)) {
                    tc_fence_after_sync();
                    const uint64_t adesc = A_MN ? sw128_mnmajor_desc(a) : sw128_kmajor_desc(a);
                    const uint64_t bdesc = B_MN ? sw128_mnmajor_desc(b) : sw128_kmajor_desc(b);
                    auto issue = [&](int kk) {
                        mma_elected(elected, d_tmem,
                                    adesc + static_cast<uint64_t>(kk) *
                                                (A_MN ? KSTEP_MNMAJOR : KSTEP_KMAJOR),
                                    bdesc + static_cast<uint64_t>(kk) *
                                                (B_MN ? KSTEP_MNMAJOR : KSTEP_KMAJOR),
                                    idesc, (kb == 0 && kk == 0) ? 0u : 1u);
                    };
                    if (left >= BLK_K) {
#pragma unroll
                        for (int kk = 0; kk < BLK_K / MMA_K; ++kk) issue(kk);
                    } else {
                        for (int kk = 0; kk < slices; ++kk) issue(kk);
                    }
                    commit_elected(elected, bar(BAR_EMPTY + stage));
                }
                __syncwarp();
                if (++stage == D) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (__all_sync(0xffffffffu, !wd.aborted)) commit_elected(elected, bar(BAR_TMEM_FULL + acc));
            __syncwarp();
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
        if (lane == 0) {
            mma_commit(bar(BAR_DRAIN));
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
        for (int use = 0; tiles0.at(grouped_read(bars, use, wd, lane), w); ++use) {
            const bool zero = w.klen == 0;
            if (!zero) {
                wd.wait(bar(BAR_TMEM_FULL + acc), acc_phase, WAIT_TMEM_FULL, w.n0, -1);
                tc_fence_after_sync();
            }
            store_tile<OP, BN, F16OUT>(tmem_base + static_cast<uint32_t>(acc * BN), zero, q, lane,
                                       staging, &tmC, p, w, sub_count, !wd.aborted);
            if (!zero) {
                tc_fence_before_sync();
                mbar_arrive(bar(BAR_TMEM_EMPTY + acc));
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            }
        }
        if (lane == 0) bulk_wait_group<0>();
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

template <int OP>
cudaError_t launch_grouped_pair(const GroupedSpec& s, cudaStream_t stream);

// Launch one of the built tile widths of form OP; each form is instantiated by
// a translation unit of its own, so that they compile in parallel.
template <int OP>
cudaError_t launch_grouped_op(const GroupedSpec& s, cudaStream_t stream)
{
    if (s.pair) return launch_grouped_pair<OP>(s, stream);
    auto kernel = s.block_n == 256
                      ? (s.f16out ? k_grouped<OP, 256, true> : k_grouped<OP, 256, false>)
                      : (s.f16out ? k_grouped<OP, 128, true> : k_grouped<OP, 128, false>);
    cudaError_t e = ensure_smem_limit(kernel, s.smem_bytes);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(static_cast<unsigned>(s.grid)), dim3(GROUPED_THREADS),
                            s.smem_bytes, 1, stream, *s.tmA, *s.tmS, *s.tmB, *s.tmC, s.p);
}

extern template cudaError_t launch_grouped_op<GROUPED_FORWARD>(const GroupedSpec&, cudaStream_t);
extern template cudaError_t launch_grouped_op<GROUPED_GRAD_INPUT>(const GroupedSpec&,
                                                                 cudaStream_t);
extern template cudaError_t launch_grouped_op<GROUPED_GRAD_WEIGHT>(const GroupedSpec&,
                                                                  cudaStream_t);

}  // namespace tg
