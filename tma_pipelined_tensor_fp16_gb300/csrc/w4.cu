// w4.cu -- products with 4-bit weights and group scales,
//
//     Y[m][n] = sum_g scale[n][g] * sum_{k in g} (q[n][k] - zero[n][g]) X[m][k],
//
// for a few rows of X (decoding), and the expansion of the weights to pairs of fp16
// numbers for many rows.
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdio>
#include <new>
#include <type_traits>

#include "../../include/tmaexperts.h"
#include "device_common.cuh"
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
    int tile_rows;         // rows of the weights per CTA (a multiple of 8, up to 128)
    int wide_scales;       // a stage's scales and zeros of a row are aligned vectors
    const int* verdicts;   // 64 columns; not nullptr: run only if one of them is not zero
    int verdict_count;
    DevStatus* status;
    int epoch;
    unsigned long long budget_ns;
    int debug_stall;  // 1: the loaders, 2: the sums wait on a barrier nothing completes
};

// ---------------------------------------------------------------- few rows
//
// Blocks of up to 64 rows of X, bound by reading the codes once.  The product runs on
// tcgen05.mma with 128 rows of the weights as the M side and the rows of X as
// the N side (16, 32 or 64).  Without experts grid.y is the block.
//
// A 32-bit word holds the codes k..k+7.  Masking the word and its shift by 8
// with 0x000f000f and 0x00f000f0 and setting the exponent of 1024 (whose unit in
// the last place is one: a common way to make floats of small integers) gives half
// pairs (k, k+4), (k+1, k+5), (k+2, k+6), (k+3, k+7) of 1024 + q or 1024 + 16 q;
// one half2 add or fused multiply-add makes them q - zero, exact in fp16.  The
// operand keeps that order, and X is stored with the same order inside each 8.
//
// No weight is rounded: the tensor core sums whole q - zero of one group into
// an accumulator of its own, and the group's sum enters the row's sum times its
// scale in fp32.
//
// The converted weights are the MMA's A operand in TMEM: a lane holds a row, so
// a worker thread converts 128 codes of its row in registers and stores them
// with tcgen05.st, and shared memory is left to the codes in flight.
//
// Bound on paper by reading the codes, in fact by the instructions of the warps that
// convert and add up (about 3100 a stage and CTA, half of them the conversion and its
// stores to TMEM; 2.6 instructions a cycle over a whole launch, DRAM 41 % used).  One
// row of 16384 x 16384, groups of 128: 38.2 us, 3.6 TB/s, 31 without the conversion; 32
// slots of 64 experts of 2048 x 4096: 32.1 us; 64 rows of 8192 x 4096, groups of 32:
// 18.1 us.
//
// Roles of a CTA, joined by mbarriers only:
//   warps 0..7    workers, two teams of four warps; warp w owns rows
//                 32 (w % 4) .. + 31 of the tile.  The teams take alternate
//                 stages of 256 codes; a team converts a stage's two blocks of
//                 128 codes one after the other into the next of A_BUFS operands
//                 each and, up to 16 rows, copies the block's part of X to shared
//                 memory.
//   warps 12..15  sums (12..19 for 64 rows of X, each half of the columns): read
//                 the groups' sums from TMEM, scale and add them.
//                 (With the workers doing this after each block, every block
//                 paid the round trip to the tensor core, about 1500 cycles:
//                 54 us for one row of 16384 x 16384.)
//   warps 8, 9    take alternate stages of 256 codes: start the TMA copy of the
//                 codes, 128 bytes a row, and for more than 16 rows of X's
//                 part, and bring the stage's scales and zero points from global
//                 memory into a table in shared memory.  (64 rows of 8192 x 8192,
//                 groups of 128: 19.4 us, and 26.1 with X by the workers; 32 rows
//                 17.0 and 18.9.  Up to 16 rows X is little work, and the cheaper
//                 conversion that its reordering allows counts for more.)
//   warps 10, 11  MMA issuers, one per team (a block's eight MMAs and the waits
//                 around them take one warp about as long as a team takes to
//                 convert it); warp 11 allocates TMEM.
//
// A tile has up to 128 rows, as few as spread the rows evenly over the SMs;
// where that is not enough, the CTAs of a cluster share the rows' length, and
// rank r sums and stores columns r, r + size, ... through distributed shared
// memory, in rank order.
//
// By expert, grid.y is the row of Y.  A row whose expert has a multiple of 16
// rows before it does that row and the expert's next 15; the others have
// nothing to do, and nothing has to be sorted.
constexpr int W4_WORKERS = 8;
constexpr int W4_TEAMS = 2;
constexpr int W4_TEAM_WARPS = W4_WORKERS / W4_TEAMS;
constexpr int W4_TILE = 128;
constexpr int W4_STAGE_K = 256;                       // codes of a row per stage
constexpr int W4_STAGE_BYTES = W4_TILE * W4_STAGE_K / 2;
constexpr int W4_BLOCK_K = 128;                       // codes of a row per team and stage
constexpr int W4_A_COLS = W4_BLOCK_K / 2;             // TMEM columns of an operand
constexpr int W4_MAX_STAGES = 8;
constexpr int W4_MAX_BUFS = 4;

// Barriers of a team's blocks, in turn: block `part` of stage n is the team's block
// m = 2 (n / 2) + part.  A wait by parity must not meet a later phase of its
// barrier.  Four turns are enough.  The turn of block b comes back with block
// b + 8.  A team writes that one after its issuer has consumed b (the operand
// buffers are a ring of all blocks).  Its MMAs wait for the sums of a block at most
// W4_SET_BLOCKS before it, which come, in order, after those of b + 3, the last one
// whose worker waits for b to be done.
constexpr int W4_TURNS = 4;
constexpr int W4_SET_BLOCKS = 4;  // blocks that all sets of accumulators hold

// Barrier slots.
enum : int {
    W4_WFULL = 0,                             // codes and scales of a stage are there
    W4_WEMPTY = W4_WFULL + W4_MAX_STAGES,     // every reader is done with them
    W4_AFULL = W4_WEMPTY + W4_MAX_STAGES,     // [team][turn] a block's operands are written
    W4_DONE = W4_AFULL + W4_TEAMS * W4_TURNS, // [team][turn] the MMAs have read them
    W4_GFULL = W4_DONE + W4_TEAMS * W4_TURNS, // a block's group sums are complete
    W4_GEMPTY = W4_GFULL + W4_MAX_BUFS,       // they have been read
    W4_DRAIN = W4_GEMPTY + W4_MAX_BUFS,       // [team]
    W4_STALL = W4_DRAIN + W4_TEAMS,           // stall test: never completed
    W4_BARRIERS
};

// CTAs per SM.  From 32 columns on the sums need more registers than two CTAs
// leave.
__host__ __device__ constexpr int w4_ctas(int cols) { return cols == 16 ? 2 : 1; }

template <int NC, int GROUP>
struct W4Layout {
    static constexpr int CTAS = w4_ctas(NC);
    // X comes by TMA with the codes, in its own order; up to 16 rows the workers
    // bring it, in the codes' order (see decode8)
    static constexpr bool X_TMA = NC > 16;
    static constexpr int STAGES = NC == 32 ? 6 : 4;
    static constexpr int GPS = W4_STAGE_K / GROUP;          // groups per stage and row
    static constexpr int GPB = W4_BLOCK_K / GROUP;          // groups per block
    static constexpr int SUMMERS = NC == 64 ? 8 : 4;        // warps that add up
    static constexpr int COLS = NC * 4 / SUMMERS;           // columns each of them has
    static constexpr int THREADS = (12 + SUMMERS) * 32;
    // A set of accumulators, the groups that one commit completes: all of a stage
    // where two such sets fit TMEM (fewer waits: half of them with groups of 128),
    // else a block's, or half a block's.
    static constexpr int TMEM_COLS = CTAS == 2 ? 256 : 512;
    static constexpr bool STAGE_SETS = 2 * GPS * NC + 2 * W4_A_COLS <= TMEM_COLS;
    static constexpr int SET_GROUPS = STAGE_SETS ? GPS : GPB * NC > 128 ? 128 / NC : GPB;
    static constexpr int SETS_PER_BLOCK = STAGE_SETS ? 1 : GPB / SET_GROUPS;
    static constexpr int SUM_COLS = SET_GROUPS * NC;        // TMEM columns of a set
    static constexpr int A_BUFS = TMEM_COLS - 3 * W4_A_COLS >= 2 * SUM_COLS ? 3 : 2;
    static constexpr int SETS =
        !STAGE_SETS && TMEM_COLS - A_BUFS * W4_A_COLS >= 4 * SUM_COLS ? 4 : 2;
    // Two issuers where every set always belongs to the same team's stages; else
    // the first one does all.
    static constexpr int ISSUERS =
        SETS % (W4_TEAMS * (STAGE_SETS ? 1 : 2 * SETS_PER_BLOCK)) == 0 ? 2 : 1;
    static constexpr int X_BYTES = NC * W4_BLOCK_K * 2;     // a block's part of X
    static constexpr int STAGE = W4_STAGE_BYTES + (X_TMA ? 2 * X_BYTES : 0);
    static constexpr int W = 0;
    static constexpr int X = X_TMA ? W + W4_STAGE_BYTES : W + STAGES * STAGE;
    // [stage][group][row]: the scale's bits, and -(1024 + zero) in fp16 above
    static constexpr int TABLE = W + STAGES * STAGE + (X_TMA ? 0 : A_BUFS * X_BYTES);
    static constexpr int TABLE_WORDS = GPS * W4_TILE;
    static constexpr int BARS = TABLE + STAGES * TABLE_WORDS * 4;
    static constexpr int LIST = BARS + (W4_BARRIERS + 1) * 8;  // rows of Y by expert
    static constexpr int TOTAL = LIST + 64 + 1024;
    static_assert(A_BUFS * W4_A_COLS + SETS * SUM_COLS <= TMEM_COLS, "TMEM columns");
    static_assert(SETS * (STAGE_SETS ? 2 : 1) <= W4_SET_BLOCKS * SETS_PER_BLOCK && A_BUFS <= 3,
                  "a wait by parity could meet a later phase");
    static_assert(NC * W4_TILE * 4 <= STAGES * STAGE, "the sums fit the code ring");
    // 228 KB an SM, 1 KB of it taken by the system per CTA
    static_assert(TOTAL <= (CTAS == 2 ? 113 : 227) * 1024, "shared memory");
};

__device__ __forceinline__ __half2 as_half2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
__device__ __forceinline__ uint32_t as_u32(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }

// q - zero of the eight codes of `w` as half pairs (k, k + 4), (k + 1, k + 5),
// (k + 2, k + 6), (k + 3, k + 7).  `z` is -(1024 + zero), twice, and z64 -(64 + zero).
__device__ __forceinline__ uint32_t code_pair(uint32_t w, uint32_t mask)
{
    // (w & mask) | the exponent of 1024, twice: one instruction, which the
    // compiler does not make of the expression
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "r"(mask), "r"(0x64006400u));
    return r;
}

__device__ __forceinline__ void decode8(uint32_t w, __half2 z, __half2 z64, uint32_t* e)
{
    const __half2 sixteenth = as_half2(0x2c002c00u);
    const uint32_t v = w >> 8;
    e[0] = as_u32(__hadd2(as_half2(code_pair(w, 0x000f000fu)), z));
    e[1] = as_u32(__hfma2(as_half2(code_pair(w, 0x00f000f0u)), sixteenth, z64));
    e[2] = as_u32(__hadd2(as_half2(code_pair(v, 0x000f000fu)), z));
    e[3] = as_u32(__hfma2(as_half2(code_pair(v, 0x00f000f0u)), sixteenth, z64));
}

// The same in the codes' own order: (k, k + 1) and so on, from one byte each, with
// 1024 + q in the lower and 1024 + 16 q in the upper half.  `z` is -(1024 + zero)
// below and -(64 + zero) above.  Three instructions a pair against two and a quarter.
__device__ __forceinline__ void decode8_in_order(uint32_t w, __half2 z, uint32_t* e)
{
    const __half2 unit = as_half2(0x2c003c00u);  // 1, 1/16
    const uint32_t sel[4] = {0x4040u, 0x4141u, 0x4242u, 0x4343u};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        e[i] = as_u32(
            __hfma2(as_half2(__byte_perm(w, 0x64646464u, sel[i]) & 0x64f0640fu), unit, z));
}

// X[k..k+7] in the order of decode8.
__device__ __forceinline__ uint4 order_x(const uint4& v)
{
    return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                      __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}

// TMEM -> registers, 32 lanes x 16 columns, complete on return.
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

// The same for 4 columns.
__device__ __forceinline__ void tmem_load_4cols(uint32_t taddr, uint32_t (&r)[4])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(taddr)
        : "memory");
}

// Registers -> TMEM, 32 lanes x 8 columns.  (One store of 32 columns ties 32
// registers together; its moves made the conversion a tenth slower.)
__device__ __forceinline__ void tmem_store_8cols(uint32_t taddr, const uint32_t (&r)[8])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// One lane of a converged warp (the same one every time): 1 there, else 0.
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t r;
    asm volatile(
        "{\n\t"
        ".reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "}\n"
        : "=r"(r));
    return r;
}

// D[tmem] (+)= A[tmem] * B[smem]^T, fp16 x fp16 -> fp32, issued by the lane with
// `elected` set.  The whole warp executes the statement: without a branch around
// it the operands stay in uniform registers (behind `if (lane == 0)` the issue of
// a block's eight MMAs took 950 cycles, more than their conversion).
__device__ __forceinline__ void mma_f16_ts(uint32_t elected, uint32_t d_tmem, uint32_t a_tmem,
                                           uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t"
        ".reg .pred p, q;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "setp.ne.b32 q, %4, 0;\n\t"
        "@p tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, q;\n\t"
        "}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(elected)
        : "memory");
}

__device__ __forceinline__ void mma_commit_elected(uint32_t elected, uint32_t bar)
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

__device__ __forceinline__ void store_y(const W4Params& p, int64_t row, int n, float v)
{
    const int64_t at = row * p.N + n;
    if (p.f16out)
        static_cast<__half*>(p.Y)[at] = __float2half_rn(v);
    else
        static_cast<float*>(p.Y)[at] = v;
}

// A bounded wait that leaves the issue slots to the warps that work: the hint
// lets the hardware suspend the thread for up to 100 us at a time.
struct W4Wait : Watchdog {
    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, int where, int tile, int kb)
    {
        if (aborted) return false;
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = globaltimer_ns();
        while (true) {
            uint32_t done;
            asm volatile(
                "{\n\t"
                ".reg .pred p;\n\t"
                "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t"
                "}\n"
                : "=r"(done)
                : "r"(bar), "r"(parity), "r"(100000u)
                : "memory");
            if (done) return true;
            if (peer_aborted()) {
                aborted = true;
                return false;
            }
            if (globaltimer_ns() - t0 > budget_ns) {
                record(where, tile, kb);
                return false;
            }
        }
    }
};

template <int NC, int GROUP>
__global__ void __launch_bounds__(W4Layout<NC, GROUP>::THREADS, W4Layout<NC, GROUP>::CTAS)
    k_w4(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
         const __grid_constant__ W4Params p)
{
    using L = W4Layout<NC, GROUP>;
    constexpr int STAGES = L::STAGES, A_BUFS = L::A_BUFS, SETS = L::SETS;
    constexpr int GPS = L::GPS, GPB = L::GPB, COLS = L::COLS;
    constexpr int FIRST_SUMMER = 12;
    constexpr int XPT = NC * (W4_BLOCK_K / 8) / 128;  // chunks of X per worker and block
    extern __shared__ __align__(1024) uint8_t w4_smem[];
    const uint32_t raw = smem_u32(w4_smem);
    const uint32_t base = align1024(raw);
    uint8_t* gen = w4_smem + (base - raw);
    const uint32_t bars = base + L::BARS;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gen + L::BARS + W4_BARRIERS * 8);
    int* list = reinterpret_cast<int*>(gen + L::LIST);
    const int tid = static_cast<int>(threadIdx.x);
    const int warp = tid >> 5;
    const uint32_t lane = lane_id();
    const uint32_t csize = gridDim.z, crank = blockIdx.z;
    const int n0 = static_cast<int>(blockIdx.x) * p.tile_rows;
    auto bar = [&](int slot) { return bars + static_cast<uint32_t>(slot) * 8u; };
    W4Wait wd;
    wd.st = p.status;
    wd.epoch = p.epoch;
    wd.budget_ns = p.budget_ns;
    wd.aborted = false;
    griddep_wait();
    if constexpr (NC == 64) {  // more rows than that are expanded
        if (p.verdicts) {
            int any = 0;
            for (int i = tid; i < p.verdict_count; i += L::THREADS) any |= p.verdicts[i];
            if (!__syncthreads_or(any)) return;  // the GEMM's result stands (k_w4_expand)
        }
    }

    // the rows of Y of this CTA: y0 and the following, or those on the list
    int expert = 0, y0 = 0, count = p.M;
    if (p.experts == 0) {
        y0 = static_cast<int>(blockIdx.y) * NC;
        count = p.M - y0 < NC ? p.M - y0 : NC;
    } else {
        const int first = static_cast<int>(blockIdx.y);
        expert = p.ids[first];
        if (expert < 0 || expert >= p.experts) {  // a dropped row
            if (crank == 0 && tid < p.tile_rows && n0 + tid < p.N)
                store_y(p, first, n0 + tid, 0.0f);
            return;
        }
        int before = 0;
        for (int r = tid; r - tid < first; r += L::THREADS)
            before += __syncthreads_count(r < first && p.ids[r] == expert);
        if (before % 16 != 0) return;
        if (warp == 0) {
            int found = 0;
            for (int r = first; r < p.M && found < 16; r += 32) {
                const int i = r + static_cast<int>(lane);
                const unsigned hit = __ballot_sync(0xffffffffu, i < p.M && p.ids[i] == expert);
                const int slot = found + __popc(hit & ((1u << lane) - 1u));
                if (((hit >> lane) & 1u) && slot < 16) list[slot] = i;
                found += __popc(hit);
            }
            if (lane < 16 && static_cast<int>(lane) >= found) list[lane] = -1;
        }
    }
    const int stages = (p.K + W4_STAGE_K - 1) / W4_STAGE_K;
    const int s_begin = static_cast<int>(static_cast<int64_t>(stages) * crank / csize);
    const int s_end = static_cast<int>(static_cast<int64_t>(stages) * (crank + 1) / csize);

    if (warp == 8 && lane == 0) {
        prefetch_tensormap(&tmW);
        if (L::X_TMA) prefetch_tensormap(&tmX);
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(bar(W4_WFULL + i), 2);  // the copies' announcement, the table
            // workers, sums and, where they read X there, the MMAs
            mbar_init(bar(W4_WEMPTY + i), W4_TEAM_WARPS + L::SUMMERS + (L::X_TMA ? 1 : 0));
        }
        for (int i = 0; i < W4_TEAMS * W4_TURNS; ++i) {
            mbar_init(bar(W4_AFULL + i), W4_TEAM_WARPS);
            mbar_init(bar(W4_DONE + i), 1);
        }
        for (int i = 0; i < SETS; ++i) {
            mbar_init(bar(W4_GFULL + i), 1);
            mbar_init(bar(W4_GEMPTY + i), L::SUMMERS);
        }
        for (int i = 0; i < W4_TEAMS; ++i) mbar_init(bar(W4_DRAIN + i), 1);
        mbar_init(bar(W4_STALL), 1);
        fence_mbar_init();
    }
    if (warp == 11) {
        tmem_alloc(smem_u32(tmem_slot), L::TMEM_COLS);
        tmem_relinquish_alloc_permit();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    griddep_launch_dependents();  // CTAs that have returned count as having done so
    const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    if (p.experts > 0) {
        count = 0;
        while (count < 16 && list[count] >= 0) ++count;
    }
    float acc[COLS];  // sums: columns col0 .. col0 + COLS - 1 of the thread's row
#pragma unroll
    for (int i = 0; i < COLS; ++i) acc[i] = 0.0f;
    const int col0 = (warp - FIRST_SUMMER) / 4 * COLS;
    const int q = warp & 3;  // workers and sums: TMEM lane quarter
    const int row = 32 * q + static_cast<int>(lane);
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t sum_tmem = tmem_base + A_BUFS * W4_A_COLS;

    if (warp < W4_WORKERS) {
        // -------------------------------------------------------- workers
        const int team = warp >> 2;
        // X: row m0, chunk c0 of the block's 16, then rows m0 + 8, m0 + 16, ...;
        // two operand tiles of 64 codes.  By expert there are two rows a thread
        // at most, so a first row and a distance describe them too.
        const int m0 = (tid & 127) >> 4, c0 = tid & 15;
        const uint32_t xdst = base + L::X + static_cast<uint32_t>(
            (c0 >> 3) * NC * 128 + m0 * 128 + (((c0 & 7) ^ m0) << 4));
        static_assert(XPT * 8 == NC, "rows of a thread");
        const __half* x = p.X;
        int64_t xnext = static_cast<int64_t>(p.K) * 8;
        if (!L::X_TMA && m0 < count) {
            const int y = p.experts > 0 ? list[m0] : y0 + m0;
            x = p.X + static_cast<int64_t>(y / p.share) * p.K + c0 * 8;
            if (p.experts > 0 && m0 + 8 < count)
                xnext = static_cast<int64_t>(list[m0 + 8] / p.share - y / p.share) * p.K;
        }
        // a warp holds rows 2 q, 2 q + 1 and 8, 16, ... on
        const bool has_x = !L::X_TMA && 2 * q < count;
        int k = (s_begin + team) * W4_STAGE_K;  // first code of the block whose X comes next
        uint4 xv[XPT];
        auto load_x = [&] {  // zeros past K
            const int left = p.K - k - c0 * 8;
#pragma unroll
            for (int i = 0; i < XPT; ++i) {
                xv[i] = make_uint4(0, 0, 0, 0);
                if (m0 + 8 * i >= count) continue;
                const __half* from = x + i * xnext + k;
                if (left > 0) xv[i] = *reinterpret_cast<const uint4*>(from);
                // the team's next stage comes from the L1 cache then
                if (left > 2 * W4_STAGE_K)
                    asm volatile("prefetch.global.L1 [%0];" ::"l"(from + 2 * W4_STAGE_K));
            }
        };
        if (has_x) load_x();
        const uint32_t sw = static_cast<uint32_t>(row & 7) << 4;
        const uint32_t a_tmem = tmem_base + lanes;
        const uint32_t* words = reinterpret_cast<const uint32_t*>(gen + L::TABLE) + row;
        const uint32_t src0 = base + L::W + row * 128;
        static_assert(STAGES % W4_TEAMS == 0, "a slot always belongs to the same team");
        for (int s = s_begin + team; s < s_end; s += W4_TEAMS) {
            const int n = s - s_begin;
            const int ws = n % STAGES;
            wd.wait(bar(W4_WFULL + ws), static_cast<uint32_t>(n / STAGES) & 1u, WAIT_FULL, s, 0);
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                if (s * W4_STAGE_K + part * W4_BLOCK_K >= p.K) break;  // no such block
                const int b = 2 * n + part, buf = b % A_BUFS;
                __half2 zero[GPB];
#pragma unroll
                for (int i = 0; i < GPB; ++i)
                    zero[i] = as_half2(__byte_perm(
                        words[ws * L::TABLE_WORDS + (part * GPB + i) * W4_TILE], 0u, 0x3232));
                if (b >= A_BUFS) {  // the block that had this buffer before
                    const int n1 = (b - A_BUFS) >> 1, m = 2 * (n1 >> 1) + ((b - A_BUFS) & 1);
                    wd.wait(bar(W4_DONE + (n1 & 1) * W4_TURNS + m % W4_TURNS),
                            static_cast<uint32_t>(m / W4_TURNS) & 1u, WAIT_EMPTY, s, b);
                }
                const uint32_t src = src0 + ws * L::STAGE;
                const uint32_t a_block = a_tmem + static_cast<uint32_t>(buf * W4_A_COLS);
#pragma unroll
                for (int c = 0; c < W4_BLOCK_K / 32; ++c) {  // 32 codes at a time
                    const uint4 w =
                        ld_shared_v4(src + ((static_cast<uint32_t>(part * 64 + c * 16)) ^ sw));
                    const __half2 z = zero[c * 32 / GROUP];
                    uint32_t e[8];
                    if constexpr (L::X_TMA) {
                        const __half2 zz = __hadd2(z, as_half2(0x63800000u));  // 0, 960
                        decode8_in_order(w.x, zz, e);
                        decode8_in_order(w.y, zz, e + 4);
                        tmem_store_8cols(a_block + c * 16, e);
                        decode8_in_order(w.z, zz, e);
                        decode8_in_order(w.w, zz, e + 4);
                    } else {
                        const __half2 z64 = __hadd2(z, as_half2(0x63806380u));
                        decode8(w.x, z, z64, e);
                        decode8(w.y, z, z64, e + 4);
                        tmem_store_8cols(a_block + c * 16, e);
                        decode8(w.z, z, z64, e);
                        decode8(w.w, z, z64, e + 4);
                    }
                    tmem_store_8cols(a_block + c * 16 + 8, e);
                }
                if (has_x) {
#pragma unroll
                    for (int i = 0; i < XPT; ++i) {
                        if (m0 + 8 * i >= count) continue;
                        const uint4 v = order_x(xv[i]);
                        st_shared_v4(xdst + buf * L::X_BYTES + i * 8 * 128, v.x, v.y, v.z, v.w);
                    }
                    fence_proxy_async_smem();
                }
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    const int m = 2 * (n >> 1) + part;
                    mbar_arrive(bar(W4_AFULL + team * W4_TURNS + m % W4_TURNS));
                }
                if (has_x) {  // the stage's second block, then the team's next stage
                    k += part == 0 ? W4_BLOCK_K : W4_TEAMS * W4_STAGE_K - W4_BLOCK_K;
                    load_x();
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(W4_WEMPTY + ws));
        }
    } else if (warp >= FIRST_SUMMER) {
        // ----------------------------------------------------------- sums
        int ws = 0, set = 0;
        uint32_t ws_phase = 0, set_phase = 0;
        const uint32_t* words = reinterpret_cast<const uint32_t*>(gen + L::TABLE) + row;
        int left = p.K - s_begin * W4_STAGE_K;
        for (int s = s_begin; s < s_end; ++s) {
            // (a stalled role waits in this place: a wait of its own costs registers)
            const bool stall = p.debug_stall == 2;
            wd.wait(bar(stall ? W4_STALL : W4_WFULL + ws), stall ? 0u : ws_phase, WAIT_FULL, s, 4);
            // read when needed: a stage's eight scales beside the sums spill
            auto scale_of = [&](int i) {
                return __half2float(__ushort_as_half(static_cast<unsigned short>(
                    words[ws * L::TABLE_WORDS + i * W4_TILE] & 0xffffu)));
            };
#pragma unroll 1
            for (int g0 = 0; g0 < GPS; g0 += L::SET_GROUPS) {
                if (g0 * GROUP / W4_BLOCK_K * W4_BLOCK_K >= left) break;  // no such block
                wd.wait(bar(W4_GFULL + set), set_phase, WAIT_TMEM_FULL, s, g0);
                tc_fence_after_sync();
                const uint32_t from =
                    sum_tmem + lanes + static_cast<uint32_t>(set * L::SUM_COLS + col0);
#pragma unroll
                for (int g = 0; g < L::SET_GROUPS; ++g) {
                    // the last stage may have one block only
                    if (L::STAGE_SETS && g >= GPB && left <= W4_BLOCK_K) break;
                    const float sg = scale_of(g0 + g);
                    // Few rows, the usual case, pay for few columns only (one row of 16384
                    // x 16384: 38.2 us and 38.8, with groups of 32 50.9 and 53.0; 16 rows
                    // lose a hundredth by the branch).
                    if (COLS == 16 && count <= 4) {
                        uint32_t v[4];
                        tmem_load_4cols(from + g * NC, v);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[j] = fmaf(sg, __uint_as_float(v[j]), acc[j]);
                        continue;
                    }
                    uint32_t v[COLS];
                    if constexpr (COLS == 16)
                        tmem_load_16cols(from + g * NC, v);
                    else
                        tmem_load_32cols(from + g * NC, v);
#pragma unroll
                    for (int j = 0; j < COLS; ++j)
                        acc[j] = fmaf(sg, __uint_as_float(v[j]), acc[j]);
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(W4_GEMPTY + set));
                if (++set == SETS) {
                    set = 0;
                    set_phase ^= 1u;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(W4_WEMPTY + ws));
            left -= W4_STAGE_K;
            if (++ws == STAGES) {
                ws = 0;
                ws_phase ^= 1u;
            }
        }
    } else if (warp < 10) {
        // ------------------------------------------------ codes and scales
        const int groups = p.K / GROUP;
        const uint32_t tx =
            static_cast<uint32_t>(p.tile_rows) * 128u + (L::X_TMA ? 2 * L::X_BYTES : 0);
        int last_n = -1;
        struct alignas(2 * GPS) Scales { unsigned short v[GPS]; };
        struct alignas(GPS) Zeros { uint8_t v[GPS]; };
        const __half* scales[W4_TILE / 32];  // of the lane's rows; rows that are not
        const uint8_t* zeros[W4_TILE / 32];  // there repeat the tile's first
#pragma unroll
        for (int i = 0; i < W4_TILE / 32; ++i) {
            const int r = 32 * i + static_cast<int>(lane);
            const int exists = r < p.tile_rows && n0 + r < p.N ? r : 0;
            const int64_t at = (static_cast<int64_t>(expert) * p.N + n0 + exists) * groups;
            scales[i] = p.scales + at;
            zeros[i] = p.zeros ? p.zeros + at : nullptr;
        }
        for (int s = s_begin + warp - 8; s < s_end; s += 2) {
            const int n = s - s_begin;
            const int ws = n % STAGES;
            const bool stall = p.debug_stall == 1;
            const bool ok =
                wd.wait(bar(stall ? W4_STALL : W4_WEMPTY + ws),
                        stall ? 0u : (static_cast<uint32_t>(n / STAGES) & 1u) ^ 1u, WAIT_EMPTY, s, 3);
            if (lane == 0 && ok) {
                mbar_arrive_expect_tx(bar(W4_WFULL + ws), tx);
                tma_load_2d(base + L::W + ws * L::STAGE, &tmW, bar(W4_WFULL + ws),
                            s * (W4_STAGE_K / 2), expert * p.N + n0);
                if constexpr (L::X_TMA) {
#pragma unroll
                    for (int i = 0; i < W4_STAGE_K / 64; ++i)  // zeros past M and K
                        tma_load_2d(base + L::X + ws * L::STAGE + i * NC * 128, &tmX,
                                    bar(W4_WFULL + ws), s * W4_STAGE_K + i * 64, y0);
                }
                last_n = n;
            }
            // an abandoned run: no arrival on a barrier whose bytes are on their way
            if (!__all_sync(0xffffffffu, ok)) break;
            uint32_t* to =
                reinterpret_cast<uint32_t*>(gen + L::TABLE) + ws * L::TABLE_WORDS + lane;
            // -(1024 + zero) in fp16 is -1024's bits plus the zero point
            if (p.wide_scales) {
                constexpr int ROWS = GPS == 8 ? 2 : W4_TILE / 32;  // as registers allow
#pragma unroll
                for (int i0 = 0; i0 < W4_TILE / 32; i0 += ROWS) {
                    Scales sc[ROWS];
                    Zeros ze[ROWS];
#pragma unroll
                    for (int i = 0; i < ROWS; ++i) {
                        sc[i] = *reinterpret_cast<const Scales*>(scales[i0 + i] + s * GPS);
                        if (zeros[i0 + i])
                            ze[i] = *reinterpret_cast<const Zeros*>(zeros[i0 + i] + s * GPS);
                    }
#pragma unroll
                    for (int i = 0; i < ROWS; ++i)
#pragma unroll
                        for (int g = 0; g < GPS; ++g)
                            to[g * W4_TILE + 32 * (i0 + i)] =
                                sc[i].v[g] | ((0xe400u + (zeros[i0 + i] ? ze[i].v[g] : 8u)) << 16);
                    __syncwarp();
                }
            } else {
#pragma unroll 1
                for (int g = 0; g < GPS; ++g) {
                    const bool inside = s * GPS + g < groups;
#pragma unroll
                    for (int i = 0; i < W4_TILE / 32; ++i) {
                        const uint32_t sc = inside ? __half_as_ushort(scales[i][s * GPS + g]) : 0u;
                        const uint32_t ze = inside && zeros[i] ? zeros[i][s * GPS + g] : 8u;
                        to[g * W4_TILE + 32 * i] = sc | ((0xe400u + ze) << 16);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(W4_WFULL + ws));
        }
        // this warp's copies in flight land before the CTA exits, whichever role may have
        // given up without waiting for them
        if (lane == 0) {
            for (int n = last_n; n >= 0 && n > last_n - STAGES; n -= 2)
                wd.drain(bar(W4_WFULL + n % STAGES), static_cast<uint32_t>(n / STAGES) & 1u);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ MMA issuer
        constexpr uint32_t idesc = idesc_f16_f32(W4_TILE, NC);
        const uint32_t elected = elect_one();
        const int issuer = warp - 10;
        const int end = s_end * W4_STAGE_K < p.K ? s_end * W4_STAGE_K : p.K;
        int k0 = s_begin * W4_STAGE_K;
        for (int b = 0; k0 < end; ++b, k0 += W4_BLOCK_K) {
            const int n = b >> 1, team = n & 1, m = 2 * (n >> 1) + (b & 1);
            if (L::ISSUERS == 2 ? team != issuer : issuer != 0) continue;
            const int buf = b % A_BUFS;
            bool ok = wd.wait(bar(W4_AFULL + team * W4_TURNS + m % W4_TURNS),
                              static_cast<uint32_t>(m / W4_TURNS) & 1u, WAIT_FULL, k0, 1);
            const uint32_t a_tmem = tmem_base + static_cast<uint32_t>(buf * W4_A_COLS);
            const int ws = n % STAGES;
            if (L::X_TMA)
                ok = ok && wd.wait(bar(W4_WFULL + ws), static_cast<uint32_t>(n / STAGES) & 1u,
                                   WAIT_FULL, k0, 2);
            const uint64_t bdesc = sw128_kmajor_desc(
                base + L::X + (L::X_TMA ? ws * L::STAGE + (b & 1) * L::X_BYTES : buf * L::X_BYTES));
#pragma unroll
            for (int h = 0; h < L::SETS_PER_BLOCK; ++h) {
                // codes of the block that go to this set, and the set's first column
                constexpr int SET_K = L::STAGE_SETS ? W4_BLOCK_K : L::SET_GROUPS * GROUP;
                const int u = L::STAGE_SETS ? n : b * L::SETS_PER_BLOCK + h, set = u % SETS;
                if (!L::STAGE_SETS || (b & 1) == 0)
                    ok = wd.wait(bar(W4_GEMPTY + set), (static_cast<uint32_t>(u / SETS) & 1u) ^ 1u,
                                 WAIT_TMEM_EMPTY, k0, h);
                if (!__all_sync(0xffffffffu, ok)) break;  // an abandoned run
                const uint32_t d_tmem =
                    sum_tmem + static_cast<uint32_t>(set * L::SUM_COLS +
                                                     (L::STAGE_SETS ? (b & 1) * GPB * NC : 0));
                tc_fence_after_sync();
#pragma unroll
                for (int i = 0; i < SET_K; i += MMA_K) {
                    const int k = h * SET_K + i;
                    mma_f16_ts(elected, d_tmem + static_cast<uint32_t>(i / GROUP * NC),
                               a_tmem + static_cast<uint32_t>(k / 2),
                               bdesc + static_cast<uint64_t>(
                                           ((k / 64) * NC * 128 + (k % 64) * 2) >> 4),
                               idesc, k % GROUP == 0 ? 0u : 1u);
                }
                if (!L::STAGE_SETS || (b & 1) == 1 || k0 + W4_BLOCK_K >= end)
                    mma_commit_elected(elected, bar(W4_GFULL + set));
            }
            if (!__all_sync(0xffffffffu, ok)) break;
            mma_commit_elected(elected, bar(W4_DONE + team * W4_TURNS + m % W4_TURNS));
            if (L::X_TMA && ((b & 1) == 1 || k0 + W4_BLOCK_K >= end))
                mma_commit_elected(elected, bar(W4_WEMPTY + ws));
        }
        mma_commit_elected(elected, bar(W4_DRAIN + issuer));  // by the lane that issued
        wd.drain(bar(W4_DRAIN + issuer), 0);
        __syncwarp();
    }

    // every MMA has been waited for and every block used up
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 11) {
        tc_fence_after_sync();
        tmem_dealloc(tmem_base, L::TMEM_COLS);
    }
    const bool summer = warp >= FIRST_SUMMER;
    const bool stores = row < p.tile_rows && n0 + row < p.N && !wd.aborted;
    if (csize == 1) {
        if (summer && stores) {
#pragma unroll
            for (int c = 0; c < COLS; ++c) {
                const int m = col0 + c;
                if (m < count) store_y(p, p.experts > 0 ? list[m] : y0 + m, n0 + row, acc[c]);
            }
        }
        return;
    }
    // this CTA's part of the length, [NC][128], over the code ring
    float* sums = reinterpret_cast<float*>(gen + L::W);
    if (summer) {
#pragma unroll
        for (int c = 0; c < COLS; ++c)
            if (col0 + c < count) sums[(col0 + c) * W4_TILE + row] = acc[c];
    }
    cluster_sync_all();
    if (stores) {
        // four warps a column
        const int step = L::THREADS / W4_TILE * static_cast<int>(csize);
        for (int m = static_cast<int>(crank) + (warp >> 2) * static_cast<int>(csize); m < count;
             m += step) {
            float v = 0.0f;
            for (uint32_t r = 0; r < csize; ++r) {
                float part;
                asm volatile("ld.shared::cluster.f32 %0, [%1];"
                             : "=f"(part)
                             : "r"(map_shared_rank(smem_u32(sums + m * W4_TILE + row), r))
                             : "memory");
                v += part;
            }
            store_y(p, p.experts > 0 ? list[m] : y0 + m, n0 + row, v);
        }
    }
    cluster_sync_all();  // nobody reads this CTA's sums any more
}

// ------------------------------------------------------------ many rows
//
// For many rows of X the GEMM multiplies expanded weights.  w = scale * (q - zero) is a
// multiple of 2^-24 with at most 11 + 8 significant bits, so
//
//     hi = w rounded to fp16 (nearest even),   lo = w - hi
//
// are both fp16 numbers and hi + lo = w: lo is a multiple of 2^-24 too, at most half a
// unit of hi.  Each chunk of eight codes becomes a chunk of hi and a chunk of lo, each
// chunk of X the same chunk twice, and the GEMM sums over twice the length: no weight
// is rounded.  (The tensor cores then do twice the work; the caller may ask for hi
// alone.)
//
// That form does not hold where hi or an entry of X is not finite: w beyond 65504, and
// infinity * lo where lo = 0.  So every CTA leaves a verdict on what it has seen, and
// the few-row kernel runs behind the GEMM: it returns at once where all verdicts are
// zero and else computes Y anew.  Every word is written in every run, so none is kept
// from one to the next.
//
// A thread expands eight codes (4 bytes) to 32 bytes, or copies a chunk of X: bound by
// the writes, which the GEMM then reads from L2 where they fit (2048 rows of 4096 x 4096,
// groups of 64: 115 us in all, 48 with rounded weights, 169 by the few-row kernel).
constexpr int W4_EXPAND_CTAS = 8;  // per SM

// Whether one of the two halves is an infinity or NaN.
__device__ __forceinline__ uint32_t not_finite(uint32_t v)
{
    return ((v & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
}

template <bool ROUNDED>
__global__ void __launch_bounds__(256)
    k_w4_expand(int64_t words, int group_shift, const uint32_t* packed, const __half* scales,
                const uint8_t* zeros, uint4* out, int64_t chunks, const uint4* X, uint4* X2,
                int* verdicts)
{
    griddep_wait();
    griddep_launch_dependents();
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    uint32_t bad = 0;
    for (int64_t i = first; i < words; i += step) {
        const int64_t at = i >> group_shift;  // a row has whole groups
        const __half2 s = __half2half2(scales[at]);
        const __half2 z = as_half2((0xe400u + (zeros ? zeros[at] : 8u)) * 0x10001u);
        uint32_t e[4], hi[4], lo[4];
        decode8_in_order(packed[i], __hadd2(z, as_half2(0x63800000u)), e);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __half2 d = as_half2(e[j]);
            const __half2 h = __hmul2(d, s);  // a product of two fp16 numbers, rounded once
            hi[j] = as_u32(h);
            if constexpr (!ROUNDED) {
                lo[j] = as_u32(__hfma2(d, s, __hneg2(h)));
                bad |= not_finite(hi[j]);
            }
        }
        if constexpr (ROUNDED) {
            out[i] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        } else {
            out[2 * i] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            out[2 * i + 1] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
    if constexpr (!ROUNDED) {
        for (int64_t i = first; i < chunks; i += step) {
            const uint4 v = X[i];
            X2[2 * i] = v;
            X2[2 * i + 1] = v;
            bad |= not_finite(v.x) | not_finite(v.y) | not_finite(v.z) | not_finite(v.w);
        }
        const int any = __syncthreads_or(static_cast<int>(bad != 0));
        if (threadIdx.x == 0) verdicts[blockIdx.x] = any;
    }
}

// One instantiation of the few-row kernel.
struct W4Kernel {
    void (*fn)(CUtensorMap, CUtensorMap, W4Params);
    unsigned smem;
    int threads;
};

template <int GROUP>
W4Kernel kernel_of_group(int cols)
{
    switch (cols) {
    case 16: return {k_w4<16, GROUP>, W4Layout<16, GROUP>::TOTAL, W4Layout<16, GROUP>::THREADS};
    case 32: return {k_w4<32, GROUP>, W4Layout<32, GROUP>::TOTAL, W4Layout<32, GROUP>::THREADS};
    default: return {k_w4<64, GROUP>, W4Layout<64, GROUP>::TOTAL, W4Layout<64, GROUP>::THREADS};
    }
}

W4Kernel kernel_of(int cols, int group)
{
    return group == 32   ? kernel_of_group<32>(cols)
           : group == 64 ? kernel_of_group<64>(cols)
                         : kernel_of_group<128>(cols);
}

// Clusters along z: the CTAs that share the rows' length.
struct W4Launch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];

    W4Launch(const W4Kernel& k, dim3 grid, cudaStream_t stream)
    {
        cfg.gridDim = grid;
        cfg.blockDim = dim3(static_cast<unsigned>(k.threads));
        cfg.dynamicSmemBytes = k.smem;
        cfg.stream = stream;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 1;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = grid.z;
        cfg.attrs = attr;
        cfg.numAttrs = grid.z > 1 ? 2 : 1;
    }
};

// Rows per tile and CTAs per cluster of the few-row kernel, and the time they are
// expected to take.  A stage of 256 codes takes a CTA the same time whatever its rows
// (the kernel is bound by the instructions and waits of its warps), a launch about 5 us
// more: so the length is shared by as many CTAs as are resident at once, and the tiles
// are as low as spread the rows evenly over those.  The table below is measured with
// one CTA per SM; two (up to 16 rows) take 1.7 times as long, each.  A second wave of
// CTAs sets up anew: 3.6 us, 7 for clusters.  How many clusters are resident with one
// CTA per SM is asked of the runtime: clusters of four and eight leave SMs of a GPC
// idle.  One row, 4096 x 14336: 13.5 us on 4 x 35 CTAs, 18.9 on 8 x 37, of which not
// all are resident; 16384 x 16384: 39 us on 2 x 147, two per SM, 71 on 1 x 293.
cudaError_t choose_w4_tile(int64_t N, int64_t K, int64_t matrices, int cols, int group, int sms,
                           int* tile_rows, int* length_ctas, double* us)
{
    const W4Kernel k = kernel_of(cols, group);
    cudaError_t e = ensure_smem_limit(k.fn, k.smem);
    if (e != cudaSuccess) return e;
    const int64_t stages = (K + W4_STAGE_K - 1) / W4_STAGE_K;
    // us per stage by columns (16, 32, 64) and group (32, 64, 128)
    static const double stage_us[3][3] = {{0.9, 0.75, 0.6}, {1.15, 0.8, 0.75}, {1.36, 1.14, 0.76}};
    const double one = stage_us[cols / 32][group / 64];
    double best = -1.0;
    for (int ctas = 1; ctas <= 8 && (ctas == 1 || ctas * 2 <= stages); ctas *= 2) {
        int resident = sms;
        if (ctas > 1) {
            W4Launch launch(k, dim3(1, 1, static_cast<unsigned>(ctas)), nullptr);
            e = cudaOccupancyMaxActiveClusters(&resident, k.fn, &launch.cfg);
            if (e != cudaSuccess) return e;
            resident = std::min(resident, sms / ctas);
            if (resident < 1) continue;
        }
        for (int per_sm = 1; per_sm <= w4_ctas(cols); ++per_sm) {
            const int64_t clusters = static_cast<int64_t>(resident) * per_sm;
            const int64_t per_matrix = std::max<int64_t>(1, clusters / matrices);
            const int64_t rows =
                std::min<int64_t>(W4_TILE, ((N + per_matrix - 1) / per_matrix + 7) / 8 * 8);
            const int64_t tiles = (N + rows - 1) / rows * matrices;
            const int64_t waves = (tiles + clusters - 1) / clusters;
            const double time =
                5.0 + static_cast<double>(waves - 1) * (ctas > 1 ? 7.0 : 3.6) +
                static_cast<double>(waves * ((stages + ctas - 1) / ctas)) * one *
                    (per_sm == 2 ? 1.7 : 1.0);
            if (best < 0.0 || time < best) {
                best = time;
                *tile_rows = static_cast<int>(rows);
                *length_ctas = ctas;
                *us = time;
            }
        }
    }
    return cudaSuccess;
}

// Expected time of the expansion and the GEMM: the weights (and X, twice) are written,
// and read by a GEMM that takes 5.8 us per 1024 of its length at least (few tiles), and
// for more rows 1500 TFLOP/s.  Few-row kernel, expansion and GEMM, rounded weights, us:
// 8192 x 8192, groups of 128: 256 rows 62, 174, 84; 512 rows 121, 170, 77; 1024 rows 211,
// 244, 111; 2048 rows 419, 396, 187.  4096 x 4096, groups of 64: 512 rows 49, 75, 35;
// 1024 rows 97, 72, 30; 2048 rows 169, 115, 48.  16384 x 4096, groups of 32: 256 rows 110,
// 144, 61; 512 rows 193, 175, 78.  1024 x 4096, groups of 128: 2048 rows 37, 68, 30.
double expanded_us(int64_t M, int64_t N, int64_t K, bool rounded)
{
    const double weights = static_cast<double>(N) * static_cast<double>(K);
    const double x = static_cast<double>(M) * static_cast<double>(K);
    const double gemm = std::max({5.8 * static_cast<double>(K) / 1024.0, weights * 2.0 / 4.7e6,
                                  2.0 * static_cast<double>(M) * weights / 1.5e9});
    if (rounded) return 3.5 + weights * 2.6 / 6.5e6 + gemm;
    return 8.0 + (weights * 5.2 + x * 6.0) / 6.5e6 + 2.0 * gemm;
}

// Whether a plan of more than one block of rows expands.  Many rows of a short length
// always do: the two are then close (few-row kernel and expansion, us: 1500 rows of 1032 x
// 1152 20.0 and 24.9, 3000 of 512 x 512 16.5 and 15.6, 2000 of 136 x 256 8.6 and 10.8).
//
// The GEMM's sum loses 1.2e-9 of its norm per product of its doubled length (the tensor
// cores' accumulator truncates: 9.6e-6 with K = 4096), where the few-row kernel's, which
// adds groups of up to 128 exact products in fp32, loses 1.5e-7 in all.  That is far below
// the rounding of an fp16 output, but not of an fp32 one, which is expanded up to a
// length only whose error is that of the grouped products, 3e-6.
bool prefers_expansion(int64_t M, int64_t N, int64_t K, int dtype, bool rounded, double rows_us)
{
    if (!rounded && dtype == GEMM_OUT_F32) return M > 1024 && K <= 1280;
    if (!rounded && K > 32768) return false;
    return (M > 1024 && K < 2048) || rows_us > expanded_us(M, N, K, rounded);
}

}  // namespace

}  // namespace tg

using namespace tg;

struct gemm_w4_plan {
    int64_t M, N, K;
    int group, experts, share, dtype;
    int device, sms;
    bool expand;      // expand + GEMM, the few-row kernel where that does not hold
    bool rounded;     // the weights rounded to fp16, no more
    int cols;         // N side of the few-row kernel's MMA
    int length_ctas;  // CTAs that share a row's length
    int tile_rows;    // rows of the weights per CTA
    DevStatus* d_status;
    unsigned epoch;
    unsigned long long budget_ns;
    int debug_stall;
    void* d_weights;  // N x 2 K fp16 (rounded: N x K)
    void* d_x;        // M x 2 K fp16
    int* d_verdicts;  // one per CTA of the expansion
    gemm_plan* gemm;
    char desc[256];
};

namespace {

// Tensor map over a row-major matrix: boxes of 128 bytes x `box_rows`, 128-byte
// swizzle, zeros outside.
int encode_rows(CUtensorMap* map, const char* what, CUtensorMapDataType type, int elt,
                const void* from, int64_t cols, int64_t rows, int box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = get_encode_fn();
    if (!enc) return fail(GEMM_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols * elt)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / elt), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, type, 2, const_cast<void*>(from), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) return GEMM_OK;
    char buf[100];
    std::snprintf(buf, sizeof(buf), "cuTensorMapEncodeTiled(%s) failed with CUresult %d", what,
                  static_cast<int>(r));
    return fail(GEMM_ERR_CUDA, buf);
}

void release(const gemm_w4_plan& p)
{
    if (p.gemm) gemm_destroy(p.gemm);
    if (p.d_weights) cudaFree(p.d_weights);
    if (p.d_x) cudaFree(p.d_x);
    if (p.d_verdicts) cudaFree(p.d_verdicts);
    if (p.d_status) cudaFree(p.d_status);
}

constexpr int64_t MAX_ROW_BLOCKS = 65535;  // grid.y

// The few-row kernel over all of a plan's rows; with `verdicts`, behind an expansion
// of so many CTAs.
int run_rows(gemm_w4_plan* plan, const void* X, const void* packed, const void* scales,
             const void* zeros, const int32_t* expert_ids, void* Y, cudaStream_t stream,
             int verdicts)
{
    W4Params p = {};
    p.N = static_cast<int>(plan->N);
    p.K = static_cast<int>(plan->K);
    p.experts = plan->experts;
    p.share = plan->share;
    p.packed = static_cast<const uint8_t*>(packed);
    p.scales = static_cast<const __half*>(scales);
    p.zeros = static_cast<const uint8_t*>(zeros);
    p.ids = expert_ids;
    p.f16out = plan->dtype == GEMM_OUT_F16;
    p.tile_rows = plan->tile_rows;
    p.wide_scales = plan->K % W4_STAGE_K == 0 && (reinterpret_cast<uintptr_t>(zeros) & 7u) == 0;
    p.verdicts = verdicts > 0 ? plan->d_verdicts : nullptr;
    p.verdict_count = verdicts;
    p.status = plan->d_status;
    p.epoch = next_epoch(&plan->epoch);
    p.budget_ns = plan->budget_ns;
    p.debug_stall = plan->debug_stall;
    CUtensorMap codes, x;
    int r = encode_rows(&codes, "packed", CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, packed, plan->K / 2,
                        plan->N * std::max(plan->experts, 1), plan->tile_rows);
    if (r != GEMM_OK) return r;
    const W4Kernel k = kernel_of(plan->cols, plan->group);
    const int64_t most = plan->experts > 0 ? plan->M : MAX_ROW_BLOCKS * plan->cols;
    for (int64_t m0 = 0; m0 < plan->M; m0 += most) {
        const int64_t rows = std::min(most, plan->M - m0);
        p.M = static_cast<int>(rows);
        p.X = static_cast<const __half*>(X) + m0 * plan->K;
        p.Y = static_cast<char*>(Y) + m0 * plan->N * (p.f16out ? 2 : 4);
        x = codes;  // not used
        if (plan->cols > 16)
            r = encode_rows(&x, "X", CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, p.X, plan->K, rows,
                            plan->cols);
        if (r != GEMM_OK) return r;
        const dim3 grid(static_cast<unsigned>((plan->N + plan->tile_rows - 1) / plan->tile_rows),
                        static_cast<unsigned>(plan->experts > 0
                                                  ? rows
                                                  : (rows + plan->cols - 1) / plan->cols),
                        static_cast<unsigned>(plan->length_ctas));
        W4Launch launch(k, grid, stream);
        const cudaError_t e = cudaLaunchKernelEx(&launch.cfg, k.fn, codes, x, p);
        if (e != cudaSuccess) return cuda_fail("w4 product launch", e);
    }
    return ok();
}

}  // namespace

extern "C" {

gemm_w4_plan* gemm_w4_create_plan(int64_t M, int64_t N, int64_t K, int group, int experts,
                                  int share, int dtype_out)
{
    return gemm_w4_create_plan_ex(M, N, K, group, experts, share, dtype_out,
                                  GEMM_W4_WEIGHTS_EXACT);
}

gemm_w4_plan* gemm_w4_create_plan_ex(int64_t M, int64_t N, int64_t K, int group, int experts,
                                     int share, int dtype_out, int weights)
{
    gemm_w4_plan* plan = nullptr;
    guarded([&] {
        const int64_t LIM = MAX_COORDINATE;
        if (M < 1 || N < 1 || K < 1 || M > LIM || N > LIM || K > LIM)
            return fail(GEMM_ERR_INVALID_ARG, "M, N, K must be in [1, 2^31-65536]");
        if (group != 32 && group != 64 && group != 128)
            return fail(GEMM_ERR_INVALID_ARG, "group must be 32, 64 or 128");
        if (dtype_out != GEMM_OUT_F32 && dtype_out != GEMM_OUT_F16)
            return fail(GEMM_ERR_INVALID_ARG,
                        "dtype_out must be GEMM_OUT_F32 (0) or GEMM_OUT_F16 (1)");
        if (weights != GEMM_W4_WEIGHTS_EXACT && weights != GEMM_W4_WEIGHTS_ROUNDED)
            return fail(GEMM_ERR_INVALID_ARG, "unknown gemm_w4_weights");
        if (experts < 0 || share < 1 || (experts == 0 && share != 1))
            return fail(GEMM_ERR_INVALID_ARG,
                        "experts must be >= 0 and share >= 1 (1 without experts)");
        if (K % group != 0)
            return fail(GEMM_ERR_UNSUPPORTED, "K must be a multiple of group");
        const int elt = dtype_out == GEMM_OUT_F16 ? 2 : 4;
        if ((N * elt) % 16 != 0)
            return fail(GEMM_ERR_UNSUPPORTED,
                        "N * sizeof(output) must be a multiple of 16 bytes");
        if (N > LIM / std::max(experts, 1))
            return fail(GEMM_ERR_UNSUPPORTED, "experts * N is too large");
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
        p.rounded = weights == GEMM_W4_WEIGHTS_ROUNDED;
        p.budget_ns = DEFAULT_WAIT_NS;
        p.cols = 16;
        while (experts == 0 && p.cols < std::min<int64_t>(M, 64)) p.cols *= 2;
        const int64_t blocks = (M + p.cols - 1) / p.cols;  // of rows, without experts
        double us = 0.0;
        cudaError_t e = choose_w4_tile(N, K, experts > 0 ? std::min<int64_t>(M, experts) : blocks,
                                       p.cols, group, p.sms, &p.tile_rows, &p.length_ctas, &us);
        if (e != cudaSuccess) return cuda_fail("choosing the tile", e);
        const int64_t depth = p.rounded ? K : 2 * K;
        p.expand = experts == 0 && blocks > 1 && depth <= LIM &&
                   std::max(M, N) <= (int64_t(1) << 45) / depth &&
                   prefers_expansion(M, N, K, dtype_out, p.rounded, us);
        int length = 0;
        if (p.expand) {
            p.gemm = gemm_create_plan(M, N, depth, dtype_out);
            if (!p.gemm) return gemm_last_status();
            length = std::snprintf(p.desc, sizeof(p.desc), "w4 expand group=%d weights=%s; %.180s",
                                   group, p.rounded ? "rounded" : "exact",
                                   gemm_plan_describe(p.gemm));
        } else {
            length = std::snprintf(p.desc, sizeof(p.desc),
                                   "w4 rows M=%lld N=%lld K=%lld group=%d experts=%d tile=%dx%d "
                                   "length_ctas=%d out=%s",
                                   static_cast<long long>(M), static_cast<long long>(N),
                                   static_cast<long long>(K), group, experts, p.tile_rows, p.cols,
                                   p.length_ctas, elt == 2 ? "f16" : "f32");
        }
        if (length < 0) p.desc[0] = '\0';
        const char* what = "allocating the device status record";
        if (!p.expand || !p.rounded) {
            e = cudaMalloc(&p.d_status, sizeof(DevStatus));
            if (e == cudaSuccess) e = cudaMemset(p.d_status, 0, sizeof(DevStatus));
        }
        if (e == cudaSuccess && p.expand) {
            what = "allocating the expanded weights";
            e = cudaMalloc(&p.d_weights, static_cast<size_t>(N) * depth * 2);
            if (e == cudaSuccess && !p.rounded)
                e = cudaMalloc(&p.d_x, static_cast<size_t>(M) * depth * 2);
            if (e == cudaSuccess && !p.rounded)
                e = cudaMalloc(&p.d_verdicts,
                               static_cast<size_t>(p.sms) * W4_EXPAND_CTAS * sizeof(int));
        }
        if (e == cudaSuccess) plan = new (std::nothrow) gemm_w4_plan(p);
        if (!plan) {
            release(p);
            return e != cudaSuccess ? cuda_fail(what, e) : fail(GEMM_ERR_CUDA, "out of host memory");
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
        if (!plan->expand)
            return run_rows(plan, X, packed, scales, zeros, expert_ids, Y, stream, 0);
        const int64_t words = plan->N * (plan->K / 8);
        const int64_t chunks = plan->rounded ? 0 : plan->M * (plan->K / 8);
        const int64_t blocks = std::min<int64_t>((std::max(words, chunks) + 255) / 256,
                                                 static_cast<int64_t>(plan->sms) * W4_EXPAND_CTAS);
        e = launch_dependent(plan->rounded ? k_w4_expand<true> : k_w4_expand<false>,
                             dim3(static_cast<unsigned>(blocks)), dim3(256), 0, 1, stream, words,
                             plan->group == 32 ? 2 : plan->group == 64 ? 3 : 4,
                             static_cast<const uint32_t*>(packed),
                             static_cast<const __half*>(scales),
                             static_cast<const uint8_t*>(zeros),
                             static_cast<uint4*>(plan->d_weights), chunks,
                             static_cast<const uint4*>(X), static_cast<uint4*>(plan->d_x),
                             plan->d_verdicts);
        if (e != cudaSuccess) return cuda_fail("weight expansion launch", e);
        const int r = gemm_run(plan->gemm, plan->rounded ? X : plan->d_x, plan->d_weights, Y,
                               cuda_stream);
        if (r != GEMM_OK || plan->rounded) return r;
        return run_rows(plan, X, packed, scales, zeros, nullptr, Y, stream,
                        static_cast<int>(blocks));
    });
}

int gemm_w4_set_wait(gemm_w4_plan* plan, int wait_budget_ms, int debug_stall)
{
    return guarded([&] {
        if (!plan) return fail(GEMM_ERR_INVALID_ARG, "plan is NULL");
        const int r = check_wait(wait_budget_ms, debug_stall);
        if (r != GEMM_OK) return r;
        plan->budget_ns = wait_ns(wait_budget_ms);
        plan->debug_stall = debug_stall;
        return ok();
    });
}

int gemm_w4_get_device_status(gemm_w4_plan* plan)
{
    return guarded([&] {
        if (!plan) return fail(GEMM_ERR_INVALID_ARG, "plan is NULL");
        const int r = plan->gemm ? gemm_get_device_status(plan->gemm) : GEMM_OK;
        return r == GEMM_OK && plan->d_status ? read_device_status(plan->d_status) : r;
    });
}

void gemm_w4_destroy(gemm_w4_plan* plan)
{
    if (!plan) return;
    release(*plan);
    delete plan;
}

const char* gemm_w4_describe(const gemm_w4_plan* plan) { return plan ? plan->desc : "(null plan)"; }

}  // extern "C"
