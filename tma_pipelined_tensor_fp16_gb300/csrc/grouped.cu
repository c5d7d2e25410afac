// grouped.cu -- host side of the grouped products: argument checks, the choice
// of the tile width, the tensor maps and the launch.
#include "grouped.h"

#include <algorithm>
#include <cstdio>
#include <cstring>
#include <memory>
#include <mutex>
#include <new>
#include <vector>

#include "../../include/tmaexperts.h"
#include "counter_slots.h"
#include "runtime.h"

using namespace tg;

struct gemm_grouped_plan {
    int64_t rows, N, K;
    int experts, op, dtype;
    int device;
    bool pair;
    int block_m, block_n, grid, pipe_depth;
    unsigned smem_bytes;
    int tiles_m, tiles_n;
    DevStatus* d_status;
    unsigned epoch;
    unsigned long long budget_ns;
    int debug_stall;
    char desc[256];
};

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Raster group height in tiles.  Lower for the weight gradient on pairs, whose stores
// then fill rows of the output sooner (16 experts of 2048 x 4096, fp32: 231 us with 8, 226
// with 4; forward and input gradient no better with 4 or 16).
constexpr int GROUP_M = 8;
constexpr int GROUP_M_PAIR_WEIGHT = 4;

// Tensor map over `planes` row-major matrices of `rows` x `cols` (planes = 0: a
// single matrix, a 2-D map), 128-byte swizzle, zero fill out of bounds.
int encode(CUtensorMap* map, CUtensorMapDataType dt, int elt, const void* base, int64_t cols,
           int64_t rows, int64_t planes, int box_cols, int box_rows, const char* what)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = get_encode_fn();
    if (!enc) return fail(GEMM_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(planes)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols * elt),
                                   static_cast<cuuint64_t>(cols * elt * rows)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols),
                               static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const bool rows_on_256 =
        (cols * elt) % 256 == 0 && reinterpret_cast<uintptr_t>(base) % 256 == 0;
    CUresult r = enc(map, dt, planes ? 3 : 2, const_cast<void*>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     rows_on_256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                 : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        char buf[160];
        std::snprintf(buf, sizeof(buf), "cuTensorMapEncodeTiled(%s) failed with CUresult %d", what,
                      static_cast<int>(r));
        return fail(GEMM_ERR_CUDA, buf);
    }
    return GEMM_OK;
}

constexpr int PAIR_DEPTH = 3;  // stages of two K blocks in the pair kernel

// Row tiles of height bm that a plan can expect: exact for GRAD_WEIGHT; else an
// expert's last tile is half full on average, and every expert has one.
int64_t expected_row_tiles(int64_t rows, int64_t N, int experts, int op, int bm)
{
    if (op == GROUPED_GRAD_WEIGHT) return ceil_div(N, bm) * experts;
    const int64_t used = std::min<int64_t>(experts, rows);
    return std::max(ceil_div(rows, bm) + used / 2, used);
}

// The automatic tile: the one whose waves of tiles (a launch that hands out its
// tiles ends half a wave after the last full one) take the least time, at each
// tile's throughput per SM relative to pairs: 0.82 for 128 x 256 on single CTAs,
// 0.70 for 128 x 128.  Measured, pairs, 128 x 256, 128 x 128: 16 even experts of 4096 x
// 4096 with 1024 rows each 334, 351, 457 us; 29 uneven experts of 1400 x 1744 with 18013
// rows, input gradient, 84, 92, 119; uneven experts of 2816 x 2048, input gradient, 32
// with 256 rows on average 97, 102, 126, and 64 with 128 rows 148, 126, 146; 4 experts
// of 488 x 2136 with 1810 rows 22, 25, 18; 41 experts of 3440 x 1920 with 78 rows in all
// 87, 77, 79.  GRAD_WEIGHT's tiles of few rows are bounded by their stores, in which
// pairs are slower (fp32, experts of 2048 x 4096: pairs 247 and 128 x 256 233 us at 512
// rows per expert, 287 and 280 at 682, 226 and 232 at 1024, 186 and 194 at 2048).
int choose_tile(int64_t rows, int64_t N, int64_t cols, int experts, int op, int sms, bool pair_fits)
{
    struct Tile {
        int kind, bm, bn, slots;
        double rate;
    };
    const Tile tiles[3] = {{GEMM_GROUPED_TILE_256X256, 256, 256, std::max(1, sms / 2), 2.0},
                           {GEMM_GROUPED_TILE_128X256, 128, 256, sms, 0.82},
                           {GEMM_GROUPED_TILE_128X128, 128, 128, sms, 0.70}};
    int best = GEMM_GROUPED_TILE_128X256;
    double best_time = -1.0;
    for (const Tile& t : tiles) {
        if (t.kind == GEMM_GROUPED_TILE_256X256 &&
            (!pair_fits || (op == GROUPED_GRAD_WEIGHT && rows < 800ll * experts)))
            continue;
        const int64_t count = expected_row_tiles(rows, N, experts, op, t.bm) * ceil_div(cols, t.bn);
        const double waves =
            count <= t.slots ? 1.0 : static_cast<double>(count) / t.slots + 0.5;
        const double time = waves * t.bm * t.bn / t.rate;
        if (best_time < 0.0 || time < best_time) {
            best_time = time;
            best = t.kind;
        }
    }
    return best;
}

const char* op_name(int op)
{
    return op == GROUPED_FORWARD      ? "forward"
           : op == GROUPED_GRAD_INPUT ? "grad_input"
                                      : "grad_weight";
}

// Output columns, and rows of one tile column of the whole output.
int64_t out_cols_of(const gemm_grouped_plan& p)
{
    return p.op == GROUPED_FORWARD ? p.N : p.K;
}

int check_grouped(int64_t rows, int64_t N, int64_t K, int experts, int op, int dtype)
{
    const int64_t LIM = MAX_COORDINATE;
    if (rows < 0 || N < 1 || K < 1 || rows > LIM || N > LIM || K > LIM)
        return fail(GEMM_ERR_INVALID_ARG,
                    "rows must be in [0, 2^31-65536], N and K in [1, 2^31-65536]");
    if (experts < 1 || experts > GROUPED_MAX_EXPERTS)
        return fail(GEMM_ERR_INVALID_ARG, "experts must be in 1..1024");
    if (op < GROUPED_FORWARD || op > GROUPED_GRAD_WEIGHT)
        return fail(GEMM_ERR_INVALID_ARG, "unknown gemm_grouped_op");
    if (dtype != GEMM_OUT_F32 && dtype != GEMM_OUT_F16)
        return fail(GEMM_ERR_INVALID_ARG, "dtype_out must be GEMM_OUT_F32 (0) or GEMM_OUT_F16 (1)");
    if (N % 8 != 0 || K % 8 != 0)
        return fail(GEMM_ERR_UNSUPPORTED,
                    "N and K must be multiples of 8: the TMA row strides must be multiples of 16 bytes");
    if (N > LIM / experts || N * K >= (int64_t(1) << 38))
        return fail(GEMM_ERR_UNSUPPORTED, "experts * N or N * K is too large");
    return GEMM_OK;
}

// A device's tile counters, all zero between runs.  Made with its first plan and kept:
// graphs may outlive every plan.
struct CounterPool {
    CounterSlots slots;
    unsigned long long* d_counters = nullptr;
};

std::mutex g_pool_mutex;
std::vector<CounterPool*> g_pools;  // by device

int make_counters(int dev)
{
    std::lock_guard<std::mutex> lock(g_pool_mutex);
    if (g_pools.size() <= static_cast<size_t>(dev)) g_pools.resize(dev + 1, nullptr);
    if (g_pools[dev]) return GEMM_OK;
    std::unique_ptr<CounterPool> pool(new CounterPool);
    constexpr size_t BYTES = CounterSlots::COUNT * sizeof(unsigned long long);
    cudaError_t e = cudaMalloc(&pool->d_counters, BYTES);
    if (e == cudaSuccess) e = fill_memory(pool->d_counters, nullptr, BYTES);
    if (e != cudaSuccess) {
        if (pool->d_counters) cudaFree(pool->d_counters);
        return cuda_fail("allocating the tile counters", e);
    }
    g_pools[dev] = pool.release();
    return GEMM_OK;
}

CounterPool& pool_of(int dev)
{
    std::lock_guard<std::mutex> lock(g_pool_mutex);
    return *g_pools[dev];
}

// A captured launch's hold on its counter, which ends with the graph.
struct CapturedSlot {
    CounterSlots* slots;
    int slot;
};

void CUDART_CB release_captured(void* p)
{
    CapturedSlot* held = static_cast<CapturedSlot*>(p);
    held->slots->release(held->slot);
    delete held;
}

// The tile counter of a run on `stream` (see counter_slots.h).
int counter_of(CounterSlots& slots, cudaStream_t stream, int* slot)
{
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(stream, &status);
    if (e != cudaSuccess) return cuda_fail("cudaStreamIsCapturing", e);
    if (status != cudaStreamCaptureStatusActive) {
        unsigned long long id = 0;
        e = cudaStreamGetId(stream, &id);
        if (e != cudaSuccess) return cuda_fail("cudaStreamGetId", e);
        bool taken_over = false;
        *slot = slots.of_stream(id, &taken_over);
        if (taken_over) e = cudaDeviceSynchronize();
        if (e == cudaSuccess) return GEMM_OK;
        slots.give_up(*slot);
        return cuda_fail("cudaDeviceSynchronize", e);
    }
    std::unique_ptr<CapturedSlot> held(new CapturedSlot{&slots, slots.of_capture()});
    *slot = held->slot;
    if (held->slot < 0)
        return fail(GEMM_ERR_UNSUPPORTED, "too many live CUDA graphs hold grouped products");
    cudaGraph_t graph = nullptr;
    cudaUserObject_t object = nullptr;
    e = cudaStreamGetCaptureInfo(stream, &status, nullptr, &graph, nullptr, nullptr, nullptr);
    if (e == cudaSuccess)
        e = cudaUserObjectCreate(&object, held.get(), release_captured, 1,
                                 cudaUserObjectNoDestructorSync);
    if (e != cudaSuccess) {
        slots.release(*slot);
        return cuda_fail("tying a tile counter to the graph", e);
    }
    held.release();  // the object's now
    e = cudaGraphRetainUserObject(graph, object, 1, cudaGraphUserObjectMove);
    if (e != cudaSuccess) {
        cudaUserObjectRelease(object, 1);
        return cuda_fail("tying a tile counter to the graph", e);
    }
    return GEMM_OK;
}

}  // namespace

extern "C" {

gemm_grouped_plan* gemm_grouped_create_plan(int64_t rows, int64_t N, int64_t K, int experts, int op,
                                            int dtype_out)
{
    return gemm_grouped_create_plan_ex(rows, N, K, experts, op, dtype_out, GEMM_GROUPED_TILE_AUTO);
}

gemm_grouped_plan* gemm_grouped_create_plan_ex(int64_t rows, int64_t N, int64_t K, int experts,
                                               int op, int dtype_out, int tile)
{
    gemm_grouped_plan* plan = nullptr;
    guarded([&] {
        int r = check_grouped(rows, N, K, experts, op, dtype_out);
        if (r != GEMM_OK) return r;
        if (tile < GEMM_GROUPED_TILE_AUTO || tile > GEMM_GROUPED_TILE_256X256)
            return fail(GEMM_ERR_INVALID_ARG, "unknown gemm_grouped_tile");
        int dev, sms, smem_optin;
        r = require_device(&dev, &sms, &smem_optin);
        if (r != GEMM_OK) return r;
        gemm_grouped_plan p = {};
        p.rows = rows;
        p.N = N;
        p.K = K;
        p.experts = experts;
        p.op = op;
        p.dtype = dtype_out;
        p.device = dev;
        p.budget_ns = DEFAULT_WAIT_NS;
        const int64_t cols = out_cols_of(p);
        const uint32_t table = grouped_table_bytes(op, experts);
        const bool pair_fits = smem_layout(2 * PAIR_DEPTH, 128, NUM_STAGING).total + table <=
                               static_cast<uint32_t>(smem_optin);
        if (tile == GEMM_GROUPED_TILE_256X256 && !pair_fits)
            return fail(GEMM_ERR_UNSUPPORTED,
                        "tiles of 256 x 256 leave no shared memory for so many experts");
        if (tile == GEMM_GROUPED_TILE_AUTO)
            tile = choose_tile(rows, N, cols, experts, op, sms, pair_fits);
        p.pair = tile == GEMM_GROUPED_TILE_256X256;
        p.block_m = p.pair ? 2 * BLK_M : BLK_M;
        p.block_n = tile == GEMM_GROUPED_TILE_128X128 ? 128 : 256;
        // at most one more tile per expert than its rows fill (and one group for
        // the rows that belong to none)
        const int64_t most = op == GROUPED_GRAD_WEIGHT
                                 ? ceil_div(N, p.block_m) * experts
                                 : rows / p.block_m + std::min<int64_t>(experts + 1, rows);
        const int64_t tn = ceil_div(cols, p.block_n);
        if (most * tn >= (int64_t(1) << 31) - 65536)
            return fail(GEMM_ERR_UNSUPPORTED, "too many output tiles");
        p.tiles_n = static_cast<int>(tn);
        p.tiles_m = static_cast<int>(ceil_div(N, p.block_m));
        if (p.pair) {
            p.grid = static_cast<int>(2 * std::max<int64_t>(1, std::min<int64_t>(sms / 2, most * tn)));
            p.pipe_depth = PAIR_DEPTH;
            p.smem_bytes = smem_layout(2 * PAIR_DEPTH, 128, NUM_STAGING).total + table;
        } else {
            p.grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(sms, most * tn)));
            for (int d = MAX_STAGES; d >= 1; --d) {
                const uint32_t need = smem_layout(d, p.block_n, NUM_STAGING).total + table;
                if (need <= static_cast<uint32_t>(smem_optin)) {
                    p.pipe_depth = d;
                    p.smem_bytes = need;
                    break;
                }
            }
            if (p.pipe_depth < 2)
                return fail(GEMM_ERR_UNSUPPORTED, "no stage count fits shared memory");
        }
        std::snprintf(p.desc, sizeof(p.desc),
                      "grouped op=%s rows=%lld N=%lld K=%lld experts=%d tile=%dx%dx%d "
                      "pipe_depth=%d smem=%u grid=%d out=%s",
                      op_name(op), static_cast<long long>(rows), static_cast<long long>(N),
                      static_cast<long long>(K), experts, p.block_m, p.block_n,
                      p.pair ? 2 * BLK_K : BLK_K, p.pipe_depth,
                      p.smem_bytes, p.grid, dtype_out == GEMM_OUT_F16 ? "f16" : "f32");
        r = make_counters(dev);
        if (r != GEMM_OK) return r;
        cudaError_t e = cudaMalloc(&p.d_status, sizeof(DevStatus));
        if (e == cudaSuccess) e = fill_memory(p.d_status, nullptr, sizeof(DevStatus));
        if (e != cudaSuccess) {
            if (p.d_status) cudaFree(p.d_status);
            return cuda_fail("allocating the device status record", e);
        }
        plan = new (std::nothrow) gemm_grouped_plan(p);
        if (!plan) {
            cudaFree(p.d_status);
            return fail(GEMM_ERR_CUDA, "out of host memory");
        }
        return ok();
    });
    return plan;
}

int gemm_grouped_run(gemm_grouped_plan* plan, const void* P, const void* Q,
                     const int32_t* offsets, void* out, void* cuda_stream)
{
    return guarded([&] {
        if (!plan) return fail(GEMM_ERR_INVALID_ARG, "plan is NULL");
        const bool weight = plan->op == GROUPED_GRAD_WEIGHT;
        if (plan->rows == 0 && !weight) return ok();
        if (!offsets || !out || (plan->rows > 0 && (!P || !Q)))
            return fail(GEMM_ERR_INVALID_ARG, "P, Q, offsets and out must be non-NULL");
        if (!aligned16(P) || !aligned16(Q) || !aligned16(out))
            return fail(GEMM_ERR_UNSUPPORTED, "P, Q and out must be 16-byte aligned (TMA)");
        if (reinterpret_cast<uintptr_t>(offsets) & 3u)
            return fail(GEMM_ERR_UNSUPPORTED, "offsets must be 4-byte aligned");
        int dev = -1;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return cuda_fail("cudaGetDevice", e);
        if (dev != plan->device)
            return fail(GEMM_ERR_INVALID_ARG, "plan was created on another device");
        cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
        const int64_t R = plan->rows, N = plan->N, K = plan->K, E = plan->experts;
        const int elt = plan->dtype == GEMM_OUT_F16 ? 2 : 4;
        const int64_t cols = out_cols_of(*plan);
        if (R == 0) {  // no rows at all: every expert's weight gradient is zero
            e = cudaMemsetAsync(out, 0, static_cast<size_t>(E) * N * K * elt, stream);
            return e == cudaSuccess ? ok() : cuda_fail("cudaMemsetAsync", e);
        }
        const CUtensorMapDataType F16 = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
        const CUtensorMapDataType OUT =
            elt == 2 ? F16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
        CUtensorMap tmA, tmS, tmB, tmC;
        int r;
        if (plan->op == GROUPED_FORWARD) {
            r = encode(&tmA, F16, 2, P, K, R, 0, BLK_K, BLK_M, "A");
            if (r == GEMM_OK)
                r = encode(&tmB, F16, 2, Q, K, N, E, BLK_K,
                           plan->pair ? plan->block_n / 2 : plan->block_n, "B");
        } else if (plan->op == GROUPED_GRAD_INPUT) {
            r = encode(&tmA, F16, 2, P, N, R, 0, BLK_K, BLK_M, "dC");
            if (r == GEMM_OK) r = encode(&tmB, F16, 2, Q, K, N, E, 64, BLK_K, "B");
        } else {
            r = encode(&tmA, F16, 2, P, N, R, 0, 64, BLK_K, "dC");
            if (r == GEMM_OK) r = encode(&tmB, F16, 2, Q, K, R, 0, 64, BLK_K, "A");
        }
        if (r == GEMM_OK && !weight && !plan->pair)
            r = encode(&tmS, F16, 2, P, plan->op == GROUPED_FORWARD ? K : N, R, 0, BLK_K,
                       GROUPED_SMALL_ROWS, "rows");
        else
            tmS = tmA;  // not used
        if (r == GEMM_OK)
            r = weight ? encode(&tmC, OUT, elt, out, K, N, E, 128 / elt, 32, "dB")
                       : encode(&tmC, OUT, elt, out, cols, R, 0, 128 / elt, 32, "out");
        if (r != GEMM_OK) return r;

        GroupedSpec s = {};
        s.op = plan->op;
        s.block_n = plan->block_n;
        s.pair = plan->pair;
        s.f16out = elt == 2;
        s.grid = plan->grid;
        s.smem_bytes = plan->smem_bytes;
        s.tmA = &tmA;
        s.tmS = &tmS;
        s.tmB = &tmB;
        s.tmC = &tmC;
        GroupedParams& p = s.p;
        p.rows = static_cast<int>(R);
        p.out_rows = static_cast<int>(weight ? N : R);
        p.out_cols = static_cast<int>(cols);
        p.depth = static_cast<int>(plan->op == GROUPED_GRAD_INPUT ? N : K);
        p.experts = plan->experts;
        p.tiles_n = plan->tiles_n;
        p.tiles_m = plan->tiles_m;
        p.group_m = weight && plan->pair ? GROUP_M_PAIR_WEIGHT : GROUP_M;
        p.pipe_depth = plan->pipe_depth;
        p.offsets = offsets;
        p.out = out;
        p.status = plan->d_status;
        int slot = -1;
        CounterPool& pool = pool_of(dev);
        r = counter_of(pool.slots, stream, &slot);
        if (r != GEMM_OK) return r;
        p.counter = pool.d_counters + slot;
        p.epoch = next_epoch(&plan->epoch);
        p.budget_ns = plan->budget_ns;
        p.debug_stall = plan->debug_stall;
        e = launch_grouped(s, stream);
        return e == cudaSuccess ? ok() : cuda_fail("grouped product launch", e);
    });
}

int gemm_grouped_set_wait(gemm_grouped_plan* plan, int wait_budget_ms, int debug_stall)
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

int gemm_grouped_get_device_status(gemm_grouped_plan* plan)
{
    return guarded([&] {
        if (!plan) return fail(GEMM_ERR_INVALID_ARG, "plan is NULL");
        return read_device_status(plan->d_status);
    });
}

void gemm_grouped_destroy(gemm_grouped_plan* plan)
{
    if (!plan) return;
    if (plan->d_status) cudaFree(plan->d_status);
    delete plan;
}

const char* gemm_grouped_describe(const gemm_grouped_plan* plan)
{
    return plan ? plan->desc : "(null plan)";
}

}  // extern "C"

namespace tg {

template <int OP>
cudaError_t launch_grouped_op(const GroupedSpec& s, cudaStream_t stream);

cudaError_t launch_grouped(const GroupedSpec& s, cudaStream_t stream)
{
    switch (s.op) {
    case GROUPED_FORWARD: return launch_grouped_op<GROUPED_FORWARD>(s, stream);
    case GROUPED_GRAD_INPUT: return launch_grouped_op<GROUPED_GRAD_INPUT>(s, stream);
    case GROUPED_GRAD_WEIGHT: return launch_grouped_op<GROUPED_GRAD_WEIGHT>(s, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace tg
