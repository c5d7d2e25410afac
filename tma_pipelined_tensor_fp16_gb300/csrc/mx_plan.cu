// mx_plan.cu -- host side of the block-scaled products: argument checks, the choice of the
// kernel, the tensor maps and the launch.
#include <algorithm>
#include <atomic>
#include <cstdio>
#include <new>

#include "../../include/tmamicro.h"
#include "mx_product.h"
#include "runtime.h"

using namespace tg;

// The status record of one plan or of several, and the number of their last run.
struct MxRecord {
    DevStatus* d_status;
    int device;
    unsigned epoch;
    std::atomic<int> plans;
};

struct gemm_mx_plan {
    int64_t M, N, K;
    int format, dtype;
    int device;
    bool pair, swapped;
    int cols, split;
    int stage_chunks, stage_groups;
    int grid_x, grid_y, pipe_depth, staging;
    unsigned smem_bytes;
    MxParams p;
    MxRecord* record;
    unsigned long long budget_ns;
    int debug_stall;
    char desc[256];
};

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int GROUP_M = 8;

// Tensor map over operand storage as rows of `row_bytes` (a chunk or a group of scales of
// 128 rows), boxes of `box_bytes` x `box_rows`; 64-bit elements, no swizzle, zero fill.
// With `blocks` a third dimension of so many blocks of `rows` rows, and boxes of two.
int encode_storage(CUtensorMap* map, const void* base, int64_t row_bytes, int64_t rows,
                   int box_bytes, int box_rows, const char* what, int64_t blocks = 0)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = get_encode_fn();
    if (!enc) return fail(GEMM_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(row_bytes / 8),
                                static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(blocks)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(row_bytes),
                                   static_cast<cuuint64_t>(row_bytes * rows)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_bytes / 8),
                               static_cast<cuuint32_t>(box_rows), 2};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT64, blocks ? 3 : 2,
                           const_cast<void*>(base), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        char buf[160];
        std::snprintf(buf, sizeof(buf), "cuTensorMapEncodeTiled(%s) failed with CUresult %d", what,
                      static_cast<int>(r));
        return fail(GEMM_ERR_CUDA, buf);
    }
    return GEMM_OK;
}

int encode_output(CUtensorMap* map, void* base, int64_t rows, int64_t cols, int elt)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = get_encode_fn();
    if (!enc) return fail(GEMM_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols * elt)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / elt), 32};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map,
                           elt == 2 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                           2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        char buf[160];
        std::snprintf(buf, sizeof(buf), "cuTensorMapEncodeTiled(C) failed with CUresult %d",
                      static_cast<int>(r));
        return fail(GEMM_ERR_CUDA, buf);
    }
    return GEMM_OK;
}

const char* format_name(int format)
{
    return format == MXFP8 ? "mxfp8" : format == MXFP4 ? "mxfp4" : "nvfp4";
}

int check_product(int64_t M, int64_t N, int64_t K, int format, int dtype, int kernel, int split)
{
    const int64_t LIM = MAX_COORDINATE;
    if (format < MXFP8 || format > NVFP4)
        return fail(GEMM_ERR_INVALID_ARG, "unknown gemm_mx_format");
    if (M < 1 || N < 1 || K < 1 || M > LIM || N > LIM || K > LIM)
        return fail(GEMM_ERR_INVALID_ARG, "M, N and K must be in [1, 2^31-65536]");
    if (dtype != GEMM_OUT_F32 && dtype != GEMM_OUT_F16)
        return fail(GEMM_ERR_INVALID_ARG, "dtype_out must be GEMM_OUT_F32 (0) or GEMM_OUT_F16 (1)");
    if (kernel < GEMM_MX_AUTO || kernel > GEMM_MX_SINGLE)
        return fail(GEMM_ERR_INVALID_ARG, "unknown gemm_mx_kernel");
    if (split != 0 && split != 1 && split != 2 && split != 4 && split != 8)
        return fail(GEMM_ERR_INVALID_ARG, "split must be 0, 1, 2, 4 or 8");
    if (N % (dtype == GEMM_OUT_F16 ? 8 : 4) != 0)
        return fail(GEMM_ERR_UNSUPPORTED, "N * sizeof(C element) must be a multiple of 16 bytes");
    for (const int64_t rows : {M, N})
        // a tile may start one block of rows behind the last
        if ((mx_row_blocks(rows) + 1) * mx_chunks(K, format) > LIM)
            return fail(GEMM_ERR_UNSUPPORTED, "an operand is too large");
    return GEMM_OK;
}

int make_record(int dev, MxRecord** made)
{
    MxRecord* r = new (std::nothrow) MxRecord{};
    if (!r) return fail(GEMM_ERR_CUDA, "out of host memory");
    r->device = dev;
    r->plans = 1;
    cudaError_t e = cudaMalloc(&r->d_status, sizeof(DevStatus));
    if (e == cudaSuccess) e = fill_memory(r->d_status, nullptr, sizeof(DevStatus));
    if (e != cudaSuccess) {
        if (r->d_status) cudaFree(r->d_status);
        delete r;
        return cuda_fail("allocating the device status record", e);
    }
    *made = r;
    return GEMM_OK;
}

void release(MxRecord* r)
{
    if (r->plans.fetch_sub(1) > 1) return;
    cudaFree(r->d_status);
    delete r;
}

// A plan with the record of `first`, or with one of its own where that is NULL.
gemm_mx_plan* make_plan(int64_t M, int64_t N, int64_t K, int format, int dtype_out, int kernel,
                        int split, const gemm_mx_plan* first)
{
    gemm_mx_plan* plan = nullptr;
    guarded([&] {
        int r = check_product(M, N, K, format, dtype_out, kernel, split);
        if (r != GEMM_OK) return r;
        int dev, sms, smem_optin;
        r = require_device(&dev, &sms, &smem_optin);
        if (r != GEMM_OK) return r;
        if (first && first->device != dev)
            return fail(GEMM_ERR_INVALID_ARG, "plan was created on another device");
        gemm_mx_plan q = {};
        q.M = M;
        q.N = N;
        q.K = K;
        q.format = format;
        q.dtype = dtype_out;
        q.device = dev;
        q.budget_ns = DEFAULT_WAIT_NS;
        MxParams& p = q.p;
        p.M = static_cast<int>(M);
        p.N = static_cast<int>(N);
        p.chunks = static_cast<int>(mx_chunks(K, format));
        p.groups = static_cast<int>(mx_groups(K, format));
        p.steps = p.chunks / mx_step_chunks(format);
        p.group_m = GROUP_M;
        const int64_t pair_tiles = ceil_div(M, 256) * ceil_div(N, 256);
        // Pairs from a quarter of a GPU of their tiles on, single CTAs below and for up to 64
        // rows.  Measured, pairs and single CTAs: 512 x 8192 x 8192 nvfp4 (64 tiles of pairs)
        // 14.1, 19.3 us; 2048 x 2048 x 2048 nvfp4 (64) 7.0, 8.6; 1024 x 4096 x 4096 mxfp8 (64)
        // 14.8, 17.7; 512 x 4096 x 4096 mxfp8 (32) 13.4, 11.1; 256 x 4096 x 4096 nvfp4 (16)
        // 7.8, 7.6; 64 x 16384 x 16384 mxfp8 46.9, 45.1; 1 x 16384 x 16384 nvfp4 25.9, 25.8.
        q.pair = kernel == GEMM_MX_PAIR ||
                 (kernel == GEMM_MX_AUTO && M > 64 && 4 * pair_tiles >= sms);
        q.stage_chunks = q.pair ? mx_pair_chunks(format) : mx_stage_chunks(format);
        q.stage_groups = q.pair ? mx_pair_groups(format) : mx_stage_groups(format);
        p.stages = static_cast<int>(ceil_div(p.chunks, q.stage_chunks));
        if (q.pair && split > 1)
            return fail(GEMM_ERR_INVALID_ARG, "only GEMM_MX_SINGLE takes a split");
        if (q.pair) {
            if (pair_tiles > MAX_COORDINATE)
                return fail(GEMM_ERR_UNSUPPORTED, "too many output tiles");
            p.tiles_m = static_cast<int>(ceil_div(M, 256));
            p.tiles_n = static_cast<int>(ceil_div(N, 256));
            q.grid_x = static_cast<int>(2 * std::min<int64_t>(std::max(1, sms / 2), pair_tiles));
            q.grid_y = 1;
            q.split = 1;
            q.cols = 256;
            const auto bytes = [&](int depth) {
                return mx_pair_layout(format, depth, q.staging).total;
            };
            // Short contractions are bound by their tiles' stores: two staging buffers a warp,
            // and a stage less.  8192 x 8192 nvfp4 to fp16, two and one: K = 384 24.7, 31.4 us;
            // 768 28.8, 33.1; 1536 40.2, 41.0; 2048 50.0, 46.4.  (mxfp8 has no room for them.)
            q.staging = 2;
            if (format == MXFP8 || p.stages > 8) q.staging = 1;
            for (q.pipe_depth = MAX_STAGES; q.pipe_depth > MX_PAIR_MIN_STAGES; --q.pipe_depth)
                if (bytes(q.pipe_depth) <= static_cast<uint32_t>(smem_optin)) break;
            q.smem_bytes = bytes(q.pipe_depth);
        } else {
            q.swapped = M <= 64;
            q.cols = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
            const int64_t tu = ceil_div(q.swapped ? N : M, MX_ROWS);
            const int64_t tv = q.swapped ? 1 : ceil_div(N, q.cols);
            if (split == 0) {
                // CTAs for two per SM with few rows, where the bytes in flight count, else for
                // one; each with a few stages at least.  Measured with split = 1, 2, 4, 8: 64 x
                // 16384 x 16384 mxfp8 50.0, 45.1, 49.4, 59.5 us; 16 x 8192 x 8192 nvfp4 11.5,
                // 9.6, 9.8, 14.0; 4 x 4096 x 4096 nvfp4 6.3, 5.2, 4.5, 5.2; 4 x 4096 x 14336
                // mxfp4 15.5, 10.3, 7.5, 7.3; 256 x 4096 x 4096 nvfp4 7.9, 7.6, 9.6, 17.9.
                const int64_t room = q.swapped ? 2 * sms : sms;
                split = 1;
                while (split < 8 && tu * tv * split * 2 <= room && p.stages >= 8 * split)
                    split *= 2;
            }
            while (split > p.stages) split /= 2;
            q.split = split;
            if (tu * split > MAX_COORDINATE || tv > 65535)
                return fail(GEMM_ERR_UNSUPPORTED, "too many output tiles");
            q.grid_x = static_cast<int>(tu * split);
            q.grid_y = static_cast<int>(tv);
            p.tiles_m = static_cast<int>(tu);
            p.tiles_n = static_cast<int>(tv);
            // two CTAs on an SM
            const uint32_t room = 113u * 1024u;
            for (q.pipe_depth = MAX_STAGES; q.pipe_depth > 2; --q.pipe_depth)
                if (mx_single_layout(format, q.cols, q.pipe_depth, q.swapped).total <= room) break;
            q.smem_bytes = mx_single_layout(format, q.cols, q.pipe_depth, q.swapped).total;
        }
        if (q.smem_bytes > static_cast<unsigned>(smem_optin))
            return fail(GEMM_ERR_UNSUPPORTED, "no stage count fits shared memory");
        p.split = q.split;
        p.pipe_depth = q.pipe_depth;
        std::snprintf(q.desc, sizeof(q.desc),
                      "mx format=%s M=%lld N=%lld K=%lld kernel=%s tile=%dx%d split=%d "
                      "pipe_depth=%d smem=%u grid=%dx%d out=%s",
                      format_name(format), static_cast<long long>(M), static_cast<long long>(N),
                      static_cast<long long>(K),
                      q.pair ? "pair" : q.swapped ? "rows" : "single", q.pair ? 256 : 128, q.cols,
                      q.split, q.pipe_depth, q.smem_bytes, q.grid_x, q.grid_y,
                      dtype_out == GEMM_OUT_F16 ? "f16" : "f32");
        if (first) {
            q.record = first->record;
            q.record->plans.fetch_add(1);
        } else {
            r = make_record(dev, &q.record);
            if (r != GEMM_OK) return r;
        }
        plan = new (std::nothrow) gemm_mx_plan(q);
        if (!plan) {
            release(q.record);
            return fail(GEMM_ERR_CUDA, "out of host memory");
        }
        return ok();
    });
    return plan;
}

}  // namespace

extern "C" {

gemm_mx_plan* gemm_mx_create_plan(int64_t M, int64_t N, int64_t K, int format, int dtype_out)
{
    return make_plan(M, N, K, format, dtype_out, GEMM_MX_AUTO, 0, nullptr);
}

gemm_mx_plan* gemm_mx_create_plan_ex(int64_t M, int64_t N, int64_t K, int format, int dtype_out,
                                     int kernel, int split)
{
    return make_plan(M, N, K, format, dtype_out, kernel, split, nullptr);
}

gemm_mx_plan* gemm_mx_create_plan_beside(const gemm_mx_plan* plan, int64_t M, int64_t N, int64_t K,
                                         int dtype_out, int kernel, int split)
{
    if (!plan) {
        guarded([&] { return fail(GEMM_ERR_INVALID_ARG, "plan is NULL"); });
        return nullptr;
    }
    return make_plan(M, N, K, plan->format, dtype_out, kernel, split, plan);
}

int gemm_mx_run(gemm_mx_plan* plan, const void* codes_a, const void* scales_a, const float* scale_a,
                const void* codes_b, const void* scales_b, const float* scale_b, void* C,
                void* cuda_stream)
{
    return guarded([&] {
        if (!plan) return fail(GEMM_ERR_INVALID_ARG, "plan is NULL");
        if (!codes_a || !scales_a || !codes_b || !scales_b || !C)
            return fail(GEMM_ERR_INVALID_ARG, "codes, scales and C must be non-NULL");
        if (!aligned16(codes_a) || !aligned16(scales_a) || !aligned16(codes_b) ||
            !aligned16(scales_b) || !aligned16(C))
            return fail(GEMM_ERR_UNSUPPORTED, "codes, scales and C must be 16-byte aligned (TMA)");
        if ((scale_a || scale_b) && plan->format != NVFP4)
            return fail(GEMM_ERR_INVALID_ARG, "only GEMM_NVFP4 has tensor scales");
        if ((reinterpret_cast<uintptr_t>(scale_a) | reinterpret_cast<uintptr_t>(scale_b)) & 3u)
            return fail(GEMM_ERR_UNSUPPORTED, "tensor scales must be 4-byte aligned");
        int dev = -1;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return cuda_fail("cudaGetDevice", e);
        if (dev != plan->device)
            return fail(GEMM_ERR_INVALID_ARG, "plan was created on another device");
        const int f = plan->format;
        const MxParams& q = plan->p;
        const int64_t a_blocks = mx_row_blocks(plan->M), b_blocks = mx_row_blocks(plan->N);
        const bool swapped = plan->swapped;
        const int v_bytes = plan->pair ? MX_CHUNK_BYTES : plan->cols * 16;
        CUtensorMap tmUc, tmUs, tmVc, tmVs, tmC;
        int r = encode_storage(&tmUc, swapped ? codes_b : codes_a, MX_CHUNK_BYTES,
                               (swapped ? b_blocks : a_blocks) * q.chunks, MX_CHUNK_BYTES,
                               plan->stage_chunks, "codes");
        if (r == GEMM_OK)
            r = encode_storage(&tmUs, swapped ? scales_b : scales_a, MX_GROUP_BYTES,
                               (swapped ? b_blocks : a_blocks) * q.groups, MX_GROUP_BYTES,
                               plan->stage_groups, "scales");
        if (r == GEMM_OK)
            r = encode_storage(&tmVc, swapped ? codes_a : codes_b, MX_CHUNK_BYTES,
                               (swapped ? a_blocks : b_blocks) * q.chunks, v_bytes,
                               plan->stage_chunks, "codes");
        if (r == GEMM_OK)
            r = plan->pair ? encode_storage(&tmVs, scales_b, MX_GROUP_BYTES, q.groups,
                                            MX_GROUP_BYTES, plan->stage_groups, "scales", b_blocks)
                           : encode_storage(&tmVs, swapped ? scales_a : scales_b, MX_GROUP_BYTES,
                                            (swapped ? a_blocks : b_blocks) * q.groups,
                                            MX_GROUP_BYTES, plan->stage_groups, "scales");
        if (r == GEMM_OK && plan->pair)
            r = encode_output(&tmC, C, plan->M, plan->N, plan->dtype == GEMM_OUT_F16 ? 2 : 4);
        if (r != GEMM_OK) return r;
        MxSpec s = {};
        s.format = f;
        s.f16out = plan->dtype == GEMM_OUT_F16;
        s.pair = plan->pair;
        s.cols = plan->cols;
        s.swapped = swapped;
        s.grid_x = plan->grid_x;
        s.grid_y = plan->grid_y;
        s.staging = plan->staging;
        s.smem_bytes = plan->smem_bytes;
        s.codes_u = &tmUc;
        s.scales_u = &tmUs;
        s.codes_v = &tmVc;
        s.scales_v = &tmVs;
        s.out = &tmC;
        s.p = q;
        s.p.scale_a = scale_a;
        s.p.scale_b = scale_b;
        s.p.C = C;
        s.p.status = plan->record->d_status;
        s.p.epoch = next_epoch(&plan->record->epoch);
        s.p.budget_ns = plan->budget_ns;
        s.p.debug_stall = plan->debug_stall;
        cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
        e = plan->pair ? launch_mx_pair(s, stream) : launch_mx_single(s, stream);
        return e == cudaSuccess ? ok() : cuda_fail("block-scaled product launch", e);
    });
}

int gemm_mx_set_wait(gemm_mx_plan* plan, int wait_budget_ms, int debug_stall)
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

int gemm_mx_get_device_status(gemm_mx_plan* plan)
{
    return guarded([&] {
        if (!plan) return fail(GEMM_ERR_INVALID_ARG, "plan is NULL");
        return read_device_status(plan->record->d_status);
    });
}

void gemm_mx_destroy(gemm_mx_plan* plan)
{
    if (!plan) return;
    release(plan->record);
    delete plan;
}

const char* gemm_mx_describe(const gemm_mx_plan* plan)
{
    return plan ? plan->desc : "(null plan)";
}

}  // extern "C"
