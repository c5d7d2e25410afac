// runtime.h -- host-side pieces every C entry point shares: the thread's error
// record behind gemm_last_error() / gemm_last_status(), the device check and
// the driver's tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <exception>
#include <string>

#include "../../include/tmagemm.h"
#include "gemm_common.h"

namespace tg {

// Record `status` and a message for this host thread; returns `status`.
int fail(int status, const std::string& msg);
// Clear the record; returns GEMM_OK.
int ok();
// GEMM_ERR_CUDA with the runtime's name and text of `e`.
int cuda_fail(const char* what, cudaError_t e);

// cuTensorMapEncodeTiled of the installed driver, or nullptr.
PFN_cuTensorMapEncodeTiled_v12000 get_encode_fn();

// The current device, its SM count and its opt-in shared memory per block;
// GEMM_ERR_NO_DEVICE when there is none or it is not sm_103.  The attributes
// are read once per device.
int require_device(int* dev, int* sms, int* smem_optin);

// Read a plan's device status record after its stream has been synchronised, and
// clear it: GEMM_OK, GEMM_ERR_TIMEOUT or GEMM_ERR_CUDA.
int read_device_status(DevStatus* record);

// Launch `kernel` as a programmatic dependent of the work before it on `stream`
// (clusters of `cluster` CTAs along x when that is above 1).  The kernel
// executes griddep_wait() in every CTA before its first global-memory access.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, dim3 block, unsigned smem_bytes,
                             int cluster, cudaStream_t stream, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem_bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// The largest size of a dimension in the expert-layer operators: a coordinate plus the
// width of a tile or the stages in flight stays within 32 bits.
constexpr int64_t MAX_COORDINATE = (int64_t(1) << 31) - 65536;

// The number of a plan's next run, > 0; threads may run one plan at the same time.
inline int next_epoch(unsigned* epoch)
{
    return static_cast<int>(__atomic_add_fetch(epoch, 1u, __ATOMIC_RELAXED) % 0x7fffffffu) + 1;
}

// The bound on a wait inside a kernel, and the checks of its setters.
constexpr unsigned long long DEFAULT_WAIT_NS = 2000ull * 1000000ull;

inline unsigned long long wait_ns(int budget_ms)
{
    return budget_ms > 0 ? static_cast<unsigned long long>(budget_ms) * 1000000ull
                         : DEFAULT_WAIT_NS;
}

inline int check_wait(int budget_ms, int debug_stall)
{
    if (budget_ms < 0) return fail(GEMM_ERR_INVALID_ARG, "wait_budget_ms must be >= 0");
    if (debug_stall < 0 || debug_stall > 2)
        return fail(GEMM_ERR_INVALID_ARG, "debug_stall must be 0, 1 or 2");
    return GEMM_OK;
}

inline bool aligned16(const void* p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// Run the body of a C entry point; a C++ exception (out of host memory)
// becomes a status instead of crossing the C boundary.
template <typename Body>
int guarded(Body body) noexcept
{
    try {
        return body();
    } catch (const std::exception&) {
        try {
            return fail(GEMM_ERR_CUDA, "out of host memory");
        } catch (...) {
            return GEMM_ERR_CUDA;
        }
    }
}

}  // namespace tg
