// runtime.cu -- the device check and the status record's reader, shared by the C
// entry points.
#include <cstdio>
#include <mutex>

#include "runtime.h"

namespace tg {

namespace {
constexpr int MAX_DEVICES = 64;
struct DeviceInfo {
    bool known;
    int major, minor, sms, smem_optin;
};
std::mutex g_device_mutex;
DeviceInfo g_devices[MAX_DEVICES] = {};
}  // namespace

int require_device(int* dev, int* sms, int* smem_optin)
{
    cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess)
        return fail(GEMM_ERR_NO_DEVICE, std::string("no CUDA device: ") + cudaGetErrorString(e));
    DeviceInfo info = {};
    std::lock_guard<std::mutex> lock(g_device_mutex);
    if (*dev < MAX_DEVICES) info = g_devices[*dev];
    if (!info.known) {
        e = cudaDeviceGetAttribute(&info.major, cudaDevAttrComputeCapabilityMajor, *dev);
        if (e == cudaSuccess)
            e = cudaDeviceGetAttribute(&info.minor, cudaDevAttrComputeCapabilityMinor, *dev);
        if (e == cudaSuccess)
            e = cudaDeviceGetAttribute(&info.sms, cudaDevAttrMultiProcessorCount, *dev);
        if (e == cudaSuccess)
            e = cudaDeviceGetAttribute(&info.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin,
                                       *dev);
        if (e != cudaSuccess) return cuda_fail("cudaDeviceGetAttribute", e);
        info.known = true;
        if (*dev < MAX_DEVICES) g_devices[*dev] = info;
    }
    if (info.major != 10 || info.minor != 3) {
        char buf[160];
        std::snprintf(buf, sizeof(buf),
                      "device %d is sm_%d%d; this library is built for sm_103a (GB300) only", *dev,
                      info.major, info.minor);
        return fail(GEMM_ERR_NO_DEVICE, buf);
    }
    if (sms) *sms = info.sms;
    if (smem_optin) *smem_optin = info.smem_optin;
    return GEMM_OK;
}

int read_device_status(DevStatus* record)
{
    DevStatus st;
    cudaError_t e = cudaMemcpy(&st, record, sizeof(st), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail("reading the device status record", e);
    DevStatus left = st;
    const int code = take_status(&left);
    if (code == DEV_OK) return ok();
    e = cudaMemcpy(record, &left, sizeof(left), cudaMemcpyHostToDevice);
    if (e != cudaSuccess) return cuda_fail("clearing the device status record", e);
    char buf[200];
    std::snprintf(buf, sizeof(buf),
                  "kernel wait timed out (where=%d block=%d tile=%d k_block=%d); the run was abandoned",
                  st.where, st.block, st.tile, st.kblock);
    return fail(code == DEV_TIMEOUT ? GEMM_ERR_TIMEOUT : GEMM_ERR_CUDA, buf);
}

}  // namespace tg
