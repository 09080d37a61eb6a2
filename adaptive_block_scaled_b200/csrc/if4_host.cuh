// Host side shared by the stream-ordered kernels: device properties, the
// checks of a dense tensor's description, and the programmatic launch.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>

#include "../../include/if4.h"

namespace {

constexpr int MAX_DEVICES = 64;

struct DeviceInfo {
    int id = 0;
    int sm_count = 0;
    int cc_major = 0;
};

bool device_info(DeviceInfo &out)
{
    static std::mutex mu;
    static DeviceInfo cache[MAX_DEVICES];
    static bool have[MAX_DEVICES] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= MAX_DEVICES) return false;
    std::lock_guard<std::mutex> lock(mu);
    if (!have[dev]) {
        DeviceInfo d;
        d.id = dev;
        if (cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return false;
        if (cudaDeviceGetAttribute(&d.cc_major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
            return false;
        cache[dev] = d;
        have[dev] = true;
    }
    out = cache[dev];
    return true;
}

int check_device(DeviceInfo &d)
{
    if (!device_info(d)) return IF4_ERR_CUDA;
    if (d.cc_major != 10) return IF4_ERR_DEVICE;
    return IF4_OK;
}

// Status of a launch.  A failed one leaves nothing in the runtime's last error,
// which the next call would take for its own.
inline int launched(cudaError_t e)
{
    if (e == cudaSuccess) return IF4_OK;
    (void)cudaGetLastError();
    return IF4_ERR_CUDA;
}

// Raises a kernel's dynamic shared-memory limit, once per device (a race only
// repeats the call; nothing here throws).
typedef std::atomic<bool> OncePerDevice[MAX_DEVICES];

template <typename Kernel>
int allow_smem(Kernel kernel, int bytes, const DeviceInfo &d, OncePerDevice &done)
{
    if (!done[d.id].load(std::memory_order_acquire)) {
        const int rc = launched(
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
        if (rc != IF4_OK) return rc;
        done[d.id].store(true, std::memory_order_release);
    }
    return IF4_OK;
}

int elem_size(int dt)
{
    switch (dt) {
    case IF4_F32: return 4;
    case IF4_BF16: return 2;
    case IF4_F16: return 2;
    default: return 0;
    }
}

struct Shape {
    uint32_t gpr = 0, ngroups = 0;
    int64_t ld_bytes = 0;
    bool contig = false, v8 = false;
};

// Validate a dense input or output tensor description.
int check_tensor(const void *p, int dt, int64_t rows, int64_t cols, int64_t ld, Shape &s)
{
    const int es = elem_size(dt);
    if (es == 0) return IF4_ERR_DTYPE;
    if (rows < 0 || cols < 0 || cols % 16 != 0 || ld < cols) return IF4_ERR_SHAPE;
    if (rows > 0 && (cols / 16) > 0 && rows > (int64_t)0x7FFFFFFF / (cols / 16)) return IF4_ERR_SHAPE;
    if (rows > 0 && cols > 0 && p == nullptr) return IF4_ERR_NULL;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (a % 16 != 0 || (ld * es) % 16 != 0) return IF4_ERR_ALIGN;
    s.gpr = (uint32_t)(cols / 16);
    s.ngroups = (uint32_t)(rows * (cols / 16));
    s.ld_bytes = ld * es;
    s.contig = (ld == cols) || rows <= 1;
    s.v8 = (a % 32 == 0) && (s.ld_bytes % 32 == 0);
    return IF4_OK;
}

int launch_status()
{
    return cudaGetLastError() == cudaSuccess ? IF4_OK : IF4_ERR_CUDA;
}

// Launch of the stream-ordered kernels (amax, scale, quantize, dequantize)
// with programmatic dependent launch: each such kernel lets the next one be
// scheduled while it drains, and waits for its predecessor's results before
// reading anything (pdl_enter), so stream order holds as usual.
template <typename... KArgs, typename... Args>
int launch_k(void (*k)(KArgs...), unsigned grid, unsigned block, cudaStream_t st, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(block, 1, 1);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return launched(cudaLaunchKernelEx(&cfg, k, args...));
}

}  // namespace
