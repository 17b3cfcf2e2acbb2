// host_util.cuh -- host-side helpers shared by the ABI implementations: pointer checks, launch
// status, opt-in shared memory, device properties.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "osdn.h"

namespace osdn {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

inline size_t io_size(osdn_dtype_t io) { return io == OSDN_BF16 ? 2 : 4; }

inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

inline osdn_status_t launch_status() {
    return cudaGetLastError() == cudaSuccess ? OSDN_OK : OSDN_ERR_CUDA;
}

template <typename KernelT>
inline bool set_smem(KernelT kernel, size_t bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)bytes) == cudaSuccess;
}

inline int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        return 148;
    return n;
}

// cuTensorMapEncodeTiled from the driver, looked up once through the runtime (the library
// does not link libcuda directly).
using EncodeTiledFn = PFN_cuTensorMapEncodeTiled_v12000;
inline EncodeTiledFn tensor_map_encoder() {
    static EncodeTiledFn fn = []() -> EncodeTiledFn {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// Reads and clears the device status word of mixer_lib.cu's kernels (each translation unit of
// the library has its own).  False if the copy fails.
bool take_mixer_status(int* value);

}  // namespace osdn
