// Host helpers of the kernels that use TMA: the tensor-map encoder's entry point and
// the opt-in to more than 48 KB of dynamic shared memory.
#pragma once

#include <atomic>
#include <mutex>

#include <cudaTypedefs.h>
#include <cuda_runtime.h>

namespace qsa {

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

inline bool set_smem_once(const void* fn, int bytes, std::atomic<bool> (&done)[128])
{
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 128) return false;
    if (!done[dev].load()) {  // setting it twice (two host threads) is harmless
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
        done[dev].store(true);
    }
    return true;
}

}  // namespace qsa
