// Host-side launch helpers shared by the translation units: the tensor-map
// encoder, dynamic shared-memory limits, launches with programmatic dependent
// launch.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <map>
#include <mutex>
#include <utility>

namespace dgen {

// ------------------------------------------------------------------ tensor maps

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiledFn g_encode = nullptr;
inline std::once_flag g_encode_once;

inline bool load_encode() {
    std::call_once(g_encode_once, [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<EncodeTiledFn>(fn);
    });
    return g_encode != nullptr;
}

// ------------------------------------------------------------------ launches

// Raise a kernel's dynamic shared-memory limit to at least `bytes` on a
// device (kept per (kernel, device) and only ever raised: a kernel whose
// dynamic size depends on the shape must not be capped by an earlier, smaller
// launch).  Keyed on the kernel's address: instantiations that differ only in
// tile size share a function type.
inline std::mutex g_attr_mu;
inline std::map<std::pair<const void*, int>, int> g_attr_bytes;

template <class K>
void set_smem_attr_once(K kern, int bytes, int dev) {
    const void* f = reinterpret_cast<const void*>(kern);
    std::lock_guard<std::mutex> lock(g_attr_mu);
    int& cur = g_attr_bytes[{f, dev}];
    if (bytes > cur) {
        cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        cur = bytes;
    }
}

// Launch with the programmatic-stream-serialization attribute: the kernel may be
// scheduled while its predecessor drains; each kernel waits (griddepcontrol)
// before touching memory the predecessor writes.
inline std::atomic<bool> g_pdl{true};  // cleared by DGEN_FLAG_NO_PDL on any handle (process-wide)

template <typename... KArgs, typename... Args>
cudaError_t launch_ex(cudaStream_t st, void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = g_pdl.load(std::memory_order_relaxed) ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace dgen
