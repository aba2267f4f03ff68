// Host helpers shared by the library's two translation units: device
// properties, error reporting, launch set-up, the tensor-map encoder.
#pragma once

#include <atomic>
#include <cstdio>
#include <cstdlib>

#include <cudaTypedefs.h>

#include "common.cuh"

namespace engram {

// Per-device host caches below are relaxed atomics: host threads that reach a
// first call together compute and store the same value.
static inline int num_sms() {
    static std::atomic<int> sms[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return 148;
    int n = sms[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        int v = 0;
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
        n = v > 0 ? v : 148;
        sms[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

static inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// With ENGRAM_DEBUG set in the environment, failed CUDA calls are reported on
// stderr with the call site (the status returned is the same either way).
static inline engram_status cuda_fail(cudaError_t e, const char *what) {
    static const bool debug = getenv("ENGRAM_DEBUG") != nullptr;
    if (debug) fprintf(stderr, "libengram: %s failed: %s\n", what, cudaGetErrorString(e));
    return ENGRAM_ECUDA;
}

// Opt a kernel in to `bytes` of dynamic shared memory once per device.
static inline engram_status ensure_smem(const void *kern, int bytes, std::atomic<bool> *attr_done) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_done[dev].load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(smem)");
        if (dev >= 0 && dev < 64) attr_done[dev].store(true, std::memory_order_relaxed);
    }
    return ENGRAM_OK;
}

static inline engram_status launch_status() {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? ENGRAM_OK : cuda_fail(e, "kernel launch");
}

static inline PFN_cuTensorMapEncodeTiled_v12000 tensormap_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }
    return fn;
}

// Reads and clears the including translation unit's error word on the current
// device.
static inline cudaError_t take_error_word(unsigned int *w) {
    const cudaError_t e = cudaMemcpyFromSymbol(w, g_error_word, sizeof(*w));
    if (e != cudaSuccess) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero));
}

namespace attn {
cudaError_t take_error(unsigned int *w);  // the attention kernels' error word
}

}  // namespace engram
