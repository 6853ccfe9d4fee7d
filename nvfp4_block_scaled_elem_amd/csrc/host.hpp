// Host-side helpers of the C entry points: checks of pointers and types, errors, scratch.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "launch.hpp"

#define NVFP4_API extern "C" __attribute__((visibility("default")))

namespace nvfp4 {

inline bool aligned(const void *p, unsigned a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool plain_dtype(int t) { return t == NVFP4_DTYPE_BF16 || t == NVFP4_DTYPE_F32; }
inline unsigned width(int t) { return t == NVFP4_DTYPE_BF16 ? 2u : t == NVFP4_DTYPE_F32 ? 4u : 1u; }

inline int status(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP; }

// Scratch of a call: the caller's workspace, or stream-ordered memory given back on the same stream. The
// library does not allocate on a capturing stream.
template <typename F>
int with_scratch(void *workspace, size_t workspace_bytes, size_t need, hipStream_t st, F &&run) {
    if (need == 0) return status(run(nullptr));
    if (workspace) return workspace_bytes < need ? (int)NVFP4_ERR_WORKSPACE : status(run(workspace));
    hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(st, &cs) != hipSuccess) return NVFP4_ERR_HIP;
    if (cs != hipStreamCaptureStatusNone) return NVFP4_ERR_UNSUPPORTED;
    void *ws = nullptr;
    if (hipMallocAsync(&ws, need, st) != hipSuccess) return NVFP4_ERR_HIP;
    const hipError_t e = run(ws);
    if (hipFreeAsync(ws, st) != hipSuccess) return NVFP4_ERR_HIP;
    return status(e);
}

}  // namespace nvfp4
