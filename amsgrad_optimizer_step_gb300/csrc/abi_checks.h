// Argument checks and trace ranges shared by the C-ABI host layers (abi.cpp for the
// optimizer step, model_abi.cpp for the model-side operators).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "fused_adamw.h"

namespace fa {

inline bool valid_dtype(fa_dtype d) { return d == FA_F32 || d == FA_F16 || d == FA_BF16; }
inline size_t dtype_bytes(fa_dtype d) { return d == FA_F32 ? 4 : 2; }

// Host-side trace ranges (NVTX): a profiler attached to the process shows each
// entry point's span around the kernels it enqueues; without one they cost nothing.
struct TraceRange {
    explicit TraceRange(const char *name) { nvtxRangePushA(name); }
    ~TraceRange() { nvtxRangePop(); }
    TraceRange(const TraceRange &) = delete;
    TraceRange &operator=(const TraceRange &) = delete;
};

// The current device, checked against the stream's device (the legacy default
// stream belongs to the current device).
inline fa_status stream_device(void *stream, int *dev) {
    if (cudaGetDevice(dev) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    if (stream) {
        // A stream that is being captured into a graph cannot report its device
        // (the query fails and ends the capture); its work is recorded for the
        // device the capture belongs to, so the check is left out then.
        cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
        if (cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &cs) != cudaSuccess) {
            cudaGetLastError();
            return FA_ERR_POINTER;
        }
        if (cs == cudaStreamCaptureStatusActive) return FA_OK;
        int sdev = -1;
        if (cudaStreamGetDevice(static_cast<cudaStream_t>(stream), &sdev) != cudaSuccess) {
            cudaGetLastError();
            return FA_ERR_POINTER;
        }
        if (sdev != *dev) return FA_ERR_POINTER;
    }
    return FA_OK;
}

// Device (or managed) memory of device ``dev``, aligned to ``align`` bytes.
inline fa_status check_device_ptr(const void *p, int dev, size_t align) {
    if (!p) return FA_ERR_NULL;
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_POINTER;
    }
    if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged) return FA_ERR_POINTER;
    if (at.device != dev) return FA_ERR_POINTER;
    if (reinterpret_cast<uintptr_t>(p) % align) return FA_ERR_ALIGN;
    return FA_OK;
}

struct Range {
    const void *p;
    size_t bytes;
};

inline bool overlap(Range a, Range b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

inline bool any_overlap(const Range *r, int count) {
    for (int i = 0; i < count; ++i)
        for (int j = i + 1; j < count; ++j)
            if (overlap(r[i], r[j])) return true;
    return false;
}

}  // namespace fa
