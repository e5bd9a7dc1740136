// What the entry points of both translation units share on the host: checks of pointers, launch
// status, the copy of an untouched state, and stream-ordered scratch.
#pragma once

#include <cstddef>
#include <cstdint>

#include "common.cuh"

namespace drscan {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool ok_ptr(const void* p) { return p != nullptr && aligned16(p); }
inline bool ok_opt(const void* p) { return p == nullptr || aligned16(p); }
inline bool dim_supported(int d) { return d == 32 || d == 64 || d == 128; }

inline int launch_status() {
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? DR_OK : DR_ERR_CUDA;
}

// State handed through unchanged when there are no tokens: S_final = S0 (or zeros).
inline int copy_state(float* dst, const float* src, size_t count, cudaStream_t stream) {
    if (!dst) return DR_OK;
    cudaError_t e = src ? cudaMemcpyAsync(dst, src, count * sizeof(float),
                                          cudaMemcpyDeviceToDevice, stream)
                        : cudaMemsetAsync(dst, 0, count * sizeof(float), stream);
    return e == cudaSuccess ? DR_OK : DR_ERR_CUDA;
}

// Defined in drscan.cu.
int scratch_alloc(void** p, size_t bytes, cudaStream_t stream);
// Defined in layer.cu: reads and clears the status word of that unit's kernels.
int layer_poll_status(int* status);

}  // namespace drscan
