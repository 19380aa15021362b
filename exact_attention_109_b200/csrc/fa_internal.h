// fa_internal.h -- host helpers that the translation units of libfa_sm100.so
// share: the one-time device set-up and the TMA tensor-map encoder.  Not part
// of the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <utility>

#include "fa.h"

namespace fa_host {

// The current device's ordinal, error word and SM count, after the one-time
// set-up; FA_OK, or why the device cannot be used.
fa_status device(int* dev, unsigned int** err_word, int* sm_count);

// Tensor map of a row-major [planes][rows][cols] tensor (elem_bytes 2: bf16,
// 4: fp32), 128-byte swizzled boxes of {box_cols, box_rows, 1}.
bool encode_map(CUtensorMap* map, const void* base, int elem_bytes, int cols, long long rows,
                long long planes, int box_cols, int box_rows);

// Launches a kernel that waits (grid_dependency_wait) before it reads or writes
// any memory that other kernels do: it may then be set up while the stream's
// previous kernel ends, which takes about a microsecond off a short call.
template <class... Params, class... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), dim3 grid, int threads, size_t smem,
                              cudaStream_t s, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

inline bool aligned(const void* p, uintptr_t bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

}  // namespace fa_host
