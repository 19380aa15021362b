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

// Launches a kernel so that it may be set up while the stream's previous kernel
// ends, which takes about a microsecond off a short call.  It starts once every
// CTA of that kernel has called grid_launch_dependents or has ended (a kernel
// that never calls it is waited for whole), and its grid_dependency_wait
// returns once that kernel has ended and its writes are visible.  So a kernel
// waits before it touches memory that any earlier one may use, with two
// exceptions among the launches of fa_fwd_paged, each of which rests on where
// the kernel before it signals:
//  * fa_own_kernel behind a prefix reads its inputs and writes its part of the
//    workspace without waiting.  fa_prefix_kernel signals after its own wait, so
//    everything before the call has ended by then, and the two write different
//    rows.  The first CTA of the line waits for the prefix grid at its end.
//  * fa_paged_merge_kernel reads seq_start before its wait.  fa_own_kernel
//    signals after its own wait or, behind a prefix, after that kernel's, and
//    neither writes seq_start.
// Each kernel's end also means the end of all before it: fa_own_kernel's of the
// prefix grid (that first CTA), every other's of the one that it waited for.  A
// kernel that signals earlier, or skips its wait, breaks those behind it.
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
