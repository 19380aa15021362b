// fa_internal.h -- host helpers that the translation units of libfa_sm100.so
// share: the one-time device set-up and the TMA tensor-map encoder.  Not part
// of the C ABI.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "fa.h"

namespace fa_host {

// The current device's ordinal, error word and SM count, after the one-time
// set-up; FA_OK, or why the device cannot be used.
fa_status device(int* dev, unsigned int** err_word, int* sm_count);

// Tensor map of a row-major [planes][rows][cols] tensor (elem_bytes 2: bf16,
// 4: fp32), 128-byte swizzled boxes of {box_cols, box_rows, 1}.
bool encode_map(CUtensorMap* map, const void* base, int elem_bytes, int cols, long long rows,
                long long planes, int box_cols, int box_rows);

inline bool aligned(const void* p, uintptr_t bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

}  // namespace fa_host
