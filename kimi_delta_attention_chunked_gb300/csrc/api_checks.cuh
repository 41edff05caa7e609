// api_checks.cuh -- argument checks that the C entries of the step operators share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kda.h"

namespace kda_host {

inline kda_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return KDA_OK;
    if (e == cudaErrorNotSupported) return KDA_ERR_UNSUPPORTED;
    return KDA_ERR_CUDA;
}

inline bool page_ok(int p) { return p == 16 || p == 32 || p == 64 || p == 128 || p == 256; }
inline bool dtype_ok(kda_dtype t) { return t == KDA_FP32 || t == KDA_BF16; }
inline int element_size(kda_dtype t) { return t == KDA_BF16 ? 2 : 4; }
inline bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Rows of `width` elements, `outer` x `inner` of them at these strides (each in either order), share no element.
inline bool rows_apart(int outer, int64_t outer_stride, int inner, int64_t inner_stride, int width) {
    const __int128 o = outer_stride, i = inner_stride;
    if ((outer > 1 && o < width) || (inner > 1 && i < width)) return false;
    if (outer <= 1 || inner <= 1) return true;
    return o >= i * (inner - 1) + width || i >= o * (outer - 1) + width;
}

}  // namespace kda_host
