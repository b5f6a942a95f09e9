// sv_host.hpp -- host-side helpers shared by the C entry points: argument
// checks, workspace alignment and the launch status.
#pragma once

#include <hip/hip_runtime.h>

#include <climits>
#include <cstddef>
#include <cstdint>

#include "specverify.h"
#include "sv_common.hpp"

namespace sv {

inline size_t align_up(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

inline int elem_size(int32_t dtype) { return dtype == SPEC_DTYPE_F32 ? 4 : 2; }

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline spec_status check_logits_shape(int32_t V, int64_t stride, int32_t dtype,
                                      float temperature) {
    if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16) return SPEC_ERR_ARG;
    if (V < 2 || stride < V) return SPEC_ERR_ARG;
    if ((stride * elem_size(dtype)) % 16 != 0) return SPEC_ERR_ARG;
    // rows are addressed with 32-bit byte offsets
    if (static_cast<int64_t>(V) * elem_size(dtype) > INT32_MAX) return SPEC_ERR_UNSUPPORTED;
    if (!(temperature >= 1e-4f && temperature <= 1e4f)) return SPEC_ERR_ARG;
    return SPEC_OK;
}

inline spec_status launch_status() {
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_ERR_HIP;
}

inline float log2e_over(float temperature) { return kLog2e / temperature; }

}  // namespace sv
