// ct_checks.h -- helpers of the entry points' host-side argument checks.
#pragma once

#include "../../include/cast_transpose.h"

#include <cuda_runtime.h>
#include <stdint.h>

namespace ct {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Range {
    uintptr_t lo, hi;   // [lo, hi)
};
inline Range range_of(const void* p, int64_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{lo, lo + static_cast<uintptr_t>(bytes)};
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? CT_OK : CT_ERR_CUDA; }

}  // namespace ct
