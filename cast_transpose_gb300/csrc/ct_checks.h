// ct_checks.h -- helpers of the entry points' host-side argument checks.
#pragma once

#include "../../include/cast_transpose.h"

#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>

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

constexpr int64_t kMaxIndex = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxElements = int64_t(1) << 40;   // of a matrix
constexpr int64_t kMaxNormHidden = 32768;

inline bool dtype_ok(int d) { return d == CT_BF16 || d == CT_FP16 || d == CT_FP32; }
inline int elem_bytes(int d) { return d == CT_FP32 ? 4 : 2; }

// A buffer of a call: null only where `optional`, aligned to `align`.
struct Buffer {
    const void* p;
    int64_t bytes;
    int align;
    bool written;
    bool optional = false;
};

// Buffers of no bytes are not checked (an empty matrix may have any pointer).
inline int check_buffers(std::initializer_list<Buffer> buffers) {
    for (const Buffer& b : buffers)
        if (!b.p && !b.optional && b.bytes > 0) return CT_ERR_NULL;
    for (const Buffer& b : buffers)
        if (b.p && b.bytes > 0 && !aligned(b.p, b.align)) return CT_ERR_ALIGN;
    for (const Buffer& w : buffers) {
        if (!w.written || !w.p) continue;
        for (const Buffer& o : buffers)
            if (&o != &w && o.p && overlap(range_of(w.p, w.bytes), range_of(o.p, o.bytes)))
                return CT_ERR_ALIAS;
    }
    return CT_OK;
}

}  // namespace ct
