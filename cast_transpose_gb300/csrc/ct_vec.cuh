// ct_vec.cuh -- eight columns of a row as four pairs of fp32 values, parameters
// and FP8 rows, for the norm kernels.
#pragma once

#include "ct_device.cuh"
#include "ct_types.cuh"

namespace ct {
namespace {

// ---- eight columns as four pairs -------------------------------------------
struct V8 {
    uint64_t p[4];
};
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void halves(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ V8 pairs(const float (&f)[8]) {
    return V8{{pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7])}};
}
__device__ __forceinline__ void floats(const V8& v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) halves(v.p[i], f[2 * i], f[2 * i + 1]);
}

// Columns past the row's end: a vector is read from column 0 instead, so that
// no load is conditional; what it adds to a sum is dropped by on(), and it is
// not stored.
template <int G>
__device__ __forceinline__ bool on(const dev::Cols<G>& c) {
    return G != 8 || c.any();
}
template <int G, typename T>
__device__ __forceinline__ V8 load_v8(const T* row, const dev::Cols<G>& c) {
    float f[8];
    if constexpr (G == 8)
        dev::unpack8(dev::load8(row + (c.any() ? c.first : 0)), f);
    else
        dev::load_cols<G>(row, c, f);
    return pairs(f);
}
template <typename T>
__device__ __forceinline__ V8 unpacked(const dev::Raw8<T>& r) {
    float f[8];
    dev::unpack8(r, f);
    return pairs(f);
}
template <int G, typename T>
__device__ __forceinline__ void store_v8(T* row, const dev::Cols<G>& c, const V8& v) {
    float f[8];
    floats(v, f);
    dev::store_cols<G>(row, c, f);
}
__device__ __forceinline__ float lanes_sum(uint64_t v) {
    float lo, hi;
    halves(v, lo, hi);
    return lo + hi;
}

// The larger one, a NaN if there is one.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// ---- parameters ------------------------------------------------------------
template <typename T>
__device__ __forceinline__ void set_param(void* p, int f32, int64_t i, float v) {
    if (f32)
        static_cast<float*>(p)[i] = v;
    else
        dev::from_f32(static_cast<T*>(p)[i], v);
}

// offset + w of the thread's columns; 1 without a weight.
template <typename T, int G>
__device__ __forceinline__ void load_param(const void* p, int f32, int64_t at, float offset,
                                           const dev::Cols<G>& c, float (&f)[8]) {
    if (!p) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = 1.0f;
        return;
    }
    if (f32)
        dev::load_cols<G>(static_cast<const float*>(p) + at, c, f);
    else
        dev::load_cols<G>(static_cast<const T*>(p) + at, c, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] += offset;
}

// b of the thread's columns; 0 without a bias.
template <typename T, int G>
__device__ __forceinline__ void load_bias(const void* p, int f32, int64_t at, const dev::Cols<G>& c,
                                          float (&f)[8]) {
    if (p) {
        load_param<T>(p, f32, at, 0.0f, c, f);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.0f;
}

// Eight FP8 codes of y * scale.
template <int G>
__device__ __forceinline__ void store_fp8(uint8_t* row, const dev::Cols<G>& c,
                                          const float (&y)[8], float scale, int fmt) {
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float lo = __fmul_rn(y[2 * j], scale), hi = __fmul_rn(y[2 * j + 1], scale);
        h[j] = fmt == 0 ? dev::cvt_fp8x2<0>(lo, hi) : dev::cvt_fp8x2<1>(lo, hi);
    }
    if constexpr (G == 8) {
        if (c.any())
            *reinterpret_cast<uint2*>(row + c.first) =
                make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c.has(j)) row[c.at(j)] = static_cast<uint8_t>(h[j >> 1] >> (8 * (j & 1)));
    }
}

// The types of u and y, and of the residual stream.
template <typename F>
cudaError_t by_types(int dtype, int res_dtype, F&& f) {
    if (dtype == 0)
        return res_dtype == 0 ? f(__nv_bfloat16{}, __nv_bfloat16{}) : f(__nv_bfloat16{}, float{});
    if (dtype == 1) return res_dtype == 1 ? f(__half{}, __half{}) : f(__half{}, float{});
    return f(float{}, float{});
}


template <typename... P>
bool all_aligned(P... p) {
    return ((reinterpret_cast<uintptr_t>(p) % 16 == 0) && ...);
}

}  // namespace
}  // namespace ct
