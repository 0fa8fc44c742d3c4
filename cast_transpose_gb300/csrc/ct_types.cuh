// ct_types.cuh -- eight columns at a time of bf16, fp16 or fp32 rows, for the
// norm and expert-movement kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace ct {
namespace dev {

// The 16-byte words that hold eight elements.
template <typename T>
struct Raw8 {
    uint4 v[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) r.v[i] = reinterpret_cast<const uint4*>(p)[i];
    return r;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

// One rounding to the stored type, to nearest even.
__device__ __forceinline__ void from_f32(float& d, float v) { d = v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(__half& d, float v) { d = __float2half_rn(v); }

__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(r.v[i].x);
        f[4 * i + 1] = __uint_as_float(r.v[i].y);
        f[4 * i + 2] = __uint_as_float(r.v[i].z);
        f[4 * i + 3] = __uint_as_float(r.v[i].w);
    }
}
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& r, float (&f)[8]) {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack8(const Raw8<__half>& r, float (&f)[8]) {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = *reinterpret_cast<const __half2*>(&w[i]);
        f[2 * i] = __low2float(h);
        f[2 * i + 1] = __high2float(h);
    }
}

__device__ __forceinline__ Raw8<float> pack8(const float (&f)[8], float) {
    Raw8<float> r;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        r.v[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                            __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]));
    return r;
}
__device__ __forceinline__ Raw8<__nv_bfloat16> pack8(const float (&f)[8], __nv_bfloat16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return Raw8<__nv_bfloat16>{{make_uint4(w[0], w[1], w[2], w[3])}};
}
__device__ __forceinline__ Raw8<__half> pack8(const float (&f)[8], __half) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 b = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return Raw8<__half>{{make_uint4(w[0], w[1], w[2], w[3])}};
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
    const Raw8<T> r = pack8(f, T{});
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = r.v[i];
}

// The eight columns of item `vi` of a row of H, in groups of G neighbours.
// G = 8: one 16-byte vector of two-byte elements (H % 8 == 0, rows 16-byte
// aligned).  Otherwise 32 items, a warp's, share 256 columns, each group 32 * G
// columns after the one before: a warp's accesses are consecutive and their
// offsets constants.  G = 2: pairs (H even, rows aligned for them); G = 1: any
// H and alignment.
template <int G>
struct Cols {
    static constexpr int kStep = 32 * G;
    int first, H;
    __device__ __forceinline__ Cols(int vi, int H_) : H(H_) {
        first = G == 8 ? vi * 8 : (vi >> 5) * 256 + (vi & 31) * G;
    }
    __device__ __forceinline__ int at(int j) const { return G == 8 ? first + j : first + j / G * kStep + j % G; }
    __device__ __forceinline__ bool any() const { return first < H; }
    __device__ __forceinline__ bool has(int j) const { return G == 8 ? first < H : at(j) < H; }
};

template <typename T>
struct Pair {
    T x, y;
};
template <>
struct __align__(4) Pair<__nv_bfloat16> {
    __nv_bfloat16 x, y;
};
template <>
struct __align__(4) Pair<__half> {
    __half x, y;
};
template <>
struct __align__(8) Pair<float> {
    float x, y;
};

template <int G, typename T>
__device__ __forceinline__ void load_cols(const T* row, const Cols<G>& c, float (&f)[8]) {
    if constexpr (G == 8) {
        if (c.any()) {
            unpack8(load8(row + c.first), f);
            return;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = 0.0f;
    } else if constexpr (G == 2) {
        const Pair<T>* p = reinterpret_cast<const Pair<T>*>(row + c.first);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool some = c.has(2 * j);
            Pair<T> v;
            if (some) v = p[32 * j];
            f[2 * j] = some ? to_f32(v.x) : 0.0f;
            f[2 * j + 1] = some ? to_f32(v.y) : 0.0f;
        }
    } else {
        const T* p = row + c.first;
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = c.has(j) ? to_f32(p[32 * j]) : 0.0f;
    }
}

template <int G, typename T>
__device__ __forceinline__ void store_cols(T* row, const Cols<G>& c, const float (&f)[8]) {
    if constexpr (G == 8) {
        if (c.any()) store8(row + c.first, f);
    } else if constexpr (G == 2) {
        Pair<T>* p = reinterpret_cast<Pair<T>*>(row + c.first);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            Pair<T> v;
            from_f32(v.x, f[2 * j]);
            from_f32(v.y, f[2 * j + 1]);
            if (c.has(2 * j)) p[32 * j] = v;
        }
    } else {
        T* p = row + c.first;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c.has(j)) from_f32(p[32 * j], f[j]);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

}  // namespace dev
}  // namespace ct
