// ct_dropout.cuh -- which elements a dropout keeps, from a counter-based
// generator: nothing is stored, and whoever knows the seed, the step and the
// place gets the same answer.
//
// The generator is Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011).  One call gives eight
// columns of a row 16 bits each: 32 bits each would double its cost, which is
// what a dropout computes (some 60 operations a call), for chances finer than
// 1/65536.
//   counter  (column / 8, row, site, step mod 2^32)      key  the seed
//   column j: half j % 2 (0: the lower) of word (j % 8) / 2
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ct_ops.h"

namespace ct {
namespace {

__device__ __forceinline__ uint4 philox_round(uint4 c, uint32_t k0, uint32_t k1) {
    const uint64_t a = uint64_t(0xD2511F53u) * c.x, b = uint64_t(0xCD9E8D57u) * c.z;
    return make_uint4(uint32_t(b >> 32) ^ c.y ^ k0, uint32_t(b), uint32_t(a >> 32) ^ c.w ^ k1, uint32_t(a));
}
constexpr int kPhiloxRounds = 10;
constexpr uint32_t kKeyStep0 = 0x9E3779B9u, kKeyStep1 = 0xBB67AE85u;     // added to the key after a round

// The generator of one call, as its kernel uses it.
struct Drops {
    uint2 key;
    uint32_t site, step;
    uint32_t cut;           // dropped: 16 bits below this / 65536
    float scale;            // of what is kept
    bool some;              // anything to drop

    __device__ __forceinline__ explicit Drops(const DropArgs& a) {
        some = a.cut != 0;
        cut = a.cut << 16;
        scale = a.scale;
        site = a.site;
        key = make_uint2(0, 0);
        step = 0;
        if (!some) return;
        const ulonglong2 s = make_ulonglong2(a.rng[0], a.rng[1]);
        key = make_uint2(uint32_t(s.x), uint32_t(s.x >> 32));
        step = uint32_t(s.y);
    }
    __device__ __forceinline__ uint4 words(uint32_t row, uint32_t group) const {
        uint4 c = make_uint4(group, row, site, step);
#pragma unroll
        for (int i = 0; i < kPhiloxRounds; ++i) c = philox_round(c, key.x + i * kKeyStep0, key.y + i * kKeyStep1);
        return c;
    }
    // Bit j: column 8 * group + j of the row is kept.
    static __device__ __forceinline__ uint32_t bits(uint4 r, uint32_t cut) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w}, over = 0u - cut;     // carries out where w >= cut
        uint32_t kept = 0;
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            asm("{\n\t.reg .u32 sum;\n\tadd.cc.u32 sum, %1, %2;\n\taddc.u32 %0, %0, %0;\n\t}" : "+r"(kept) : "r"(w[i]), "r"(over));
            asm("{\n\t.reg .u32 sum;\n\tadd.cc.u32 sum, %1, %2;\n\taddc.u32 %0, %0, %0;\n\t}" : "+r"(kept) : "r"(w[i] << 16), "r"(over));
        }
        return kept;
    }
    // v of the thread's columns Cols<G>(vi), dropped or scaled.  With G = 8 they are
    // the group's own; where they are spread over the warp's 32 groups, of which
    // the lane's has the number `group`, the lanes pass each other a bit for each
    // column.  The whole warp has to call it.
    template <int G>
    __device__ __forceinline__ void apply(uint32_t row, uint32_t group, float (&v)[8]) const {
        const uint4 r = words(row, group);
        if constexpr (G == 8) {
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = (w[i] << 16) >= cut ? v[2 * i] * scale : 0.0f;
                v[2 * i + 1] = w[i] >= cut ? v[2 * i + 1] * scale : 0.0f;
            }
        } else {
            static_assert(G == 1, "pairs are not used");
            const uint32_t own = bits(r, cut);
            const int lane = threadIdx.x & 31;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t other = __shfl_sync(0xFFFFFFFFu, own, 4 * j + (lane >> 3));
                v[j] = (other >> (lane & 7)) & 1 ? v[j] * scale : 0.0f;
            }
        }
    }
};

}  // namespace
}  // namespace ct
