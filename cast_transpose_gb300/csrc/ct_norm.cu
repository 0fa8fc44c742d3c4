// ct_norm.cu -- the junction between two blocks: norm, gate, residual sum and
// norm, forward and backward.
//
// Both passes are bound by HBM: forward reads u and res and writes res_out and
// y, backward reads dy, dres_out, u and res_out and writes du and dres, with
// some ten operations per element.  Each row needs two sums over its columns,
// the second of which depends on the first, so what has to be avoided is
// memory standing still while a row waits for them, and per-row work (sums
// across warps, barriers, addresses) outweighing that on the columns.  The
// design, common to both:
//   - a cluster of blocks owns a contiguous run of rows, each of its blocks a
//     fixed slice of the columns, each thread 16 fixed columns: parameters stay
//     in the thread's own shared memory, the backward pass's column sums in
//     its registers;
//   - rows arrive in a ring of shared-memory stages by bulk copies that one
//     thread issues rows ahead, so loads are in flight during every barrier;
//   - the first sum of row i+1 and the second sum of row i are exchanged
//     together, and the first sum of row i+2 is taken while they travel;
//   - arithmetic on pairs of columns (f32x2).
// Rows of up to 16 columns a thread take one block; longer ones a cluster of
// 2, 4 or 8 that exchange partial sums through distributed shared memory.  Rows
// that are not whole 16-byte blocks take the same path, copied as the aligned
// blocks that cover them.  Launches of no more rows than clusters fit take a
// kernel of one row per cluster, without loops and rings.
//
// Measured, bf16, of the measured copy rate: forward 8191x6144 68.8 us (403 MB,
// 0.86), backward with its join 8192x6144 102.6 us (604 MB, 0.87), 8192x12288
// 189.8 us (1208 MB, 0.94).  What is left is the chain of a row (two sums, each
// over the block, around 16 columns' arithmetic a thread), of which only as
// many fit an SM as its registers (backward) and the parameters' shared memory
// (forward) allow.
#include "ct_device.cuh"
#include "ct_ops.h"
#include "ct_types.cuh"

#include <algorithm>
#include <mutex>

namespace ct {
namespace {

constexpr int kPer = 2;               // groups of eight columns per thread
// Threads of a block: forward, two blocks with 80 registers a thread (512 with
// 64 do not hold a row's u: 8191x6144 72.5 us, so: 68.8); backward, one with
// 168, which its column sums and the compiler's room to interleave columns need
// (8192x6144, 512 with 128: 109 us, so: 106; 12288x4096: 131, so: 119, where
// blocks of 256 threads leave a third of the registers unused).
constexpr int kForwardThreads = 384, kBackwardThreads = 384;
constexpr int kMaxThreads = kForwardThreads;
constexpr int kMaxCluster = 8;
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kMaxStages = 6;         // of either ring
constexpr int kSmemPerSm = 227 * 1024;
constexpr int kSmemFixed = 3328;      // static shared memory and the system's, per block

// How a launch divides the work.
struct NormShape {
    int cluster;        // blocks per row
    int width;          // columns per block, a multiple of 8
    int lead, trail;    // stages of the rings; 0: one row per cluster, no rings
    int clusters;       // runs of rows
};

// Bits as of the cast kernels' diagnostic word (ct_internal.h).
__device__ unsigned int g_norm_error;

// Rows [first, last) of run c out of `runs`.
__host__ __device__ __forceinline__ int64_t run_begin(int64_t rows, int64_t c, int64_t runs) {
    return rows * c / runs;
}
// The run that row r is in.
__device__ __forceinline__ int64_t run_of(int64_t rows, int64_t r, int64_t runs) {
    return ((r + 1) * runs - 1) / rows;
}

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

// alpha * gate * a(w_post): what the normed u is multiplied by.
template <typename T, int G, typename Args>
__device__ __forceinline__ void branch_factor(const Args& a, int64_t gate_row, int col0,
                                              const dev::Cols<G>& c, float (&f)[8]) {
    float w[8];
    load_param<T>(a.gate, a.param_f32, gate_row * a.hidden + col0, 0.0f, c, f);
    load_param<T>(a.post ? a.w_post : nullptr, a.param_f32, col0, a.weight_offset, c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= a.branch_scale * w[j];
}

// fp32 values of a thread's columns in shared memory that no other thread
// reads: one float4 per thread and plane, so that a warp's accesses are
// consecutive.
struct Own {
    float4* base;
    __device__ __forceinline__ float4* at(int slot, int p) const {
        return base + (slot * kPer + p) * 2 * blockDim.x + threadIdx.x;
    }
    __device__ __forceinline__ void put(int slot, int p, const float (&f)[8]) const {
        float4* q = at(slot, p);
        q[0] = make_float4(f[0], f[1], f[2], f[3]);
        q[blockDim.x] = make_float4(f[4], f[5], f[6], f[7]);
    }
    __device__ __forceinline__ V8 get(int slot, int p) const {
        const ulonglong2* q = reinterpret_cast<const ulonglong2*>(at(slot, p));
        const ulonglong2 a = q[0], b = q[blockDim.x];
        return V8{{a.x, a.y, b.x, b.y}};
    }
};
enum { kBranch, kPre, kOwnSlots };    // alpha gate a(w_post), a(w_pre)
constexpr int kOwnBytes = 32 * kPer * kOwnSlots;   // per thread

// ---- waits -----------------------------------------------------------------
// Every thread polls a barrier for itself and gives up for itself (`lost`):
// its neighbours may see the same barrier complete.  A thread that is lost goes
// through the rest of its rows without waiting, so that it meets the others at
// every shuffle and block barrier, but from then on it arrives at no barrier,
// sends nothing and fetches nothing: a phase that it has not seen end must not
// be entered a second time.  Whoever needs its part gives up in turn, so that
// all of the cluster gets to RowSums::end, where each lost thread reports.

// CLUSTER: for a barrier that other blocks of the cluster complete.
template <bool CLUSTER>
__device__ __forceinline__ bool try_wait(uint64_t* bar, uint32_t parity) {
    if constexpr (!CLUSTER) return dev::mbar_try_wait(bar, parity);
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(dev::smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}

// As dev::mbar_wait_bounded, with a last try after the limit: a block that did
// not run for that long finds its barriers complete.
template <bool CLUSTER>
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
    if (try_wait<CLUSTER>(bar, parity)) return true;
    const uint64_t t0 = dev::globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
        if (try_wait<CLUSTER>(bar, parity)) return true;
        if ((i & 63u) == 0 && dev::globaltimer_ns() - t0 > limit_ns) return try_wait<CLUSTER>(bar, parity);
    }
}

// Sums of a and b over the cluster's blocks, the same in every thread, in a
// fixed order, in two steps so that work can go on between them: send() leaves
// the warps' sums in every block, get() waits for all of them and adds them
// up.  Lanes 0..15 work on a, lanes 16..31 on b.  Two sets of slots and
// barriers take turns: whoever sends the second time after a get() knows that
// everyone has finished that get().
struct RowSums {
    float (*slots)[2][kMaxCluster * kMaxWarps];
    uint64_t* bars;
    int cluster, rank;
    uint64_t limit_ns = dev::kWaitLimitNs;
    int turn = 0;
    uint32_t parity = 0;

    // The arrivals of a turn: one per warp, or thread 0's with the bytes that
    // the cluster's warps send.
    __device__ __forceinline__ void init() const {
        for (int i = 0; i < 2; ++i) dev::mbar_init(bars + i, cluster == 1 ? blockDim.x >> 5 : 1);
    }
    static __device__ __forceinline__ float half_sum(float v) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        return v;
    }
    // `lost`: a wait gave up earlier; then nothing is sent.
    __device__ __forceinline__ void send(float a, float b, bool lost) {
        const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const bool upper = lane >= 16;
        float v = upper ? b : a;
        v = half_sum(v + __shfl_xor_sync(0xFFFFFFFFu, upper ? a : b, 16));
        float* slot = slots[turn][upper] + rank * warps + warp;
        if (cluster == 1) {
            if ((lane & 15) == 0 && !lost) *slot = v;
            __syncwarp();
            if (lane == 0 && !lost) dev::mbar_arrive(bars + turn);
        } else {
            if (threadIdx.x == 0 && !lost) dev::mbar_arrive_expect_tx(bars + turn, cluster * warps * 8);
            if ((lane & 15) < cluster && !lost) {
                uint32_t to, bar;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                             : "=r"(to) : "r"(dev::smem_u32(slot)), "r"(lane & 15));
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                             : "=r"(bar) : "r"(dev::smem_u32(bars + turn)), "r"(lane & 15));
                asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];"
                             ::"r"(to), "r"(__float_as_uint(v)), "r"(bar) : "memory");
            }
        }
    }
    // `lost`: a wait gave up, here or earlier; then nothing is waited for.
    __device__ __forceinline__ float2 get(bool& lost) {
        const int n = cluster * (blockDim.x >> 5), lane = threadIdx.x & 31;
        if (!lost)
            lost = !(cluster == 1 ? wait_bounded<false>(bars + turn, parity, limit_ns)
                                  : wait_bounded<true>(bars + turn, parity, limit_ns));
        const float* half = slots[turn][lane >= 16];
        parity ^= turn;
        turn ^= 1;
        float v = 0.0f;
        for (int i = lane & 15; i < n; i += 16) v += half[i];
        v = half_sum(v);
        return make_float2(__shfl_sync(0xFFFFFFFFu, v, 0), __shfl_sync(0xFFFFFFFFu, v, 16));
    }

    // Every block of the cluster has begun and set up its shared memory, or is
    // done with the others'.
    __device__ __forceinline__ void meet() const {
        if (cluster == 1)
            __syncthreads();
        else
            asm volatile("barrier.cluster.arrive.release;\n\t"
                         "barrier.cluster.wait.acquire;" ::: "memory");
    }
    // The block's last step.  Its shared memory stays until its peers have sent
    // their last sums, and, where a wait gave up, until what had been sent has
    // landed: nothing tells how many sends an unfinished turn got, so a lost
    // thread stays for kLandNs, a thousand times what a send takes.  Every thread
    // that gave up reports it, whichever it is.
    static constexpr uint64_t kLandNs = 1000000;
    __device__ __forceinline__ void end(bool lost, unsigned error) const {
        if (cluster > 1) meet();
        if (!lost) return;
        atomicOr(&g_norm_error, error);
        if (cluster > 1)
            for (const uint64_t t0 = dev::globaltimer_ns(); dev::globaltimer_ns() - t0 < kLandNs;) {
            }
    }
};
__device__ __forceinline__ float lanes_sum(uint64_t v) {
    float lo, hi;
    halves(v, lo, hi);
    return lo + hi;
}

// ---- rows ------------------------------------------------------------------
// A ring of stages that hold one row's slices of one or two tensors, one after
// the other.  Thread 0 issues the copies; everyone waits on the stage's
// barrier.  With G = 1 a slice is copied as the aligned 16-byte blocks that
// cover it, and lies (address mod 16) bytes into its place.
//
// A launch has two: the leading ring for what a row's first sum needs, which
// is taken two rows ahead, and the trailing ring for the rest; the leading one
// is longer by about that much.
struct Ring {
    uint64_t* full;
    uint8_t* base;
    uint32_t stage_bytes;
    int stages;
    int stage = 0;
    uint32_t parity = 0;
    int fetched = 0;        // thread 0: fetches so far, number f to stage f % stages

    __device__ __forceinline__ void next() {
        if (++stage == stages) {
            stage = 0;
            parity ^= 1;
        }
    }
    // Where thread 0 gave up: every stage's last copies have to land, or another
    // limit run out, before the block ends.  (A thread 0 that did not has waited
    // for every row, and so for every copy.)
    __device__ __forceinline__ void drain() const {
        for (int f = max(0, fetched - stages); f < fetched; ++f)
            if (!wait_bounded<false>(full + f % stages, (f / stages) & 1, dev::kWaitLimitNs)) return;
    }
    __device__ __forceinline__ void init() const {
        for (int i = 0; i < stages; ++i) dev::mbar_init(full + i, 1);
    }
    // `lost`: a wait gave up, here or earlier; then nothing is waited for.
    __device__ __forceinline__ void wait(bool& lost) const {
        if (!lost) lost = !wait_bounded<false>(full + stage, parity, dev::kWaitLimitNs);
    }
    __device__ __forceinline__ const uint8_t* at() const { return base + stage * stage_bytes; }
    static __device__ __forceinline__ uint32_t blocks_bytes(const void* src, uint32_t bytes) {
        return (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(src) & 15) + bytes + 15) & ~15u;
    }
    __device__ __forceinline__ void copy(int to, uint32_t offset, const void* src, uint32_t bytes) const {
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
            ::"r"(dev::smem_u32(base) + to * stage_bytes + offset),
            "l"(reinterpret_cast<uintptr_t>(src) & ~uintptr_t(15)), "r"(blocks_bytes(src, bytes)),
            "r"(dev::smem_u32(full + to)) : "memory");
    }
    // Stage `to` becomes the slices at p and q (either may be null).
    __device__ __forceinline__ void fetch(int to, const void* p, uint32_t p_bytes, uint32_t q_place,
                                          const void* q, uint32_t q_bytes) {
        ++fetched;
        dev::mbar_arrive_expect_tx(full + to, (p ? blocks_bytes(p, p_bytes) : 0) +
                                                  (q ? blocks_bytes(q, q_bytes) : 0));
        if (p) copy(to, 0, p, p_bytes);
        if (q) copy(to, q_place, q, q_bytes);
    }
};

// Bytes of a tensor's place in a stage.
template <int G, typename T>
__host__ __device__ constexpr uint32_t place_bytes(int width) {
    return width * sizeof(T) + (G == 8 ? 0 : 32);
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


// y, as it is or as FP8 with the largest magnitude in `most`.
template <typename T, int G>
__device__ __forceinline__ void put_y(const NormArgs& a, int64_t at, const dev::Cols<G>& c, const V8& v,
                                      float scale, unsigned& most) {
    if (!a.scale) {
        store_v8<G>(static_cast<T*>(a.y) + at, c, v);
        return;
    }
    float f[8];
    floats(v, f);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (on(c)) most = max(most, __float_as_uint(f[j]) & 0x7FFFFFFFu);
    store_fp8<G>(static_cast<uint8_t*>(a.y) + at, c, f, scale, a.fmt);
}

// The block's largest magnitude joins amax, unless a thread's wait gave up: the
// history outlives the call.  The first block writes scale_inv.
__device__ __forceinline__ void put_amax(const NormArgs& a, unsigned most, float scale, unsigned* block_max,
                                         bool lost) {
    if (!a.scale) return;
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if ((threadIdx.x & 31) == 0) atomicMax(block_max, most);
    const bool wrong = __syncthreads_or(lost);
    if (threadIdx.x == 0) {
        if (*block_max && !wrong) atomicMax(reinterpret_cast<unsigned*>(a.amax), *block_max);
        if (blockIdx.x == 0) *a.scale_inv = __fdiv_rn(1.0f, scale);
    }
}

// With G = 1 the 16-byte blocks that cover a row's slice may begin or end up
// to 15 bytes outside it: rows that near to the tensors' ends are read from
// global memory instead.
template <int G>
__device__ __forceinline__ bool in_ring(int64_t row, int64_t rows, int H) {
    return G == 8 || (row * H >= 8 && (rows - 1 - row) * H >= 8);   // of two bytes at least
}

// Where a row's slice is read from: its place in a stage, or itself.
template <int G, typename T>
__device__ __forceinline__ const T* row_at(const uint8_t* stage, uint32_t offset, const T* global, bool staged) {
    if (G != 8 && !staged) return global;
    stage += offset;
    if (G != 8) stage += reinterpret_cast<uintptr_t>(global) & 15;
    return reinterpret_cast<const T*>(stage);
}

// The next kernel of the stream is let in when a block's rows are done, not
// at once: blocks of it that came to wait beside these would take the room of
// the last of them, which would then run as a second wave.
//
// FULL: u, both norms and (backward) dres_out are there, known to the compiler.

// Forward.  Per row: sum u^2 -> rstd_post; res_out and sum res_out^2 ->
// rstd_pre; y.
//
// KEEP: a row's u stays in registers between its two uses, two rows apart, so
// that its stage is free for a row on its way (two-byte types: 16 registers).
template <typename T, typename R, int G, bool FULL>
__global__ void __launch_bounds__(kForwardThreads, 2) block_norm_kernel(const NormArgs a,
                                                                    const NormShape s) {
    constexpr bool KEEP = FULL && G == 8 && sizeof(T) == 2;
    struct Kept {
        dev::Raw8<T> v[KEEP ? kPer : 1];
    };
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float slots[2][2][kMaxCluster * kMaxWarps];
    __shared__ __align__(8) uint64_t full[2 * kMaxStages + 2];
    __shared__ unsigned block_max;
    const bool has_u = FULL || a.u, post = FULL || a.post, pre = FULL || a.pre;
    const int tid = threadIdx.x, H = a.hidden;
    const int rank = blockIdx.x % s.cluster, run = blockIdx.x / s.cluster;
    const int col0 = rank * s.width, W = min(s.width, H - col0);
    auto cols = [&](int p) { return dev::Cols<G>(p * blockDim.x + tid, W); };
    const int64_t begin = run_begin(a.rows, run, s.clusters), end = run_begin(a.rows, run + 1, s.clusters);
    const T* u = static_cast<const T*>(a.u) + col0;
    const R* res = static_cast<const R*>(a.res) + col0;
    Ring lead{full, smem, place_bytes<G, T>(s.width), s.lead};                  // u
    Ring trail{full + kMaxStages, smem + lead.stages * lead.stage_bytes,
               place_bytes<G, R>(s.width), s.trail};                                  // res
    bool lost = false;       // a wait gave up: no more waiting, the error is reported
    const Own own{reinterpret_cast<float4*>(trail.base + trail.stages * trail.stage_bytes)};
    RowSums sums{slots, full + 2 * kMaxStages, s.cluster, rank};

    if (tid == 0) {
        block_max = 0;
        sums.init();
        lead.init();
        trail.init();
        dev::fence_barrier_init();
    }
    sums.meet();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    auto fetch_lead = [&](int64_t row, int to) {
        const bool staged = has_u && in_ring<G>(row, a.rows, H);
        lead.fetch(to, staged ? u + row * H : nullptr, W * sizeof(T), 0, nullptr, 0);
    };
    auto fetch_trail = [&](int64_t row, int to) {
        trail.fetch(to, in_ring<G>(row, a.rows, H) ? res + row * H : nullptr, W * sizeof(R), 0, nullptr, 0);
    };
    if (tid == 0)
        for (int i = 0; i < max(lead.stages, trail.stages) && begin + i < end; ++i) {
            if (i < lead.stages) fetch_lead(begin + i, i);
            if (i < trail.stages) fetch_trail(begin + i, i);
        }
    int64_t gate_row = a.gate ? begin / a.rows_per_gate : 0;
    int64_t gate_end = a.gate ? (gate_row + 1) * a.rows_per_gate : a.rows;
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
        float f[8];
        if (has_u) {
            branch_factor<T>(a, gate_row, col0, cols(p), f);
            own.put(kBranch, p, f);
        }
        if (pre) {
            load_param<T>(a.w_pre, a.param_f32, col0, a.weight_offset, cols(p), f);
            own.put(kPre, p, f);
        }
    }
    const float scale = a.scale ? *a.scale : 0.0f;
    const float per_column = 1.0f / H;
    const uint64_t beta = pair(a.residual_scale, a.residual_scale);
    unsigned most = 0;

    // sum u^2 of the next row of the leading ring; KEEP: with the row itself
    auto sum_u = [&](int64_t row, Kept& kept) {
        lead.wait(lost);
        if (!post) {
            lead.next();
            return 0.0f;
        }
        const T* x = row_at<G>(lead.at(), 0, u + row * H, in_ring<G>(row, a.rows, H));
        lead.next();
        float sum = 0.0f;
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
            V8 v;
            if constexpr (KEEP) {
                kept.v[p] = dev::load8(x + (cols(p).any() ? cols(p).first : 0));
                v = unpacked(kept.v[p]);
            } else {
                v = load_v8<G>(x, cols(p));
            }
            uint64_t part = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) part = fma2(v.p[j], v.p[j], part);
            sum += on(cols(p)) ? lanes_sum(part) : 0.0f;
        }
        return sum;
    };
    const bool writes_rstd = rank == 0 && tid == 0;
    float rstd_u = 1.0f;
    Kept u_now, u_next;
    const float first_sum = sum_u(begin, u_now);
    int u_stage = 0;        // the leading stage that is done with next: this row's, KEEP: the next one's
    if (post) {
        sums.send(first_sum, 0.0f, lost);
        rstd_u = rsqrtf(sums.get(lost).x * per_column + a.eps);
        if (a.rstd_post && writes_rstd) a.rstd_post[begin] = rstd_u;
        if (KEEP) {
            if (tid == 0 && !lost && begin + lead.stages < end) fetch_lead(begin + lead.stages, u_stage);
            ++u_stage;
        }
    }
    float next_u = begin + 1 < end ? sum_u(begin + 1, u_next) : 0.0f;
    for (int64_t row = begin; row < end; ++row) {
        const int64_t at = row * H;
        const bool staged = in_ring<G>(row, a.rows, H);
        if (has_u && row == gate_end) {
            gate_end += a.rows_per_gate;
            ++gate_row;
#pragma unroll
            for (int p = 0; p < kPer; ++p) {
                float f[8];
                branch_factor<T>(a, gate_row, col0, cols(p), f);
                own.put(kBranch, p, f);
            }
        }
        V8 v[kPer];
        float sum_v = 0.0f;
        trail.wait(lost);
        const R* r = row_at<G>(trail.at(), 0, res + at, staged);
        const T* x = row_at<G>(lead.base + u_stage * lead.stage_bytes, 0, u + at, staged);
        const uint64_t rstd2 = pair(rstd_u, rstd_u);
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
            v[p] = load_v8<G>(r, cols(p));
            if (has_u) {
                V8 xv;
                if constexpr (KEEP)
                    xv = unpacked(u_now.v[p]);
                else
                    xv = load_v8<G>(x, cols(p));
                const V8 g = own.get(kBranch, p);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[p].p[j] = fma2(mul2(xv.p[j], rstd2), g.p[j], mul2(beta, v[p].p[j]));
                store_v8<G>(static_cast<R*>(a.res_out) + at + col0, cols(p), v[p]);
            }
            uint64_t part = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) part = fma2(v[p].p[j], v[p].p[j], part);
            sum_v += on(cols(p)) ? lanes_sum(part) : 0.0f;
        }
        sums.send(next_u, sum_v, lost);
        if constexpr (KEEP) u_now = u_next;
        if (row + 2 < end) next_u = sum_u(row + 2, u_next);
        const float2 sum = sums.get(lost);
        // everyone has read this row's stages; KEEP: of u, the next row's
        if (tid == 0 && !lost) {
            const int64_t far = row + lead.stages + (KEEP ? 1 : 0);
            if (far < end) fetch_lead(far, u_stage);
            if (row + trail.stages < end) fetch_trail(row + trail.stages, trail.stage);
        }
        trail.next();
        if (++u_stage == lead.stages) u_stage = 0;
        if (post) {
            rstd_u = rsqrtf(sum.x * per_column + a.eps);
            if (a.rstd_post && writes_rstd && row + 1 < end) a.rstd_post[row + 1] = rstd_u;
        }
        if (!pre) continue;
        const float rstd = rsqrtf(sum.y * per_column + a.eps);
        if (a.rstd_pre && writes_rstd) a.rstd_pre[row] = rstd;
        const uint64_t rstd_v = pair(rstd, rstd);
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
            const V8 w = own.get(kPre, p);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[p].p[j] = mul2(mul2(v[p].p[j], rstd_v), w.p[j]);
            put_y<T>(a, at + col0, cols(p), v[p], scale, most);
        }
    }
    dev::pdl_launch_dependents();
    if (pre) put_amax(a, most, scale, &block_max, lost);
    if (lost && tid == 0) {
        lead.drain();
        trail.drain();
    }
    sums.end(lost, kErrWaitTimeout);
}

// Forward, one row per cluster: for launches of no more rows than clusters fit.
// Everything is loaded at once, then summed twice (4x4096 to FP8: 4.6 us, the
// ring's kernel with plain loads 5.4).  From more rows on the ring is ahead:
// 1000x4096 12.6 us against 20.6, 1200x6144 16.9 against 46.
template <typename T, typename R, int G>
__global__ void __launch_bounds__(kForwardThreads, 1) block_norm_row_kernel(const NormArgs a,
                                                                        const NormShape s) {
    __shared__ float slots[2][2][kMaxCluster * kMaxWarps];
    __shared__ __align__(8) uint64_t bars[2];
    __shared__ unsigned block_max;
    const int tid = threadIdx.x, H = a.hidden;
    const int rank = blockIdx.x % s.cluster, col0 = rank * s.width, W = min(s.width, H - col0);
    const int64_t row = blockIdx.x / s.cluster, at = row * H + col0;
    auto cols = [&](int p) { return dev::Cols<G>(p * blockDim.x + tid, W); };
    RowSums sums{slots, bars, s.cluster, rank};
    bool lost = false;
    dev::pdl_launch_dependents();
    if (tid == 0) {
        block_max = 0;
        sums.init();
        dev::fence_barrier_init();
    }
    sums.meet();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const float scale = a.scale ? *a.scale : 0.0f, per_column = 1.0f / H;
    const int64_t gate_row = a.gate ? row / a.rows_per_gate : 0;
    V8 u[kPer], v[kPer], branch[kPer], w[kPer];
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
        float f[8];
        v[p] = load_v8<G>(static_cast<const R*>(a.res) + at, cols(p));
        if (a.u) {
            u[p] = load_v8<G>(static_cast<const T*>(a.u) + at, cols(p));
            branch_factor<T>(a, gate_row, col0, cols(p), f);
            branch[p] = pairs(f);
        }
        if (a.pre) {
            load_param<T>(a.w_pre, a.param_f32, col0, a.weight_offset, cols(p), f);
            w[p] = pairs(f);
        }
    }
    auto sum_squares = [&](const V8 (&x)[kPer]) {
        float sum = 0.0f;
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
            uint64_t part = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) part = fma2(x[p].p[j], x[p].p[j], part);
            sum += on(cols(p)) ? lanes_sum(part) : 0.0f;
        }
        return sum;
    };
    if (a.u) {
        float rstd = 1.0f;
        if (a.post) {
            sums.send(sum_squares(u), 0.0f, lost);
            rstd = rsqrtf(sums.get(lost).x * per_column + a.eps);
            if (a.rstd_post && rank == 0 && tid == 0) a.rstd_post[row] = rstd;
        }
        const uint64_t rstd2 = pair(rstd, rstd), beta = pair(a.residual_scale, a.residual_scale);
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[p].p[j] = fma2(mul2(u[p].p[j], rstd2), branch[p].p[j], mul2(beta, v[p].p[j]));
            store_v8<G>(static_cast<R*>(a.res_out) + at, cols(p), v[p]);
        }
    }
    if (a.pre) {
        sums.send(0.0f, sum_squares(v), lost);
        const float rstd = rsqrtf(sums.get(lost).y * per_column + a.eps);
        if (a.rstd_pre && rank == 0 && tid == 0) a.rstd_pre[row] = rstd;
        const uint64_t rstd2 = pair(rstd, rstd);
        unsigned most = 0;
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[p].p[j] = mul2(mul2(v[p].p[j], rstd2), w[p].p[j]);
            put_y<T>(a, at, cols(p), v[p], scale, most);
        }
        put_amax(a, most, scale, &block_max, lost);
    }
    sums.end(lost, kErrWaitTimeout);
}

// What the workspace holds for the backward pass, [clusters][H] each: partial
// column sums of dw_pre and dw_post, and those of dgate for the first and the
// last gate row of a run, where they belong to other runs too.
enum { kSumPre, kSumPost, kSumGateFirst, kSumGateLast, kSums };

// Backward.  With xh = res_out rstd_pre, G = dy a_pre, uh = u rstd_post:
//   D  = dres_out + rstd_pre (G - xh mean(G xh))      dres = beta D
//   P  = alpha gate a_post D                           du = rstd_post (P - uh mean(P uh))
//   dw_pre = sum dy xh
//   S  = sum D uh over a gate row's rows: dgate = alpha a_post S, dw_post = sum alpha gate S
template <typename T, typename R, int G, bool FULL>
__global__ void __launch_bounds__(kBackwardThreads, 1)
    block_norm_backward_kernel(const NormBackwardArgs a, const NormShape s) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float slots[2][2][kMaxCluster * kMaxWarps];
    __shared__ __align__(8) uint64_t full[2 * kMaxStages + 2];
    const bool has_u = FULL || a.u, post = FULL || a.post, pre = FULL || a.pre;
    const bool has_dres = FULL || a.dres_out;
    const int tid = threadIdx.x, H = a.hidden;
    const int rank = blockIdx.x % s.cluster, run = blockIdx.x / s.cluster;
    const int col0 = rank * s.width, W = min(s.width, H - col0);
    auto cols = [&](int p) { return dev::Cols<G>(p * blockDim.x + tid, W); };
    const int64_t begin = run_begin(a.rows, run, s.clusters), end = run_begin(a.rows, run + 1, s.clusters);
    constexpr uint32_t kT = sizeof(T), kR = sizeof(R);
    const uint32_t second = place_bytes<G, R>(s.width);    // in a stage: of type R, then of type T
    const uint32_t stage_bytes = second + place_bytes<G, T>(s.width);
    Ring lead{full, smem, stage_bytes, s.lead};        // res_out, dy
    Ring trail{full + kMaxStages, smem + lead.stages * stage_bytes, stage_bytes, s.trail};   // dres_out, u
    bool lost = false;
    const Own own{reinterpret_cast<float4*>(trail.base + trail.stages * stage_bytes)};
    RowSums sums{slots, full + 2 * kMaxStages, s.cluster, rank};
    const R* res_out = static_cast<const R*>(a.res_out) + col0;
    const R* dres_out = static_cast<const R*>(a.dres_out) + col0;
    const T* dy = static_cast<const T*>(a.dy) + col0;
    const T* u = static_cast<const T*>(a.u) + col0;

    if (tid == 0) {
        sums.init();
        lead.init();
        trail.init();
        dev::fence_barrier_init();
    }
    sums.meet();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    auto fetch_lead = [&](int64_t row, int to) {
        const bool staged = pre && in_ring<G>(row, a.rows, H);
        lead.fetch(to, staged ? res_out + row * H : nullptr, W * kR, second, staged ? dy + row * H : nullptr, W * kT);
    };
    auto fetch_trail = [&](int64_t row, int to) {
        const bool staged = in_ring<G>(row, a.rows, H);
        trail.fetch(to, staged && has_dres ? dres_out + row * H : nullptr, W * kR, second,
                    staged && has_u ? u + row * H : nullptr, W * kT);
    };
    if (tid == 0)
        for (int i = 0; i < max(lead.stages, trail.stages) && begin + i < end; ++i) {
            if (i < lead.stages) fetch_lead(begin + i, i);
            if (i < trail.stages) fetch_trail(begin + i, i);
        }
    const float beta1 = has_u ? a.residual_scale : 1.0f;
    const uint64_t beta = pair(beta1, beta1);
    const int64_t first_gate = a.gate ? begin / a.rows_per_gate : 0;
    int64_t gate_row = first_gate;
    int64_t gate_end = a.gate ? (gate_row + 1) * a.rows_per_gate : a.rows;
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
        float f[8];
        if (has_u) {
            branch_factor<T>(a, gate_row, col0, cols(p), f);
            own.put(kBranch, p, f);
        }
        if (pre) {
            load_param<T>(a.w_pre, a.param_f32, col0, a.weight_offset, cols(p), f);
            own.put(kPre, p, f);
        }
    }
    const float per_column = 1.0f / H;
    V8 dw_pre[kPer] = {}, dots[kPer] = {};   // sums of dy xh, and S

    // sum of G xh over the next row of the leading ring, and its part of dw_pre
    auto first_sum = [&](int64_t row, float rstd) {
        lead.wait(lost);
        const uint8_t* stage = lead.at();
        lead.next();
        if (!pre) return 0.0f;
        const bool staged = in_ring<G>(row, a.rows, H);
        const T* g = row_at<G>(stage, second, dy + row * H, staged);
        const R* x = row_at<G>(stage, 0, res_out + row * H, staged);
        const uint64_t rstd2 = pair(rstd, rstd);
        float sum = 0.0f;
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
            uint64_t part = 0;
            const V8 gv = load_v8<G>(g, cols(p)), xv = load_v8<G>(x, cols(p)), w = own.get(kPre, p);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint64_t t = mul2(gv.p[j], xv.p[j]);
                dw_pre[p].p[j] = fma2(t, rstd2, dw_pre[p].p[j]);
                part = fma2(t, w.p[j], part);
            }
            sum += on(cols(p)) ? lanes_sum(part) : 0.0f;
        }
        return sum * rstd;
    };
    // Ends a gate row: its part of dw_post joins the run's, which this thread
    // alone touches in the workspace; dgate goes out where all its rows are
    // this run's, else to the workspace.
    auto end_gate = [&] {
        const bool whole = gate_row * a.rows_per_gate >= begin && min(gate_end, a.rows) <= end;
        float* post_sums = a.workspace + (int64_t(kSumPost) * s.clusters + run) * H + col0;
        float* gate_sums = a.workspace +
            (int64_t(gate_row == first_gate ? kSumGateFirst : kSumGateLast) * s.clusters + run) * H + col0;
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
            const dev::Cols<G> c = cols(p);
            float f[8], w[8];
            floats(dots[p], f);
            dots[p] = V8{};
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= a.branch_scale;
            if (a.dw_post) {
                float sum[8] = {};
                if (gate_row != first_gate) dev::load_cols<G>(post_sums, c, sum);
                load_param<T>(a.gate, a.param_f32, gate_row * H + col0, 0.0f, c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] = fmaf(w[j], f[j], sum[j]);
                dev::store_cols<G>(post_sums, c, sum);
            }
            if (a.dgate) {
                load_param<T>(post ? a.w_post : nullptr, a.param_f32, col0, a.weight_offset, c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] *= w[j];
                const int64_t at = gate_row * H + col0;
                if (!whole)
                    dev::store_cols<G>(gate_sums, c, f);
                else if (a.param_f32)
                    dev::store_cols<G>(static_cast<float*>(a.dgate) + at, c, f);
                else
                    dev::store_cols<G>(static_cast<T*>(a.dgate) + at, c, f);
            }
        }
    };

    // rstd of this row and the next two
    auto rstd_at = [&](bool norm, const float* rstd, int64_t row, float none) {
        return norm && row < end ? rstd[row] : none;
    };
    float rstd_x = rstd_at(pre, a.rstd_pre, begin, 0.0f), rstd_u = rstd_at(post, a.rstd_post, begin, 1.0f);
    float next_x = rstd_at(pre, a.rstd_pre, begin + 1, 0.0f);
    float mean_x = 0.0f;
    {
        const float sum = first_sum(begin, rstd_x);
        if (pre) {
            sums.send(sum, 0.0f, lost);
            mean_x = sums.get(lost).x * per_column;
        }
    }
    float sum_x = begin + 1 < end ? first_sum(begin + 1, next_x) : 0.0f;
    int x_stage = 0;        // the stage of this row's res_out: the leading ring itself is rows ahead
    for (int64_t row = begin; row < end; ++row) {
        const int64_t at = row * H;
        const bool staged = in_ring<G>(row, a.rows, H);
        const float far_x = rstd_at(pre, a.rstd_pre, row + 2, 0.0f);
        const float next_u = rstd_at(post, a.rstd_post, row + 1, 1.0f);
        if (has_u && row == gate_end) {
            end_gate();
            gate_end += a.rows_per_gate;
            ++gate_row;
#pragma unroll
            for (int p = 0; p < kPer; ++p) {
                float f[8];
                branch_factor<T>(a, gate_row, col0, cols(p), f);
                own.put(kBranch, p, f);
            }
        }
        V8 branch[kPer], hat[kPer];          // P, uh
        float sum_p = 0.0f;
        trail.wait(lost);
        const uint8_t* stage = lead.base + x_stage * stage_bytes;
        const R* x = row_at<G>(stage, 0, res_out + at, staged);
        const T* g = row_at<G>(stage, second, dy + at, staged);
        const R* r = row_at<G>(trail.at(), 0, dres_out + at, staged);
        const T* y = row_at<G>(trail.at(), second, u + at, staged);
        const float back1 = -rstd_x * rstd_x * mean_x;
        const uint64_t back = pair(back1, back1), rx2 = pair(rstd_x, rstd_x), ru2 = pair(rstd_u, rstd_u);
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
            V8 d = {};
            if (has_dres) d = load_v8<G>(r, cols(p));
            if (pre) {
                const V8 gv = load_v8<G>(g, cols(p)), xv = load_v8<G>(x, cols(p)), w = own.get(kPre, p);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    d.p[j] = fma2(xv.p[j], back, fma2(mul2(gv.p[j], rx2), w.p[j], d.p[j]));
            }
            V8 out;
#pragma unroll
            for (int j = 0; j < 4; ++j) out.p[j] = mul2(beta, d.p[j]);
            store_v8<G>(static_cast<R*>(a.dres) + at + col0, cols(p), out);
            if (has_u) {
                hat[p] = load_v8<G>(y, cols(p));
                branch[p] = own.get(kBranch, p);
                uint64_t part = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    hat[p].p[j] = mul2(hat[p].p[j], ru2);
                    dots[p].p[j] = fma2(d.p[j], hat[p].p[j], dots[p].p[j]);
                    branch[p].p[j] = mul2(branch[p].p[j], d.p[j]);
                    part = fma2(branch[p].p[j], hat[p].p[j], part);
                }
                sum_p += on(cols(p)) ? lanes_sum(part) : 0.0f;
            }
        }
        sums.send(sum_x, sum_p, lost);
        if (row + 2 < end) sum_x = first_sum(row + 2, far_x);
        const float2 sum = sums.get(lost);
        // everyone has read this row's stages
        if (tid == 0 && !lost) {
            if (row + lead.stages < end) fetch_lead(row + lead.stages, x_stage);
            if (row + trail.stages < end) fetch_trail(row + trail.stages, trail.stage);
        }
        trail.next();
        if (++x_stage == lead.stages) x_stage = 0;
        if (has_u) {
            const float mean = post ? -sum.y * per_column : 0.0f;
            const uint64_t mean2 = pair(mean, mean);
#pragma unroll
            for (int p = 0; p < kPer; ++p) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    branch[p].p[j] = mul2(ru2, fma2(hat[p].p[j], mean2, branch[p].p[j]));
                store_v8<G>(static_cast<T*>(a.du) + at + col0, cols(p), branch[p]);
            }
        }
        mean_x = sum.x * per_column;
        rstd_x = next_x;
        next_x = far_x;
        rstd_u = next_u;
    }
    dev::pdl_launch_dependents();
    if (has_u) end_gate();
    if (a.dw_pre) {
        float* part = a.workspace + (int64_t(kSumPre) * s.clusters + run) * H + col0;
#pragma unroll
        for (int p = 0; p < kPer; ++p) store_v8<G>(part, cols(p), dw_pre[p]);
    }
    if (lost && tid == 0) {
        lead.drain();
        trail.drain();
    }
    sums.end(lost, kErrWaitTimeout);
}

// Backward, one row per cluster, likewise: its column sums are the row's terms
// (500x777 with the join 14.6 us, the ring's kernel with plain loads 20.1).
template <typename T, typename R, int G>
__global__ void __launch_bounds__(kBackwardThreads, 1)
    block_norm_backward_row_kernel(const NormBackwardArgs a, const NormShape s) {
    __shared__ float slots[2][2][kMaxCluster * kMaxWarps];
    __shared__ __align__(8) uint64_t bars[2];
    const int tid = threadIdx.x, H = a.hidden;
    const int rank = blockIdx.x % s.cluster, col0 = rank * s.width, W = min(s.width, H - col0);
    const int64_t row = blockIdx.x / s.cluster, at = row * H + col0;
    auto cols = [&](int p) { return dev::Cols<G>(p * blockDim.x + tid, W); };
    RowSums sums{slots, bars, s.cluster, rank};
    bool lost = false;
    dev::pdl_launch_dependents();
    if (tid == 0) {
        sums.init();
        dev::fence_barrier_init();
    }
    sums.meet();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const float rstd_x = a.pre ? a.rstd_pre[row] : 0.0f, rstd_u = a.post ? a.rstd_post[row] : 1.0f;
    const float beta1 = a.u ? a.residual_scale : 1.0f, per_column = 1.0f / H;
    const uint64_t rx2 = pair(rstd_x, rstd_x), ru2 = pair(rstd_u, rstd_u), beta = pair(beta1, beta1);
    const int64_t gate_row = a.gate ? row / a.rows_per_gate : 0;
    auto sums_of = [&](int kind) { return a.workspace + (int64_t(kind) * s.clusters + row) * H + col0; };
    V8 d[kPer], g[kPer], x[kPer], hat[kPer], gate[kPer], w_post[kPer];
    float sum = 0.0f;
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
        float f[8];
        d[p] = V8{};
        if (a.dres_out) d[p] = load_v8<G>(static_cast<const R*>(a.dres_out) + at, cols(p));
        if (a.u) {
            hat[p] = load_v8<G>(static_cast<const T*>(a.u) + at, cols(p));
            load_param<T>(a.gate, a.param_f32, gate_row * H + col0, 0.0f, cols(p), f);
            gate[p] = pairs(f);
            load_param<T>(a.post ? a.w_post : nullptr, a.param_f32, col0, a.weight_offset, cols(p), f);
            w_post[p] = pairs(f);
        }
        if (a.pre) {
            g[p] = load_v8<G>(static_cast<const T*>(a.dy) + at, cols(p));
            x[p] = load_v8<G>(static_cast<const R*>(a.res_out) + at, cols(p));
            load_param<T>(a.w_pre, a.param_f32, col0, a.weight_offset, cols(p), f);
            const V8 w = pairs(f);
            V8 terms;
            uint64_t part = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[p].p[j] = mul2(x[p].p[j], rx2);                // xh
                terms.p[j] = mul2(g[p].p[j], x[p].p[j]);
                part = fma2(terms.p[j], w.p[j], part);
                g[p].p[j] = mul2(g[p].p[j], w.p[j]);             // G
            }
            sum += on(cols(p)) ? lanes_sum(part) : 0.0f;
            if (a.dw_pre) store_v8<G>(sums_of(kSumPre), cols(p), terms);
        }
    }
    float mean = 0.0f;
    if (a.pre) {
        sums.send(sum, 0.0f, lost);
        mean = -sums.get(lost).x * per_column;
    }
    const uint64_t mean_x = pair(mean, mean), alpha = pair(a.branch_scale, a.branch_scale);
    sum = 0.0f;
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
        V8 out;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (a.pre) d[p].p[j] = fma2(rx2, fma2(x[p].p[j], mean_x, g[p].p[j]), d[p].p[j]);
            out.p[j] = mul2(beta, d[p].p[j]);
        }
        store_v8<G>(static_cast<R*>(a.dres) + at, cols(p), out);
        if (!a.u) continue;
        V8 post_terms, gate_terms;
        uint64_t part = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            hat[p].p[j] = mul2(hat[p].p[j], ru2);                // uh
            const uint64_t dots = mul2(alpha, mul2(d[p].p[j], hat[p].p[j]));
            post_terms.p[j] = mul2(gate[p].p[j], dots);
            gate_terms.p[j] = mul2(w_post[p].p[j], dots);
            d[p].p[j] = mul2(mul2(alpha, mul2(gate[p].p[j], d[p].p[j])), w_post[p].p[j]);   // P
            part = fma2(d[p].p[j], hat[p].p[j], part);
        }
        sum += on(cols(p)) ? lanes_sum(part) : 0.0f;
        if (a.dw_post) store_v8<G>(sums_of(kSumPost), cols(p), post_terms);
        if (a.dgate) {
            if (gate_row * a.rows_per_gate != row || min((gate_row + 1) * a.rows_per_gate, a.rows) != row + 1)
                store_v8<G>(sums_of(kSumGateFirst), cols(p), gate_terms);
            else if (a.param_f32)
                store_v8<G>(static_cast<float*>(a.dgate) + gate_row * H + col0, cols(p), gate_terms);
            else
                store_v8<G>(static_cast<T*>(a.dgate) + gate_row * H + col0, cols(p), gate_terms);
        }
    }
    if (a.u) {
        mean = 0.0f;
        if (a.post) {
            sums.send(0.0f, sum, lost);
            mean = -sums.get(lost).y * per_column;
        }
        const uint64_t mean_p = pair(mean, mean);
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
#pragma unroll
            for (int j = 0; j < 4; ++j) d[p].p[j] = mul2(ru2, fma2(hat[p].p[j], mean_p, d[p].p[j]));
            store_v8<G>(static_cast<T*>(a.du) + at, cols(p), d[p]);
        }
    }
    sums.end(lost, kErrWaitTimeout);
}

// The give-up path by itself: a cluster exchanges sums three times, and after
// the second time one thread of its first block goes on as if that wait had run
// out.  Its warp's third sums are then missing where it would have sent them.
constexpr int kSelftestThreads = 64;

__global__ void __launch_bounds__(kSelftestThreads) norm_wait_selftest_kernel(int thread, uint64_t limit_ns) {
    __shared__ float slots[2][2][kMaxCluster * kMaxWarps];
    __shared__ __align__(8) uint64_t bars[2];
    RowSums sums{slots, bars, static_cast<int>(gridDim.x), static_cast<int>(blockIdx.x), limit_ns};
    bool lost = false;
    if (threadIdx.x == 0) {
        sums.init();
        dev::fence_barrier_init();
    }
    sums.meet();
    dev::pdl_wait();      // so that what follows it in the stream follows what came before, too
    for (int i = 0; i < 3; ++i) {
        sums.send(1.0f, 2.0f, lost);
        sums.get(lost);
        if (i == 1 && blockIdx.x == 0 && threadIdx.x == thread) lost = true;
    }
    sums.end(lost, kErrSelftestTimeout);
}

// Joins the runs' column sums, in run order.  blockIdx.y 0, 1: dw_pre, dw_post;
// from 2 on the gate rows that more than one run has rows of, by gate row
// (few of them, perhaps of many runs), else by the run they begin in.
//
// A block takes `cols` columns (32, or 8, one sector, of short rows) and gives
// each blockDim / cols threads, which add up every so many-th run.
constexpr int kJoinThreads = 512;      // at most

template <typename T>
__global__ void __launch_bounds__(kJoinThreads)
    block_norm_join_kernel(const NormBackwardArgs a, int64_t runs, int cols, int by_gate_row) {
    __shared__ float parts[kJoinThreads];
    dev::pdl_launch_dependents();
    dev::pdl_wait();
    if (a.noop && *a.noop != 0.0f) return;
    const int H = a.hidden, x = threadIdx.x % cols, y = threadIdx.x / cols;
    const int shares = blockDim.x / cols, which = blockIdx.y;
    int64_t first = 0, last = runs - 1, at = 0;   // the runs to add up
    int col = blockIdx.x * cols + x;
    void* out = which == 0 ? a.dw_pre : which == 1 ? a.dw_post : a.dgate;
    if (!out) return;
    // where the first run's sums are, and the others'
    int kind_first = which == 0 ? kSumPre : kSumPost, kind = kind_first;
    if (which >= 2) {
        int64_t gate_row;
        if (by_gate_row) {
            gate_row = which - 2;
            first = run_of(a.rows, gate_row * a.rows_per_gate, runs);
        } else {
            // blockDim.x columns of the gate row that run `which - 2` ends in,
            // if it begins there
            col = blockIdx.x * blockDim.x + threadIdx.x;
            first = which - 2;
            gate_row = (run_begin(a.rows, first + 1, runs) - 1) / a.rows_per_gate;
            if (gate_row * a.rows_per_gate < run_begin(a.rows, first, runs)) return;
        }
        last = run_of(a.rows, min((gate_row + 1) * a.rows_per_gate, a.rows) - 1, runs);
        if (first == last) return;                // written by its run
        at = gate_row * H;
        // a gate row is the last one of its first run, unless it is that run's
        // first one too, and the first one of the others
        kind = kSumGateFirst;
        kind_first = run_begin(a.rows, first, runs) / a.rows_per_gate == gate_row ? kSumGateFirst : kSumGateLast;
    }
    const float* sums = a.workspace + int64_t(kind) * runs * H + col;
    const float* sums_first = a.workspace + (int64_t(kind_first) * runs + first) * H + col;
    float sum = 0.0f;
    if (which >= 2 && !by_gate_row) {
        if (col >= H) return;
        sum = *sums_first;
        for (int64_t r = first + 1; r <= last; ++r) sum += sums[r * H];
        set_param<T>(out, a.param_f32, at + col, sum);
        return;
    }
    if (col < H && first <= last) {
        if (y == 0) sum = *sums_first;
        const int64_t step = int64_t(shares) * H;
        const float* p = sums + (first + (y == 0 ? shares : y)) * H;
        int left = static_cast<int>((last - first - (y == 0 ? shares : y) + shares) / shares);
#pragma unroll 8
        for (; left > 0; --left, p += step) sum += *p;
    }
    parts[threadIdx.x] = sum;
    for (int n = shares / 2; n > 0; n /= 2) {
        __syncthreads();
        if (y < n) parts[threadIdx.x] += parts[threadIdx.x + n * cols];
    }
    if (y == 0 && col < H) set_param<T>(out, a.param_f32, at + col, parts[x]);
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

int round_up(int v, int to) { return (v + to - 1) / to * to; }
int threads_of(int width) { return std::max(32, round_up((width + 8 * kPer - 1) / (8 * kPer), 32)); }
int slice(int64_t hidden, int cluster) {
    return std::max(8, round_up(static_cast<int>((hidden + cluster - 1) / cluster), 8));
}

// The most runs of rows a backward launch makes: the workspace has room for them.
int64_t max_clusters(int64_t rows, int64_t hidden) {
    int cluster = 1;
    while (threads_of(slice(hidden, cluster)) > kBackwardThreads) cluster *= 2;
    return std::min<int64_t>(rows, int64_t(sm_count()) * (kBackwardThreads / threads_of(slice(hidden, cluster))) / cluster);
}

// Picks the fewest blocks per row whose rings hold enough, then as many blocks
// per SM as the registers and then the rings allow.  lead_bytes, trail_bytes:
// of one column in a stage, of `tensors` tensors; min_lead: rows that hold a
// leading stage at a time; max_threads, sm_threads: of a block, and those that
// an SM's registers hold; most: runs of rows, at most.
NormShape shape_of(int64_t rows, int hidden, int lead_bytes, int trail_bytes, int tensors, int min_lead,
                   bool vec, int max_threads, int sm_threads, int64_t most, size_t* smem) {
    NormShape s = {};
    const int pad = vec ? 0 : 32 * tensors;
    auto own = [&] { return kOwnBytes * threads_of(s.width); };
    auto rings = [&](int lead, int trail) {
        return lead * (s.width * lead_bytes + pad) + trail * (s.width * trail_bytes + pad);
    };
    // Stages for `per_sm` blocks; false with fewer than the rows that are in use
    // at a time in the leading ring and two in the trailing one.
    auto fill = [&](int per_sm) {
        const int room = kSmemPerSm / per_sm - kSmemFixed - own();
        s.lead = min_lead;
        s.trail = 2;
        if (rings(s.lead, s.trail) > room) return false;
        for (;;) {
            if (s.lead < kMaxStages && rings(s.lead + 1, s.trail) <= room) ++s.lead;
            else return true;
            if (s.trail < kMaxStages && rings(s.lead, s.trail + 1) <= room) ++s.trail;
        }
    };
    for (s.cluster = 1;; s.cluster *= 2) {
        s.width = slice(hidden, s.cluster);
        if (threads_of(s.width) <= max_threads && (s.cluster == kMaxCluster || fill(1))) break;
    }
    int per_sm = std::min(sm_threads / threads_of(s.width), 32);
    while (per_sm > 1 && !fill(per_sm)) --per_sm;
    s.clusters = static_cast<int>(
        std::min({rows, most, int64_t(std::max(1, sm_count() * per_sm / s.cluster))}));
    fill(per_sm);
    *smem = size_t(own()) + rings(s.lead, s.trail);
    if (rows <= s.clusters) {
        s.lead = s.trail = 0;
        *smem = 0;
    }
    return s;
}

// The launch configuration of a shape; `attr` has to live as long as it.
cudaLaunchConfig_t config_of(const NormShape& s, size_t smem, cudaStream_t stream, cudaLaunchAttribute (&attr)[2]) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(s.clusters * s.cluster));
    cfg.blockDim = dim3(static_cast<unsigned>(threads_of(s.width)));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(s.cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = s.cluster > 1 ? 2 : 1;
    return cfg;
}

// Before a kernel's first launch on a device with this much shared memory:
// allows it, and asks for as much shared memory as the SM has.  Limits the
// runs to the clusters that can be resident: those of 4 or 8 blocks do not
// fill every SM, and a second wave of runs would double the time.
cudaError_t prepare(const void* kernel, NormShape& s, size_t smem) {
    struct Known {
        const void* kernel;
        int device, cluster, threads;
        size_t smem;
        int most;
    };
    // the latest shapes; one that has been displaced is looked up again
    constexpr int kKnown = 256;
    static std::mutex mutex;
    static Known known[kKnown];
    static unsigned remembered = 0;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mutex);
    const int count = static_cast<int>(std::min(remembered, unsigned(kKnown)));
    for (int i = 0; i < count; ++i) {
        const Known& k = known[i];
        if (k.kernel == kernel && k.device == device && k.cluster == s.cluster &&
            k.threads == threads_of(s.width) && k.smem == smem) {
            if (s.lead) s.clusters = std::min(s.clusters, k.most);
            return cudaSuccess;
        }
    }
    Known k = {kernel, device, s.cluster, threads_of(s.width), smem, s.clusters};
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerSm - kSmemFixed);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                 cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    k.most = 1 << 30;
    if (s.cluster > 1) {
        cudaLaunchAttribute attr[2];
        const cudaLaunchConfig_t cfg = config_of(s, smem, nullptr, attr);
        int most = 0;
        e = cudaOccupancyMaxActiveClusters(&most, kernel, &cfg);
        if (e != cudaSuccess) return e;
        k.most = std::max(most, 1);
    }
    known[remembered++ % kKnown] = k;
    if (remembered == 2u * kKnown) remembered = kKnown;   // so that it never wraps
    if (s.lead) s.clusters = std::min(s.clusters, k.most);
    return cudaSuccess;
}

template <typename Args>
cudaError_t launch_rows(void (*kernel)(const Args, const NormShape), const Args& a, const NormShape& s,
                        size_t smem, cudaStream_t stream) {
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = config_of(s, smem, stream, attr);
    return cudaLaunchKernelEx(&cfg, kernel, a, s);
}

}  // namespace

cudaError_t read_norm_error(unsigned* value, bool clear) {
    const cudaError_t e = cudaMemcpyFromSymbol(value, g_norm_error, sizeof(unsigned));
    if (e != cudaSuccess || !clear) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_norm_error, &zero, sizeof(unsigned));
}

cudaError_t launch_norm_wait_selftest(int blocks, int thread, uint32_t limit_us, cudaStream_t stream) {
    NormShape s = {};
    s.cluster = blocks;
    s.clusters = 1;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = config_of(s, 0, stream, attr);
    cfg.blockDim = dim3(kSelftestThreads);
    return cudaLaunchKernelEx(&cfg, norm_wait_selftest_kernel, thread, uint64_t(limit_us) * 1000);
}

cudaError_t launch_block_norm(const NormArgs& a, int dtype, int res_dtype, cudaStream_t stream) {
    const bool vec = a.hidden % 8 == 0 && all_aligned(a.u, a.res, a.w_post, a.w_pre, a.gate,
                                                      a.res_out, a.y);
    return by_types(dtype, res_dtype, [&](auto t, auto r) {
        using T = decltype(t);
        using R = decltype(r);
        size_t smem;
        const bool full = a.u && a.post && a.pre;
        // rows i+1, i+2, and i unless it is kept
        const int min_lead = full && vec && sizeof(T) == 2 ? 2 : 3;
        NormShape s = shape_of(a.rows, a.hidden, sizeof(T), sizeof(R), 1, min_lead, vec, kForwardThreads,
                               2 * kForwardThreads, a.rows, &smem);
        auto* kernel = s.lead ? (vec ? (full ? block_norm_kernel<T, R, 8, true> : block_norm_kernel<T, R, 8, false>)
                                     : block_norm_kernel<T, R, 1, false>)
                              : (vec ? block_norm_row_kernel<T, R, 8> : block_norm_row_kernel<T, R, 1>);
        const cudaError_t e = prepare(reinterpret_cast<const void*>(kernel), s, smem);
        return e != cudaSuccess ? e : launch_rows(kernel, a, s, smem, stream);
    });
}

size_t norm_backward_workspace(int64_t rows, int64_t hidden) {
    return static_cast<size_t>(max_clusters(rows, hidden) * kSums * hidden) * sizeof(float) / 16 * 16 + 16;
}

cudaError_t launch_block_norm_backward(const NormBackwardArgs& a, int dtype, int res_dtype,
                                       cudaStream_t stream) {
    const bool vec = a.hidden % 8 == 0 &&
                     all_aligned(a.dy, a.dres_out, a.u, a.res_out, a.w_post, a.w_pre, a.gate, a.du,
                                 a.dres, a.dgate);
    return by_types(dtype, res_dtype, [&](auto t, auto r) {
        using T = decltype(t);
        using R = decltype(r);
        size_t smem;
        NormShape s = shape_of(a.rows, a.hidden, sizeof(T) + sizeof(R), sizeof(T) + sizeof(R), 2, 3, vec,
                               kBackwardThreads, kBackwardThreads, max_clusters(a.rows, a.hidden), &smem);
        if (a.rows > 0) {
            const bool full = a.u && a.post && a.pre && a.dres_out;
            auto* kernel = s.lead ? (vec ? (full ? block_norm_backward_kernel<T, R, 8, true>
                                                 : block_norm_backward_kernel<T, R, 8, false>)
                                         : block_norm_backward_kernel<T, R, 1, false>)
                                  : (vec ? block_norm_backward_row_kernel<T, R, 8>
                                         : block_norm_backward_row_kernel<T, R, 1>);
            cudaError_t e = prepare(reinterpret_cast<const void*>(kernel), s, smem);
            if (e == cudaSuccess) e = launch_rows(kernel, a, s, smem, stream);
            if (e != cudaSuccess) return e;
        }
        if (!a.dw_pre && !a.dw_post && !a.dgate) return cudaSuccess;
        const int64_t gates = a.dgate ? (a.rows + a.rows_per_gate - 1) / a.rows_per_gate : 0;
        const bool by_gate_row = gates <= s.clusters / 2;
        const int64_t joins = !a.dgate ? 0 : by_gate_row ? gates : s.clusters - 1;
        // Shorter sums where runs are many, smaller blocks where they are few; the
        // whole backward pass, us, with 128 / 256 / 512 threads: 76 runs of 12288
        // columns 189.4 / 191.5 / -, 152 of 6144 103.3 / 102.6 / -, 912 of 1024
        // - / 105.1 / 102.9.
        const int cols = s.clusters > 256 && a.hidden < 1024 ? 8 : 32;
        const int threads = s.clusters > 256 ? kJoinThreads : s.clusters > 100 ? 256 : 128;
        return launch_pdl(block_norm_join_kernel<T>,
                          dim3((a.hidden + cols - 1) / cols, static_cast<unsigned>(2 + joins)),
                          dim3(threads), 0, stream, a, int64_t(s.clusters), cols, by_gate_row ? 1 : 0);
    });
}

}  // namespace ct
