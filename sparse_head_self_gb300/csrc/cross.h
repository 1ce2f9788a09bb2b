// Internal declarations of the cross attention (queries of one sequence,
// keys and values of another) and of the query/key norm with rotation.  The
// operations and every argument rule are documented in include/fibatt.h.
#pragma once

#include <algorithm>
#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

#include "fibatt.h"
#include "fibatt_internal.h"
#include "per_device.h"

namespace fibatt {

// One head tensor as a kernel sees it: element [b, h, n, d] at
// p + b sb + h sh + n sn + d (strides in elements).
template <typename T>
struct Rows {
    T *p;
    int64_t sb, sh, sn;
    __host__ __device__ T *row(int64_t b, int64_t h, int64_t n) const { return p + b * sb + h * sh + n * sn; }
};

template <typename T>
Rows<T> rows_of(const fibatt_heads &v) {
    return Rows<T>{static_cast<T *>(v.ptr), v.stride_b, v.stride_h, v.stride_n};
}

// Which keys a sequence attends: k < len[b] and mask[b][k] != 0.
struct KeySet {
    const int32_t *len;      // [B] or null
    const uint8_t *mask;     // [B][Nk] or null
    int64_t mask_sb;
    int Nk;
#ifdef __CUDACC__
    // keys at or behind the result are not attended
    __device__ int bound(int b) const { return len ? max(0, min(__ldg(len + b), Nk)) : Nk; }
    __device__ bool has(int b, int k) const { return !mask || __ldg(mask + b * mask_sb + k) != 0; }
#endif
};

// A number that a call reads on the device.
__host__ __device__ __forceinline__ int32_t load_number(const int32_t *p) {
#ifdef __CUDA_ARCH__
    return __ldg(p);
#else
    return *p;
#endif
}
__host__ __device__ __forceinline__ int least(int a, int b) { return a < b ? a : b; }
__host__ __device__ __forceinline__ int most(int a, int b) { return a < b ? b : a; }

// Attention over a sliding window with sinks: the query at position p of its
// sequence attends the keys k <= p with k > p - window or k < sinks.  Positions
// outside the sequence attend nothing, which p = -1 stands for below.  (Sizes and
// the window are at most 2^30, so that sums of two stay in 32 bits.)
struct Band {
    const int32_t *start;    // [B]: position of a sequence's first query, or null: Nk - Nq
    int Nq, Nk, window, sinks;
    // (a start further out leaves no query a position, wherever it is)
    __host__ __device__ __forceinline__ int first(int b) const {
        return start ? most(-Nq, least(load_number(start + b), Nk)) : Nk - Nq;
    }
    __host__ __device__ __forceinline__ bool sees(int p, int k) const { return k <= p && (k > p - window || k < sinks); }
};

// Division of numbers below 2^31 by a divisor that a call has once: with s = ceil(log2 d) and m = 2^32 (2^s - d) / d
// rounded down, plus 1, the quotient is (n m / 2^32 + n) / 2^s, both rounded down (Granlund and Montgomery,
// Division by Invariant Integers using Multiplication, 1994).  The processors have no division: one takes 30
// instructions or so.
struct Div {
    uint32_t d, m, s;
    explicit Div(uint32_t by = 1) : d(by), s(0) {
        while ((1ull << s) < d) ++s;
        m = (uint32_t)((((1ull << s) - d) << 32) / d + 1);
    }
    __host__ __device__ __forceinline__ int of(int n) const {
#ifdef __CUDA_ARCH__
        return (int)((__umulhi(m, (uint32_t)n) + (uint32_t)n) >> s);
#else
        return (int)((((uint64_t)m * (uint32_t)n >> 32) + (uint32_t)n) >> s);
#endif
    }
    __host__ __device__ __forceinline__ int rest(int n) const { return n - of(n) * (int)d; }
};

// Bits below n: none for n <= 0, all for n >= 32.
__host__ __device__ __forceinline__ uint32_t bits_below(int n) {
#ifdef __CUDA_ARCH__
    uint32_t above;
    asm("shl.b32 %0, 0xffffffff, %1;" : "=r"(above) : "r"(max(n, 0)));     // (0 from 32 on)
    return ~above;
#else
    return n <= 0 ? 0u : n >= 32 ? ~0u : ~(~0u << n);
#endif
}
// Bit i: the query at position p attends key k0 + i.
__host__ __device__ __forceinline__ uint32_t keys_of(const Band &w, int p, int k0) {
    return bits_below(p + 1 - k0) & (~bits_below(p + 1 - w.window - k0) | bits_below(w.sinks - k0));
}
// Bit i: a query at one of the positions lo to hi attends key k0 + i.
__host__ __device__ __forceinline__ uint32_t keys_between(const Band &w, int lo, int hi, int k0) {
    return lo > hi ? 0u : bits_below(hi + 1 - k0) & (~bits_below(lo + 1 - w.window - k0) | bits_below(w.sinks - k0));
}
// Bit i: the query at position p0 + i, if that is below `end`, attends key k.
__host__ __device__ __forceinline__ uint32_t queries_of(const Band &w, int k, int p0, int end) {
    return bits_below((k < w.sinks ? end : least(end, k + w.window)) - p0) & ~bits_below(k - p0);
}

// The T-key tiles that hold the keys of the queries at positions lo to hi: first those of
// the sinks, then the windows', from the oldest key in one of them on, so that they are as few as can
// be.
template <int T>
struct KeyWalk {
    int sinks, oldest, n;    // tiles of the sinks, first key behind them, tiles of the walk
    __host__ __device__ __forceinline__ KeyWalk() {}
    __host__ __device__ __forceinline__ KeyWalk(const Band &w, int lo, int hi) : sinks(0), oldest(0), n(0) {
        if (lo > hi) return;
        oldest = most(0, lo - w.window + 1);
        sinks = (w.sinks + T - 1) / T;
        n = sinks + (hi - oldest) / T + 1;
        if (oldest > w.sinks && n < hi / T + 1) return;
        sinks = oldest = 0;          // from the first key on: no more tiles than in two parts
        n = hi / T + 1;
    }
    __host__ __device__ __forceinline__ int key(int i) const { return i < sinks ? i * T : oldest + (i - sinks) * T; }
    // By which tile i's keys are attended: a tile of the sinks by them alone (its other keys come again
    // with the windows).
    __host__ __device__ __forceinline__ Band band(Band w, int i) const {
        if (i < sinks) w.window = 0;
        return w;
    }
};

// The same in whole pages: those that hold sinks, then the others of the windows.
template <int T>
struct BandWalk {
    int sinks, gap, n;       // tiles of the sinks, tiles between them and the windows', tiles of the walk
    __host__ __device__ __forceinline__ BandWalk() {}
    __host__ __device__ __forceinline__ BandWalk(const Band &w, int lo, int hi) : sinks(0), gap(0), n(0) {
        if (lo > hi) return;
        const int oldest = most(0, lo - w.window + 1) / T;
        sinks = least((w.sinks + T - 1) / T, oldest);
        gap = oldest - sinks;
        n = hi / T + 1 - gap;
    }
    __host__ __device__ __forceinline__ int tile(int i) const { return i < sinks ? i : i + gap; }
};

struct CrossArgs {
    int B, Hq, Hkv, Nq, Nk;
    fibatt_dtype dtype;
    float scale;
    KeySet keys;
    bool banded;             // the queries attend by `band`, of the keys below keys.len
    Band band;
    fibatt_heads Q, K, V, O, dO, dQ, dK, dV;
    float *LSE;              // [B, Hq, Nq]
    float2 *stats;           // backward's workspace: (LSE log2 e, D) of every query row, and more in 16 bits
    cudaStream_t stream;
};

// Streaming multiprocessors of the current device.
int sm_count();
// The current device, -1 if it cannot be told.
inline int current_device() {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess ? dev : -1;
}

// How many clusters of `c` CTAs of kernel K the current device holds at once (-1:
// none).  More than eight CTAs have to be asked for, on each device.
template <auto K>
int clusters_held(int c, unsigned threads, size_t smem) {
    if (c > 8 && cudaFuncSetAttribute(K, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
        (void)cudaGetLastError();
        return -1;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)c;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)c);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int held = 0;
    if (cudaOccupancyMaxActiveClusters(&held, K, &cfg) != cudaSuccess) (void)cudaGetLastError();
    return held > 0 ? held : -1;
}

// CTAs of a cluster for `units` units that walk over `walk` tiles each: until
// `places` CTAs, which the GPU holds at once, are taken, as long as each keeps a tile.
inline int cluster_for(int64_t units, int64_t walk, int64_t places, int most = 8) {
    int c = 1;
    while (c < most && units * c * 2 <= places && walk >= 2 * c) c *= 2;
    return c;
}
// A backward pass has two kinds of unit, whose walks may differ much (a few queries on
// many keys: hundreds of units of one tile, and one of hundreds).  They go in one
// launch, or in one of each kind with clusters of its own where the longest walk, or
// all tiles over the places, is estimated to be over sooner.  In tiles: `unit`, what a
// unit costs beside its walk, and `start`, another launch.
struct Launches {
    bool two;
    int c, c_query, c_key;
    Launches(int64_t query_units, int64_t query_walk, int64_t key_units, int64_t key_walk, int64_t places, int unit,
             int start, int most = 8) {
        const auto time = [&](int64_t units, int64_t walk, int c) {
            return std::max((walk + c - 1) / c + unit, units * (walk + unit) / places);
        };
        c = cluster_for(query_units + key_units, std::max(query_walk, key_walk), places, most);
        c_query = cluster_for(query_units, query_walk, places, most);
        c_key = cluster_for(key_units, key_walk, places, most);
        const int64_t longest = (std::max(query_walk, key_walk) + c - 1) / c + unit,
                      all = query_units * (query_walk + unit) + key_units * (key_walk + unit),
                      one = std::max(longest, all / places);
        two = time(query_units, query_walk, c_query) + time(key_units, key_walk, c_key) + start < one;
    }
};

// Launch `kern` on clusters of `c` CTAs along x, programmatic dependent when
// the library launches that way.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kern)(KArgs...), unsigned grid, unsigned c, unsigned threads, size_t smem,
                            cudaStream_t stream, Args &&...args) {
    const ProfileLaunch prof(stream, reinterpret_cast<const void *>(kern));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = c;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

// Before the first launch of kernel K on a device: its shared memory, and a
// check of its registers (0: none).  A kernel that shares its registers out
// anew (setmaxnreg) is written for the number it is launched with; shares that
// do not add up would wait for ever.
template <auto K>
cudaError_t prepare_kernel(size_t smem, int regs) {
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    cudaFuncAttributes at;
    if ((e = cudaFuncGetAttributes(&at, K)) != cudaSuccess) return e;
    if (regs && at.numRegs != regs) return cudaErrorInvalidKernelImage;
    e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_release);
    return e;
}

// ---- launchers (return the CUDA launch status) -----------------------------
cudaError_t launch_cross_fwd_f32(const CrossArgs &a);
cudaError_t launch_cross_bwd_f32(const CrossArgs &a);
cudaError_t launch_cross_fwd_mma(const CrossArgs &a);   // bf16
cudaError_t launch_cross_bwd_mma(const CrossArgs &a);   // bf16
size_t cross_bwd_mma_workspace(int B, int Hq, int Nq);
size_t window_bwd_mma_workspace(int B, int Hq, int Hkv, int Nq, int Nk, int window, int sinks);
bool cross_rows_takes(const CrossArgs &a);               // few enough query rows for the next
cudaError_t launch_cross_rows(const CrossArgs &a);

struct QkNormArgs {
    int B, N, Hq, Hk, Hv;
    fibatt_dtype dtype;
    const void *X;
    int64_t x_sb, x_sn;      // elements
    const void *wq, *wk;     // [64] in the I/O type, or null: that part is not normalised
    float eps;
    int rot;                 // leading dims rotated (0: none)
    int interleaved;
    const float *cos, *sin;  // [P, rot / 2]
    int P;
    const int32_t *pos;      // [B, N] with batch stride pos_sb (0: one row for all), or null: 0..N-1
    int64_t pos_sb;
    void *Q, *K, *V;         // [B, H, N, 64]
    const void *dQ, *dK, *dV;
    void *dX;
    int64_t dx_sb, dx_sn;
    void *dwq, *dwk;         // [64] in the I/O type
    float *ws;
    cudaStream_t stream;
};
size_t qk_norm_bwd_workspace();
cudaError_t launch_qk_norm_fwd(const QkNormArgs &a);
cudaError_t launch_qk_norm_bwd(const QkNormArgs &a);

}  // namespace fibatt
