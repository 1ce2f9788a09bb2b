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

struct CrossArgs {
    int B, Hq, Hkv, Nq, Nk;
    fibatt_dtype dtype;
    float scale;
    KeySet keys;
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
