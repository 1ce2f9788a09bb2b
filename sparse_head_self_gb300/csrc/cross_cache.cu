// A paged cache of keys and values in 8 bits: storing tokens, loading them, and the
// attention of a sequence's newest tokens to what it holds.
//
// A page has 64 tokens of every key/value head.  A head's part of it is 8 KB in one
// piece, its keys token by token and its values dim by dim, each 4096 e4m3 bytes
// with a scale of their own: a power of two, so that dividing by it and
// raising it later are exact (but for what falls below the type's smallest step).
#include <algorithm>

#include "cluster.cuh"
#include "cross_cache.h"
#include "cross_tiles.cuh"

namespace fibatt {
namespace {

constexpr float kNegInf = -__builtin_inff();
constexpr unsigned kErrPage = 16u;       // a token or key whose page the table or the cache has not

// ---- 8-bit values ------------------------------------------------------------------
// Two values rounded to nearest, ties to even, beyond the largest to the largest; lo in the low byte.
__device__ __forceinline__ uint32_t to_e4m3(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// The values of the two low bytes, exactly, as two halves.
__device__ __forceinline__ uint32_t halves_of(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}
__device__ __forceinline__ float2 floats_of(uint32_t two) {
    const uint32_t h = halves_of(two);
    float2 f;
    asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.f32.f16 %0, lo; cvt.f32.f16 %1, hi; }" : "=f"(f.x), "=f"(f.y) : "r"(h));
    return f;
}

// 2^e, e in [-126, 127]
__device__ __forceinline__ float two_to(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ int exponent_of(float x) { return (__float_as_int(x) >> 23 & 255) - 127; }
// The exponent of the smallest power of two whose 448th multiple (448 = 1.75 2^8) reaches x >= 0; -100 at least.
__device__ __forceinline__ int scale_exponent(float x) {
    const int e = exponent_of(x) - 8 + ((__float_as_int(x) & 0x7fffff) > 0x600000);
    return max(e, -100);
}
// A page's scale as the store wrote it: a power of two.  (Whatever else stands there is read as one.)
__device__ __forceinline__ int stored_exponent(float s) { return max(-100, min(exponent_of(s), 120)); }

// ---- storing and loading -----------------------------------------------------------
constexpr int kStoreThreads = 128;       // two a token, 32 dims each
constexpr int kLine = 80;                // bytes between the dims' lines of a page's values in shared memory

__device__ __forceinline__ void load32(const float *p, float (&x)[32]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float4 t = __ldg(reinterpret_cast<const float4 *>(p) + i);
        x[4 * i] = t.x, x[4 * i + 1] = t.y, x[4 * i + 2] = t.z, x[4 * i + 3] = t.w;
    }
}
__device__ __forceinline__ void load32(const __nv_bfloat16 *p, float (&x)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 t = __ldg(reinterpret_cast<const uint4 *>(p) + i);
        const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) x[8 * i + 2 * k] = bf16_lo(w[k]), x[8 * i + 2 * k + 1] = bf16_hi(w[k]);
    }
}
__device__ __forceinline__ void store32(float *p, const float (&x)[32]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) reinterpret_cast<float4 *>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
__device__ __forceinline__ void store32(__nv_bfloat16 *p, const float (&x)[32]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        reinterpret_cast<uint4 *>(p)[i] = make_uint4(pack_bf16x2(x[8 * i], x[8 * i + 1]), pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                                                     pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
}

// Four values times f, rounded again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
    const float2 a = floats_of(w & 0xffff), b = floats_of(w >> 16);
    return to_e4m3(a.x * f, a.y * f) | to_e4m3(b.x * f, b.y * f) << 16;
}

// Tokens into a page's keys or values.  A page that the call begins gets the
// scale that its tokens here need; one that held tokens before keeps its scale, or
// has it raised and those tokens rounded again.
template <typename T>
__global__ void __launch_bounds__(kStoreThreads) cache_store_kernel(const __grid_constant__ CacheArgs a) {
    __shared__ float tops[kStoreThreads / 32];
    __shared__ __align__(16) uint8_t lines[kHeadDim * kLine];
    grid_dep_wait();
    grid_dep_launch();
    const Spot s(a, blockIdx.x);
    if (s.lost && threadIdx.x == 0) atomicOr(&g_device_error, kErrPage);
    if (s.page < 0) return;
    const int t = threadIdx.x >> 1, half = threadIdx.x & 1;
    const bool mine = t >= s.lo && t < s.hi;
    float x[32], top = 0.f;
    if (mine) {
        const Rows<const T> rows{static_cast<const T *>(s.kind ? a.V.ptr : a.K.ptr), s.kind ? a.V.stride_b : a.K.stride_b,
                                 s.kind ? a.V.stride_h : a.K.stride_h, s.kind ? a.V.stride_n : a.K.stride_n};
        load32(rows.row(s.b, s.hk, s.token + t) + 32 * half, x);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float m = fabsf(x[i]);
            if (m < __builtin_inff()) top = fmaxf(top, m);
        }
    }
#pragma unroll
    for (int m = 16; m; m >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, m));
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
    float *scale = a.scales + 2 * a.place(s.page, s.hk) + s.kind;
    const int had = s.lo > 0 ? stored_exponent(*scale) : -100;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kStoreThreads / 32; ++w) top = fmaxf(top, tops[w]);
    const int need = scale_exponent(top), e = max(had, need);
    const bool raised = s.lo > 0 && e > had;
    const float f = two_to(-e), again = raised ? two_to(max(had - e, -126)) : 1.f;
    if (threadIdx.x == 0 && (s.lo == 0 || raised)) *scale = two_to(e);
    uint8_t *page = a.data + (a.place(s.page, s.hk) * 2 + s.kind) * kPageBytes;
    uint32_t y[8];
    if (mine) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] = to_e4m3(x[4 * i] * f, x[4 * i + 1] * f) | to_e4m3(x[4 * i + 2] * f, x[4 * i + 3] * f) << 16;
    }
    if (s.kind == 0) {
        uint4 *row = reinterpret_cast<uint4 *>(page + t * kHeadDim + 32 * half);
        if (!mine && raised && t < s.lo) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 w = row[i];
                row[i] = make_uint4(rescale4(w.x, again), rescale4(w.y, again), rescale4(w.z, again), rescale4(w.w, again));
            }
        }
        if (mine) {
            row[0] = make_uint4(y[0], y[1], y[2], y[3]);
            row[1] = make_uint4(y[4], y[5], y[6], y[7]);
        }
        return;
    }
    if (mine) {
#pragma unroll
        for (int i = 0; i < 32; ++i) lines[(32 * half + i) * kLine + t] = (uint8_t)(y[i >> 2] >> (8 * (i & 3)));
    }
    __syncthreads();
    // a dim's 64 tokens: four pieces of 16
    for (int i = threadIdx.x; i < kHeadDim * 4; i += kStoreThreads) {
        const int dim = i >> 2, t0 = 16 * (i & 3);
        uint8_t *to = page + dim * kPage + t0;
        const uint8_t *from = lines + dim * kLine + t0;
        if (t0 >= s.lo && t0 + 16 <= s.hi) {
            *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(from);
            continue;
        }
        for (int k = 0; k < 16; ++k) {
            if (t0 + k >= s.lo && t0 + k < s.hi) to[k] = from[k];
            else if (raised && t0 + k < s.lo) to[k] = (uint8_t)rescale4(to[k], again);
        }
    }
}

// Tokens from a page's keys or values, as the values they stand for; zeros from the sequence's count on.
template <typename T>
__global__ void __launch_bounds__(kStoreThreads) cache_load_kernel(const __grid_constant__ CacheArgs a) {
    __shared__ __align__(16) uint8_t lines[kHeadDim * kLine];
    grid_dep_wait();
    grid_dep_launch();
    const Spot s(a, blockIdx.x);
    if (s.lost && threadIdx.x == 0) atomicOr(&g_device_error, kErrPage);
    const int t = threadIdx.x >> 1, half = threadIdx.x & 1, n = s.token + t;
    float x[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = 0.f;
    if (s.page >= 0) {
        const float f = two_to(stored_exponent(__ldg(a.scales + 2 * a.place(s.page, s.hk) + s.kind)));
        const uint8_t *page = a.data + (a.place(s.page, s.hk) * 2 + s.kind) * kPageBytes;
        uint32_t y[8] = {};
        if (s.kind == 0) {
            const uint4 *row = reinterpret_cast<const uint4 *>(page + t * kHeadDim + 32 * half);
            const uint4 u = row[0], v = row[1];
            y[0] = u.x, y[1] = u.y, y[2] = u.z, y[3] = u.w, y[4] = v.x, y[5] = v.y, y[6] = v.z, y[7] = v.w;
        } else {
            for (int i = threadIdx.x; i < kHeadDim * 4; i += kStoreThreads)
                *reinterpret_cast<uint4 *>(lines + (i >> 2) * kLine + 16 * (i & 3)) = reinterpret_cast<const uint4 *>(page)[i];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i >> 2] |= (uint32_t)lines[(32 * half + i) * kLine + t] << (8 * (i & 3));
        }
        if (t < s.hi) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 v = floats_of(y[i >> 1] >> (16 * (i & 1)) & 0xffff);
                x[2 * i] = v.x * f, x[2 * i + 1] = v.y * f;
            }
        }
    }
    if (n < 0 || n >= a.N) return;
    const Rows<T> rows{static_cast<T *>(s.kind ? a.V.ptr : a.K.ptr), s.kind ? a.V.stride_b : a.K.stride_b,
                       s.kind ? a.V.stride_h : a.K.stride_h, s.kind ? a.V.stride_n : a.K.stride_n};
    store32(rows.row(s.b, s.hk, n) + 32 * half, x);
}

// ---- attention ---------------------------------------------------------------------
// Up to 16 rows (query heads of a key head by tokens) read a sequence's pages once, and
// the time is that of reading them.  A cluster of CTAs takes such a block of rows, its
// warps every so many-th page each: a warp has its own ring of stages, which a bulk copy
// of 8 KB fills, and keeps the running maximum, sum and weighted values of its own
// keys until the end, when they are joined in shared memory and over the cluster,
// in a fixed order.
//
// Scores and weighted values are warp-wide products of halves: an e4m3 value is
// one exactly, a bf16 query too, after a power of two has moved its row's largest to
// [2^8, 2^9) (32-bit queries and weights are two halves, 22 bits), a 16-bit call's weight is rounded to
// 11 bits.  The layout of a page makes every operand's fragment a piece of 16 bytes in
// it: lane (g, c) of a product has keys 16 (g / 2) + 2 t + (g mod 2) of tile t with
// dims 16 c to 16 c + 15, four at a time in the order in which the rows have them;
// its scores are then those of keys 16 c to 16 c + 15, and its 16 bytes of a dim's line of values
// are those same keys.  No shuffles, and no conflicts in shared memory.
constexpr int kWarps = 4, kStages = 3;
constexpr int kThreads = 32 * kWarps;
constexpr int kBlocks = 2;                           // CTAs a SM
constexpr size_t kSmem = 128 + (size_t)kWarps * kStages * 2 * kPageBytes;
constexpr float kLift = 7.f;                         // weights are held times 2^7, ...
constexpr float kRaise = 15.f;                       // and stay below 2^15: within a half's range, far from its smallest step

struct AttendArgs {
    CacheArgs c;
    Band band;
    int G, rows, blocks;                             // heads of a group, rows of a key head, blocks of rows
    float scale_log2;
    int units;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t h) {
    float2 f;
    asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.f32.f16 %0, lo; cvt.f32.f16 %1, hi; }" : "=f"(f.x), "=f"(f.y) : "r"(h));
    return f;
}
__device__ __forceinline__ void store2(__nv_bfloat16 *p, float2 v) { *reinterpret_cast<uint32_t *>(p) = pack_bf16x2(v.x, v.y); }
__device__ __forceinline__ void store2(float *p, float2 v) { *reinterpret_cast<float2 *>(p) = v; }
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float (&x)[4]) {
    const uint2 t = __ldg(reinterpret_cast<const uint2 *>(p));
    x[0] = bf16_lo(t.x), x[1] = bf16_hi(t.x), x[2] = bf16_lo(t.y), x[3] = bf16_hi(t.y);
}
__device__ __forceinline__ void load4(const float *p, float (&x)[4]) {
    const float4 t = __ldg(reinterpret_cast<const float4 *>(p));
    x[0] = t.x, x[1] = t.y, x[2] = t.z, x[3] = t.w;
}
// Bytes whose bit is set.
__device__ __forceinline__ uint32_t bytes_of(uint32_t four) {
    return ((four & 1) | (four & 2) << 7 | (four & 4) << 14 | (four & 8) << 21) * 0xffu;
}

// HALVES: 1 (at most 8 rows; the products' lower rows are not looked at) or 2.
template <typename T, int HALVES>
__global__ void __launch_bounds__(kThreads, kBlocks)
cache_fwd_kernel(const __grid_constant__ AttendArgs a, Rows<const T> Q, Rows<T> O) {
    constexpr int R = 8 * HALVES, kParts = sizeof(T) == 4 ? 2 : 1;     // halves of an operand
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((128 - (smem_u32(smem_raw) & 127)) & 127);
    __shared__ uint64_t full[kWarps][kStages];
    __shared__ float2 scale_of[kWarps][kStages];      // of a stage's keys and values; 0: no page
    __shared__ int abort_flag;
    __shared__ float sm[kWarps][R], sl[kWarps][R];
    __shared__ float cm[R], cl[R];                    // the CTA's, read by the cluster
    __shared__ float2 co[R][32];
    static_assert(kWarps * R * 32 * sizeof(float2) <= kSmem - 128, "the warps' sums fit");
    volatile int *abort = &abort_flag;
    const int warp = warp_number(), lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int C = (int)cluster_size(), rank = (int)cluster_rank();
    if (threadIdx.x < kWarps * kStages) mbar_init(&full[0][0] + threadIdx.x, 1);
    if (threadIdx.x == 0) abort_flag = 0;
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();

    const int unit = blockIdx.x / C, rb = unit % a.blocks, hk = unit / a.blocks % a.c.Hkv, b = unit / a.blocks / a.c.Hkv;
    const int r0 = 16 * rb, rows = min(R, a.rows - r0);
    const int start = a.c.first(b), n = a.c.tokens(b), end = a.c.table_len * kPage;
    // positions of the block's first and last queries that attend keys
    const int first = max(0, start + r0 / a.G), last = min(end, start + min(n, (r0 + rows - 1) / a.G + 1)) - 1;
    if (start + n > end && threadIdx.x == 0) atomicOr(&g_device_error, kErrPage);
    const BandWalk<kPage> walk(a.band, first, last);
    const int at = rank * kWarps + warp, step = C * kWarps, mine = max(0, (walk.n - at + step - 1) / step);

    // row r of the block: query head g(r) of the group at token n(r), tokens apart
    const auto position = [&](int r) {
        const int p = start + (r0 + r) / a.G;
        return r < rows && p <= last ? p : -1;
    };
    // ---- copies: this warp's pages in turn
    uint8_t *stages = ring + (size_t)warp * kStages * 2 * kPageBytes;
    int pages = -1;                                  // of page numbers 32 and 32 on, one a lane, with its scales
    float2 scales = make_float2(0.f, 0.f);
    const auto issue = [&](int k) {
        if ((k & 31) == 0) {
            pages = -1;
            scales = make_float2(0.f, 0.f);
            if (k + lane < mine) {
                pages = a.c.page(b, walk.tile(at + (k + lane) * step));
                if (pages >= 0) scales = __ldg(reinterpret_cast<const float2 *>(a.c.scales) + a.c.place(pages, hk));
                else atomicOr(&g_device_error, kErrPage);
            }
        }
        const int page = __shfl_sync(kFullMask, pages, k & 31), s = k % kStages;
        const float sk = __shfl_sync(kFullMask, scales.x, k & 31), sv = __shfl_sync(kFullMask, scales.y, k & 31);
        if (lane == 0) {
            scale_of[warp][s] = page < 0 ? make_float2(0.f, 0.f) : make_float2(two_to(stored_exponent(sk)), two_to(stored_exponent(sv)));
            if (page < 0) {
                mbar_arrive(&full[warp][s]);
            } else {
                mbar_expect_tx(&full[warp][s], 2 * kPageBytes);
                bulk_g2s(stages + (size_t)s * 2 * kPageBytes, a.c.data + a.c.place(page, hk) * 2 * kPageBytes, 2 * kPageBytes,
                         &full[warp][s]);
            }
        }
        __syncwarp();
    };
    int issued = 0;
    for (; issued < min(mine, kStages); ++issued) issue(issued);

    // ---- the rows as operands of four steps of 16 dims, and what their scores are multiplied with
    uint32_t q[kParts][4][4];
    float factor[HALVES], m[HALVES], l[HALVES], o[8][4];
    int p[HALVES];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float x[16];
        float top = 0.f;
        const int r = g + 8 * i;
        if (i < HALVES && r < rows) {
            const T *src = Q.row(b, hk * a.G + (r0 + r) % a.G, (r0 + r) / a.G) + 16 * c;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float y[4];
                load4(src + 4 * j, y);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    x[4 * j + k] = y[k];
                    top = fmaxf(top, fabsf(y[k]));
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = 0.f;
        }
        top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
        const int e = max(-100, min(exponent_of(top), 120)) - 8;
        const float f = two_to(-e);
        if (i < HALVES) {
            factor[i] = a.scale_log2 * two_to(e);
            m[i] = kNegInf;
            l[i] = 0.f;
            p[i] = position(r);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float u = x[4 * j + 2 * k] * f, v = x[4 * j + 2 * k + 1] * f;
                const uint32_t hi = pack_f16x2(u, v);
                q[0][j][i + 2 * k] = hi;
                if (kParts == 2) {
                    const float2 h = unpack_f16x2(hi);
                    q[kParts - 1][j][i + 2 * k] = pack_f16x2(u - h.x, v - h.y);
                }
            }
    }
#pragma unroll
    for (int d = 0; d < 8; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d][i] = 0.f;

    int done = 0;
    for (; done < mine; ++done) {
        const int s = done % kStages;
        if (!pipe_wait(&full[warp][s], (done / kStages) & 1, abort)) break;
        __syncwarp();
        const float2 scale = scale_of[warp][s];
        if (scale.x > 0.f) {
            const uint8_t *keys = stages + (size_t)s * 2 * kPageBytes, *values = keys + kPageBytes;
            const int k0 = walk.tile(at + done * step) * kPage, k1 = k0 + kPage - 1;
            const bool whole = k1 <= first && (k0 > last - a.band.window || k1 < a.band.sinks);
            float x[8][4];
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const uint4 w = *reinterpret_cast<const uint4 *>(keys + (16 * (g >> 1) + 2 * t + (g & 1)) * kHeadDim + 16 * c);
                const uint32_t four[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) x[t][i] = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t b0 = halves_of(four[j] & 0xffff), b1 = halves_of(four[j] >> 16);
                    if (kParts == 2) mma_f16(x[t], q[kParts - 1][j], b0, b1);
                    mma_f16(x[t], q[0][j], b0, b1);
                }
            }
            uint32_t live = 0xffffu;              // this lane's keys that a row of the block attends
            uint32_t w[kParts][4][4];             // the weights as operands of four steps of 16 keys
#pragma unroll
            for (int i = 0; i < HALVES; ++i) {
                const float f = factor[i] * scale.x;
                uint32_t seen = 0xffffu;
                if (!whole) {
                    seen = keys_of(a.band, p[i], k0 + 16 * c);
                    live = keys_between(a.band, first, last, k0 + 16 * c);
                }
                float top = kNegInf;
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float &y = x[t][2 * i + k];
                        y = (seen >> (2 * t + k)) & 1 ? y * f : kNegInf;
                        top = fmaxf(top, y);
                    }
                top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
                top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
                if (__any_sync(kFullMask, top > m[i] + kRaise)) {      // m: 2^7 below the maximum when it was set
                    const float next = fmaxf(top - kLift, m[i]), keep = next == kNegInf ? 1.f : fast_exp2(m[i] - next);
                    m[i] = next;
                    l[i] *= keep;
#pragma unroll
                    for (int d = 0; d < 8; ++d) {
                        o[d][2 * i] *= keep;
                        o[d][2 * i + 1] *= keep;
                    }
                }
                const float base = m[i] == kNegInf ? 0.f : m[i];
                float sum[2] = {0.f, 0.f};
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const float u = fast_exp2(x[t][2 * i] - base), v = fast_exp2(x[t][2 * i + 1] - base);
                    sum[t & 1] += u + v;
                    const uint32_t hi = pack_f16x2(u, v);
                    w[0][t >> 1][i + 2 * (t & 1)] = hi;
                    if (kParts == 2) {
                        const float2 h = unpack_f16x2(hi);
                        w[kParts - 1][t >> 1][i + 2 * (t & 1)] = pack_f16x2(u - h.x, v - h.y);
                    }
                }
                l[i] += sum[0] + sum[1];
            }
            if (HALVES == 1) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int k = 0; k < kParts; ++k) w[k][j][1] = w[k][j][3] = 0u;
            }
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                const uint4 v = *reinterpret_cast<const uint4 *>(values + (8 * d + g) * kPage + 16 * c);
                uint32_t four[4] = {v.x, v.y, v.z, v.w};
                if (!whole) {                     // a weight of 0 meets no NaN
#pragma unroll
                    for (int j = 0; j < 4; ++j) four[j] &= bytes_of(live >> (4 * j) & 15);
                }
                // a page's sum by itself, and into the running one by an addition that rounds
                float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t b0 = halves_of(four[j] & 0xffff), b1 = halves_of(four[j] >> 16);
                    if (kParts == 2) mma_f16(part, w[kParts - 1][j], b0, b1);
                    mma_f16(part, w[0][j], b0, b1);
                }
#pragma unroll
                for (int i = 0; i < 2 * HALVES; ++i) o[d][i] = fmaf(part[i], scale.y, o[d][i]);
            }
        }
        __syncwarp();
        if (issued < mine) issue(issued++);
    }
    if (lane == 0)   // leave no copy in flight
        for (int i = done; i < issued; ++i) mbar_drain(&full[warp][i % kStages], (i / kStages) & 1);
    __syncthreads();      // the ring is free: it takes the warps' sums

    float2(*so)[R][32] = reinterpret_cast<float2(*)[R][32]>(ring);
#pragma unroll
    for (int i = 0; i < HALVES; ++i) {
        l[i] += __shfl_xor_sync(kFullMask, l[i], 1);
        l[i] += __shfl_xor_sync(kFullMask, l[i], 2);
        const int r = g + 8 * i;
#pragma unroll
        for (int d = 0; d < 8; ++d) so[warp][r][4 * d + c] = make_float2(o[d][2 * i], o[d][2 * i + 1]);
        if (c == 0) {
            sm[warp][r] = m[i];
            sl[warp][r] = l[i];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * 32; i += kThreads) {
        const int r = i >> 5, d = i & 31;
        float top = kNegInf;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w][r]);
        const float base = top == kNegInf ? 0.f : top;
        float sum = 0.f;
        float2 x = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = fast_exp2(sm[w][r] - base);
            sum = fmaf(f, sl[w][r], sum);
            x = fma2(make_float2(f, f), so[w][r][d], x);
        }
        co[r][d] = x;
        if (d == 0) {
            cm[r] = top;
            cl[r] = sum;
        }
    }
    cluster_sync();
    // row r is finished by CTA r mod C
    for (int i = threadIdx.x; i < rows * 32; i += kThreads) {
        const int r = i >> 5, d = i & 31;
        if (r % C != rank) continue;
        float top = kNegInf;
        for (int k = 0; k < C; ++k) top = fmaxf(top, ld_cluster(cluster_addr(cm + r, k)));
        const float base = top == kNegInf ? 0.f : top;
        float sum = 0.f;
        float2 x = make_float2(0.f, 0.f);
        for (int k = 0; k < C; ++k) {
            const float f = fast_exp2(ld_cluster(cluster_addr(cm + r, k)) - base);
            sum = fmaf(f, ld_cluster(cluster_addr(cl + r, k)), sum);
            x = fma2(make_float2(f, f), ld_cluster2(cluster_addr(&co[r][d], k)), x);
        }
        const int h = hk * a.G + (r0 + r) % a.G, at_n = (r0 + r) / a.G;
        const bool none = position(r) < 0 || sum == 0.f;
        const float inv = none ? 0.f : 1.f / sum;
        store2(O.row(b, h, at_n) + 2 * d, none ? make_float2(0.f, 0.f) : make_float2(x.x * inv, x.y * inv));
        if (d == 0) a.c.LSE[((int64_t)b * a.c.Hq + h) * a.c.N + at_n] = none ? kNegInf : (top + log2f(sum)) * kLn2;
    }
    cluster_sync();   // the others may still read this CTA's part
}

template <typename T, int HALVES>
cudaError_t attend(const AttendArgs &f) {
    const cudaError_t e = prepare_kernel<cache_fwd_kernel<T, HALVES>>(kSmem, 0);
    if (e != cudaSuccess) return e;
    // CTAs of a cluster: as many as the GPU holds at once, as long as a warp keeps a page
    const int64_t keys = std::min<int64_t>((int64_t)f.c.table_len * kPage, (int64_t)f.band.window + f.band.sinks + f.c.N);
    int c = 1;
    while (c < 8 && (int64_t)f.units * c * 2 <= kBlocks * sm_count() && keys > (int64_t)c * kWarps * kPage) c *= 2;
    return launch_clusters(cache_fwd_kernel<T, HALVES>, (unsigned)(f.units * c), c, kThreads, kSmem, f.c.stream, f,
                           rows_of<const T>(f.c.Q), rows_of<T>(f.c.O));
}

}  // namespace

cudaError_t launch_cache_store(const CacheArgs &a) {
    const int64_t blocks = 2 * (int64_t)a.B * a.Hkv * pages_of(a.N);
    return a.dtype == FIBATT_F32 ? launch_clusters(cache_store_kernel<float>, (unsigned)blocks, 1, kStoreThreads, 0, a.stream, a)
                                 : launch_clusters(cache_store_kernel<__nv_bfloat16>, (unsigned)blocks, 1, kStoreThreads, 0, a.stream, a);
}

cudaError_t launch_cache_load(const CacheArgs &a) {
    const int64_t blocks = 2 * (int64_t)a.B * a.Hkv * pages_of(a.N);
    return a.dtype == FIBATT_F32 ? launch_clusters(cache_load_kernel<float>, (unsigned)blocks, 1, kStoreThreads, 0, a.stream, a)
                                 : launch_clusters(cache_load_kernel<__nv_bfloat16>, (unsigned)blocks, 1, kStoreThreads, 0, a.stream, a);
}

cudaError_t launch_cache_fwd(const CacheArgs &a) {
    AttendArgs f;
    f.c = a;
    f.band = Band{nullptr, a.N, a.table_len * kPage, a.window, a.sinks};
    f.G = a.Hq / a.Hkv;
    f.rows = f.G * a.N;
    f.blocks = (f.rows + 15) / 16;
    f.scale_log2 = a.scale * kLog2e;
    f.units = a.B * a.Hkv * f.blocks;
    if (a.dtype == FIBATT_F32) return f.rows <= 8 ? attend<float, 1>(f) : attend<float, 2>(f);
    return f.rows <= 8 ? attend<__nv_bfloat16, 1>(f) : attend<__nv_bfloat16, 2>(f);
}

FIBATT_DEFINE_ERROR_READER(read_error_cross_cache, "cross_cache.cu")

}  // namespace fibatt
