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
constexpr int kLargestScale = 120;
__device__ __forceinline__ int stored_exponent(float s) { return max(-100, min(exponent_of(s), kLargestScale)); }
// The largest multiple of the largest scale that 16 and 32 bits hold.
constexpr float kLargestValue = 0x1.ep127f;

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
// has it raised and those tokens rounded again.  One block for each page, head and kind, since the
// scale is of them all: it reads its tokens once, holds them in registers, finds the largest,
// and writes the bytes; values go through shared memory, to leave dim by dim in pieces of 16 tokens.
// Far from the bytes' time: a block has a chain of reads (start, table, scale), then one round of loads in flight, and
// nothing of another page asked for meanwhile.  2 x 16385 tokens of 4 heads 15.1 us (3.3 TB/s, half of a copy's
// rate), 8 x 1569 7.0 (1664 blocks on 9 places a SM, 42% of issue slots), 64 x 1 3.8.  fp32: 22.3 us (3.8 TB/s), 11.8, 3.8.
template <typename T>
__global__ void __launch_bounds__(kStoreThreads) cache_store_kernel(const __grid_constant__ CacheArgs a) {
    __shared__ float tops[kStoreThreads / 32];
    __shared__ __align__(16) uint8_t lines[kHeadDim * kLine];
    grid_dep_wait();
    grid_dep_launch();
    const Spot s(a, blockIdx.x);
    if (s.lost && threadIdx.x == 0) atomicOr(&g_device_error, kErrPage);
    if (s.page < 0 || !FIBATT_CHECKED(s.b < a.B && s.page < a.pages && s.lo >= 0 && s.hi <= kPage)) return;
    const int t = threadIdx.x >> 1, half = threadIdx.x & 1;
    const bool mine = t >= s.lo && t < s.hi && FIBATT_CHECKED(s.token + t >= 0 && s.token + t < a.N);
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
    if (mine && e == kLargestScale) {     // finite values come back as such
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (fabsf(x[i]) < __builtin_inff()) x[i] = fmaxf(-kLargestValue, fminf(x[i], kLargestValue));
    }
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
// The store's blocks the other way round, and held up as they are: 13.4 us, 6.4, 2.8; fp32 24.5, 10.5, 2.8.
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
    if (n < 0 || n >= a.N || !FIBATT_CHECKED(s.b < a.B && s.page < a.pages)) return;
    const Rows<T> rows{static_cast<T *>(s.kind ? a.V.ptr : a.K.ptr), s.kind ? a.V.stride_b : a.K.stride_b,
                       s.kind ? a.V.stride_h : a.K.stride_h, s.kind ? a.V.stride_n : a.K.stride_n};
    store32(rows.row(s.b, s.hk, n) + 32 * half, x);
}

// ---- attention ---------------------------------------------------------------------
// Up to 16 rows (query heads of a key head by tokens) read a sequence's pages once, and
// the time is that of reading them.  A cluster of CTAs takes such a block of rows, its
// pairs of warps every so many-th page each: a pair has a ring of stages of its own, which bulk
// copies of 8 KB fill, a warp 32 tokens of each page, of which it keeps the running maximum, sum and
// weighted values until the end, when the warps are joined in shared memory and the
// CTAs over the cluster, in a fixed order.
//
// Scores and weighted values are warp-wide products of halves: an e4m3 value is
// one exactly, a bf16 query too, after a power of two has moved its row's largest to
// [2^8, 2^9) (32-bit queries and weights are two halves, 22 bits), a 16-bit call's weight is rounded to
// 11 bits.  The layout of a page makes every operand's fragment one piece of
// it: lane (g, c) of a product has keys 8 (g / 2) + 2 t + (g mod 2) of its 32 in tile t with
// dims 16 c to 16 c + 15, four at a time in the order in which the rows have them;
// its scores are then those of keys 8 c to 8 c + 7, and its 8 bytes of a dim's line of values
// are those same keys.  No shuffles, and no conflicts in shared memory.
//
// (The warp-wide instructions, since the rows would leave a tile of 128 unused 7/8 and more, and e4m3
// becomes half in registers by one conversion of two values, which needs no second copy in shared memory.  Three
// stages a pair: 24 KB on the way for each, 192 KB a SM; in 32 bits with 16 rows 96.)
// Measured: 16 sequences of up to 16385, 16 heads on 4, one token: 23.1 us, 4.4 TB/s (50% of the DRAM's cycles under the
// profiler, issue slots 37%; 256 CTAs have 304 places, and a cluster has one sequence, whose mean length is 3/4 of the
// longest); 64 sequences, 4 tokens, window 1024, 4 sinks: 13.6, 2.6 TB/s (5 pages a pair of warps: start, join and
// end are half of it); one sequence 10.2; fp32 31.9 (twice the products), 21.1, 13.3.
constexpr int kPairs = 4, kStages = 3;
constexpr int kWarps = 2 * kPairs, kThreads = 32 * kWarps;
constexpr size_t kSmem = 128 + (size_t)kPairs * kStages * 2 * kPageBytes;
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
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
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
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float *x) {
    const uint2 t = __ldg(reinterpret_cast<const uint2 *>(p));
    x[0] = bf16_lo(t.x), x[1] = bf16_hi(t.x), x[2] = bf16_lo(t.y), x[3] = bf16_hi(t.y);
}
__device__ __forceinline__ void load4(const float *p, float *x) {
    const float4 t = __ldg(reinterpret_cast<const float4 *>(p));
    x[0] = t.x, x[1] = t.y, x[2] = t.z, x[3] = t.w;
}
// A write to another CTA's shared memory; the two halves of the cluster's barrier.
__device__ __forceinline__ void st_cluster2(uint32_t at, float2 v) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Bytes whose bit is set.
__device__ __forceinline__ uint32_t bytes_of(uint32_t four) {
    return ((four & 1) | (four & 2) << 7 | (four & 4) << 14 | (four & 8) << 21) * 0xffu;
}

// HALVES: 1 (at most 8 rows; the products' lower rows are not looked at) or 2.  (One token of 16
// heads on 4, 16 sequences of 16385: 23.0 us with 1, 26.6 with 2; 64 of 1569: 13.1 and 14.9; fp32 31.9 and 43.5.)
template <typename T, int HALVES>
struct Attend {
    static constexpr int kParts = sizeof(T) == 4 ? 2 : 1;             // halves of an operand
    static constexpr int kBlocks = kParts * HALVES == 4 ? 1 : 2;      // CTAs a SM
};

template <typename T, int HALVES>
__global__ void __launch_bounds__(kThreads, Attend<T, HALVES>::kBlocks)
cache_fwd_kernel(const __grid_constant__ AttendArgs a, Rows<const T> Q, Rows<T> O) {
    constexpr int R = 8 * HALVES, kParts = Attend<T, HALVES>::kParts;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = smem_raw + ((128 - (smem_u32(smem_raw) & 127)) & 127);
    __shared__ uint64_t full[kPairs][kStages];
    __shared__ int abort_flag;
    __shared__ float sm[kWarps][R], sl[kWarps][R], sf[kWarps][R];     // the warps' maxima, sums and factors
    __shared__ float2 cml[R], co[R][32];              // from the cluster's CTAs: maxima and sums, weighted values
    __shared__ float2 row_ml[R];                      // a row's maximum and sum
    static_assert(kWarps * R * 32 * sizeof(float2) <= kSmem - 128, "the warps' sums fit");
    volatile int *abort = &abort_flag;
    const int warp = warp_number(), pair = warp >> 1, sub = warp & 1, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const unsigned C = cluster_size(), rank = cluster_rank();
    if (!FIBATT_CHECKED(blockIdx.x / C < (unsigned)a.units)) return;       // whole clusters
    if (threadIdx.x < kPairs * kStages) mbar_init(&full[0][0] + threadIdx.x, 1);
    if (threadIdx.x == 0) abort_flag = 0;
    if (C > 1) cluster_arrive();      // (waited for below, before the first write to another CTA)
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();

    const unsigned unit = blockIdx.x / C, bh = unit / (unsigned)a.blocks;
    const int rb = (int)(unit - bh * a.blocks), b = (int)(bh / (unsigned)a.c.Hkv), hk = (int)(bh - (unsigned)b * a.c.Hkv);
    const int r0 = 16 * rb, rows = min(R, a.rows - r0);
    const auto token = [&](int r) { return (int)((unsigned)(r0 + r) / (unsigned)a.G); };      // of the block's row r
    // the rows' values are on their way while the pages are looked up
    float x[2][16];
#pragma unroll
    for (int i = 0; i < HALVES; ++i) {
        const int r = min(g + 8 * i, rows - 1), n = token(r);
        const T *src = Q.row(b, hk * a.G + (r0 + r - n * a.G), n) + 16 * c;
#pragma unroll
        for (int j = 0; j < 4; ++j) load4(src + 4 * j, x[i] + 4 * j);
    }
    const int start = a.c.first(b), n = a.c.tokens(b), end = a.c.table_len * kPage;
    // positions of the block's first and last queries that attend keys
    const int first = max(0, start + token(0)), last = min(end, start + min(n, token(rows - 1) + 1)) - 1;
    if (n > 0 && (start < 0 || start + n > end) && threadIdx.x == 0) atomicOr(&g_device_error, kErrPage);
    const BandWalk<kPage> walk(a.band, first, last);
    const int at = (int)rank * kPairs + pair, step = (int)C * kPairs, mine = max(0, (walk.n - at + step - 1) / step);
    const auto position = [&](int r) {
        const int p = start + token(r);
        return r < rows && p <= last ? p : -1;
    };

    // ---- copies: the pair's pages in turn.  A lane has the number and the scales of every 32nd.
    uint8_t *stages = ring + (size_t)pair * kStages * 2 * kPageBytes;
    int pages = -1;                                  // of those being copied
    float2 scales = make_float2(0.f, 0.f), used = scales;    // of those, and of those being used; 0: no page
    const auto issue = [&](int k) {
        if ((k & 31) == 0) {
            pages = -1;
            if (k + lane < mine) {
                pages = a.c.page(b, walk.tile(at + (k + lane) * step));
                if (pages < 0 && sub == 0) atomicOr(&g_device_error, kErrPage);
                if (!FIBATT_CHECKED(pages < a.c.pages)) pages = -1;
            }
            scales = make_float2(0.f, 0.f);
            if (pages >= 0) scales = __ldg(reinterpret_cast<const float2 *>(a.c.scales) + a.c.place(pages, hk));
        }
        const int page = __shfl_sync(kFullMask, pages, k & 31), s = k % kStages;
        if (sub == 0 && lane == 0) {
            if (page < 0) {
                mbar_arrive(&full[pair][s]);
            } else {
                mbar_expect_tx(&full[pair][s], 2 * kPageBytes);
                bulk_g2s(stages + (size_t)s * 2 * kPageBytes, a.c.data + a.c.place(page, hk) * 2 * kPageBytes, 2 * kPageBytes,
                         &full[pair][s]);
            }
        }
        __syncwarp();
    };
    int issued = 0;
    for (; issued < min(mine, kStages); ++issued) issue(issued);

    // ---- the rows as operands of four steps of 16 dims, and what their scores are multiplied with
    uint32_t q[kParts][4][4];
    float factor[HALVES], m[HALVES], l[HALVES], o[8][2 * HALVES];
    int p[HALVES];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float f = 0.f;
        if (i < HALVES) {
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(x[i][k]));
            top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
            top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
            const int e = max(-100, min(exponent_of(top), 120)) - 8;
            f = two_to(-e);
            factor[i] = a.scale_log2 * two_to(e);
            m[i] = kNegInf;
            l[i] = 0.f;
            p[i] = position(g + 8 * i);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float u = i < HALVES ? x[i][4 * j + 2 * k] * f : 0.f, v = i < HALVES ? x[i][4 * j + 2 * k + 1] * f : 0.f;
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
        for (int i = 0; i < 2 * HALVES; ++i) o[d][i] = 0.f;

    // (No wait's failure ends the loop: a warp's partner at the named barrier must find it there.  What
    // follows is not trusted, since the error word is set.)
    for (int done = 0; done < mine; ++done) {
        const int s = done % kStages;
        if ((done & 31) == 0) {
            used = make_float2(0.f, 0.f);
            if (pages >= 0) used = make_float2(two_to(stored_exponent(scales.x)), two_to(stored_exponent(scales.y)));
        }
        const float sk = __shfl_sync(kFullMask, used.x, done & 31), sv = __shfl_sync(kFullMask, used.y, done & 31);
        pipe_wait(&full[pair][s], (done / kStages) & 1, abort);
        __syncwarp();
        if (sk > 0.f) {
            const uint8_t *keys = stages + (size_t)s * 2 * kPageBytes + 32 * sub * kHeadDim;
            const uint8_t *values = stages + (size_t)s * 2 * kPageBytes + kPageBytes + 32 * sub;
            const int k0 = walk.tile(at + done * step) * kPage + 32 * sub, k1 = k0 + 31;
            const bool whole = k1 <= first && (k0 > last - a.band.window || k1 < a.band.sinks);
            // (products that add to one sum lie apart: each waits for the one before it)
            float y[4][4];
            uint32_t four[4][4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const uint4 w = *reinterpret_cast<const uint4 *>(keys + (8 * (g >> 1) + 2 * t + (g & 1)) * kHeadDim + 16 * c);
                four[t][0] = w.x, four[t][1] = w.y, four[t][2] = w.z, four[t][3] = w.w;
#pragma unroll
                for (int i = 0; i < 4; ++i) y[t][i] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int k = kParts - 1; k >= 0; --k)
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        mma_f16(y[t], q[k][j], halves_of(four[t][j] & 0xffff), halves_of(four[t][j] >> 16));
            uint2 v[8];
#pragma unroll
            for (int d = 0; d < 8; ++d) v[d] = *reinterpret_cast<const uint2 *>(values + (8 * d + g) * kPage + 8 * c);
            if (!whole) {                         // a weight of 0 meets no NaN
                const uint32_t live = keys_between(a.band, first, last, k0 + 8 * c);
                const uint32_t lo = bytes_of(live & 15), hi = bytes_of(live >> 4 & 15);
#pragma unroll
                for (int d = 0; d < 8; ++d) v[d].x &= lo, v[d].y &= hi;
            }
            uint32_t w[kParts][2][4];             // the weights as operands of two steps of 16 keys
#pragma unroll
            for (int i = 0; i < HALVES; ++i) {
                const float f = factor[i] * sk;
                const uint32_t seen = whole ? 0xffu : keys_of(a.band, p[i], k0 + 8 * c);
                float top = kNegInf;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float &z = y[t][2 * i + k];
                        z = (seen >> (2 * t + k)) & 1 ? z * f : kNegInf;
                        top = fmaxf(top, z);
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
                for (int t = 0; t < 4; ++t) {
                    const float u = fast_exp2(y[t][2 * i] - base), e = fast_exp2(y[t][2 * i + 1] - base);
                    sum[t & 1] += u + e;
                    const uint32_t hi = pack_f16x2(u, e);
                    w[0][t >> 1][i + 2 * (t & 1)] = hi;
                    if (kParts == 2) {
                        const float2 h = unpack_f16x2(hi);
                        w[kParts - 1][t >> 1][i + 2 * (t & 1)] = pack_f16x2(u - h.x, e - h.y);
                    }
                }
                l[i] += sum[0] + sum[1];
            }
            if (HALVES == 1) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < kParts; ++k) w[k][j][1] = w[k][j][3] = 0u;
            }
            // a page's sums by themselves, and into the running ones by additions that round
#pragma unroll
            for (int d0 = 0; d0 < 8; d0 += 4) {
                float part[4][4];
#pragma unroll
                for (int d = 0; d < 4; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i) part[d][i] = 0.f;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = kParts - 1; k >= 0; --k)
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            const uint32_t two = j ? v[d0 + d].y : v[d0 + d].x;
                            mma_f16(part[d], w[k][j], halves_of(two & 0xffff), halves_of(two >> 16));
                        }
#pragma unroll
                for (int d = 0; d < 4; ++d)
#pragma unroll
                    for (int i = 0; i < 2 * HALVES; ++i) o[d0 + d][i] = fmaf(part[d][i], sv, o[d0 + d][i]);
            }
        }
        named_sync(1 + pair, 64);       // both have read the stage
        if (issued < mine) issue(issued++);
    }
    if (sub == 0 && lane == 0)   // leave no copy in flight
        for (int i = max(0, issued - kStages); i < issued; ++i) mbar_drain(&full[pair][i % kStages], (i / kStages) & 1);
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
    // The CTA's maximum, factors and sum of each row; the cluster's, of those it finishes: row r is CTA
    // r mod C's, to whose shared memory the others write what they have of it.
    const unsigned share = R / C;        // rows that a CTA finishes (of R, a multiple of C)
    if (threadIdx.x < rows) {
        const int r = threadIdx.x;
        float top = kNegInf, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w][r]);
        const float base = top == kNegInf ? 0.f : top;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = fast_exp2(sm[w][r] - base);
            sf[w][r] = f;
            sum = fmaf(f, sl[w][r], sum);
        }
        row_ml[r] = make_float2(top, sum);
    }
    __syncthreads();
    if (C > 1) cluster_wait();
    const auto finish = [&](int r, int d, float2 x) {
        if (!FIBATT_CHECKED(r < rows && token(r) < a.c.N)) return;
        const float2 ml = row_ml[r];
        const int n = token(r), h = hk * a.G + (r0 + r - n * a.G), p = start + n;
        const bool none = p > last || ml.y == 0.f;
        const float inv = none ? 0.f : 1.f / ml.y;
        store2(O.row(b, h, n) + 2 * d, none ? make_float2(0.f, 0.f) : make_float2(x.x * inv, x.y * inv));
        if (d == 0) a.c.LSE[((int64_t)b * a.c.Hq + h) * a.c.N + n] = none ? kNegInf : (ml.x + log2f(ml.y)) * kLn2;
    };
    for (int i = threadIdx.x; i < rows * 32; i += kThreads) {
        const int r = i >> 5, d = i & 31;
        float2 x = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) x = fma2(make_float2(sf[w][r], sf[w][r]), so[w][r][d], x);
        if (C == 1) {
            finish(r, d, x);
        } else {
            const unsigned to = rank * share + r / C;
            st_cluster2(cluster_addr(&co[to][d], r % C), x);
            if (d == 0) st_cluster2(cluster_addr(&cml[to], r % C), row_ml[r]);
        }
    }
    if (C == 1) return;
    __syncwarp();
    cluster_sync();
    for (int i = threadIdx.x; i < (int)share * 32; i += kThreads) {
        const int j = i >> 5, d = i & 31, r = j * (int)C + (int)rank;
        if (r >= rows) continue;
        float top = kNegInf, sum = 0.f;
        for (unsigned k = 0; k < C; ++k) top = fmaxf(top, cml[k * share + j].x);
        const float base = top == kNegInf ? 0.f : top;
        float2 x = make_float2(0.f, 0.f);
        for (unsigned k = 0; k < C; ++k) {
            const float2 ml = cml[k * share + j], y = co[k * share + j][d];
            const float f = fast_exp2(ml.x - base);
            sum = fmaf(f, ml.y, sum);
            x = fma2(make_float2(f, f), y, x);
        }
        __syncwarp();
        if (d == 0) row_ml[r] = make_float2(top, sum);
        __syncwarp();
        finish(r, d, x);
    }
}

template <typename T, int HALVES>
cudaError_t attend(const AttendArgs &f) {
    const cudaError_t e = prepare_kernel<cache_fwd_kernel<T, HALVES>>(kSmem, 0);
    if (e != cudaSuccess) return e;
    // CTAs of a cluster: as many as the GPU holds at once, as long as a pair of warps keeps a page.  (Us with 1, 2, 4, 8:
    // 16 sequences of 16385 52, 29, 22.7, 26.5; one 50, 29, 16, 10.1; 64 of 1569 13.2, 19, 27, 42; 4 of them 8.2, 6.6, 5.3, 5.0.)
    const int64_t keys = std::min<int64_t>((int64_t)f.c.table_len * kPage, (int64_t)f.band.window + f.band.sinks + f.c.N);
    int c = 1;
    while (c < 8 && (int64_t)f.units * c * 2 <= Attend<T, HALVES>::kBlocks * sm_count() && keys > (int64_t)c * kPairs * kPage) c *= 2;
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
