// Cross attention on the FP32 units: 32-bit inputs, whose 24-bit products
// the tensor cores do not form in one pass.
//
// A CTA of 128 threads owns 64 "own" rows and walks over the 64-row tiles of
// the other side; thread (tr, tc) of an 8 x 16 grid holds an 8 x 4 piece of
// each 64 x 64 product in registers.  The three products that occur,
//   nt: acc += A B^T   (scores, dP)        A, B [64][64] rows
//   nn: acc += A B     (P V, dS K, ...)    A [64][64] weights, B [64][64] rows
// read their operands from shared memory with 16-byte loads, rows 68 floats
// apart, so that the 16 columns of a warp's load fall on different banks.
//
// Forward: own rows are queries, with the running maximum and sum of an
// online softmax per row.  Backward, query pass: own rows are queries, dQ +=
// dS K.  Key pass: own rows are keys, the tiles are the queries of every
// head that shares the key head, and the products are formed transposed
// (S^T = K Q^T), so dV += P^T dO and dK += dS^T Q are "nn" products again and
// no two CTAs add to the same gradient row: no atomics, a fixed order.
//
// With fewer CTAs than the GPU holds, the walk is cut over a thread-block
// cluster and the partial results are joined through distributed shared
// memory, in rank order.
#include <algorithm>

#include "cluster.cuh"
#include "cross.h"
#include "device_common.cuh"
#include "row_math.cuh"

namespace fibatt {
namespace {

constexpr int kT = 64;          // rows of a tile
constexpr int kLd = 68;         // floats between rows in shared memory
constexpr int kThreads = 128;
constexpr int kTile = kT * kLd; // floats of one staged tile
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ float4 load4(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }
__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }

// Rows [n0, n0 + 64) of a head into `dst`; rows that `ok` (one bit a row)
// leaves out are zeros, whatever memory holds there.
__device__ __forceinline__ void stage(float *dst, const float *head, int64_t sn, int n0, uint64_t ok) {
    for (int i = threadIdx.x; i < kT * 16; i += kThreads) {
        const int r = i >> 4, c = (i & 15) * 4;
        const float4 v = (ok >> r) & 1 ? load4(head + (int64_t)(n0 + r) * sn + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4 *>(dst + r * kLd + c) = v;
    }
}

__device__ __forceinline__ uint64_t first_bits(int n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}

// One bit for each key of [n0, n0 + 64) that sequence b attends, the same in
// every thread.
__device__ __forceinline__ uint64_t key_bits(const KeySet &ks, int b, int n0, int bound) {
    const uint64_t in = first_bits(bound - n0);
    if (!ks.mask || in == 0) return in;
    const int lane = threadIdx.x & 31;
    const bool lo = ((in >> lane) & 1) && ks.has(b, n0 + lane);
    const bool hi = ((in >> (lane + 32)) & 1) && ks.has(b, n0 + lane + 32);
    return (uint64_t)__ballot_sync(kFullMask, lo) | ((uint64_t)__ballot_sync(kFullMask, hi) << 32);
}

// acc[i][j] = <A row 8 tr + i, B row tc + 16 j>, j < J (0 for the others)
template <int J>
__device__ __forceinline__ void mm_nt_of(float (&acc)[8][4], const float *A, const float *B, int tr, int tc) {
    float2 s[8][J];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j) s[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int d = 0; d < 64; d += 4) {
        float4 b[J];
#pragma unroll
        for (int j = 0; j < J; ++j) b[j] = *reinterpret_cast<const float4 *>(B + (tc + 16 * j) * kLd + d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 a = *reinterpret_cast<const float4 *>(A + (8 * tr + i) * kLd + d);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                s[i][j] = fma2(make_float2(a.x, a.y), make_float2(b[j].x, b[j].y), s[i][j]);
                s[i][j] = fma2(make_float2(a.z, a.w), make_float2(b[j].z, b[j].w), s[i][j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = j < J ? s[i][j < J ? j : 0].x + s[i][j < J ? j : 0].y : 0.f;
}

// The columns' tile holds `cols` rows.
__device__ __forceinline__ void mm_nt(float (&acc)[8][4], const float *A, const float *B, int tr, int tc, int cols) {
    if (cols <= 16) mm_nt_of<1>(acc, A, B, tr, tc);
    else mm_nt_of<4>(acc, A, B, tr, tc);
}

// acc[i] += sum_k W[8 tr + i][k] B[k][4 tc .. 4 tc + 3] over the first `rows` k (to the next four)
__device__ __forceinline__ void mm_nn(float4 (&acc)[8], const float *W, const float *B, int tr, int tc, int rows) {
#pragma unroll 2
    for (int k = 0; k < rows; k += 4) {
        float4 b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4 *>(B + (k + j) * kLd + 4 * tc);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 w = *reinterpret_cast<const float4 *>(W + (8 * tr + i) * kLd + k);
            const float wk[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[i].x = fmaf(wk[j], b[j].x, acc[i].x);
                acc[i].y = fmaf(wk[j], b[j].y, acc[i].y);
                acc[i].z = fmaf(wk[j], b[j].z, acc[i].z);
                acc[i].w = fmaf(wk[j], b[j].w, acc[i].w);
            }
        }
    }
}

// W[8 tr + i][tc + 16 j] = v[i][j]; read back by the same warp only.
__device__ __forceinline__ void put_weights(float *W, const float (&v)[8][4], int tr, int tc) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) W[(8 * tr + i) * kLd + tc + 16 * j] = v[i][j];
    __syncwarp();
}

// Over the 16 threads that share a row (half a warp).
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) x = fmaxf(x, __shfl_xor_sync(kFullMask, x, m));
    return x;
}
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) x += __shfl_xor_sync(kFullMask, x, m);
    return x;
}

// The part of `tiles` that CTA `r` of `c` walks over.
__device__ __forceinline__ int part(int tiles, int r, int c) { return (int)((int64_t)tiles * r / c); }

__global__ void __launch_bounds__(kThreads, 2)
cross_fwd_simt_kernel(int Hq, int Hkv, int Nq, KeySet ks, Rows<const float> Q, Rows<const float> K, Rows<const float> V, Rows<float> O,
                      float *__restrict__ LSE, float scale_log2, int qtiles) {
    extern __shared__ float4 smem4[];
    float *sq = reinterpret_cast<float *>(smem4), *sk = sq + kTile, *sv = sk + kTile, *sw = sv + kTile;
    __shared__ float sm[kT], sl[kT];
    const int tid = threadIdx.x, tr = tid >> 4, tc = tid & 15;
    const int C = (int)cluster_size(), rank = (int)cluster_rank();
    const int64_t unit = blockIdx.x / C;
    const int qt = (int)(unit % qtiles), h = (int)(unit / qtiles % Hq), b = (int)(unit / qtiles / Hq);
    const int hk = h / (Hq / Hkv), q0 = qt * kT;

    grid_dep_wait();
    const int bound = ks.bound(b), tiles = (bound + kT - 1) / kT;
    const int lo = part(tiles, rank, C), hi = part(tiles, rank + 1, C);
    const uint64_t rows = first_bits(Nq - q0);
    const bool mine = (tid & ~31) / 2 < Nq - q0;     // the warp's 16 rows begin within the queries
    stage(sq, Q.row(b, h, 0), Q.sn, q0, rows);
    float m[8], l[8];
    float4 acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        m[i] = kNegInf;
        l[i] = 0.f;
        acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int t = lo; t < hi; ++t) {
        const uint64_t ok = key_bits(ks, b, t * kT, bound);
        if (ok == 0) continue;
        __syncthreads();
        stage(sk, K.row(b, hk, 0), K.sn, t * kT, ok);
        stage(sv, V.row(b, hk, 0), V.sn, t * kT, ok);
        __syncthreads();
        if (!mine) continue;
        const int cols = min(kT, bound - t * kT);
        float s[8][4];
        mm_nt(s, sq, sk, tr, tc, cols);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float top = kNegInf;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = (ok >> (tc + 16 * j)) & 1 ? s[i][j] * scale_log2 : kNegInf;
                top = fmaxf(top, s[i][j]);
            }
            const float next = fmaxf(m[i], row_max(top));
            const float base = next == kNegInf ? 0.f : next;
            const float keep = exp2f(m[i] - base);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = exp2f(s[i][j] - base);
                sum += s[i][j];
            }
            l[i] = l[i] * keep + sum;      // this thread's columns only
            m[i] = next;
            acc[i].x *= keep;
            acc[i].y *= keep;
            acc[i].z *= keep;
            acc[i].w *= keep;
        }
        put_weights(sw, s, tr, tc);
        mm_nn(acc, sw, sv, tr, tc, cols);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) l[i] = row_sum(l[i]);

    if (C == 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 8 * tr + i, n = q0 + r;
            if (n >= Nq) continue;
            const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
            store4(O.row(b, h, n) + 4 * tc,
                   make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv));
            if (tc == 0) LSE[((int64_t)b * Hq + h) * Nq + n] = l[i] == 0.f ? kNegInf : (m[i] + log2f(l[i])) * kLn2;
        }
        return;
    }
    // join the cluster's parts: CTA r finishes every C-th row
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = 8 * tr + i;
        *reinterpret_cast<float4 *>(sk + r * kLd + 4 * tc) = acc[i];
        if (tc == 0) {
            sm[r] = m[i];
            sl[r] = l[i];
        }
    }
    cluster_sync();
    for (int r = rank + C * tr; r < kT; r += C * 8) {
        const int n = q0 + r;
        if (n >= Nq) break;
        float top = kNegInf;
        for (int c = 0; c < C; ++c) top = fmaxf(top, ld_cluster(cluster_addr(sm + r, c)));
        const float base = top == kNegInf ? 0.f : top;
        float sum = 0.f;
        float2 x = make_float2(0.f, 0.f), y = x;
        for (int c = 0; c < C; ++c) {
            const float w = exp2f(ld_cluster(cluster_addr(sm + r, c)) - base);
            sum = fmaf(w, ld_cluster(cluster_addr(sl + r, c)), sum);
            const uint32_t at = cluster_addr(sk + r * kLd + 4 * tc, c);
            x = fma2(make_float2(w, w), ld_cluster2(at), x);
            y = fma2(make_float2(w, w), ld_cluster2(at + 8), y);
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        store4(O.row(b, h, n) + 4 * tc, make_float4(x.x * inv, x.y * inv, y.x * inv, y.y * inv));
        if (tc == 0) LSE[((int64_t)b * Hq + h) * Nq + n] = sum == 0.f ? kNegInf : (top + log2f(sum)) * kLn2;
    }
    cluster_sync();   // the others may still read this CTA's part
}

// (LSE log2 e, D = <dO, O>) of every query row; a row without keys gets
// +infinity, which makes each of its weights exp2(s - inf) = 0.
__global__ void __launch_bounds__(256)
cross_stats_kernel(int Hq, int Nq, int64_t rows, Rows<const float> O, Rows<const float> dO, const float *__restrict__ LSE,
                   float2 *__restrict__ stats) {
    grid_dep_wait();
    const int64_t row = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    const int c = (threadIdx.x & 15) * 4;
    if (row >= rows) return;   // whole half warps: the shuffles below stay within 16 lanes
    const int64_t n = row % Nq, h = row / Nq % Hq, b = row / Nq / Hq;
    const float4 o = load4(O.row(b, h, n) + c), g = load4(dO.row(b, h, n) + c);
    float d = o.x * g.x + o.y * g.y + (o.z * g.z + o.w * g.w);
    const unsigned half = 0xffffu << (threadIdx.x & 16);
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) d += __shfl_xor_sync(half, d, m);
    if (c == 0) {
        const float lse = LSE[row];
        stats[row] = lse == kNegInf ? make_float2(-kNegInf, 0.f) : make_float2(lse * kLog2e, d);
    }
}

// Sum over the cluster of the 64 x 64 accumulator (`part` in shared memory,
// 64 rows of kLd floats), times `scale`, into rows n0.. of `out`.
__device__ __forceinline__ void finish(float4 (&acc)[8], float *parts, Rows<float> out, int64_t b, int64_t h, int n0, int N,
                                       float scale, int tr, int tc) {
    const int C = (int)cluster_size(), rank = (int)cluster_rank();
    if (C == 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int n = n0 + 8 * tr + i;
            if (n < N)
                store4(out.row(b, h, n) + 4 * tc,
                       make_float4(acc[i].x * scale, acc[i].y * scale, acc[i].z * scale, acc[i].w * scale));
        }
        return;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<float4 *>(parts + (8 * tr + i) * kLd + 4 * tc) = acc[i];
    cluster_sync();
    for (int r = rank + C * tr; r < kT; r += C * 8) {
        if (n0 + r >= N) break;
        float2 x = make_float2(0.f, 0.f), y = x;
        for (int c = 0; c < C; ++c) {
            const uint32_t at = cluster_addr(parts + r * kLd + 4 * tc, c);
            x = add2(x, ld_cluster2(at));
            y = add2(y, ld_cluster2(at + 8));
        }
        store4(out.row(b, h, n0 + r) + 4 * tc, make_float4(x.x * scale, x.y * scale, y.x * scale, y.y * scale));
    }
    cluster_sync();
}

struct BwdArgs32 {
    int Hq, Hkv, Nq;
    KeySet ks;
    Rows<const float> Q, K, V, dO;
    const float2 *stats;
    Rows<float> dQ, dK, dV;
    float scale;
    int qtiles, ktiles;
    int key_units;        // units that hold keys; the others hold queries
};

// Holds 64 queries and walks over the keys.
__device__ __forceinline__ void hold_queries(const BwdArgs32 &a, float *smem, int64_t unit) {
    float *sq = smem, *sg = sq + kTile, *sk = sg + kTile, *sv = sk + kTile, *sw = sv + kTile;
    const int tid = threadIdx.x, tr = tid >> 4, tc = tid & 15;
    const int C = (int)cluster_size(), rank = (int)cluster_rank();
    const int qt = (int)(unit % a.qtiles), h = (int)(unit / a.qtiles % a.Hq), b = (int)(unit / a.qtiles / a.Hq);
    const int hk = h / (a.Hq / a.Hkv), q0 = qt * kT;
    const float scale_log2 = a.scale * kLog2e;
    const int bound = a.ks.bound(b), tiles = (bound + kT - 1) / kT;
    const int lo = part(tiles, rank, C), hi = part(tiles, rank + 1, C);
    const uint64_t rows = first_bits(a.Nq - q0);
    const bool mine = (tid & ~31) / 2 < a.Nq - q0;     // the warp's 16 rows begin within the queries
    stage(sq, a.Q.row(b, h, 0), a.Q.sn, q0, rows);
    stage(sg, a.dO.row(b, h, 0), a.dO.sn, q0, rows);
    float2 st[8];
    float4 acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int n = q0 + 8 * tr + i;
        st[i] = n < a.Nq ? a.stats[((int64_t)b * a.Hq + h) * a.Nq + n] : make_float2(-kNegInf, 0.f);
        acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int t = lo; t < hi; ++t) {
        const uint64_t ok = key_bits(a.ks, b, t * kT, bound);
        if (ok == 0) continue;
        __syncthreads();
        stage(sk, a.K.row(b, hk, 0), a.K.sn, t * kT, ok);
        stage(sv, a.V.row(b, hk, 0), a.V.sn, t * kT, ok);
        __syncthreads();
        if (!mine) continue;
        const int cols = min(kT, bound - t * kT);
        float s[8][4], dp[8][4];
        mm_nt(s, sq, sk, tr, tc, cols);
        mm_nt(dp, sg, sv, tr, tc, cols);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(fmaf(s[i][j], scale_log2, -st[i].x));
                s[i][j] = (ok >> (tc + 16 * j)) & 1 ? p * (dp[i][j] - st[i].y) : 0.f;
            }
        put_weights(sw, s, tr, tc);
        mm_nn(acc, sw, sk, tr, tc, cols);
    }
    finish(acc, sv, a.dQ, b, h, q0, a.Nq, a.scale, tr, tc);
}

// Holds 64 keys and walks over the queries of every head that shares them.
__device__ __forceinline__ void hold_keys(const BwdArgs32 &a, float *smem, int64_t unit) {
    float *sk = smem, *sv = sk + kTile, *sq = sv + kTile, *sg = sq + kTile, *sw = sg + kTile;
    const int tid = threadIdx.x, tr = tid >> 4, tc = tid & 15;
    const int C = (int)cluster_size(), rank = (int)cluster_rank();
    const int kt = (int)(unit % a.ktiles), hk = (int)(unit / a.ktiles % a.Hkv), b = (int)(unit / a.ktiles / a.Hkv);
    const int G = a.Hq / a.Hkv, k0 = kt * kT, qtiles = a.qtiles;
    const float scale_log2 = a.scale * kLog2e;
    const int bound = a.ks.bound(b);
    const uint64_t ok = key_bits(a.ks, b, k0, bound);
    const bool mine = (tid & ~31) / 2 < bound - k0;    // the warp's 16 rows begin within the keys
    // the walk: the query tiles of each of the G heads in turn; none for a tile without keys
    const int64_t tiles = ok ? (int64_t)G * qtiles : 0;
    const int64_t lo = tiles * rank / C, hi = tiles * (rank + 1) / C;
    stage(sk, a.K.row(b, hk, 0), a.K.sn, k0, ok);
    stage(sv, a.V.row(b, hk, 0), a.V.sn, k0, ok);
    float4 ak[8], av[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) ak[i] = av[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int64_t t = lo; t < hi; ++t) {
        const int h = hk * G + (int)(t / qtiles), q0 = (int)(t % qtiles) * kT;
        const uint64_t rows = first_bits(a.Nq - q0);
        __syncthreads();
        stage(sq, a.Q.row(b, h, 0), a.Q.sn, q0, rows);
        stage(sg, a.dO.row(b, h, 0), a.dO.sn, q0, rows);
        float2 st[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = q0 + tc + 16 * j;
            st[j] = n < a.Nq ? a.stats[((int64_t)b * a.Hq + h) * a.Nq + n] : make_float2(-kNegInf, 0.f);
        }
        __syncthreads();
        if (!mine) continue;
        const int cols = min(kT, a.Nq - q0);
        float p[8][4], ds[8][4];
        mm_nt(p, sk, sq, tr, tc, cols);
        mm_nt(ds, sv, sg, tr, tc, cols);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool in = (ok >> (8 * tr + i)) & 1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                p[i][j] = in ? exp2f(fmaf(p[i][j], scale_log2, -st[j].x)) : 0.f;
                ds[i][j] = in ? p[i][j] * (ds[i][j] - st[j].y) : 0.f;
            }
        }
        put_weights(sw, p, tr, tc);
        mm_nn(av, sw, sg, tr, tc, cols);
        put_weights(sw, ds, tr, tc);
        mm_nn(ak, sw, sq, tr, tc, cols);
    }
    finish(av, sg, a.dV, b, hk, k0, a.ks.Nk, 1.f, tr, tc);
    finish(ak, sq, a.dK, b, hk, k0, a.ks.Nk, a.scale, tr, tc);
}

// Both kinds of unit in one launch, the longer ones (keys) first.
__global__ void __launch_bounds__(kThreads, 2) cross_bwd_simt_kernel(const __grid_constant__ BwdArgs32 a) {
    extern __shared__ float4 smem4[];
    float *smem = reinterpret_cast<float *>(smem4);
    grid_dep_wait();
    const int64_t unit = blockIdx.x / cluster_size();
    if (unit < a.key_units) hold_keys(a, smem, unit);
    else hold_queries(a, smem, unit - a.key_units);
}

// CTAs of a cluster for `units` units of `tiles` tiles each: enough to give
// every SM its two CTAs, as long as each CTA keeps a tile.
int split(int64_t units, int64_t tiles) {
    int c = 1;
    while (c < 8 && units * c * 2 <= 2 * sm_count() && tiles >= 2 * c) c *= 2;
    return c;
}

}  // namespace

cudaError_t launch_cross_fwd_simt(const CrossArgs &a) {
    constexpr size_t smem = 4 * kTile * sizeof(float);
    const cudaError_t e = prepare_kernel<cross_fwd_simt_kernel>(smem, 0);
    if (e != cudaSuccess) return e;
    const int qtiles = (a.Nq + kT - 1) / kT;
    const int64_t units = (int64_t)a.B * a.Hq * qtiles;
    const int c = split(units, (a.Nk + kT - 1) / kT);
    return launch_clusters(cross_fwd_simt_kernel, (unsigned)(units * c), c, kThreads, smem, a.stream, a.Hq, a.Hkv, a.Nq,
                           a.keys, rows_of<const float>(a.Q), rows_of<const float>(a.K), rows_of<const float>(a.V),
                           rows_of<float>(a.O), a.LSE, a.scale * kLog2e, qtiles);
}

cudaError_t launch_cross_bwd_simt(const CrossArgs &a) {
    constexpr size_t smem = 5 * kTile * sizeof(float);
    cudaError_t e = prepare_kernel<cross_bwd_simt_kernel>(smem, 0);
    if (e != cudaSuccess) return e;
    BwdArgs32 f;
    f.Hq = a.Hq, f.Hkv = a.Hkv, f.Nq = a.Nq;
    f.ks = a.keys;
    f.Q = rows_of<const float>(a.Q), f.K = rows_of<const float>(a.K), f.V = rows_of<const float>(a.V);
    f.dO = rows_of<const float>(a.dO);
    f.stats = a.stats;
    f.dQ = rows_of<float>(a.dQ), f.dK = rows_of<float>(a.dK), f.dV = rows_of<float>(a.dV);
    f.scale = a.scale;
    f.qtiles = (a.Nq + kT - 1) / kT, f.ktiles = (a.Nk + kT - 1) / kT;
    const int64_t rows = (int64_t)a.B * a.Hq * a.Nq;
    e = launch_clusters(cross_stats_kernel, (unsigned)((rows + 15) / 16), 1, 256, 0, a.stream, a.Hq, a.Nq, rows,
                        rows_of<const float>(a.O), f.dO, static_cast<const float *>(a.LSE), a.stats);
    if (e != cudaSuccess) return e;
    const int64_t key_units = (int64_t)a.B * a.Hkv * f.ktiles, units = key_units + (int64_t)a.B * a.Hq * f.qtiles;
    f.key_units = (int)key_units;
    const int c = split(units, std::max<int64_t>(f.ktiles, (int64_t)(a.Hq / a.Hkv) * f.qtiles));
    return launch_clusters(cross_bwd_simt_kernel, (unsigned)(units * c), c, kThreads, smem, a.stream, f);
}

FIBATT_DEFINE_ERROR_READER(read_error_cross_simt, "cross_simt.cu")

}  // namespace fibatt
