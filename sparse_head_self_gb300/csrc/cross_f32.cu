// Cross attention of 32-bit inputs.
//
// The products keep 22 of an operand's 24 bits: each value is split into a TF32
// part (its upper 11 bits) and the rest, and a product is the three warp-wide
// matrix instructions hi lo + lo hi + hi hi, with fp32 sums; what is left out,
// lo lo, is below 2^-22 of the product.  At 301 TFLOP/s of these instructions
// (measured) that is 100 TFLOP/s of products, where the FP32 units give 80 at most and
// gave 34 here, held up by the shared memory's bandwidth.  (The 5th-generation
// cores' TF32 form would need every tile twice in shared memory, its upper and its lower bits, and for P V
// and dS K, whose second operand lies across the summed index, the swizzle in pieces of 32
// bytes that there is for 32-bit types.  Not built.)
// Measured: gradient of 4 sequences, 12 heads, 197 x 197, masked: 64 us (FP32 units:
// 85.5), 384 blocks of which some SMs have three and some two, the warp-wide
// instructions 33% busy: a scheduler's three warps wait for their own chains of cuts and
// products, for their copies, and for instructions.
//
// A CTA of four warps holds 64 rows and walks over the 64-row tiles of the
// other side, a warp 16 rows by all 64 columns:
//   nt: C = A B^T      (scores, dP)          A, B rows in shared memory
//   nn: O += W B       (P V, dS K, ...)      W in registers, B rows in shared memory
// Lane (g, t) of an instruction gives k-places t and t + 4 the elements 2 t and
// 2 t + 1 of both operands (the order of a sum does not matter): nt then reads
// 8-byte pairs, and the fragment of C, columns 2 t and 2 t + 1, is W's
// operand as it stands.  Rows are 72 floats apart: the pairs of nt fall on
// different banks, the columns of nn on 16 of them.
//
// Forward: the rows are queries, with the running maximum and sum of an
// online softmax per row.  Backward, queries held: dQ += dS K.  Keys held: the
// tiles are the queries of every head that shares the key head, and the
// products are formed transposed (S^T = K Q^T), so dV += P^T dO and dK +=
// dS^T Q are nn again and no two CTAs add to the same gradient row: no
// atomics, a fixed order.
//
// With fewer CTAs than the GPU holds, the walk is cut over a thread-block
// cluster and the partial results are joined through distributed shared
// memory, in rank order.
//
// Attention over a window with sinks (BAND): walks over the tiles that the windows meet; within a tile
// each warp's products start and end at the columns that its 16 rows may attend, in steps of 32 and 8,
// since at three instructions a product what is left out counts (gradient of 4 sequences, 12
// heads, up to 197 tokens, window 65, 1 sink: 54 -> 45.2 us; units worked out without divisions and shorter code, 43.1).
// There a SM has 3 CTAs of 4 warps, the warp-wide instructions are 17% busy, and the time goes to the waits for copies at the
// CTA's barriers: walks have 2 or 3 tiles.  2 sequences, 16 heads on 4, 1569 tokens, window 512, 4 sinks: forward
// 179 us (31 TFLOP/s of 100), gradient 920.
#include <algorithm>

#include "cluster.cuh"
#include "cross.h"
#include "device_common.cuh"
#include "row_math.cuh"

namespace fibatt {
namespace {

constexpr int kT = 64;          // rows of a tile
constexpr int kLd = 72;         // floats between rows in shared memory
constexpr int kThreads = 128;
constexpr int kTile = kT * kLd; // floats of one staged tile
constexpr int kFwdBlocks = 4, kBwdBlocks = 3;   // a SM
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ float4 load4(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }
__device__ __forceinline__ void store2(float *p, float2 v) { *reinterpret_cast<float2 *>(p) = v; }

// Rows [n0, n0 + 64) of a head into `dst`; rows that `ok` (one bit a row)
// leaves out are zeros, whatever memory holds there.  staged() before the
// CTA's barrier.
__device__ __forceinline__ void stage(float *dst, const float *head, int64_t sn, int n0, uint64_t ok) {
#pragma unroll
    for (int k = 0; k < kT * 16 / kThreads; ++k) {
        const int i = threadIdx.x + k * kThreads, r = i >> 4, c = (i & 15) * 4;
        float *to = dst + r * kLd + c;
        if ((ok >> r) & 1)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
                         "l"(head + (int64_t)(n0 + r) * sn + c)
                         : "memory");
        else
            *reinterpret_cast<float4 *>(to) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
}
__device__ __forceinline__ void staged() { asm volatile("cp.async.wait_all;" ::: "memory"); }

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

// The same for the keys that queries at positions lo to hi attend.
__device__ __forceinline__ uint64_t band_bits(const Band &w, int lo, int hi, int n0) {
    if (lo > hi) return 0ull;
    return first_bits(hi + 1 - n0) & (~first_bits(lo + 1 - w.window - n0) | first_bits(w.sinks - n0));
}

// x = hi + lo, hi rounded to 11 bits (half a step added to the pattern, the
// others cleared); of lo 11 are read.  With hi cut off instead, lo always has x's
// sign, and the products lo lo that are left out add up: 1.4e-6 of the gradients'
// norm where this leaves 3.8e-7, as 32-bit products do.
__device__ __forceinline__ void cut(float x, uint32_t &hi, uint32_t &lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2], const float (&c)[4]) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
// c[i] += a b[i] to 22 bits for four b: the instructions that add to one sum lie
// four apart, since each waits for the one before it.  The sums inside the
// instructions are cut off, not rounded, so only these three go into one; the
// running sum is kept outside, where additions round (inside, 2.6e-6).
__device__ __forceinline__ void mma3(float (&c0)[4], float (&c1)[4], float (&c2)[4], float (&c3)[4], const uint32_t (&ah)[4],
                                     const uint32_t (&al)[4], const float2 (&b)[4]) {
    uint32_t h[4][2], l[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        cut(b[i].x, h[i][0], l[i][0]);
        cut(b[i].y, h[i][1], l[i][1]);
    }
    float s[4][4];
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) mma(s[i], ah, l[i], zero);
#pragma unroll
    for (int i = 0; i < 4; ++i) mma(s[i], al, h[i], s[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) mma(s[i], ah, h[i], s[i]);
    float(*const c[4])[4] = {&c0, &c1, &c2, &c3};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
            const float2 t = add2(make_float2((*c[i])[k], (*c[i])[k + 1]), make_float2(s[i][k], s[i][k + 1]));
            (*c[i])[k] = t.x;
            (*c[i])[k + 1] = t.y;
        }
}

// A lane's fragment of 16 rows by 64 columns: [j][0], [j][1] are row g (of the
// warp's 16), columns 8 j + 2 t and the next, [j][2], [j][3] row g + 8.
struct Lane {
    int w, g, t;
    __device__ __forceinline__ Lane() : w(threadIdx.x >> 5), g((threadIdx.x & 31) >> 2), t(threadIdx.x & 3) {}
    __device__ __forceinline__ int row(int half) const { return 16 * w + g + 8 * half; }
    __device__ __forceinline__ int col(int j, int k) const { return 8 * j + 2 * t + k; }
};

// The columns [from, cols) of a tile of keys from k0 on that 16 queries from position p on may attend.
__device__ __forceinline__ void seen_columns(const Band &w, int p, int k0, int &from, int &cols) {
    if (k0 >= w.sinks) from = max(0, p + 1 - w.window - k0);
    cols = min(cols, p + 16 - k0);
}

// c = A B^T: rows of A from the warp's first; columns: rows `from` to `cols` of B
// (from the 32 before, to the next 32; 0 for the others).  TURNS of the loop laid out: 2 for the forward; the
// gradients, whose longer code waits for its instructions, are 1 to 4% faster with 1.
template <int TURNS>
__device__ __forceinline__ void nt(float (&c)[8][4], const float *A, const float *B, const Lane &l, int cols, int from = 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[j][i] = 0.f;
    const float *pa = A + l.row(0) * kLd + 2 * l.t, *pb = B + l.g * kLd + 2 * l.t;
#pragma unroll TURNS
    for (int k = 0; k < 64; k += 8) {
        const float2 u = *reinterpret_cast<const float2 *>(pa + k);
        const float2 v = *reinterpret_cast<const float2 *>(pa + 8 * kLd + k);
        uint32_t ah[4], al[4];
        cut(u.x, ah[0], al[0]);
        cut(v.x, ah[1], al[1]);
        cut(u.y, ah[2], al[2]);
        cut(v.y, ah[3], al[3]);
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
            if (8 * j >= cols) break;
            if (8 * j + 32 <= from) continue;
            float2 b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = *reinterpret_cast<const float2 *>(pb + 8 * (j + i) * kLd + k);
            mma3(c[j], c[j + 1], c[j + 2], c[j + 3], ah, al, b);
        }
    }
}

// o += W B over rows `from` to `rows` of B (from the eight before, to the next eight); W as nt leaves it.
__device__ __forceinline__ void nn(float (&o)[8][4], const float (&W)[8][4], const float *B, const Lane &l, int rows, int from = 0) {
    const float *pb = B + 2 * l.t * kLd + l.g;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (8 * j >= rows) break;
        if (8 * j + 8 <= from) continue;
        uint32_t ah[4], al[4];
        cut(W[j][0], ah[0], al[0]);
        cut(W[j][2], ah[1], al[1]);
        cut(W[j][1], ah[2], al[2]);
        cut(W[j][3], ah[3], al[3]);
#pragma unroll
        for (int n = 0; n < 8; n += 4) {
            float2 b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                b[i] = make_float2(pb[8 * j * kLd + 8 * (n + i)], pb[(8 * j + 1) * kLd + 8 * (n + i)]);
            mma3(o[n], o[n + 1], o[n + 2], o[n + 3], ah, al, b);
        }
    }
}

// Over the four lanes that share a row.
__device__ __forceinline__ float row_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(kFullMask, x, 1));
    return fmaxf(x, __shfl_xor_sync(kFullMask, x, 2));
}
__device__ __forceinline__ float row_sum(float x) {
    x += __shfl_xor_sync(kFullMask, x, 1);
    return x + __shfl_xor_sync(kFullMask, x, 2);
}

__device__ __forceinline__ void clear(float (&o)[8][4]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
}

// The part of `tiles` that CTA `r` of `c`, a power of two, walks over.
__device__ __forceinline__ int part(int tiles, int r, int c) { return (int)((int64_t)tiles * r >> (__ffs(c) - 1)); }

template <bool BAND>
__global__ void __launch_bounds__(kThreads, kFwdBlocks)
cross_fwd_f32_kernel(int Hq, int Nq, KeySet ks, Band band, Rows<const float> Q, Rows<const float> K, Rows<const float> V,
                     Rows<float> O, float *__restrict__ LSE, float scale_log2, Div by_qtiles, Div by_hq, Div by_group, int units) {
    extern __shared__ float4 smem4[];
    float *sq = reinterpret_cast<float *>(smem4), *sk = sq + kTile, *sv = sk + kTile;
    __shared__ float sm[kT], sl[kT];
    const Lane ln;
    const int C = (int)cluster_size(), rank = (int)cluster_rank();
    const int unit = (int)(blockIdx.x >> (__ffs(C) - 1));
    if (!FIBATT_CHECKED(unit < units)) return;      // whole clusters
    int qt, b, h, hk;
    if constexpr (BAND) {      // (without a window 1% slower so, for registers)
        const int bh = by_qtiles.of(unit);
        qt = by_qtiles.rest(unit), b = by_hq.of(bh), h = by_hq.rest(bh), hk = by_group.of(h);
    } else {
        qt = unit % (int)by_qtiles.d, h = unit / (int)by_qtiles.d % Hq, b = unit / (int)by_qtiles.d / Hq, hk = h / (int)by_group.d;
    }
    const int q0 = qt * kT;

    grid_dep_wait();
    const int bound = ks.bound(b);
    int tiles = (bound + kT - 1) / kT, p[2] = {-1, -1}, p0 = 0, first = 0, last = 0;   // positions: of the lane's rows, of query 0, of the tile's
    KeyWalk<kT> walk;
    if constexpr (BAND) {
        p0 = band.first(b);
        first = max(0, p0 + q0);
        last = min(bound, p0 + min(Nq, q0 + kT)) - 1;
        walk = KeyWalk<kT>(band, first, last);
        tiles = walk.n;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (p0 + q0 + ln.row(i) <= last) p[i] = p0 + q0 + ln.row(i);
    }
    const int lo = part(tiles, rank, C), hi = part(tiles, rank + 1, C);
    const bool mine = 16 * ln.w < Nq - q0;     // the warp's 16 rows begin within the queries
    stage(sq, Q.row(b, h, 0), Q.sn, q0, first_bits(Nq - q0));
    float m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f}, o[8][4];
    clear(o);
    for (int x = lo; x < hi; ++x) {
        const int k0 = BAND ? walk.key(x) : x * kT;
        const Band w = BAND ? walk.band(band, x) : band;
        const uint64_t ok = BAND ? band_bits(w, first, last, k0) : key_bits(ks, b, k0, bound);
        if (ok == 0) continue;
        __syncthreads();
        stage(sk, K.row(b, hk, 0), K.sn, k0, ok);
        stage(sv, V.row(b, hk, 0), V.sn, k0, ok);
        staged();
        __syncthreads();
        if (!mine) continue;
        int cols = min(kT, bound - k0), from = 0;
        if constexpr (BAND) seen_columns(w, p0 + q0 + 16 * ln.w, k0, from, cols);
        float s[8][4];
        nt<2>(s, sq, sk, ln, cols, from);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float top = kNegInf;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float &x = s[j][2 * i + k];
                    const bool in = BAND ? w.sees(p[i], k0 + ln.col(j, k)) : (ok >> ln.col(j, k)) & 1;
                    x = in ? x * scale_log2 : kNegInf;
                    top = fmaxf(top, x);
                }
            const float next = fmaxf(m[i], row_max(top));
            const float base = next == kNegInf ? 0.f : next;
            const float keep = exp2f(m[i] - base);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    s[j][2 * i + k] = exp2f(s[j][2 * i + k] - base);
                    sum += s[j][2 * i + k];
                    o[j][2 * i + k] *= keep;
                }
            }
            l[i] = l[i] * keep + sum;      // this lane's columns only
            m[i] = next;
        }
        nn(o, s, sv, ln, cols, from);
    }
    l[0] = row_sum(l[0]);
    l[1] = row_sum(l[1]);

    if (C == 1) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int n = q0 + ln.row(i);
            if (n >= Nq) continue;
            const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
            float *out = O.row(b, h, n) + 2 * ln.t;
#pragma unroll
            for (int j = 0; j < 8; ++j) store2(out + 8 * j, make_float2(o[j][2 * i] * inv, o[j][2 * i + 1] * inv));
            if (ln.t == 0) LSE[((int64_t)b * Hq + h) * Nq + n] = l[i] == 0.f ? kNegInf : (m[i] + log2f(l[i])) * kLn2;
        }
        return;
    }
    // join the cluster's parts: CTA r finishes every C-th row
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = ln.row(i);
#pragma unroll
        for (int j = 0; j < 8; ++j) store2(sk + r * kLd + ln.col(j, 0), make_float2(o[j][2 * i], o[j][2 * i + 1]));
        if (ln.t == 0) {
            sm[r] = m[i];
            sl[r] = l[i];
        }
    }
    cluster_sync();
    const int c4 = (threadIdx.x & 15) * 4;
    for (int r = rank + C * (int)(threadIdx.x >> 4); r < kT; r += C * (kThreads / 16)) {
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
            const uint32_t at = cluster_addr(sk + r * kLd + c4, c);
            x = fma2(make_float2(w, w), ld_cluster2(at), x);
            y = fma2(make_float2(w, w), ld_cluster2(at + 8), y);
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<float4 *>(O.row(b, h, n) + c4) = make_float4(x.x * inv, x.y * inv, y.x * inv, y.y * inv);
        if (c4 == 0) LSE[((int64_t)b * Hq + h) * Nq + n] = sum == 0.f ? kNegInf : (top + log2f(sum)) * kLn2;
    }
    cluster_sync();   // the others may still read this CTA's part
}

// (LSE log2 e, D = <dO, O>) of every query row; a row without keys gets
// +infinity, which makes each of its weights exp2(s - inf) = 0.
__global__ void __launch_bounds__(256)
cross_stats_kernel(Div by_hq, Div by_nq, int64_t rows, Rows<const float> O, Rows<const float> dO, const float *__restrict__ LSE,
                   float2 *__restrict__ stats) {
    grid_dep_wait();
    const int64_t row = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    const int c = (threadIdx.x & 15) * 4;
    if (row >= rows) return;   // whole half warps: the shuffles below stay within 16 lanes
    const int bh = by_nq.of((int)row), n = by_nq.rest((int)row), b = by_hq.of(bh), h = by_hq.rest(bh);
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

// Sum over the cluster of the lanes' fragments (by way of `parts` in shared
// memory), times `scale`, into rows n0.. of `out`.
__device__ __forceinline__ void finish(const float (&o)[8][4], float *parts, Rows<float> out, int64_t b, int64_t h, int n0,
                                       int N, float scale, const Lane &ln) {
    const int C = (int)cluster_size(), rank = (int)cluster_rank();
    if (C == 1) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int n = n0 + ln.row(i);
            if (n >= N) continue;
            float *to = out.row(b, h, n) + 2 * ln.t;
#pragma unroll
            for (int j = 0; j < 8; ++j) store2(to + 8 * j, make_float2(o[j][2 * i] * scale, o[j][2 * i + 1] * scale));
        }
        return;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            store2(parts + ln.row(i) * kLd + ln.col(j, 0), make_float2(o[j][2 * i], o[j][2 * i + 1]));
    cluster_sync();
    const int c4 = (threadIdx.x & 15) * 4;
    for (int r = rank + C * (int)(threadIdx.x >> 4); r < kT; r += C * (kThreads / 16)) {
        if (n0 + r >= N) break;
        float2 x = make_float2(0.f, 0.f), y = x;
        for (int c = 0; c < C; ++c) {
            const uint32_t at = cluster_addr(parts + r * kLd + c4, c);
            x = add2(x, ld_cluster2(at));
            y = add2(y, ld_cluster2(at + 8));
        }
        *reinterpret_cast<float4 *>(out.row(b, h, n0 + r) + c4) =
            make_float4(x.x * scale, x.y * scale, y.x * scale, y.y * scale);
    }
    cluster_sync();
}

struct BwdF32Args {
    int Hq, Nq;
    KeySet ks;
    Band band;            // BAND
    Rows<const float> Q, K, V, dO;
    const float2 *stats;
    Rows<float> dQ, dK, dV;
    float scale;
    int qtiles;
    Div by_qtiles, by_ktiles, by_hq, by_hkv, by_group;
    int key_units;        // units that hold keys; the others hold queries
    int units;            // all of them
    int first;            // unit of the launch
};

// Holds 64 queries and walks over the keys.
template <bool BAND>
__device__ __forceinline__ void hold_queries(const BwdF32Args &a, float *smem, int unit) {
    float *sq = smem, *sg = sq + kTile, *sk = sg + kTile, *sv = sk + kTile;
    const Lane ln;
    const int C = (int)cluster_size(), rank = (int)cluster_rank();
    const int bh = a.by_qtiles.of(unit), qt = a.by_qtiles.rest(unit), b = a.by_hq.of(bh), h = a.by_hq.rest(bh);
    const int hk = a.by_group.of(h), q0 = qt * kT;
    const float scale_log2 = a.scale * kLog2e;
    const int bound = a.ks.bound(b);
    int tiles = (bound + kT - 1) / kT, p[2] = {-1, -1}, p0 = 0, first = 0, last = 0;   // positions: of the lane's rows, of query 0, of the tile's
    KeyWalk<kT> walk;
    if constexpr (BAND) {
        p0 = a.band.first(b);
        first = max(0, p0 + q0);
        last = min(bound, p0 + min(a.Nq, q0 + kT)) - 1;
        walk = KeyWalk<kT>(a.band, first, last);
        tiles = walk.n;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (p0 + q0 + ln.row(i) <= last) p[i] = p0 + q0 + ln.row(i);
    }
    const int lo = part(tiles, rank, C), hi = part(tiles, rank + 1, C);
    const bool mine = 16 * ln.w < a.Nq - q0;     // the warp's 16 rows begin within the queries
    stage(sq, a.Q.row(b, h, 0), a.Q.sn, q0, first_bits(a.Nq - q0));
    stage(sg, a.dO.row(b, h, 0), a.dO.sn, q0, first_bits(a.Nq - q0));
    float2 st[2];
    float acc[8][4];
    clear(acc);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int n = q0 + ln.row(i);
        st[i] = n < a.Nq ? a.stats[((int64_t)b * a.Hq + h) * a.Nq + n] : make_float2(-kNegInf, 0.f);
    }
    for (int y = lo; y < hi; ++y) {
        const int k0 = BAND ? walk.key(y) : y * kT;
        const Band w = BAND ? walk.band(a.band, y) : a.band;
        const uint64_t ok = BAND ? band_bits(w, first, last, k0) : key_bits(a.ks, b, k0, bound);
        if (ok == 0) continue;
        __syncthreads();
        stage(sk, a.K.row(b, hk, 0), a.K.sn, k0, ok);
        stage(sv, a.V.row(b, hk, 0), a.V.sn, k0, ok);
        staged();
        __syncthreads();
        if (!mine) continue;
        int cols = min(kT, bound - k0), from = 0;
        if constexpr (BAND) seen_columns(w, p0 + q0 + 16 * ln.w, k0, from, cols);
        float s[8][4], dp[8][4];
        nt<1>(s, sq, sk, ln, cols, from);
        nt<1>(dp, sg, sv, ln, cols, from);
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = st[i >> 1];
                const float e = exp2f(fmaf(s[j][i], scale_log2, -x.x));
                const bool in = BAND ? w.sees(p[i >> 1], k0 + ln.col(j, i & 1)) : (ok >> ln.col(j, i & 1)) & 1;
                s[j][i] = in ? e * (dp[j][i] - x.y) : 0.f;
            }
        nn(acc, s, sk, ln, cols, from);
    }
    finish(acc, sv, a.dQ, b, h, q0, a.Nq, a.scale, ln);
}

// Holds 64 keys and walks over the queries of every head that shares them.
template <bool BAND>
__device__ __forceinline__ void hold_keys(const BwdF32Args &a, float *smem, float2 *sst, int unit) {
    float *sk = smem, *sv = sk + kTile, *sq = sv + kTile, *sg = sq + kTile;
    const Lane ln;
    const int C = (int)cluster_size(), rank = (int)cluster_rank();
    const int bh = a.by_ktiles.of(unit), kt = a.by_ktiles.rest(unit), b = a.by_hkv.of(bh), hk = a.by_hkv.rest(bh);
    const int G = (int)a.by_group.d, k0 = kt * kT;
    const float scale_log2 = a.scale * kLog2e;
    const int bound = a.ks.bound(b);
    uint64_t ok;
    int p0 = 0, first = 0, last = 0;      // positions: of query 0, of the queries that attend keys of the tile
    int from = 0, qtiles = a.qtiles;      // the query tiles of a head that hold those
    if constexpr (BAND) {
        p0 = a.band.first(b);
        const int k1 = min(k0 + kT, bound) - 1, end = min(bound, p0 + a.Nq);
        first = max(p0, k0);
        last = k0 > k1 ? first - 1 : (k0 < a.band.sinks ? end : min(end, k1 + a.band.window)) - 1;
        from = first <= last ? (first - p0) / kT : 0;
        qtiles = first <= last ? (last - p0) / kT + 1 - from : 0;
        ok = band_bits(a.band, first, last, k0);
    } else {
        ok = key_bits(a.ks, b, k0, bound);
    }
    const bool mine = 16 * ln.w < bound - k0;    // the warp's 16 rows begin within the keys
    // the walk: the query tiles of each of the G heads in turn; none for a tile without keys
    const int tiles = ok ? G * qtiles : 0, lo = part(tiles, rank, C), hi = part(tiles, rank + 1, C);
    stage(sk, a.K.row(b, hk, 0), a.K.sn, k0, ok);
    stage(sv, a.V.row(b, hk, 0), a.V.sn, k0, ok);
    float ak[8][4], av[8][4];
    clear(ak);
    clear(av);
    const bool in[2] = {((ok >> ln.row(0)) & 1) != 0, ((ok >> ln.row(1)) & 1) != 0};
    for (int t = lo, g = lo < hi ? lo / qtiles : 0, at = lo - g * qtiles; t < hi; ++t) {
        const int h = hk * G + g, q0 = (from + at) * kT;
        if (++at == qtiles) at = 0, ++g;
        uint64_t rows = first_bits(a.Nq - q0);
        if constexpr (BAND) rows &= first_bits(bound - p0 - q0) & ~first_bits(-p0 - q0);    // queries of the sequence
        __syncthreads();
        stage(sq, a.Q.row(b, h, 0), a.Q.sn, q0, rows);
        stage(sg, a.dO.row(b, h, 0), a.dO.sn, q0, rows);
        if (threadIdx.x < kT) {
            const int n = q0 + (int)threadIdx.x;
            sst[threadIdx.x] = (rows >> threadIdx.x) & 1 ? a.stats[((int64_t)b * a.Hq + h) * a.Nq + n] : make_float2(-kNegInf, 0.f);
        }
        staged();
        __syncthreads();
        if (!mine) continue;
        int cols = min(kT, a.Nq - q0), since = 0;
        if constexpr (BAND) {       // the queries that attend one of the warp's 16 keys
            const int k = k0 + 16 * ln.w;
            since = max(0, k - p0 - q0);
            if (k >= a.band.sinks) cols = min(cols, k + 15 + a.band.window - p0 - q0);
        }
        float p[8][4], ds[8][4];
        nt<1>(p, sk, sq, ln, cols, since);
        nt<1>(ds, sv, sg, ln, cols, since);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float4 st = *reinterpret_cast<const float4 *>(sst + ln.col(j, 0));     // of both columns
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float lse = i & 1 ? st.z : st.x, d = i & 1 ? st.w : st.y;
                bool on = in[i >> 1];
                if constexpr (BAND) on = on && a.band.sees(p0 + q0 + ln.col(j, i & 1), k0 + ln.row(i >> 1));
                p[j][i] = on ? exp2f(fmaf(p[j][i], scale_log2, -lse)) : 0.f;
                ds[j][i] = on ? p[j][i] * (ds[j][i] - d) : 0.f;
            }
        }
        nn(av, p, sg, ln, cols, since);
        nn(ak, ds, sq, ln, cols, since);
    }
    // keys that are not attended have no gradient, whatever the rows that others' weights are for hold (0 times a NaN)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (in[i]) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) ak[j][2 * i] = ak[j][2 * i + 1] = av[j][2 * i] = av[j][2 * i + 1] = 0.f;
    }
    finish(av, sg, a.dV, b, hk, k0, a.ks.Nk, 1.f, ln);
    finish(ak, sq, a.dK, b, hk, k0, a.ks.Nk, a.scale, ln);
}

// Both kinds of unit in one launch, those that hold keys first.
template <bool BAND>
__global__ void __launch_bounds__(kThreads, kBwdBlocks) cross_bwd_f32_kernel(const __grid_constant__ BwdF32Args a) {
    extern __shared__ float4 smem4[];
    __shared__ __align__(16) float2 sst[kT];
    float *smem = reinterpret_cast<float *>(smem4);
    grid_dep_wait();
    const int unit = a.first + (int)(blockIdx.x >> (__ffs(cluster_size()) - 1));
    if (!FIBATT_CHECKED(unit < a.units)) return;    // whole clusters
    if (unit < a.key_units) hold_keys<BAND>(a, smem, sst, unit);
    else hold_queries<BAND>(a, smem, unit - a.key_units);
}

// The largest cluster of this kernel: 16 CTAs where the current device takes them, else 8.
template <auto Kernel>
int largest_cluster(size_t smem) {
    static PerDevice known;
    return known.get(current_device(), [=] { return clusters_held<Kernel>(16, kThreads, smem) > 0 ? 16 : 8; });
}

// Key tiles that a query tile walks over, at most.
template <bool BAND>
int64_t key_tiles(const CrossArgs &a) {
    const int64_t all = (a.Nk + kT - 1) / kT;
    return BAND ? std::min<int64_t>(all, ((int64_t)a.band.window + kT) / kT + 1 + (a.band.sinks + kT - 1) / kT) : all;
}

template <bool BAND>
cudaError_t fwd(const CrossArgs &a) {
    constexpr size_t smem = 3 * kTile * sizeof(float);
    const cudaError_t e = prepare_kernel<cross_fwd_f32_kernel<BAND>>(smem, 0);
    if (e != cudaSuccess) return e;
    const int qtiles = (a.Nq + kT - 1) / kT;
    const int64_t units = (int64_t)a.B * a.Hq * qtiles;
    // (one head, 100 queries on 16385 keys: clusters of 16 85 us, of 8 161)
    const int c = cluster_for(units, key_tiles<BAND>(a), kFwdBlocks * sm_count(), largest_cluster<cross_fwd_f32_kernel<BAND>>(smem));
    return launch_clusters(cross_fwd_f32_kernel<BAND>, (unsigned)(units * c), c, kThreads, smem, a.stream, a.Hq, a.Nq,
                           a.keys, a.band, rows_of<const float>(a.Q), rows_of<const float>(a.K), rows_of<const float>(a.V),
                           rows_of<float>(a.O), a.LSE, a.scale * kLog2e, Div((uint32_t)qtiles), Div((uint32_t)a.Hq),
                           Div((uint32_t)(a.Hq / a.Hkv)), (int)units);
}

template <bool BAND>
cudaError_t bwd(const CrossArgs &a) {
    constexpr size_t smem = 4 * kTile * sizeof(float);
    cudaError_t e = prepare_kernel<cross_bwd_f32_kernel<BAND>>(smem, 0);
    if (e != cudaSuccess) return e;
    BwdF32Args f;
    f.Hq = a.Hq, f.Nq = a.Nq;
    f.ks = a.keys;
    f.band = a.band;
    f.Q = rows_of<const float>(a.Q), f.K = rows_of<const float>(a.K), f.V = rows_of<const float>(a.V);
    f.dO = rows_of<const float>(a.dO);
    f.stats = a.stats;
    f.dQ = rows_of<float>(a.dQ), f.dK = rows_of<float>(a.dK), f.dV = rows_of<float>(a.dV);
    f.scale = a.scale;
    const int ktiles = (a.Nk + kT - 1) / kT;
    f.qtiles = (a.Nq + kT - 1) / kT;
    f.by_qtiles = Div((uint32_t)f.qtiles), f.by_ktiles = Div((uint32_t)ktiles), f.by_hq = Div((uint32_t)a.Hq);
    f.by_hkv = Div((uint32_t)a.Hkv), f.by_group = Div((uint32_t)(a.Hq / a.Hkv));
    const int64_t rows = (int64_t)a.B * a.Hq * a.Nq;
    e = launch_clusters(cross_stats_kernel, (unsigned)((rows + 15) / 16), 1, 256, 0, a.stream, f.by_hq, Div((uint32_t)a.Nq), rows,
                        rows_of<const float>(a.O), f.dO, static_cast<const float *>(a.LSE), a.stats);
    if (e != cudaSuccess) return e;
    const int64_t key_units = (int64_t)a.B * a.Hkv * ktiles, query_units = (int64_t)a.B * a.Hq * f.qtiles;
    f.key_units = (int)key_units;
    f.units = (int)(key_units + query_units);
    f.first = 0;
    // (one head, 100 queries on 16385 keys: 147 us in two launches, 275 with clusters of 8
    // at most, 1937 in one)
    int64_t key_walk = f.qtiles;
    if (BAND && a.band.sinks == 0) key_walk = std::min<int64_t>(key_walk, ((int64_t)a.band.window + kT) / kT + 1);
    const Launches l(query_units, key_tiles<BAND>(a), key_units, (a.Hq / a.Hkv) * key_walk, kBwdBlocks * sm_count(), 1,
                     2, largest_cluster<cross_bwd_f32_kernel<BAND>>(smem));
    if (!l.two) {
        int c = l.c;
        if constexpr (BAND) {
            // Walks differ (a tile with sinks meets every later query): cut over more CTAs than find a place
            // at once, while that ends the longest before all of them, in tiles, with 1.3 for a CTA (its held
            // rows, the join).  (us with clusters of 1, 2, 4, 8, - the one taken -: 4 sequences, 12 heads, 197 tokens,
            // window 65, 1 sink 51, -41-, 55, 112; 4, 4 heads, 246, all keys 53, 35, -30-, 59; 8, 16 heads on 8, 495, window
            // 53 -142-, 161, 261, 554; 8, 12 heads on 4, 600, window 128, 4 sinks 461, -329-, 309, 523.  Over 25 forms 4.5% off
            // the best in the mean; with a quarter for a CTA 21%.)
            const int64_t group = a.Hq / a.Hkv, query_walk = key_tiles<BAND>(a),
                          others = group * std::min<int64_t>(f.qtiles, ((int64_t)a.band.window + kT) / kT + 1),
                          longest = std::max(query_walk, a.band.sinks ? group * f.qtiles : others),
                          all = (query_units * query_walk + key_units * others) * 3 / 4;
            const auto time = [&](int n) {
                return std::max<double>((double)longest / n + 1, (all + 1.3 * (double)(query_units + key_units) * n) / (kBwdBlocks * sm_count()));
            };
            while (c < 8 && time(2 * c) < time(c)) c *= 2;
        }
        return launch_clusters(cross_bwd_f32_kernel<BAND>, (unsigned)((key_units + query_units) * c), c, kThreads, smem,
                               a.stream, f);
    }
    e = launch_clusters(cross_bwd_f32_kernel<BAND>, (unsigned)(key_units * l.c_key), l.c_key, kThreads, smem, a.stream, f);
    if (e != cudaSuccess) return e;
    f.first = f.key_units;
    return launch_clusters(cross_bwd_f32_kernel<BAND>, (unsigned)(query_units * l.c_query), l.c_query, kThreads, smem, a.stream, f);
}

}  // namespace

cudaError_t launch_cross_fwd_f32(const CrossArgs &a) { return a.banded ? fwd<true>(a) : fwd<false>(a); }
cudaError_t launch_cross_bwd_f32(const CrossArgs &a) { return a.banded ? bwd<true>(a) : bwd<false>(a); }

FIBATT_DEFINE_ERROR_READER(read_error_cross_f32, "cross_f32.cu")

}  // namespace fibatt
