// Cross attention forward for a few query rows (a token being decoded, or a
// handful): at most kMaxRows rows read one key/value head, and the time is that
// of reading its keys and values once.
//
// A cluster of CTAs takes one key/value head of one sequence, a CTA a contiguous
// part of its keys, a warp every eighth group of 4 U keys of the part.  Eight
// lanes share a key (16 or 32 bytes of it each), hold the query rows' dims in
// registers, and form one score per row with three shuffles; a group of
// eight lanes keeps the running maximum, sum and weighted values of its own keys, so
// nothing is exchanged until the end: the groups of a warp are joined with
// shuffles, the warps in shared memory, the CTAs through distributed shared
// memory, always in the same order.  A warp has 2 U loads of 512 bytes (16-bit; 1 KB
// 32-bit) in flight.
#include <algorithm>

#include "cluster.cuh"
#include "cross.h"
#include "device_common.cuh"
#include "row_math.cuh"

namespace fibatt {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr float kNegInf = -__builtin_inff();

// Eight consecutive values of a row: one lane's share.
template <typename T>
struct Share;
template <>
struct Share<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float2 (&x)[4]) const {
        x[0] = make_float2(bf16_lo(w.x), bf16_hi(w.x));
        x[1] = make_float2(bf16_lo(w.y), bf16_hi(w.y));
        x[2] = make_float2(bf16_lo(w.z), bf16_hi(w.z));
        x[3] = make_float2(bf16_lo(w.w), bf16_hi(w.w));
    }
    __device__ __forceinline__ float dot(const Share &o) const {
        return dot2_bf16(w.x, o.w.x, dot2_bf16(w.y, o.w.y, 0.f)) + dot2_bf16(w.z, o.w.z, dot2_bf16(w.w, o.w.w, 0.f));
    }
};
template <>
struct Share<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = __ldg(reinterpret_cast<const float4 *>(p));
        b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float2 (&x)[4]) const {
        x[0] = make_float2(a.x, a.y), x[1] = make_float2(a.z, a.w);
        x[2] = make_float2(b.x, b.y), x[3] = make_float2(b.z, b.w);
    }
    __device__ __forceinline__ float dot(const Share &o) const {
        float2 s = mul2(make_float2(a.x, a.y), make_float2(o.a.x, o.a.y));
        s = fma2(make_float2(a.z, a.w), make_float2(o.a.z, o.a.w), s);
        s = fma2(make_float2(b.x, b.y), make_float2(o.b.x, o.b.y), s);
        s = fma2(make_float2(b.z, b.w), make_float2(o.b.z, o.b.w), s);
        return s.x + s.y;
    }
};

__device__ __forceinline__ void store2(__nv_bfloat16 *p, float2 v) {
    *reinterpret_cast<uint32_t *>(p) = pack_bf16x2(v.x, v.y);
}
__device__ __forceinline__ void store2(float *p, float2 v) { *reinterpret_cast<float2 *>(p) = v; }

// R rows (the last ones may be copies of the last real row); U keys a lane group.
template <typename T, int R, int U>
__global__ void __launch_bounds__(kThreads)
cross_rows_kernel(int Hq, int Hkv, int Nq, int rows, KeySet ks, Rows<const T> Q, Rows<const T> K, Rows<const T> V,
                  Rows<T> O, float *__restrict__ LSE, float c) {
    __shared__ float sm[kWarps][R], sl[kWarps][R];
    __shared__ float2 so[kWarps][R][32];
    __shared__ float cm[R], cl[R];            // the CTA's, read by the cluster
    __shared__ float2 co[R][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & 7, grp = lane >> 3;
    const int C = (int)cluster_size(), rank = (int)cluster_rank();
    const int unit = blockIdx.x / C, hk = unit % Hkv, b = unit / Hkv;
    const int G = Hq / Hkv;

    grid_dep_wait();
    grid_dep_launch();
    const int bound = ks.bound(b);
    const int per = ((bound + C - 1) / C + 4 * U - 1) / (4 * U) * (4 * U);   // keys of a CTA
    const int lo = (int)min((int64_t)bound, (int64_t)per * rank), hi = min(bound, lo + per);
    Share<T> q[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = min(r, rows - 1);
        q[r].load(Q.row(b, hk * G + i / Nq, i % Nq) + 8 * sub);
    }
    float m[R], l[R];
    float2 acc[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r] = kNegInf;
        l[r] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][i] = make_float2(0.f, 0.f);
    }
    const T *kp = K.row(b, hk, 0) + 8 * sub, *vp = V.row(b, hk, 0) + 8 * sub;
    for (int k0 = lo + warp * 4 * U; k0 < hi; k0 += kWarps * 4 * U) {
        Share<T> k[U], v[U];
        bool in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = k0 + 4 * u + grp;
            in[u] = at < hi;
            const int64_t off = min(at, hi - 1);
            k[u].load(kp + off * K.sn);
            v[u].load(vp + off * V.sn);
        }
        if (ks.mask)
#pragma unroll
            for (int u = 0; u < U; ++u) in[u] = in[u] && ks.has(b, min(k0 + 4 * u + grp, hi - 1));
        float s[R][U];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < R; ++r) s[r][u] = q[r].dot(k[u]);
#pragma unroll
        for (int x = 1; x < 8; x <<= 1)
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int r = 0; r < R; ++r) s[r][u] += __shfl_xor_sync(kFullMask, s[r][u], x);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float top = kNegInf;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s[r][u] = in[u] ? s[r][u] * c : kNegInf;
                top = fmaxf(top, s[r][u]);
            }
            if (top > m[r]) {
                const float keep = fast_exp2(m[r] - top);
                m[r] = top;
                l[r] *= keep;
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[r][i] = mul2(acc[r][i], make_float2(keep, keep));
            }
            const float base = m[r] == kNegInf ? 0.f : m[r];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s[r][u] = fast_exp2(s[r][u] - base);
                l[r] += s[r][u];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!in[u]) v[u].zero();      // a weight of 0 meets no NaN
            float2 x[4];
            v[u].get(x);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[r][i] = fma2(make_float2(s[r][u], s[r][u]), x[i], acc[r][i]);
        }
    }
    // the four groups of the warp, then the warps, then the CTAs
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float top = fmaxf(m[r], __shfl_xor_sync(kFullMask, m[r], 8));
        top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 16));
        const float w = fast_exp2(m[r] - (top == kNegInf ? 0.f : top));
        l[r] *= w;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][i] = mul2(acc[r][i], make_float2(w, w));
#pragma unroll
        for (int x = 8; x < 32; x <<= 1) {
            l[r] += __shfl_xor_sync(kFullMask, l[r], x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[r][i].x += __shfl_xor_sync(kFullMask, acc[r][i].x, x);
                acc[r][i].y += __shfl_xor_sync(kFullMask, acc[r][i].y, x);
            }
        }
        if (lane < 8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) so[warp][r][4 * sub + i] = acc[r][i];
            if (lane == 0) {
                sm[warp][r] = top;
                sl[warp][r] = l[r];
            }
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
        float2 o = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = fast_exp2(sm[w][r] - base);
            sum = fmaf(f, sl[w][r], sum);
            o = fma2(make_float2(f, f), so[w][r][d], o);
        }
        co[r][d] = o;
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
        float2 o = make_float2(0.f, 0.f);
        for (int k = 0; k < C; ++k) {
            const float f = fast_exp2(ld_cluster(cluster_addr(cm + r, k)) - base);
            sum = fmaf(f, ld_cluster(cluster_addr(cl + r, k)), sum);
            o = fma2(make_float2(f, f), ld_cluster2(cluster_addr(&co[r][d], k)), o);
        }
        const int h = hk * G + r / Nq, n = r % Nq;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        store2(O.row(b, h, n) + 2 * d, make_float2(o.x * inv, o.y * inv));
        if (d == 0) LSE[((int64_t)b * Hq + h) * Nq + n] = sum == 0.f ? kNegInf : (top + log2f(sum)) * kLn2;
    }
    cluster_sync();   // the others may still read this CTA's part
}

template <typename T, int R, int U>
cudaError_t run(const CrossArgs &a, int rows) {
    const int64_t units = (int64_t)a.B * a.Hkv;
    // CTAs of a cluster: until the GPU has six a SM, as long as a CTA keeps one
    // round of its warps
    int c = 1;
    while (c < 8 && units * c < 6 * sm_count() && a.Nk > 2 * c * kWarps * 4 * U) c *= 2;
    return launch_clusters(cross_rows_kernel<T, R, U>, (unsigned)(units * c), c, kThreads, 0, a.stream, a.Hq, a.Hkv,
                           a.Nq, rows, a.keys, rows_of<const T>(a.Q), rows_of<const T>(a.K), rows_of<const T>(a.V),
                           rows_of<T>(a.O), a.LSE, a.scale * kLog2e);
}

}  // namespace

bool cross_rows_takes(const CrossArgs &a) {
    const int64_t rows = (int64_t)(a.Hq / a.Hkv) * a.Nq;
    return rows <= (a.dtype == FIBATT_F32 ? 8 : 4) && (int64_t)a.B * a.Hkv < 0x7fffffff / 8;
}

cudaError_t launch_cross_rows(const CrossArgs &a) {
    const int rows = a.Hq / a.Hkv * a.Nq;
    if (a.dtype == FIBATT_F32)
        return rows == 1   ? run<float, 1, 4>(a, rows)
               : rows == 2 ? run<float, 2, 4>(a, rows)
               : rows <= 4 ? run<float, 4, 4>(a, rows)
                           : run<float, 8, 2>(a, rows);
    return rows == 1   ? run<__nv_bfloat16, 1, 4>(a, rows)
           : rows == 2 ? run<__nv_bfloat16, 2, 4>(a, rows)
                       : run<__nv_bfloat16, 4, 4>(a, rows);
}

FIBATT_DEFINE_ERROR_READER(read_error_cross_rows, "cross_rows.cu")

}  // namespace fibatt
