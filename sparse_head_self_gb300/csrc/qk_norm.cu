// Norms of the query and key heads with the position rotation, from the
// packed projection [B, N, (Hq + Hk + Hv) 64] to Q, K, V [B, H, N, 64] in one
// pass, and the gradient back into the packed layout.
//
// One head's 64 values x with weight w, position angle a (first `rot` dims in
// pairs):
//   r = 1 / sqrt(<x, x> / 64 + eps),  n = r x,  y = w n,
//   (z1, z2) = (y1 cos a - y2 sin a, y1 sin a + y2 cos a)
// and, for the gradient dz:
//   (dy1, dy2) = (dz1 cos a + dz2 sin a, -dz1 sin a + dz2 cos a),
//   dw = sum over rows of dy n,  g = w dy,  dx = r (g - n <g, n> / 64).
//
// Both directions only move data: they read and write each element once, and
// with 16-bit elements the instructions a head takes cost about as much as its
// bytes.  Eight lanes share a head, a lane has two runs of four dims, chosen so
// that both values of every rotated pair are its own (halves: dims 4 i.. and
// rot / 2 + 4 i..), which leaves the two sums over a head as the only exchange;
// the arithmetic is on packed pairs of floats.  A warp takes four heads of one
// token per step, kSteps steps at once, and the next ones' loads are in flight
// while these are worked on; a token's angles are loaded once for its heads.
// Every head row is a whole 128- or 256-byte segment, so all traffic is full
// sectors.  The values' heads are copied unconverted.
//
// dw: each lane keeps sums of its eight dims, the block joins its warps in
// shared memory, and a second kernel adds the blocks' sums in block order:
// no atomics, the same result on every run.
#include <algorithm>

#include "cross.h"
#include "device_common.cuh"
#include "row_math.cuh"

namespace fibatt {
namespace {

constexpr int kWarps = 8;
constexpr int kSteps = 2;             // head groups of four that a warp loads at once
constexpr int kMaxBlocks = 1024;      // rows of the dw partial sums
constexpr unsigned kErrPosition = 8u; // a position at or behind the end of the tables

// A lane's eight dims of a head: runs of four at a0 and a1 (elements).
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
    uint2 u, v;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, int a0, int a1) {
        u = __ldg(reinterpret_cast<const uint2 *>(p + a0));
        v = __ldg(reinterpret_cast<const uint2 *>(p + a1));
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p, int a0, int a1) const {
        *reinterpret_cast<uint2 *>(p + a0) = u;
        *reinterpret_cast<uint2 *>(p + a1) = v;
    }
    __device__ __forceinline__ void zero() { u = v = make_uint2(0, 0); }
    __device__ __forceinline__ void get(float2 (&x)[4]) const {
        x[0] = make_float2(bf16_lo(u.x), bf16_hi(u.x));
        x[1] = make_float2(bf16_lo(u.y), bf16_hi(u.y));
        x[2] = make_float2(bf16_lo(v.x), bf16_hi(v.x));
        x[3] = make_float2(bf16_lo(v.y), bf16_hi(v.y));
    }
    __device__ __forceinline__ void put(const float2 (&x)[4]) {   // the only rounding of a result
        u = make_uint2(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y));
        v = make_uint2(pack_bf16x2(x[2].x, x[2].y), pack_bf16x2(x[3].x, x[3].y));
    }
};
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p, int a0, int a1) {
        a = __ldg(reinterpret_cast<const float4 *>(p + a0));
        b = __ldg(reinterpret_cast<const float4 *>(p + a1));
    }
    __device__ __forceinline__ void store(float *p, int a0, int a1) const {
        *reinterpret_cast<float4 *>(p + a0) = a;
        *reinterpret_cast<float4 *>(p + a1) = b;
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float2 (&x)[4]) const {
        x[0] = make_float2(a.x, a.y), x[1] = make_float2(a.z, a.w);
        x[2] = make_float2(b.x, b.y), x[3] = make_float2(b.z, b.w);
    }
    __device__ __forceinline__ void put(const float2 (&x)[4]) {
        a = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
        b = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
    }
};

// What a kernel needs besides its tensors (see QkNormArgs).
template <typename T>
struct NormArgs {
    int N, Hq, Hk, Hv;
    const T *wq, *wk;
    float eps;
    int rot;
    const float *cos, *sin;
    int P;
    const int32_t *pos;
    int64_t pos_sb;
};

// Where lane `sub` of a head has its two runs of four dims.
template <bool PAIRS_INSIDE>
__device__ __forceinline__ void lane_dims(int rot, int sub, int &a0, int &a1) {
    const bool split = !PAIRS_INSIDE && 8 * sub < rot;
    a0 = split ? 4 * sub : 8 * sub;
    a1 = split ? rot / 2 + 4 * sub : 8 * sub + 4;
}

// The angles of one token for a lane's four pairs: value i of the first run
// and of the second (halves), or neighbours (PAIRS_INSIDE).
template <bool PAIRS_INSIDE>
struct Turn {
    float c[4], s[4];

    template <typename T>
    __device__ __forceinline__ void load(const NormArgs<T> &a, int64_t b, int n, int sub) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i] = 1.f;
            s[i] = 0.f;
        }
        if (8 * sub >= a.rot) return;
        const int p = a.pos ? __ldg(a.pos + b * a.pos_sb + n) : n;
        if (p < 0) return;         // not rotated
        if (p >= a.P) {
            atomicOr(&g_device_error, kErrPosition);
            return;
        }
        const int64_t at = (int64_t)p * (a.rot / 2) + 4 * sub;
        const float4 vc = __ldg(reinterpret_cast<const float4 *>(a.cos + at));
        const float4 vs = __ldg(reinterpret_cast<const float4 *>(a.sin + at));
        c[0] = vc.x, c[1] = vc.y, c[2] = vc.z, c[3] = vc.w;
        s[0] = vs.x, s[1] = vs.y, s[2] = vs.z, s[3] = vs.w;
    }
    // BACK: by minus the angle
    template <bool BACK>
    __device__ __forceinline__ void apply(float2 (&y)[4]) const {
        if (PAIRS_INSIDE) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float t = BACK ? -s[i] : s[i];
                y[i] = fma2(y[i], make_float2(c[i], c[i]), mul2(make_float2(y[i].y, y[i].x), make_float2(-t, t)));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 cc = make_float2(c[2 * i], c[2 * i + 1]);
                const float2 ss = make_float2(BACK ? -s[2 * i] : s[2 * i], BACK ? -s[2 * i + 1] : s[2 * i + 1]);
                const float2 u = y[i], v = y[2 + i];
                y[i] = fma2(u, cc, mul2(v, make_float2(-ss.x, -ss.y)));
                y[2 + i] = fma2(v, cc, mul2(u, ss));
            }
        }
    }
};

__device__ __forceinline__ float sum8(float x) {   // over the eight lanes of a head
    x += __shfl_xor_sync(kFullMask, x, 1);
    x += __shfl_xor_sync(kFullMask, x, 2);
    return x + __shfl_xor_sync(kFullMask, x, 4);
}

// wq and wk as floats in shared memory (ones where there is none).
template <typename T>
__device__ __forceinline__ void stage_weights(const NormArgs<T> &a, float (*sw)[64]) {
    if (threadIdx.x < 128) {
        const T *w = threadIdx.x < 64 ? a.wq : a.wk;
        sw[threadIdx.x >> 6][threadIdx.x & 63] = w ? (float)w[threadIdx.x & 63] : 1.f;
    }
    __syncthreads();
}

// The head groups (four heads) that a warp works through: those of one token
// after another, kSteps at a time; a token's groups are shared by `chunks`
// warps where there are fewer tokens than warps.
struct Walk {
    int64_t u, units, step;
    int N, chunks, groups;
    int64_t b;
    int n, g, end;         // token and groups [g, end) left of it
    bool first;            // at the first groups of its part
    __device__ __forceinline__ Walk(int64_t u, int64_t units, int64_t step, int N, int chunks, int groups)
        : u(u), units(units), step(step), N(N), chunks(chunks), groups(groups) {
        enter();
    }
    __device__ __forceinline__ bool left() const { return u < units; }
    __device__ __forceinline__ void enter() {
        const int64_t token = u / chunks;
        const int c = (int)(u - token * chunks);
        b = token / N;
        n = (int)(token - b * N);
        g = (int)((int64_t)groups * c / chunks);
        end = (int)((int64_t)groups * (c + 1) / chunks);
        first = true;
    }
    __device__ __forceinline__ void next() {
        first = false;
        g += kSteps;
        if (g < end) return;
        u += step;
        if (left()) enter();
    }
};

// A token's rows within Q, K and V (dense).
template <typename T>
struct HeadRows {
    T *q, *k, *v;
    __device__ __forceinline__ void token(T *Q, T *K, T *V, int Hq, int Hk, int Hv, int64_t b, int n, int N) {
        q = Q + (b * Hq * N + n) * 64;
        k = K + (b * Hk * N + n) * 64;
        v = V + (b * Hv * N + n) * 64;
    }
    __device__ __forceinline__ T *row(int h, int Hq, int Hn, int N) const {
        T *p = h < Hq ? q : h < Hn ? k : v;
        const int i = h < Hq ? h : h < Hn ? h - Hq : h - Hn;
        return p + (int64_t)i * N * 64;
    }
};

__device__ __forceinline__ float squares(const float2 (&x)[4]) {
    float2 s = mul2(x[0], x[0]);
#pragma unroll
    for (int e = 1; e < 4; ++e) s = fma2(x[e], x[e], s);
    return s.x + s.y;
}
__device__ __forceinline__ void weights(const float *sw, int a0, int a1, float2 (&w)[4]) {
    const float4 u = *reinterpret_cast<const float4 *>(sw + a0), v = *reinterpret_cast<const float4 *>(sw + a1);
    w[0] = make_float2(u.x, u.y), w[1] = make_float2(u.z, u.w);
    w[2] = make_float2(v.x, v.y), w[3] = make_float2(v.z, v.w);
}

template <typename T, bool PAIRS_INSIDE>
__global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 2 ? 4 : 3)
qk_norm_fwd_kernel(const __grid_constant__ NormArgs<T> a, const T *__restrict__ X, int64_t x_sb, int64_t x_sn,
                   T *__restrict__ Q, T *__restrict__ K, T *__restrict__ V, int64_t units, int chunks) {
    __shared__ __align__(16) float sw[2][64];
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31, sub = lane & 7, grp = lane >> 3;
    const int Hn = a.Hq + a.Hk, H = Hn + a.Hv;
    int a0, a1;
    lane_dims<PAIRS_INSIDE>(a.rot, sub, a0, a1);
    Walk t((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), units, (int64_t)gridDim.x * kWarps, a.N, chunks,
           (H + 3) / 4);
    Eight<T> raw[kSteps], ahead[kSteps];
    const auto load = [&](Eight<T> (&r)[kSteps]) {
        const T *row = X + t.b * x_sb + t.n * x_sn;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int h = 4 * (t.g + i) + grp;
            if (t.g + i < t.end && h < H) r[i].load(row + h * 64, a0, a1);
            else r[i].zero();
        }
    };
    if (t.left()) load(raw);
    stage_weights(a, sw);
    Turn<PAIRS_INSIDE> turn;
    HeadRows<T> out;
    while (t.left()) {
        if (t.first) {
            turn.load(a, t.b, t.n, sub);
            out.token(Q, K, V, a.Hq, a.Hk, a.Hv, t.b, t.n, a.N);
        }
        const int g0 = t.g, end = t.end;
        const HeadRows<T> to = out;
        t.next();
        if (t.left()) load(ahead);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int g = g0 + i, h = 4 * g + grp;
            if (g >= end) break;
            if (4 * g < Hn) {   // some head of the group is a query or a key
                float2 x[4];
                raw[i].get(x);
                const bool isq = h < a.Hq;
                const float r = (isq ? a.wq : a.wk) ? rsqrtf(sum8(squares(x)) * (1.f / 64.f) + a.eps) : 1.f;
                float2 w[4];
                weights(sw[isq ? 0 : 1], a0, a1, w);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = mul2(x[e], mul2(w[e], make_float2(r, r)));
                turn.template apply<false>(x);
                if (h < Hn) raw[i].put(x);
            }
            if (h < H) raw[i].store(to.row(h, a.Hq, Hn, a.N), a0, a1);
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) raw[i] = ahead[i];
    }
}

template <typename T, bool PAIRS_INSIDE>
__global__ void __launch_bounds__(kWarps * 32, 2)
qk_norm_bwd_kernel(const __grid_constant__ NormArgs<T> a, const T *__restrict__ X, int64_t x_sb, int64_t x_sn,
                   const T *__restrict__ dQ, const T *__restrict__ dK, const T *__restrict__ dV, T *__restrict__ dX,
                   int64_t dx_sb, int64_t dx_sn, float *__restrict__ partial, int64_t units, int chunks) {
    __shared__ __align__(16) float sw[2][64];
    __shared__ float part[kWarps][128];
    grid_dep_wait();
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & 7, grp = lane >> 3;
    const int Hn = a.Hq + a.Hk, H = Hn + a.Hv;
    int a0, a1;
    lane_dims<PAIRS_INSIDE>(a.rot, sub, a0, a1);
    float2 dwq[4], dwk[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) dwq[e] = dwk[e] = make_float2(0.f, 0.f);
    Walk t((int64_t)blockIdx.x * kWarps + warp, units, (int64_t)gridDim.x * kWarps, a.N, chunks, (H + 3) / 4);
    Eight<T> raw[kSteps], grad[kSteps], raw_ahead[kSteps], grad_ahead[kSteps];
    const auto load = [&](Eight<T> (&r)[kSteps], Eight<T> (&d)[kSteps]) {
        const T *row = X + t.b * x_sb + t.n * x_sn;
        HeadRows<const T> from;
        from.token(dQ, dK, dV, a.Hq, a.Hk, a.Hv, t.b, t.n, a.N);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int h = 4 * (t.g + i) + grp;
            r[i].zero();
            d[i].zero();
            if (t.g + i < t.end && h < H) {
                if (h < Hn) r[i].load(row + h * 64, a0, a1);
                d[i].load(from.row(h, a.Hq, Hn, a.N), a0, a1);
            }
        }
    };
    if (t.left()) load(raw, grad);
    stage_weights(a, sw);
    Turn<PAIRS_INSIDE> turn;
    while (t.left()) {
        if (t.first) turn.load(a, t.b, t.n, sub);
        T *drow = dX + t.b * dx_sb + t.n * dx_sn;
        const int g0 = t.g, end = t.end;
        t.next();
        if (t.left()) load(raw_ahead, grad_ahead);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int g = g0 + i, h = 4 * g + grp;
            if (g >= end) break;
            if (4 * g < Hn) {
                float2 x[4], dy[4], w[4];
                raw[i].get(x);
                grad[i].get(dy);
                const bool isq = h < a.Hq, isk = !isq && h < Hn;
                turn.template apply<true>(dy);
                const bool norm = (isq ? a.wq : a.wk) != nullptr;
                const float r = norm ? rsqrtf(sum8(squares(x)) * (1.f / 64.f) + a.eps) : 1.f;
                weights(sw[isq ? 0 : 1], a0, a1, w);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = mul2(x[e], make_float2(r, r));
                if (4 * g + 4 <= a.Hq) {            // four queries
#pragma unroll
                    for (int e = 0; e < 4; ++e) dwq[e] = fma2(dy[e], x[e], dwq[e]);
                } else if (4 * g >= a.Hq && 4 * g + 4 <= Hn) {     // four keys
#pragma unroll
                    for (int e = 0; e < 4; ++e) dwk[e] = fma2(dy[e], x[e], dwk[e]);
                } else {
                    // selected, not multiplied by 0: another kind's NaN stays out
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 d = mul2(dy[e], x[e]);
                        dwq[e] = add2(dwq[e], make_float2(isq ? d.x : 0.f, isq ? d.y : 0.f));
                        dwk[e] = add2(dwk[e], make_float2(isk ? d.x : 0.f, isk ? d.y : 0.f));
                    }
                }
                float2 dot = make_float2(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    dy[e] = mul2(dy[e], w[e]);
                    dot = fma2(dy[e], x[e], dot);
                }
                const float m = sum8(dot.x + dot.y) * (norm ? -1.f / 64.f : 0.f);
#pragma unroll
                for (int e = 0; e < 4; ++e) dy[e] = mul2(make_float2(r, r), fma2(x[e], make_float2(m, m), dy[e]));
                if (h < Hn) grad[i].put(dy);
            }
            if (h < H) grad[i].store(drow + h * 64, a0, a1);
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            raw[i] = raw_ahead[i];
            grad[i] = grad_ahead[i];
        }
    }
    // the block's sums: over the four heads of a warp, then over its warps
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int m = 8; m < 32; m <<= 1) {
            dwq[e].x += __shfl_xor_sync(kFullMask, dwq[e].x, m);
            dwq[e].y += __shfl_xor_sync(kFullMask, dwq[e].y, m);
            dwk[e].x += __shfl_xor_sync(kFullMask, dwk[e].x, m);
            dwk[e].y += __shfl_xor_sync(kFullMask, dwk[e].y, m);
        }
        if (lane < 8) {
            const int d = (e < 2 ? a0 : a1) + 2 * (e & 1);
            part[warp][d] = dwq[e].x;
            part[warp][d + 1] = dwq[e].y;
            part[warp][64 + d] = dwk[e].x;
            part[warp][64 + d + 1] = dwk[e].y;
        }
    }
    __syncthreads();
    if (threadIdx.x < 128) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += part[w][threadIdx.x];
        partial[(int64_t)blockIdx.x * 128 + threadIdx.x] = s;
    }
}

// dw from the blocks' sums: eight threads a column, each over every eighth
// block, joined in thread order.
template <typename T>
__global__ void __launch_bounds__(1024) qk_norm_dw_kernel(const float *__restrict__ partial, int blocks,
                                                          T *__restrict__ dwq, T *__restrict__ dwk) {
    __shared__ float part[8][128];
    grid_dep_wait();
    const int c = threadIdx.x & 127, k = threadIdx.x >> 7;
    float s = 0.f;
    for (int b = k; b < blocks; b += 8) s += partial[(int64_t)b * 128 + c];
    part[k][c] = s;
    __syncthreads();
    if (k) return;
#pragma unroll
    for (int i = 1; i < 8; ++i) s += part[i][c];
    T *out = c < 64 ? dwq : dwk;
    if (out) out[c & 63] = (T)s;
}

// One wave of blocks, each warp walking over its tokens: the next groups are
// loaded while these are worked on.  Fewer tokens than warps: a token's
// groups are cut into chunks of at least kSteps.
template <auto Kernel>
int resident_blocks() {
    static std::atomic<int> per_sm{0};
    int n = per_sm.load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, Kernel, kWarps * 32, 0) != cudaSuccess || n < 1) n = 1;
        per_sm.store(n, std::memory_order_relaxed);
    }
    return std::min(kMaxBlocks, n * sm_count());
}

struct Grid {
    int chunks;
    int64_t units;
    unsigned blocks;
    Grid(const QkNormArgs &q, int resident) {
        const int groups = (q.Hq + q.Hk + q.Hv + 3) / 4, most = (groups + kSteps - 1) / kSteps;
        const int64_t tokens = (int64_t)q.B * q.N, warps = (int64_t)resident * kWarps;
        chunks = (int)std::min<int64_t>(most, std::max<int64_t>(1, (warps + tokens - 1) / tokens));
        units = tokens * chunks;
        blocks = (unsigned)std::min<int64_t>((units + kWarps - 1) / kWarps, resident);
    }
};

template <typename T>
NormArgs<T> norm_args(const QkNormArgs &q) {
    return NormArgs<T>{q.N,   q.Hq,  q.Hk,  q.Hv, static_cast<const T *>(q.wq), static_cast<const T *>(q.wk), q.eps,
                       q.rot, q.cos, q.sin, q.P,  q.pos,                        q.pos_sb};
}

template <typename T, bool PAIRS_INSIDE>
cudaError_t fwd(const QkNormArgs &q) {
    const Grid g(q, resident_blocks<qk_norm_fwd_kernel<T, PAIRS_INSIDE>>());
    const cudaError_t e = launch_kernel(qk_norm_fwd_kernel<T, PAIRS_INSIDE>, dim3(g.blocks), dim3(kWarps * 32), 0,
                                        q.stream, pdl_enabled(), norm_args<T>(q), static_cast<const T *>(q.X), q.x_sb,
                                        q.x_sn, static_cast<T *>(q.Q), static_cast<T *>(q.K), static_cast<T *>(q.V),
                                        g.units, g.chunks);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

template <typename T, bool PAIRS_INSIDE>
cudaError_t bwd(const QkNormArgs &q) {
    const Grid g(q, resident_blocks<qk_norm_bwd_kernel<T, PAIRS_INSIDE>>());
    cudaError_t e = launch_kernel(qk_norm_bwd_kernel<T, PAIRS_INSIDE>, dim3(g.blocks), dim3(kWarps * 32), 0, q.stream,
                                  pdl_enabled(), norm_args<T>(q), static_cast<const T *>(q.X), q.x_sb, q.x_sn,
                                  static_cast<const T *>(q.dQ), static_cast<const T *>(q.dK),
                                  static_cast<const T *>(q.dV), static_cast<T *>(q.dX), q.dx_sb, q.dx_sn, q.ws, g.units,
                                  g.chunks);
    if (e != cudaSuccess) return e;
    count_launches(1);
    if (!q.dwq && !q.dwk) return cudaSuccess;
    e = launch_kernel(qk_norm_dw_kernel<T>, dim3(1), dim3(1024), 0, q.stream, pdl_enabled(),
                      static_cast<const float *>(q.ws), (int)g.blocks, static_cast<T *>(q.dwq),
                      static_cast<T *>(q.dwk));
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace

size_t qk_norm_bwd_workspace() { return (size_t)kMaxBlocks * 128 * sizeof(float); }

cudaError_t launch_qk_norm_fwd(const QkNormArgs &q) {
    if (q.interleaved) return q.dtype == FIBATT_F32 ? fwd<float, true>(q) : fwd<__nv_bfloat16, true>(q);
    return q.dtype == FIBATT_F32 ? fwd<float, false>(q) : fwd<__nv_bfloat16, false>(q);
}
cudaError_t launch_qk_norm_bwd(const QkNormArgs &q) {
    if (q.interleaved) return q.dtype == FIBATT_F32 ? bwd<float, true>(q) : bwd<__nv_bfloat16, true>(q);
    return q.dtype == FIBATT_F32 ? bwd<float, false>(q) : bwd<__nv_bfloat16, false>(q);
}

FIBATT_DEFINE_ERROR_READER(read_error_qk_norm, "qk_norm.cu")

}  // namespace fibatt
