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
// Both directions only move data: they read and write each element once.
// Eight lanes share a head (eight dims each), a warp takes four heads of one
// token per step and up to kSteps steps at once, so that a warp has up to
// 2 KB (16-bit) or 4 KB of loads in flight; the token's angles are loaded once
// for its heads.  Token rows of X are contiguous and every head row of Q, K
// and V is a whole 128- or 256-byte segment, so all traffic is full sectors.
// The values' heads are copied unconverted.
//
// dw: each lane keeps sums of its eight dims, the block joins its warps in
// shared memory, and a second kernel adds the blocks' sums in block order:
// no atomics, the same result on every run.
#include <algorithm>

#include "cross.h"
#include "device_common.cuh"

namespace fibatt {
namespace {

constexpr int kWarps = 8;
constexpr int kSteps = 4;             // head groups of four that a warp loads at once
constexpr int kMaxBlocks = 1024;      // rows of the dw partial sums
constexpr unsigned kErrPosition = 8u; // a position at or behind the end of the tables

template <typename T>
struct Eight;   // eight consecutive elements of a lane
template <>
struct Eight<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint4 *>(p) = w; }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(v[i]);
            x[2 * i + 1] = bf16_hi(v[i]);
        }
    }
    __device__ __forceinline__ void put(const float (&x)[8]) {   // the only rounding of a result
        w = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                       pack_bf16x2(x[6], x[7]));
    }
};
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = __ldg(reinterpret_cast<const float4 *>(p));
        b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void store(float *p) const {
        reinterpret_cast<float4 *>(p)[0] = a;
        reinterpret_cast<float4 *>(p)[1] = b;
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    __device__ __forceinline__ void put(const float (&x)[8]) {
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
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

// The angles of one token for a lane's eight dims.  Pairs of halves: dim d
// and d + rot / 2, the partner's values come from lane `peer`; neighbours:
// dims 2 i and 2 i + 1, both in the lane (c[i], s[i] of pair i).
template <bool PAIRS_INSIDE>
struct Turn {
    float c[PAIRS_INSIDE ? 4 : 8], s[PAIRS_INSIDE ? 4 : 8];
    int peer;

    __device__ __forceinline__ void none(int lane) {
#pragma unroll
        for (int i = 0; i < (PAIRS_INSIDE ? 4 : 8); ++i) {
            c[i] = 1.f;
            s[i] = 0.f;
        }
        peer = lane;
    }
    template <typename T>
    __device__ __forceinline__ void load(const NormArgs<T> &a, int64_t b, int n, int lane) {
        none(lane);
        const int sub = lane & 7;
        if (8 * sub >= a.rot) return;
        const int half = a.rot / 2, hl = half / 8;
        int at = PAIRS_INSIDE ? 4 * sub : 8 * sub;
        float sign = 1.f;
        if (!PAIRS_INSIDE) {
            const bool second = sub >= hl;
            peer = second ? lane - hl : lane + hl;
            if (second) at -= half;
            else sign = -1.f;      // z1 = y1 c - y2 s
        }
        const int p = a.pos ? __ldg(a.pos + b * a.pos_sb + n) : n;
        if (p < 0) return;         // not rotated
        if (p >= a.P) {
            atomicOr(&g_device_error, kErrPosition);
            return;
        }
        const float4 *pc = reinterpret_cast<const float4 *>(a.cos + (int64_t)p * half + at);
        const float4 *ps = reinterpret_cast<const float4 *>(a.sin + (int64_t)p * half + at);
#pragma unroll
        for (int i = 0; i < (PAIRS_INSIDE ? 1 : 2); ++i) {
            const float4 vc = __ldg(pc + i), vs = __ldg(ps + i);
            c[4 * i] = vc.x, c[4 * i + 1] = vc.y, c[4 * i + 2] = vc.z, c[4 * i + 3] = vc.w;
            s[4 * i] = sign * vs.x, s[4 * i + 1] = sign * vs.y, s[4 * i + 2] = sign * vs.z, s[4 * i + 3] = sign * vs.w;
        }
    }
    // Every lane of the warp calls it; dir = -1 turns back.
    __device__ __forceinline__ void apply(float (&y)[8], float dir) const {
        if (PAIRS_INSIDE) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u = y[2 * i], v = y[2 * i + 1], t = dir * s[i % (PAIRS_INSIDE ? 4 : 8)];
                y[2 * i] = u * c[i] - v * t;
                y[2 * i + 1] = u * t + v * c[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float o = __shfl_sync(kFullMask, y[i], peer);
                y[i] = y[i] * c[i % (PAIRS_INSIDE ? 4 : 8)] + dir * s[i % (PAIRS_INSIDE ? 4 : 8)] * o;
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

// A unit of a warp: one token, `steps` groups of four heads from group g0.
struct Unit {
    int64_t b;
    int n, g0, steps;
    __device__ __forceinline__ Unit(int64_t u, int N, int chunks, int groups) {
        const int64_t token = u / chunks;
        const int c = (int)(u - token * chunks);
        b = token / N;
        n = (int)(token - b * N);
        g0 = (int)((int64_t)groups * c / chunks);
        steps = (int)((int64_t)groups * (c + 1) / chunks) - g0;
    }
};

template <typename T, bool PAIRS_INSIDE>
__global__ void __launch_bounds__(kWarps * 32)
qk_norm_fwd_kernel(const __grid_constant__ NormArgs<T> a, const T *__restrict__ X, int64_t x_sb, int64_t x_sn,
                   T *__restrict__ Q, T *__restrict__ K, T *__restrict__ V, int64_t units, int chunks) {
    __shared__ float sw[2][64];
    grid_dep_wait();
    stage_weights(a, sw);
    const int lane = threadIdx.x & 31, sub = lane & 7;
    const int H = a.Hq + a.Hk + a.Hv, groups = (H + 3) / 4;
    for (int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += (int64_t)gridDim.x * kWarps) {
        const Unit t(u, a.N, chunks, groups);
        const T *row = X + t.b * x_sb + t.n * x_sn + sub * 8;
        Eight<T> raw[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int h = 4 * (t.g0 + i) + (lane >> 3);
            if (i < t.steps && h < H) raw[i].load(row + (int64_t)h * 64);
            else raw[i].zero();
        }
        Turn<PAIRS_INSIDE> turn;
        turn.load(a, t.b, t.n, lane);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            if (i >= t.steps) break;
            const int g = t.g0 + i, h = 4 * g + (lane >> 3);
            if (4 * g < a.Hq + a.Hk) {   // some head of the group is a query or a key
                float x[8], y[8];
                raw[i].get(x);
                const bool isq = h < a.Hq;
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
                ss = sum8(ss);
                const float r = (isq ? a.wq : a.wk) ? rsqrtf(ss * (1.f / 64.f) + a.eps) : 1.f;
                const float4 *w4 = reinterpret_cast<const float4 *>(sw[isq ? 0 : 1] + sub * 8);
                const float4 wa = w4[0], wb = w4[1];
                const float w[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = x[e] * r * w[e];
                turn.apply(y, 1.f);
                if (h < a.Hq + a.Hk) raw[i].put(y);
            }
            if (h < H) {
                T *out = h < a.Hq          ? Q + ((t.b * a.Hq + h) * a.N + t.n) * 64
                         : h < a.Hq + a.Hk ? K + ((t.b * a.Hk + (h - a.Hq)) * a.N + t.n) * 64
                                           : V + ((t.b * a.Hv + (h - a.Hq - a.Hk)) * a.N + t.n) * 64;
                raw[i].store(out + sub * 8);
            }
        }
    }
}

template <typename T, bool PAIRS_INSIDE>
__global__ void __launch_bounds__(kWarps * 32)
qk_norm_bwd_kernel(const __grid_constant__ NormArgs<T> a, const T *__restrict__ X, int64_t x_sb, int64_t x_sn,
                   const T *__restrict__ dQ, const T *__restrict__ dK, const T *__restrict__ dV, T *__restrict__ dX,
                   int64_t dx_sb, int64_t dx_sn, float *__restrict__ partial, int64_t units, int chunks) {
    __shared__ float sw[2][64];
    __shared__ float part[kWarps][128];
    grid_dep_wait();
    stage_weights(a, sw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & 7;
    const int H = a.Hq + a.Hk + a.Hv, groups = (H + 3) / 4;
    float dwq[8], dwk[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dwq[e] = dwk[e] = 0.f;
    for (int64_t u = (int64_t)blockIdx.x * kWarps + warp; u < units; u += (int64_t)gridDim.x * kWarps) {
        const Unit t(u, a.N, chunks, groups);
        const T *row = X + t.b * x_sb + t.n * x_sn + sub * 8;
        T *drow = dX + t.b * dx_sb + t.n * dx_sn + sub * 8;
        Eight<T> raw[kSteps], grad[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int h = 4 * (t.g0 + i) + (lane >> 3);
            raw[i].zero();
            grad[i].zero();
            if (i < t.steps && h < H) {
                if (h < a.Hq + a.Hk) raw[i].load(row + (int64_t)h * 64);
                const T *src = h < a.Hq          ? dQ + ((t.b * a.Hq + h) * a.N + t.n) * 64
                               : h < a.Hq + a.Hk ? dK + ((t.b * a.Hk + (h - a.Hq)) * a.N + t.n) * 64
                                                 : dV + ((t.b * a.Hv + (h - a.Hq - a.Hk)) * a.N + t.n) * 64;
                grad[i].load(src + sub * 8);
            }
        }
        Turn<PAIRS_INSIDE> turn;
        turn.load(a, t.b, t.n, lane);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            if (i >= t.steps) break;
            const int g = t.g0 + i, h = 4 * g + (lane >> 3);
            if (4 * g < a.Hq + a.Hk) {
                float x[8], dy[8];
                raw[i].get(x);
                grad[i].get(dy);
                const bool isq = h < a.Hq, isk = !isq && h < a.Hq + a.Hk;
                turn.apply(dy, -1.f);
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
                ss = sum8(ss);
                const bool norm = (isq ? a.wq : a.wk) != nullptr;
                const float r = norm ? rsqrtf(ss * (1.f / 64.f) + a.eps) : 1.f;
                const float4 *w4 = reinterpret_cast<const float4 *>(sw[isq ? 0 : 1] + sub * 8);
                const float4 wa = w4[0], wb = w4[1];
                const float w[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
                float dot = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float n = x[e] * r, d = dy[e] * n;
                    dwq[e] += isq ? d : 0.f;   // selected, not multiplied: another head's NaN stays out
                    dwk[e] += isk ? d : 0.f;
                    x[e] = n;
                    dy[e] *= w[e];
                    dot = fmaf(dy[e], n, dot);
                }
                dot = sum8(dot) * (norm ? 1.f / 64.f : 0.f);
#pragma unroll
                for (int e = 0; e < 8; ++e) dy[e] = r * (dy[e] - x[e] * dot);
                if (h < a.Hq + a.Hk) grad[i].put(dy);
            }
            if (h < H) grad[i].store(drow + (int64_t)h * 64);
        }
    }
    // the block's sums: over the four heads of a warp, then over its warps
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
        for (int m = 8; m < 32; m <<= 1) {
            dwq[e] += __shfl_xor_sync(kFullMask, dwq[e], m);
            dwk[e] += __shfl_xor_sync(kFullMask, dwk[e], m);
        }
        if (lane < 8) {
            part[warp][sub * 8 + e] = dwq[e];
            part[warp][64 + sub * 8 + e] = dwk[e];
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

// Units of work and blocks: chunks of a token's heads small enough for
// kSteps, four blocks an SM at most (a block then takes several units).
struct Grid {
    int chunks;
    int64_t units;
    unsigned blocks;
    explicit Grid(const QkNormArgs &q) {
        const int groups = (q.Hq + q.Hk + q.Hv + 3) / 4;
        chunks = (groups + kSteps - 1) / kSteps;
        units = (int64_t)q.B * q.N * chunks;
        blocks = (unsigned)std::min<int64_t>((units + kWarps - 1) / kWarps, std::min(kMaxBlocks, 4 * sm_count()));
    }
};

template <typename T>
NormArgs<T> norm_args(const QkNormArgs &q) {
    return NormArgs<T>{q.N,   q.Hq,  q.Hk,  q.Hv, static_cast<const T *>(q.wq), static_cast<const T *>(q.wk), q.eps,
                       q.rot, q.cos, q.sin, q.P,  q.pos,                        q.pos_sb};
}

template <typename T>
cudaError_t fwd(const QkNormArgs &q) {
    const Grid g(q);
    const auto kern = q.interleaved ? qk_norm_fwd_kernel<T, true> : qk_norm_fwd_kernel<T, false>;
    const cudaError_t e = launch_kernel(kern, dim3(g.blocks), dim3(kWarps * 32), 0, q.stream, pdl_enabled(),
                                        norm_args<T>(q), static_cast<const T *>(q.X), q.x_sb, q.x_sn,
                                        static_cast<T *>(q.Q), static_cast<T *>(q.K), static_cast<T *>(q.V), g.units,
                                        g.chunks);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

template <typename T>
cudaError_t bwd(const QkNormArgs &q) {
    const Grid g(q);
    const auto kern = q.interleaved ? qk_norm_bwd_kernel<T, true> : qk_norm_bwd_kernel<T, false>;
    cudaError_t e = launch_kernel(kern, dim3(g.blocks), dim3(kWarps * 32), 0, q.stream, pdl_enabled(), norm_args<T>(q),
                                  static_cast<const T *>(q.X), q.x_sb, q.x_sn, static_cast<const T *>(q.dQ),
                                  static_cast<const T *>(q.dK), static_cast<const T *>(q.dV), static_cast<T *>(q.dX),
                                  q.dx_sb, q.dx_sn, q.ws, g.units, g.chunks);
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
    return q.dtype == FIBATT_F32 ? fwd<float>(q) : fwd<__nv_bfloat16>(q);
}
cudaError_t launch_qk_norm_bwd(const QkNormArgs &q) {
    return q.dtype == FIBATT_F32 ? bwd<float>(q) : bwd<__nv_bfloat16>(q);
}

FIBATT_DEFINE_ERROR_READER(read_error_qk_norm, "qk_norm.cu")

}  // namespace fibatt
