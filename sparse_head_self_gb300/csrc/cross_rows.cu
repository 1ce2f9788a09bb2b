// Cross attention forward for a few query rows (a token being decoded, or a
// handful): at most 16 rows (8 in 32 bits) read one key/value head, and the time
// is that of reading its keys and values once.
//
// A cluster of CTAs takes one key/value head of one sequence, a CTA a contiguous
// part of its keys.  One warp brings the keys and values in by tensor copies, a
// ring of 32 KB stages (128 keys in 16 bits, 64 in 32), so that up to 96 KB a CTA are
// on their way whatever the others do; eight warps take a share of each stage and
// keep the running maximum, sum and weighted values of their own keys, so nothing
// is exchanged until the end, when the warps are joined in shared memory and the
// CTAs through distributed shared memory, always in the same order.
//
// 16 bits: a warp's 16 keys of a stage are two products of the rows (padded to
// 16) with warp-wide matrix instructions, whose score fragments are the weights'
// operand of the second product.  (These are far below the 5th-generation tensor
// cores' rate, but need no tile of 128 rows, and the rows leave it unused:
// 16385 keys, 64 key heads, 4 rows each: 55 us with scalar products, bound by
// their instructions; 34.3 with these, 5.6 TB/s, as the copies alone.)
// 32 bits: eight lanes share a key and form one score per row with three
// shuffles.
#include <algorithm>

#include "cluster.cuh"
#include "cross_tiles.cuh"

namespace fibatt {
namespace {

constexpr int kWarps = 8;                  // and one that copies
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kStages = 3;
constexpr int kStageBytes = 32768;         // half of them keys
constexpr size_t kSmem = 1024 + kStages * kStageBytes;
constexpr float kNegInf = -__builtin_inff();

// One lane's eight values of a 32-bit row: dims 4 sub.. and 32 + 4 sub.., so that
// the lanes of a load touch consecutive banks.
struct Share {
    float4 a, b;
    __device__ __forceinline__ void load(const float *row, int sub) {
        a = *reinterpret_cast<const float4 *>(row + 4 * sub);
        b = *reinterpret_cast<const float4 *>(row + 32 + 4 * sub);
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
    __device__ static __forceinline__ int pair(int sub, int i) { return (i < 2 ? 0 : 14) + 2 * sub + i; }
};

__device__ __forceinline__ void store2(__nv_bfloat16 *p, float2 v) {
    *reinterpret_cast<uint32_t *>(p) = pack_bf16x2(v.x, v.y);
}
__device__ __forceinline__ void store2(float *p, float2 v) { *reinterpret_cast<float2 *>(p) = v; }

struct RowsArgs {
    TensorArg k, v;
    int Hq, Hkv, Nq, rows;
    KeySet ks;
    float *LSE;
    float c;
};

// What both kernels have around their products.
template <int R, int KEYS>
struct Part {
    const RowsArgs &a;
    uint8_t *ring;
    uint64_t *full, *empty;
    volatile int *abort;
    int hk, b, G, rank, C, bound, lo, hi, stages;

    __device__ __forceinline__ Part(const RowsArgs &a, uint8_t *smem_raw, uint64_t *full, uint64_t *empty, int *abort_flag)
        : a(a), full(full), empty(empty), abort(abort_flag) {
        ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
        C = (int)cluster_size();
        rank = (int)cluster_rank();
        const int unit = blockIdx.x / C;
        hk = unit % a.Hkv;
        b = unit / a.Hkv;
        G = a.Hq / a.Hkv;
        if (threadIdx.x == 0) {
            for (int s = 0; s < kStages; ++s) {
                mbar_init(&full[s], 1);
                mbar_init(&empty[s], kWarps);
            }
            *abort_flag = 0;
            prefetch_map(&a.k.map);
            prefetch_map(&a.v.map);
        }
        __syncthreads();
        grid_dep_wait();
        grid_dep_launch();
        bound = a.ks.bound(b);
        const int per = ((bound + C - 1) / C + 31) / 32 * 32;            // keys of a CTA
        lo = (int)min((int64_t)bound, (int64_t)per * rank);
        hi = min(bound, lo + per);
        stages = (hi - lo + KEYS - 1) / KEYS;
    }
    // the copying warp
    __device__ __forceinline__ void copy() {
        int j = 0;
        for (; j < stages; ++j) {
            const int s = j % kStages, last = j - kStages;
            if (last >= 0 && !pipe_wait(&empty[s], (last / kStages) & 1, abort)) break;
            if (elect_one()) {
                uint8_t *dst = ring + s * kStageBytes;
                mbar_expect_tx(&full[s], kStageBytes);
                load_tile(dst, a.k, lo + j * KEYS, hk, b, &full[s]);
                load_tile(dst + kStageBytes / 2, a.v, lo + j * KEYS, hk, b, &full[s]);
            }
            __syncwarp();
        }
        if ((threadIdx.x & 31) == 0)   // leave no copy in flight
            for (int i = max(0, j - kStages); i < j; ++i) mbar_drain(&full[i % kStages], (i / kStages) & 1);
    }
    // The warps' (m, l, O) of `rows` rows in shared memory -> O and LSE.
    template <typename T>
    __device__ __forceinline__ void join(const float (*sm)[R], const float (*sl)[R], const float2 (*so)[R][32], float *cm,
                                         float *cl, float2 (*co)[32], Rows<T> O) {
        __syncthreads();
        const int rows = FIBATT_CHECKED(a.rows <= R && a.rows == G * a.Nq) ? a.rows : 0;     // the kernel's room
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
            const int h = hk * G + r / a.Nq, n = r % a.Nq;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            store2(O.row(b, h, n) + 2 * d, make_float2(o.x * inv, o.y * inv));
            if (d == 0) a.LSE[((int64_t)b * a.Hq + h) * a.Nq + n] = sum == 0.f ? kNegInf : (top + log2f(sum)) * kLn2;
        }
        cluster_sync();   // the others may still read this CTA's part
    }
};

// ---- 16 bits ---------------------------------------------------------------------
// Four 8 x 8 matrices of 16-bit values, lane i giving row i mod 8 of matrix i / 8.
template <bool ACROSS>
__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], const void *row) {
    if (ACROSS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(smem_u32(row))
                     : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(smem_u32(row))
                     : "memory");
}

// R: 8 (the products' lower rows are not looked at) or 16.
template <int R>
__global__ void __launch_bounds__(kThreads, 2)
cross_rows_mma_kernel(const __grid_constant__ RowsArgs a, Rows<const __nv_bfloat16> Q, Rows<__nv_bfloat16> O) {
    constexpr int kKeys = 128, kHalves = R / 8;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ int abort_flag;
    __shared__ float sm[kWarps][R], sl[kWarps][R];
    __shared__ float cm[R], cl[R];            // the CTA's, read by the cluster
    __shared__ float2 co[R][32];
    Part<R, kKeys> p(a, smem_raw, full, empty, &abort_flag);
    const int warp = warp_number(), lane = threadIdx.x & 31, row = lane >> 2, pair = lane & 3;

    float m[kHalves], l[kHalves], o[8][4];
#pragma unroll
    for (int i = 0; i < kHalves; ++i) {
        m[i] = kNegInf;
        l[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
    if (warp == kWarps) {
        p.copy();
    } else {
        uint32_t q[4][4];                     // the rows as operands of four k-steps
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = row + 8 * i;
            const uint32_t *src = reinterpret_cast<const uint32_t *>(
                r < a.rows ? Q.row(p.b, p.hk * p.G + r / a.Nq, r % a.Nq) : nullptr);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                q[k][i] = src ? __ldg(src + 8 * k + pair) : 0u;
                q[k][2 + i] = src ? __ldg(src + 8 * k + 4 + pair) : 0u;
            }
        }
        for (int j = 0; j < p.stages; ++j) {
            const int st = j % kStages, k0 = p.lo + j * kKeys + 16 * warp;
            const int key = k0 + (lane & 15);
            const uint32_t in =
                __ballot_sync(kFullMask, key < p.hi && a.ks.has(p.b, min(key, p.hi - 1))) & 0xffffu;
            pipe_wait(&full[st], (j / kStages) & 1, p.abort);
            uint8_t *kt = p.ring + st * kStageBytes + 16 * warp * 128, *vt = kt + kStageBytes / 2;
            if (in != 0xffffu && lane < 16 && !((in >> lane) & 1)) {   // a weight of 0 meets no NaN
                uint4 *v = reinterpret_cast<uint4 *>(vt + lane * 128);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[(i + lane) & 7] = make_uint4(0, 0, 0, 0);
                fence_smem_async();      // before the next copy into the stage
            }
            __syncwarp();
            float s[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[t][i] = 0.f;
#pragma unroll
                for (int h = 0; h < 2; ++h) {       // 32 dims of 8 keys
                    uint32_t f[4];
                    const int r = lane & 7, ch = 4 * h + (lane >> 3);
                    load_matrices<false>(f, kt + (8 * t + r) * 128 + ((ch ^ r) << 4));
                    warp_mma(s[t], q[2 * h], f[0], f[1]);
                    warp_mma(s[t], q[2 * h + 1], f[2], f[3]);
                }
            }
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < kHalves; ++i) {
                float x[4] = {s[0][2 * i] * a.c, s[0][2 * i + 1] * a.c, s[1][2 * i] * a.c, s[1][2 * i + 1] * a.c};
                if (in != 0xffffu) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (!((in >> (2 * pair + (k & 1) + 8 * (k >> 1))) & 1)) x[k] = kNegInf;
                }
                float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
                top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
                if (__any_sync(kFullMask, top > m[i] + 8.f)) {     // raised seldom: weights stay below 2^8
                    const float next = fmaxf(top, m[i]), keep = next == kNegInf ? 1.f : fast_exp2(m[i] - next);
                    m[i] = next;
                    l[i] *= keep;
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        o[t][2 * i] *= keep;
                        o[t][2 * i + 1] *= keep;
                    }
                }
                const float base = m[i] == kNegInf ? 0.f : m[i];
#pragma unroll
                for (int k = 0; k < 4; ++k) x[k] = fast_exp2(x[k] - base);
                l[i] += (x[0] + x[1]) + (x[2] + x[3]);
                w[i] = pack_bf16x2(x[0], x[1]);
                w[2 + i] = pack_bf16x2(x[2], x[3]);
            }
            if (kHalves == 1) w[1] = w[3] = 0u;
#pragma unroll
            for (int t = 0; t < 8; t += 2) {        // 16 dims
                uint32_t f[4];
                const int r = 8 * ((lane >> 3) & 1) + (lane & 7), ch = t + (lane >> 4);
                load_matrices<true>(f, vt + r * 128 + ((ch ^ (r & 7)) << 4));
                warp_mma(o[t], w, f[0], f[1]);
                warp_mma(o[t + 1], w, f[2], f[3]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
        }
    }
    __syncthreads();      // the ring is free: it takes the warps' sums
    float2(*so)[R][32] = reinterpret_cast<float2(*)[R][32]>(p.ring);
    if (warp < kWarps) {
#pragma unroll
        for (int i = 0; i < kHalves; ++i) {
            l[i] += __shfl_xor_sync(kFullMask, l[i], 1);
            l[i] += __shfl_xor_sync(kFullMask, l[i], 2);
            const int r = row + 8 * i;
#pragma unroll
            for (int t = 0; t < 8; ++t) so[warp][r][4 * t + pair] = make_float2(o[t][2 * i], o[t][2 * i + 1]);
            if (pair == 0) {
                sm[warp][r] = m[i];
                sl[warp][r] = l[i];
            }
        }
    }
    p.join(sm, sl, so, cm, cl, co, O);
}

// ---- 32 bits ---------------------------------------------------------------------
// R rows (the last ones may be copies of the last real row).
template <int R>
__global__ void __launch_bounds__(kThreads, R > 4 ? 1 : 2)
cross_rows_kernel(const __grid_constant__ RowsArgs a, Rows<const float> Q, Rows<float> O) {
    constexpr int kKeys = 64, U = kKeys / kWarps / 4;     // keys of a stage, of a group of lanes
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ int abort_flag;
    __shared__ float sm[kWarps][R], sl[kWarps][R];
    __shared__ float2 so[kWarps][R][32];
    __shared__ float cm[R], cl[R];            // the CTA's, read by the cluster
    __shared__ float2 co[R][32];
    Part<R, kKeys> p(a, smem_raw, full, empty, &abort_flag);
    const int warp = warp_number(), lane = threadIdx.x & 31, sub = lane & 7, grp = lane >> 3;
    if (warp == kWarps) p.copy();
    Share q[R];
    float m[R], l[R];
    float2 acc[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = min(r, a.rows - 1);
        q[r].load(Q.row(p.b, p.hk * p.G + i / a.Nq, i % a.Nq), sub);
        m[r] = kNegInf;
        l[r] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][i] = make_float2(0.f, 0.f);
    }
    for (int j = 0; warp < kWarps && j < p.stages; ++j) {
        const int st = j % kStages, k0 = p.lo + j * kKeys + warp * 4 * U + grp;
        bool in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) in[u] = k0 + 4 * u < p.hi && a.ks.has(p.b, min(k0 + 4 * u, p.hi - 1));
        pipe_wait(&full[st], (j / kStages) & 1, p.abort);
        const float *kr = reinterpret_cast<const float *>(p.ring + st * kStageBytes) + (warp * 4 * U + grp) * 64;
        const float *vr = kr + kKeys * 64;
        float s[R][U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Share k;
            k.load(kr + 4 * u * 64, sub);
#pragma unroll
            for (int r = 0; r < R; ++r) s[r][u] = q[r].dot(k);
        }
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
                s[r][u] = in[u] ? s[r][u] * a.c : kNegInf;
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
            Share v;
            v.load(vr + 4 * u * 64, sub);
            if (!in[u]) v.zero();         // a weight of 0 meets no NaN
            float2 x[4];
            v.get(x);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[r][i] = fma2(make_float2(s[r][u], s[r][u]), x[i], acc[r][i]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
    }
    if (warp < kWarps) {
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
            for (int i = 0; i < 4; ++i) so[warp][r][Share::pair(sub, i)] = acc[r][i];
            if (lane == 0) {
                sm[warp][r] = top;
                sl[warp][r] = l[r];
            }
        }
    }
    }
    p.join(sm, sl, so, cm, cl, co, O);
}

template <typename T, auto Kernel>
cudaError_t run(const CrossArgs &a, int rows) {
    constexpr int kKeys = kStageBytes / 2 / (64 * (int)sizeof(T));
    RowsArgs f;
    if (!make_tensor(&f.k, a.K, a.B, a.Hkv, a.Nk, kKeys, 1, a.dtype, sizeof(T) == 2) ||
        !make_tensor(&f.v, a.V, a.B, a.Hkv, a.Nk, kKeys, 1, a.dtype, sizeof(T) == 2))
        return cudaErrorInvalidValue;
    f.Hq = a.Hq, f.Hkv = a.Hkv, f.Nq = a.Nq, f.rows = rows;
    f.ks = a.keys;
    f.LSE = a.LSE;
    f.c = a.scale * kLog2e;
    const cudaError_t e = prepare_kernel<Kernel>(kSmem, 0);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)a.B * a.Hkv;
    // CTAs of a cluster: as many as the GPU holds at once (two a SM), as long as a CTA
    // keeps a stage (64 units: clusters of four 33.6 us, of eight, in two waves, 35.2)
    int c = 1;
    while (c < 8 && units * c * 2 <= 2 * sm_count() && a.Nk > c * kKeys) c *= 2;
    return launch_clusters(Kernel, (unsigned)(units * c), c, kThreads, kSmem, a.stream, f, rows_of<const T>(a.Q),
                           rows_of<T>(a.O));
}

}  // namespace

bool cross_rows_takes(const CrossArgs &a) {
    const int64_t rows = (int64_t)(a.Hq / a.Hkv) * a.Nq;
    return rows <= (a.dtype == FIBATT_F32 ? 8 : 16) && (int64_t)a.B * a.Hkv < 0x7fffffff / 8;
}

cudaError_t launch_cross_rows(const CrossArgs &a) {
    const int rows = a.Hq / a.Hkv * a.Nq;
    if (a.dtype == FIBATT_F32)
        return rows == 1   ? run<float, cross_rows_kernel<1>>(a, rows)
               : rows == 2 ? run<float, cross_rows_kernel<2>>(a, rows)
               : rows <= 4 ? run<float, cross_rows_kernel<4>>(a, rows)
                           : run<float, cross_rows_kernel<8>>(a, rows);
    return rows <= 8 ? run<__nv_bfloat16, cross_rows_mma_kernel<8>>(a, rows)
                     : run<__nv_bfloat16, cross_rows_mma_kernel<16>>(a, rows);
}

FIBATT_DEFINE_ERROR_READER(read_error_cross_rows, "cross_rows.cu")

}  // namespace fibatt
