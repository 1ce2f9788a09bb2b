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
// bytes.  A block takes 16 consecutive tokens at a time (over the sequences'
// ends: a token's rows are found once) and some or all heads, its warps eight of the
// tokens and every fourth head, so that a warp's head is of one kind.  Eight lanes share a
// head row; a lane has two runs of four dims, chosen so that both values of
// every rotated pair are its own (halves: dims 4 i.. and rot / 2 + 4 i..),
// which leaves the two sums over a head as the only exchange; the arithmetic
// is on packed pairs of floats.  Rows arrive by asynchronous copies in a ring of
// each warp's own, two or three heads ahead and over the items' ends, without holding
// registers; the tokens' angles are brought into shared memory once for all heads.
// Every head row is a whole 128- or 256-byte segment, so all traffic is full
// sectors.  The values' heads are copied unconverted.
//
// Measured: 64 sequences of 197 tokens, 36 heads, bf16, forward: 23.7 us, 4.9 TB/s
// (72% of a copy's rate; the issue slots 61% taken, most stalls fixed latencies of
// a head's chain of sums), fp32 41 us, 5.7 TB/s; 256 sequences, bf16, backward: 125 us,
// 5.0 TB/s; 2 x 16385 tokens, 48 heads, fp32, half of each head rotated, backward: 189 us,
// 5.7 TB/s; 8 tokens, forward: 2.9 us.
//
// dw: each lane sums its eight dims, the block joins its warps in shared memory, and
// a second kernel adds the blocks' sums in block order: no atomics, the same result
// on every run.  For a result of 32 bits a lane's sum goes over one unit only, and the
// units' sums into totals that keep what their additions round off, so that the error
// does not grow with the rows: against 64 bits, 2 x 16385 tokens, 16 heads of each
// kind, dw 1.1e-7 (one sum a lane, and of the blocks: 3.0e-7); it costs 1 to 3 us of 190.
// A result of 16 bits is rounded far above that: one sum a lane.
#include <algorithm>

#include "cross.h"
#include "device_common.cuh"
#include "row_math.cuh"

namespace fibatt {
namespace {

constexpr int kWarps = 8;
constexpr int kTokens = 16;           // of a unit
constexpr int kSteps = 2;             // four tokens each: a warp's half of a unit
// Heads in a warp's ring, whose rows are of RT tensors.  The fp32 backward has three, with
// which an SM holds two blocks: 2 x 16385 tokens, 48 heads, of which 32 dims are rotated, 187 us
// where four and one block take 209; with all 64 rotated, halves paired, 190 and 183.
template <typename T, int RT>
constexpr int ring_depth() {
    return sizeof(T) == 4 && RT == 2 ? 3 : 4;
}
constexpr int kMaxBlocks = 1024;      // rows of the dw partial sums
constexpr unsigned kErrPosition = 8u; // a position at or behind the end of the tables

__device__ __forceinline__ void copy_async(void *smem, const void *gmem) {   // 16 bytes
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(gmem)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest N groups of this thread's copies have arrived.
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A lane's eight dims of a head row: runs of four at a0 and a1 (elements).
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
    uint2 u, v;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, int a0, int a1) {
        u = *reinterpret_cast<const uint2 *>(p + a0);
        v = *reinterpret_cast<const uint2 *>(p + a1);
    }
    __device__ __forceinline__ void store(__nv_bfloat16 *p, int a0, int a1) const {
        *reinterpret_cast<uint2 *>(p + a0) = u;
        *reinterpret_cast<uint2 *>(p + a1) = v;
    }
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
        a = *reinterpret_cast<const float4 *>(p + a0);
        b = *reinterpret_cast<const float4 *>(p + a1);
    }
    __device__ __forceinline__ void store(float *p, int a0, int a1) const {
        *reinterpret_cast<float4 *>(p + a0) = a;
        *reinterpret_cast<float4 *>(p + a1) = b;
    }
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

    // from a token's 32 cosines and 32 sines in shared memory (8 sub < rot)
    __device__ __forceinline__ void load(const float *angles, int sub) {
        const float4 vc = *reinterpret_cast<const float4 *>(angles + 4 * sub);
        const float4 vs = *reinterpret_cast<const float4 *>(angles + 32 + 4 * sub);
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

// A sum that keeps what its additions round off (the two-sum of Knuth).
struct Total {
    float sum = 0.f, lost = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float s = sum + x, part = s - sum;
        lost += (sum - (s - part)) + (x - part);
        sum = s;
    }
    // of an infinite sum, what it lost is no number
    __device__ __forceinline__ float kept() const { return isfinite(lost) ? lost : 0.f; }
    __device__ __forceinline__ float value() const { return sum + kept(); }
};
// Over the four heads (lanes 8 apart) of a warp's sums d of four pairs; lane's
// result: pair lane / 8.
__device__ __forceinline__ float2 sum_groups(const float2 (&d)[4]) {
    const bool far = threadIdx.x & 16, near = threadIdx.x & 8;
    float2 k[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 give = far ? d[i] : d[2 + i];
        k[i] = add2(far ? d[2 + i] : d[i], make_float2(__shfl_xor_sync(kFullMask, give.x, 16), __shfl_xor_sync(kFullMask, give.y, 16)));
    }
    const float2 give = near ? k[0] : k[1];
    return add2(near ? k[1] : k[0], make_float2(__shfl_xor_sync(kFullMask, give.x, 8), __shfl_xor_sync(kFullMask, give.y, 8)));
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

// Bring the angles of the unit's 16 tokens into `to` [16][64]: thread 16 i + j
// copies the j-th 16 bytes of token i's cosines (j < 8) and sines.  `turned` [16]:
// which of them are rotated; the others' values are left as they are (an angle of
// 0 would make NaN of a pair with an infinity).  The rotation stands in a branch on it:
// 64 x 197 tokens, bf16, forward 24.1 us; selecting between turned and not, 25.2.
template <typename T>
__device__ __forceinline__ void stage_angles(const NormArgs<T> &a, float *to, uint8_t *turned, unsigned unit, unsigned tokens) {
    const int i = threadIdx.x >> 4, j = threadIdx.x & 15, half = a.rot / 2, at = 4 * (j & 7);
    const unsigned token = unit * kTokens + i;
    if (at >= half || token >= tokens) return;
    const unsigned b = token / (unsigned)a.N;
    const int n = (int)(token - b * a.N);
    const int p = a.pos ? __ldg(a.pos + b * a.pos_sb + n) : n;
    const bool on = p >= 0 && p < a.P;
    if (on) copy_async(to + 64 * i + 4 * j, (j < 8 ? a.cos : a.sin) + (int64_t)p * half + at);
    else if (p >= a.P) atomicOr(&g_device_error, kErrPosition);
    if (j == 0) turned[i] = on;
}

// A lane's two tokens of a unit, and where their rows are.
struct Tokens {
    unsigned b[kSteps], n[kSteps];
    bool in[kSteps];
    __device__ __forceinline__ void set(unsigned unit, unsigned tokens, int N) {
        const unsigned first = (threadIdx.x >> 5 & 1) * 8 + (threadIdx.x >> 3 & 3);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const unsigned t = unit * kTokens + first + 4 * s;
            in[s] = t < tokens;
            b[s] = t / (unsigned)N;
            n[s] = t - b[s] * N;
        }
    }
    // in the packed tensor
    __device__ __forceinline__ int64_t packed(int s, int h, int64_t sb, int64_t sn) const {
        return (int64_t)b[s] * sb + (int64_t)n[s] * sn + h * 64;
    }
    // head h of H in a dense [B, H, N, 64] tensor
    __device__ __forceinline__ int64_t dense(int s, int h, int H, int N) const {
        return (((int64_t)b[s] * H + h) * N + n[s]) * 64;
    }
};

// The tensor of head h (the same kind for the whole warp): its heads, and h's
// number among them.
template <typename T>
__device__ __forceinline__ T *kind_of(T *q, T *k, T *v, int Hq, int Hk, int Hv, int h, int &i, int &H) {
    if (h < Hq) {
        i = h, H = Hq;
        return q;
    }
    if (h < Hq + Hk) {
        i = h - Hq, H = Hk;
        return k;
    }
    i = h - Hq - Hk, H = Hv;
    return v;
}

// One head row of 64 elements from `src` into the warp's slot: lane's share of
// 16-byte copies.
template <typename T>
__device__ __forceinline__ void copy_row(T *dst, const T *src) {
    constexpr int kPer = 16 / sizeof(T);
    const int sub = threadIdx.x & 7;
#pragma unroll
    for (int i = 0; i < 8 / kPer; ++i) copy_async(dst + (8 * i + sub) * kPer, src + (8 * i + sub) * kPer);
}

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

// Shared memory of a block: two units' angles, and every warp's ring of heads of RT
// tensors, eight rows each.
template <typename T, int RT>
constexpr size_t ring_bytes() {
    return 2 * kTokens * 64 * sizeof(float) + (size_t)kWarps * ring_depth<T, RT>() * RT * 8 * 64 * sizeof(T);
}

// Where a warp is in its sequence of heads: an item is a unit's tokens and one of
// `chunks` parts of the heads, [lo, hi).
struct Place {
    unsigned item, unit;
    int h, lo, hi;
    __device__ __forceinline__ Place(int H, int chunks) { enter(blockIdx.x, H, chunks); }
    __device__ __forceinline__ void enter(unsigned i, int H, int chunks) {
        item = i;
        unit = i / (unsigned)chunks;
        const int c = (int)(i - unit * chunks);
        lo = H * c / chunks;
        hi = H * (c + 1) / chunks;
        h = lo + (threadIdx.x >> 6);
    }
    // the next head; true when the item changed
    __device__ __forceinline__ bool next(int H, int chunks) {
        h += kWarps / 2;
        if (h < hi) return false;
        enter(item + gridDim.x, H, chunks);
        return true;
    }
};

// CUT: the heads are cut into `cuts` chunks; else cuts is not looked at.
template <typename T, bool PAIRS_INSIDE, bool CUT>
__global__ void __launch_bounds__(kWarps * 32, 3)
qk_norm_fwd_kernel(const __grid_constant__ NormArgs<T> a, const T *__restrict__ X, int64_t x_sb, int64_t x_sn,
                   T *__restrict__ Q, T *__restrict__ K, T *__restrict__ V, unsigned tokens, unsigned items, int cuts) {
    extern __shared__ float4 smem4[];
    __shared__ __align__(16) float sw[2][64];
    __shared__ uint8_t turned[2][kTokens];
    constexpr int kDepth = ring_depth<T, 1>();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & 7, grp = lane >> 3;
    float *angles = reinterpret_cast<float *>(smem4);
    T *ring = reinterpret_cast<T *>(angles + 2 * kTokens * 64) + (size_t)warp * kDepth * 8 * 64;
    const int Hn = a.Hq + a.Hk, H = Hn + a.Hv, chunks = CUT ? cuts : 1;
    const bool few = H / chunks < 4 * kDepth;     // a warp may have fewer heads of an item than its ring holds
    int a0, a1;
    lane_dims<PAIRS_INSIDE>(a.rot, sub, a0, a1);
    grid_dep_wait();
    grid_dep_launch();

    Tokens ahead, here;
    Place load(H, chunks), work(H, chunks);
    // copies of the next (unit, head) into slot `slot`; one group each, empty at the end
    const auto fetch = [&](int slot) {
        if (load.item < items && load.h < load.hi) {
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                if (ahead.in[s])
                    copy_row(ring + (slot * 8 + 4 * s + grp) * 64, X + ahead.packed(s, load.h, x_sb, x_sn));
            if (load.next(H, chunks)) ahead.set(load.unit, tokens, a.N);
        }
        copies_commit();
    };
    if (a.rot) stage_angles(a, angles, turned[0], work.unit, tokens);
    copies_commit();
    ahead.set(work.unit, tokens, a.N);
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) fetch(i);
    stage_weights(a, sw);

    int slot = 0;
    for (int buf = 0; work.item < items; buf ^= 1) {
        const unsigned item = work.item, after = item + gridDim.x;
        here.set(work.unit, tokens, a.N);
        // this unit's angles: the oldest group at the start; later they were asked for
        // with the first head of the unit before, at least kDepth groups ago
        if (few) copies_wait<0>();
        else copies_wait<kDepth - 1>();
        __syncthreads();
        if (a.rot && after < items)
            stage_angles(a, angles + (buf ^ 1) * kTokens * 64, turned[buf ^ 1], after / (unsigned)chunks, tokens);
        if (few) copies_commit();
        bool turns[kSteps];       // this lane's dims of its two tokens are rotated
#pragma unroll
        for (int s = 0; s < kSteps; ++s) turns[s] = 8 * sub < a.rot && turned[buf][(warp & 1) * 8 + 4 * s + grp] != 0;
        // nearly always the whole warp's: a branch that all of it takes costs less (24.0 and 23.5 us; the
        // backward is slower with it, 124.4 and 125.4)
        const bool all = __all_sync(kFullMask, turns[0] && turns[1]);
        while (work.item == item && work.h < work.hi) {
            fetch((slot + kDepth - 1) % kDepth);     // also takes along the next unit's angles
            copies_wait<kDepth - 1>();
            __syncwarp();
            int hi, Hs;
            T *out = kind_of(Q, K, V, a.Hq, a.Hk, a.Hv, work.h, hi, Hs);
            const bool isq = work.h < a.Hq, isn = work.h < Hn, norm = (isq ? a.wq : a.wk) != nullptr;
            float2 w[4];
            weights(sw[isq ? 0 : 1], a0, a1, w);
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                Eight<T> raw;
                raw.load(ring + (slot * 8 + 4 * s + grp) * 64, a0, a1);
                if (isn) {
                    float2 x[4];
                    raw.get(x);
                    const float r = norm ? rsqrtf(sum8(squares(x)) * (1.f / 64.f) + a.eps) : 1.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = mul2(x[e], mul2(w[e], make_float2(r, r)));
                    const auto rotate = [&] {
                        Turn<PAIRS_INSIDE> turn;
                        turn.load(angles + (buf * kTokens + (warp & 1) * 8 + 4 * s + grp) * 64, sub);
                        turn.template apply<false>(x);
                    };
                    if (all) rotate();
                    else if (turns[s]) rotate();
                    raw.put(x);
                }
                if (here.in[s] && FIBATT_CHECKED(hi >= 0 && hi < Hs && here.n[s] < (unsigned)a.N)) raw.store(out + here.dense(s, hi, Hs, a.N), a0, a1);
            }
            __syncwarp();
            slot = (slot + 1) % kDepth;
            work.next(H, chunks);
        }
        if (work.item == item) work.enter(after, H, chunks);    // a warp without heads
    }
    copies_wait<0>();
}

template <typename T, bool PAIRS_INSIDE, bool CUT>
__global__ void __launch_bounds__(kWarps * 32, 2)
qk_norm_bwd_kernel(const __grid_constant__ NormArgs<T> a, const T *__restrict__ X, int64_t x_sb, int64_t x_sn,
                   const T *__restrict__ dQ, const T *__restrict__ dK, const T *__restrict__ dV, T *__restrict__ dX,
                   int64_t dx_sb, int64_t dx_sn, float *__restrict__ partial, unsigned tokens, unsigned items, int cuts) {
    extern __shared__ float4 smem4[];
    __shared__ __align__(16) float sw[2][64];
    __shared__ uint8_t turned[2][kTokens];
    __shared__ float part[kWarps][128];
    constexpr int kDepth = ring_depth<T, 2>();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & 7, grp = lane >> 3;
    float *angles = reinterpret_cast<float *>(smem4);
    T *ring = reinterpret_cast<T *>(angles + 2 * kTokens * 64) + (size_t)warp * kDepth * 2 * 8 * 64;
    const int Hn = a.Hq + a.Hk, H = Hn + a.Hv, chunks = CUT ? cuts : 1;
    const bool few = H / chunks < 4 * kDepth;     // a warp may have fewer heads of an item than its ring holds
    int a0, a1;
    lane_dims<PAIRS_INSIDE>(a.rot, sub, a0, a1);
    grid_dep_wait();
    grid_dep_launch();

    Tokens ahead, here;
    Place load(H, chunks), work(H, chunks);
    // the next (unit, head): its rows of the gradient and, where there is a norm, of X (what
    // else X holds does not matter to the gradient: an infinity there would give 0 inf)
    const auto fetch = [&](int slot) {
        if (load.item < items && load.h < load.hi) {
            int hi, Hs;
            const T *src = kind_of(dQ, dK, dV, a.Hq, a.Hk, a.Hv, load.h, hi, Hs);
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                if (ahead.in[s]) {
                    T *dst = ring + (slot * 16 + 4 * s + grp) * 64;
                    if (load.h < Hn && (load.h < a.Hq ? a.wq : a.wk))
                        copy_row(dst, X + ahead.packed(s, load.h, x_sb, x_sn));
                    copy_row(dst + 8 * 64, src + ahead.dense(s, hi, Hs, a.N));
                }
            if (load.next(H, chunks)) ahead.set(load.unit, tokens, a.N);
        }
        copies_commit();
    };
    if (a.rot) stage_angles(a, angles, turned[0], work.unit, tokens);
    copies_commit();
    ahead.set(work.unit, tokens, a.N);
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) fetch(i);
    stage_weights(a, sw);
    constexpr bool kEachItem = sizeof(T) == 4;
    float2 dwq[4], dwk[4];       // of the item, or of all
#pragma unroll
    for (int e = 0; e < 4; ++e) dwq[e] = dwk[e] = make_float2(0.f, 0.f);
    Total total[4];              // of pair grp: wq, wk
    const auto collect = [&] {
        const float2 q = sum_groups(dwq), k = sum_groups(dwk);
        total[0].add(q.x);
        total[1].add(q.y);
        total[2].add(k.x);
        total[3].add(k.y);
    };

    int slot = 0;
    for (int buf = 0; work.item < items; buf ^= 1) {
        const unsigned item = work.item, after = item + gridDim.x;
        here.set(work.unit, tokens, a.N);
        if (few) copies_wait<0>();
        else copies_wait<kDepth - 1>();
        __syncthreads();
        if (a.rot && after < items)
            stage_angles(a, angles + (buf ^ 1) * kTokens * 64, turned[buf ^ 1], after / (unsigned)chunks, tokens);
        if (few) copies_commit();
        bool turns[kSteps];       // this lane's dims of its two tokens are rotated
#pragma unroll
        for (int s = 0; s < kSteps; ++s) turns[s] = 8 * sub < a.rot && turned[buf][(warp & 1) * 8 + 4 * s + grp] != 0;
        while (work.item == item && work.h < work.hi) {
            fetch((slot + kDepth - 1) % kDepth);
            copies_wait<kDepth - 1>();
            __syncwarp();
            const bool isq = work.h < a.Hq, isn = work.h < Hn, norm = (isq ? a.wq : a.wk) != nullptr;
            float2 w[4];
            weights(sw[isq ? 0 : 1], a0, a1, w);
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const T *src = ring + (slot * 16 + 4 * s + grp) * 64;
                Eight<T> grad;
                grad.load(src + 8 * 64, a0, a1);
                if (isn) {
                    float2 dy[4];
                    grad.get(dy);
                    if (turns[s]) {
                        Turn<PAIRS_INSIDE> turn;
                        turn.load(angles + (buf * kTokens + (warp & 1) * 8 + 4 * s + grp) * 64, sub);
                        turn.template apply<true>(dy);
                    }
                    if (norm) {
                        Eight<T> raw;
                        raw.load(src, a0, a1);
                        float2 x[4];
                        raw.get(x);
                        const float r = rsqrtf(sum8(squares(x)) * (1.f / 64.f) + a.eps);
                        float2 dot = make_float2(0.f, 0.f);
                        const bool in = here.in[s];      // the slot of no token holds anything: its sums are left out
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[e] = mul2(x[e], make_float2(r, r));
                            if (in && isq) dwq[e] = fma2(dy[e], x[e], dwq[e]);
                            else if (in) dwk[e] = fma2(dy[e], x[e], dwk[e]);
                            dy[e] = mul2(dy[e], w[e]);
                            dot = fma2(dy[e], x[e], dot);
                        }
                        const float m = sum8(dot.x + dot.y) * (-1.f / 64.f);
#pragma unroll
                        for (int e = 0; e < 4; ++e) dy[e] = mul2(make_float2(r, r), fma2(x[e], make_float2(m, m), dy[e]));
                    }
                    grad.put(dy);
                }
                if (here.in[s] && FIBATT_CHECKED(work.h < H && here.n[s] < (unsigned)a.N)) grad.store(dX + here.packed(s, work.h, dx_sb, dx_sn), a0, a1);
            }
            __syncwarp();
            slot = (slot + 1) % kDepth;
            work.next(H, chunks);
        }
        if (work.item == item) work.enter(after, H, chunks);    // a warp without heads
        if (kEachItem && (a.wq || a.wk)) {
            collect();
#pragma unroll
            for (int e = 0; e < 4; ++e) dwq[e] = dwk[e] = make_float2(0.f, 0.f);
        }
    }
    copies_wait<0>();
    if (!kEachItem) collect();
    // the block's sums
    const int d = (grp < 2 ? a0 : a1) + 2 * (grp & 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) part[warp][64 * (i >> 1) + d + (i & 1)] = total[i].value();
    __syncthreads();
    if (threadIdx.x < 128 && FIBATT_CHECKED(blockIdx.x < kMaxBlocks)) {      // the workspace's rows
        Total t;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) t.add(part[w][threadIdx.x]);
        partial[(int64_t)blockIdx.x * 128 + threadIdx.x] = t.value();
    }
}

// dw from the blocks' sums: eight threads a column, each over every eighth
// block, joined in thread order.
template <typename T>
__global__ void __launch_bounds__(1024) qk_norm_dw_kernel(const float *__restrict__ partial, int blocks,
                                                          T *__restrict__ dwq, T *__restrict__ dwk) {
    __shared__ float2 part[8][128];     // sums and what they lost
    grid_dep_wait();
    const int c = threadIdx.x & 127, k = threadIdx.x >> 7;
    Total t;
    for (int b = k; b < blocks; b += 8) t.add(partial[(int64_t)b * 128 + c]);
    part[k][c] = make_float2(t.sum, t.kept());
    __syncthreads();
    if (k) return;
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        t.add(part[i][c].x);
        t.add(part[i][c].y);
    }
    T *out = c < 64 ? dwq : dwk;
    if (out) out[c & 63] = (T)t.value();
}

// The launch of `Kernel`: one wave of blocks, each walking over its items.  With
// fewer units than blocks the heads are cut into chunks, of four at least (one
// token of eight sequences, 24 heads: 5.9 -> 3.0 us); with more they are not,
// since a warp's ring drains at an item's end when the item is shorter than the
// ring (ViT-B, B=64, in chunks of eight heads: 36 us instead of 27).
struct Launch {
    unsigned tokens, items, blocks;
    int chunks;
};
template <auto Kernel>
cudaError_t plan(const QkNormArgs &q, size_t smem, Launch *l) {
    cudaError_t e = prepare_kernel<Kernel>(smem, 0);
    if (e != cudaSuccess) return e;
    static std::atomic<int> per_sm{0};
    int n = per_sm.load(std::memory_order_relaxed);
    if (n == 0) {
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, Kernel, kWarps * 32, smem);
        if (e != cudaSuccess) return e;
        n = std::max(n, 1);
        per_sm.store(n, std::memory_order_relaxed);
    }
    const int64_t resident = std::min(kMaxBlocks, n * sm_count());
    const int H = q.Hq + q.Hk + q.Hv;
    l->tokens = (unsigned)q.B * (unsigned)q.N;
    const int64_t units = ((int64_t)l->tokens + kTokens - 1) / kTokens;
    l->chunks = units < resident ? (int)std::min<int64_t>(std::max(1, H / 4), (resident + units - 1) / units) : 1;
    l->items = (unsigned)(units * l->chunks);
    l->blocks = (unsigned)std::min<int64_t>(l->items, resident);
    return cudaSuccess;
}

template <typename T>
NormArgs<T> norm_args(const QkNormArgs &q) {
    return NormArgs<T>{q.N,   q.Hq,  q.Hk,  q.Hv, static_cast<const T *>(q.wq), static_cast<const T *>(q.wk), q.eps,
                       q.rot, q.cos, q.sin, q.P,  q.pos,                        q.pos_sb};
}

template <typename T, bool PAIRS_INSIDE, bool CUT>
cudaError_t fwd(const QkNormArgs &q) {
    constexpr size_t smem = ring_bytes<T, 1>();
    Launch l;
    cudaError_t e = plan<qk_norm_fwd_kernel<T, PAIRS_INSIDE, CUT>>(q, smem, &l);
    if (e != cudaSuccess) return e;
    if (!CUT && l.chunks > 1) return fwd<T, PAIRS_INSIDE, true>(q);
    e = launch_kernel(qk_norm_fwd_kernel<T, PAIRS_INSIDE, CUT>, dim3(l.blocks), dim3(kWarps * 32), smem, q.stream,
                      pdl_enabled(), norm_args<T>(q), static_cast<const T *>(q.X), q.x_sb, q.x_sn,
                      static_cast<T *>(q.Q), static_cast<T *>(q.K), static_cast<T *>(q.V), l.tokens, l.items, l.chunks);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

template <typename T, bool PAIRS_INSIDE, bool CUT>
cudaError_t bwd(const QkNormArgs &q) {
    constexpr size_t smem = ring_bytes<T, 2>();
    Launch l;
    cudaError_t e = plan<qk_norm_bwd_kernel<T, PAIRS_INSIDE, CUT>>(q, smem, &l);
    if (e != cudaSuccess) return e;
    if (!CUT && l.chunks > 1) return bwd<T, PAIRS_INSIDE, true>(q);
    e = launch_kernel(qk_norm_bwd_kernel<T, PAIRS_INSIDE, CUT>, dim3(l.blocks), dim3(kWarps * 32), smem, q.stream,
                      pdl_enabled(), norm_args<T>(q), static_cast<const T *>(q.X), q.x_sb, q.x_sn,
                      static_cast<const T *>(q.dQ), static_cast<const T *>(q.dK), static_cast<const T *>(q.dV),
                      static_cast<T *>(q.dX), q.dx_sb, q.dx_sn, q.ws, l.tokens, l.items, l.chunks);
    if (e != cudaSuccess) return e;
    count_launches(1);
    if (!q.dwq && !q.dwk) return cudaSuccess;
    e = launch_kernel(qk_norm_dw_kernel<T>, dim3(1), dim3(1024), 0, q.stream, pdl_enabled(),
                      static_cast<const float *>(q.ws), (int)l.blocks, static_cast<T *>(q.dwq),
                      static_cast<T *>(q.dwk));
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace

size_t qk_norm_bwd_workspace() { return (size_t)kMaxBlocks * 128 * sizeof(float); }

cudaError_t launch_qk_norm_fwd(const QkNormArgs &q) {
    if (q.interleaved) return q.dtype == FIBATT_F32 ? fwd<float, true, false>(q) : fwd<__nv_bfloat16, true, false>(q);
    return q.dtype == FIBATT_F32 ? fwd<float, false, false>(q) : fwd<__nv_bfloat16, false, false>(q);
}
cudaError_t launch_qk_norm_bwd(const QkNormArgs &q) {
    if (q.interleaved) return q.dtype == FIBATT_F32 ? bwd<float, true, false>(q) : bwd<__nv_bfloat16, true, false>(q);
    return q.dtype == FIBATT_F32 ? bwd<float, false, false>(q) : bwd<__nv_bfloat16, false, false>(q);
}

FIBATT_DEFINE_ERROR_READER(read_error_qk_norm, "qk_norm.cu")

}  // namespace fibatt
