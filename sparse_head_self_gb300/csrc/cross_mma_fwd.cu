// Cross attention forward on the tensor cores (bf16).
//
// A CTA holds NT tiles of 128 query rows of one key/value head and walks over
// the 128-key tiles of its sequence:
//   S = Q K^T          128 x 128, fp32 in tensor memory (2 x 128 x 128 x 64 flops)
//   P = exp2(c S - m)  two threads own a row, 64 columns each, and exchange their
//                      maxima through shared memory
//   O += P V           P back to tensor memory as bf16, V across its rows
// Warps: 8 per tile for the softmax (four on every scheduler hide each other's
// waits), one that copies (tensor copies into a ring of K/V stages), one that
// finds each tile's attended keys and clears the other value rows, two that
// issue the matrix instructions, one for S and one for O, so that neither waits
// for what the other needs.  S of the next key tile is formed while the softmax
// works on this one (S and P have columns of their own), so the tensor cores and
// the exponentials, which take about as long at a head dim of 64, overlap.
//
// The running maximum is raised only when a score exceeds it by more than
// 2^8 (P stays below 256, exact enough in fp32 sums and as relative bf16), so
// O is almost never rescaled; a rescaling reads and rewrites O in tensor memory
// between two products.  P is rounded to bf16 for its product (relative
// 2^-8 a weight, averaging out over the keys); l adds the unrounded weights.
//
// With few units, or a last round of them that leaves most SMs idle, the keys are
// cut over a cluster, whose CTAs join their (m, l, O) through distributed shared
// memory in rank order.  CTAs of one tile are one wave, two a SM, that walks over
// the units: copies and scores run ahead into the next unit while the softmax
// finishes this one (768 units of 65 x 197: 19.1 -> 16.5 us).  CTAs of two tiles
// are not: their softmax has no register to spare for the walk, which cost 10% of
// every tile.
//
// Measured: 2 sequences, 16 heads, 1569 x 16385: 227 us, 927 TFLOP/s (clusters of
// two; one CTA a unit, 1.47 rounds: 266); 16 heads, 4096 x 4096: 75 us, 919; 8
// sequences, 12 heads, 197 x 1569: 21 us; 64 sequences, 12 heads, 65 x 197, masked:
// 20.0 us.  A pair of tiles takes about 1900 cycles: 1094 of matrix instructions
// (128 x 128 x 64 from shared memory 257, 128 x 64 x 128 with P in tensor memory
// 290), 1024 of exponentials (4 cycles a warp and scheduler), which overlap but for
// the waits between them; the issue slots are 59% taken.  The short shapes are bound by the
// latencies of a unit's start and end.
#include <algorithm>

#include "cluster.cuh"
#include "cross_tiles.cuh"

namespace fibatt {
namespace {

constexpr float kNegInf = -__builtin_inff();
constexpr float kRaise = 8.f;    // log2 units
constexpr int kJoinLd = 68;      // floats between rows of a partial O in shared memory

template <int NT>
struct Cfg {
    static constexpr int kSoftmaxWarps = 8 * NT;
    static constexpr int kCopyWarp = kSoftmaxWarps, kKeysWarp = kSoftmaxWarps + 1;
    static constexpr int kScoreWarp = kSoftmaxWarps + 2, kValueWarp = kSoftmaxWarps + 3;
    static constexpr int kThreads = 32 * (kSoftmaxWarps + 4);   // whole warp groups
    static constexpr int kStages = NT == 2 ? 5 : 2;
    static constexpr uint32_t kCols = NT * 256;        // S 128, P 64, O 64 a tile
    static constexpr size_t kSmem = 1024 + NT * kTileBytes + kStages * 2 * kTileBytes;
    static constexpr int kMinBlocks = NT == 2 ? 1 : 2;
    static constexpr bool kWalks = NT == 1;            // one wave of CTAs for all units
    // registers a thread: at launch, and after the softmax warps took what the others gave
    static constexpr int kRegs = NT == 2 ? 96 : 80, kRegsFew = 32, kRegsMany = NT == 2 ? 112 : 104;
    static_assert(2 * NT * kRegsMany + kRegsFew == (2 * NT + 1) * kRegs, "the shares add up");
    static_assert(NT * kTileRows * kJoinLd * 4 <= NT * kTileBytes + kStages * 2 * kTileBytes, "partial O fits");
};

struct FwdMmaArgs {
    TensorArg q, k, v;
    QueryTiles qt;
    KeySet ks;
    Rows<__nv_bfloat16> O;
    float *LSE;
    int Hq, Hkv;
    int pairs;               // NT-tile units of one key/value head
    int units;               // of all heads and sequences
    float c;                 // |scale| log2 e (> 0)
    int negative;            // scale < 0
    FwdMmaArgs() : qt(1, 1, false) {}
};

// One unit of work: NT query tiles of one key/value head, ...
template <int NT>
struct Place {
    int t0, nt, hk, b;
    __device__ __forceinline__ Place() {}
    __device__ __forceinline__ Place(const FwdMmaArgs &a, int unit) {
        t0 = unit % a.pairs * NT;
        hk = unit / a.pairs % a.Hkv;
        b = unit / a.pairs / a.Hkv;
        nt = min(NT, a.qt.tiles - t0);      // tiles of this unit
    }
};
// ... and the part of its sequence's key tiles that this CTA of the cluster walks
// over.  CTAs that walk over their units have them from the copying warp.
template <int NT>
struct Unit : Place<NT> {
    int bound, lo, n;
    __device__ __forceinline__ Unit() {}
    __device__ __forceinline__ Unit(const FwdMmaArgs &a, const Place<NT> &p) : Place<NT>(p) { set(a); }
    __device__ __forceinline__ void set(const FwdMmaArgs &a) {
        const Place<NT> &p = *this;
        bound = a.ks.bound(p.b);
        const int ktiles = (bound + kTileRows - 1) / kTileRows, CS = (int)cluster_size(), rank = (int)cluster_rank();
        lo = (int)((int64_t)ktiles * rank / CS);
        n = (int)((int64_t)ktiles * (rank + 1) / CS) - lo;
    }
};

// A named barrier of `threads` threads (whole warps), and whether `p` holds in all of them.
__device__ __forceinline__ bool all_of(int id, int threads, bool p) {
    int r;
    asm volatile("{ .reg .pred p, q; setp.ne.s32 p, %1, 0; bar.red.and.pred q, %2, %3, p; selp.s32 %0, 1, 0, q; }"
                 : "=r"(r)
                 : "r"((int)p), "r"(id), "r"(threads)
                 : "memory");
    return r != 0;
}

template <int NT>
__global__ void __launch_bounds__(Cfg<NT>::kThreads, Cfg<NT>::kMinBlocks)
cross_fwd_mma_kernel(const __grid_constant__ FwdMmaArgs a) {
    using C = Cfg<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *sq = smem, *skv = smem + NT * kTileBytes;   // stage s: K at skv + 2 s tiles, V behind it
    __shared__ uint64_t bar_q, bar_qfree, bar_full[C::kStages], bar_ready[C::kStages], bar_empty[C::kStages];
    __shared__ uint64_t bar_s[NT], bar_sfree[NT], bar_p[NT], bar_o[NT], bar_end[2];
    __shared__ uint64_t bar_unit[2], bar_unitfree[2];
    __shared__ Unit<NT> units[2];       // of a CTA that walks, in turn; n < 0: no more
    __shared__ uint4 keys[C::kStages];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    __shared__ float join_m[NT * kTileRows], join_l[NT * kTileRows];
    // what the halves of a row exchange: maxima, [turn][half], and sums at a unit's end
    __shared__ float half_of[2][2][NT * kTileRows], sum_of[2][NT * kTileRows];
    volatile int *abort = &abort_flag;

    const int warp = warp_number(), lane = threadIdx.x & 31;
    const int CS = (int)cluster_size(), rank = (int)cluster_rank();
    // the CTA's units: a cluster has one, the CTAs of one wave walk over all of them
    const int first = (int)(blockIdx.x / CS), step = (int)(gridDim.x / CS);
    const Place<NT> first_place(a, first);

    if (threadIdx.x == 0) {
        mbar_init(&bar_q, 1);
        mbar_init(&bar_qfree, 1);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&bar_full[s], 1);
            mbar_init(&bar_ready[s], 1);
            mbar_init(&bar_empty[s], 1);
        }
        for (int t = 0; t < NT; ++t) {
            mbar_init(&bar_s[t], 1);
            mbar_init(&bar_sfree[t], 8);
            mbar_init(&bar_p[t], 8);
            mbar_init(&bar_o[t], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar_end[i], 1);
            mbar_init(&bar_unit[i], 1);
            mbar_init(&bar_unitfree[i], C::kSoftmaxWarps + 3);
        }
        abort_flag = 0;
        prefetch_map(&a.q.map);
        prefetch_map(&a.k.map);
        prefetch_map(&a.v.map);
    }
    if (warp == C::kValueWarp) tmem_alloc(&tmem_base, C::kCols);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = tmem_base;
    const uint32_t col_s = tmem, col_p = tmem + NT * 128, col_o = tmem + NT * 192;

    grid_dep_wait();
    grid_dep_launch();

    // body(unit) for each of the CTA's units
    const auto each = [&](auto body) {
        if constexpr (C::kWalks) {
#pragma unroll 1
            for (int k = 0;; ++k) {
                bool go = pipe_wait(&bar_unit[k & 1], (k >> 1) & 1, abort);
                __syncwarp();
                // the softmax warps meet at barriers within a unit: all of them go on, or none
                if (warp < C::kSoftmaxWarps) go = all_of(2, 32 * C::kSoftmaxWarps, go);
                if (!go || units[k & 1].n < 0) break;
                body(units[k & 1]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_unitfree[k & 1]);
            }
        } else {
            body(Unit<NT>(a, first_place));
        }
    };
    // `ring` counts the key tiles over all units of the CTA: tile `ring` is in stage
    // ring mod kStages.  A query tile's barriers complete a phase for each key tile of
    // the units that have it, which `it` counts.
    if (warp < C::kSoftmaxWarps) {
        take_registers<C::kRegsMany>();
        // ---- softmax: two threads a row, in warps four apart, 64 columns each ----------------------
        // (No wait's failure ends the loop over a unit's tiles: a warp's partner at the named barriers must find it
        // there; what follows is not trusted, since the error word is set.)
        const int t = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3, r = quarter * 32 + lane;
        const int at = t * kTileRows + r, pair_bar = 3 + 4 * t + quarter;
        const uint32_t lanes = (uint32_t)quarter << 21;   // 32 lanes, in the upper 16 bits
        const uint32_t ts = col_s + t * 128 + 64 * half + lanes, tp = col_p + t * 64 + 32 * half + lanes;
        const uint32_t to = col_o + t * 64 + 32 * half + lanes;
        int it = 0, skipped = 0;
        each([&](const Unit<NT> &u) {
            if (t >= u.nt) {
                skipped += u.n;
                return;
            }
            const int n = u.n, whole = a.ks.mask ? 0 : u.bound / kTileRows - u.lo;   // the tiles attended wholly come first
            float m = kNegInf, l = 0.f;
            uint32_t o[32];
            for (int j = 0; j < n; ++j, ++it) {
                pipe_wait(&bar_s[t], it & 1, abort);
                tc_after_sync();
                uint32_t s[2][32];
                tmem_ld32(s[0], ts);
                tmem_ld32(s[1], ts + 32);
                tmem_wait_ld(s[0]);
                tmem_pin(s[1]);
                tc_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_sfree[t]);
                if (j >= whole) {
                    const int ring = it + skipped, st = ring % C::kStages;
                    pipe_wait(&bar_ready[st], (ring / C::kStages) & 1, abort);   // keys[st] is written
                    const uint4 w = keys[st];
                    const uint32_t words[2] = {half ? w.z : w.x, half ? w.w : w.y};
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!((words[i] >> k) & 1)) s[i][k] = __float_as_uint(kNegInf);
                }
                float top[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t *x = s[i >> 1] + 16 * (i & 1);
                    top[i] = __uint_as_float(x[0]);
#pragma unroll
                    for (int k = 1; k < 15; k += 2) top[i] = max3(top[i], __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
                    top[i] = fmaxf(top[i], __uint_as_float(x[15]));
                }
                const float mine = fmaxf(max3(top[0], top[1], top[2]), top[3]);
                half_of[it & 1][half][at] = mine;
                named_sync(pair_bar, 64);
                const float next = fmaxf(mine, half_of[it & 1][half ^ 1][at]) * a.c;
                const bool free = j == 0 || pipe_ready(&bar_o[t], (it - 1) & 1);
                const bool raise = next > m + kRaise;     // also the first finite maximum: m = -inf
                const float keep = raise ? fast_exp2(m - next) : 1.f;
                if (raise) m = next;
                const float base = m == kNegInf ? 0.f : -m;
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                uint32_t p[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const int i = k >> 4, e = 2 * (k & 15);
                    const float2 x = fma2(make_float2(__uint_as_float(s[i][e]), __uint_as_float(s[i][e + 1])),
                                          make_float2(a.c, a.c), make_float2(base, base));
                    const float2 y = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                    sum[k & 1] = add2(sum[k & 1], y);
                    p[k] = pack_bf16x2(y.x, y.y);
                }
                // the product with the last P has read it and written O
                if (!free) pipe_wait(&bar_o[t], (it - 1) & 1, abort);
                tc_after_sync();
                if (j > 0 && __any_sync(kFullMask, raise)) {
                    l *= keep;
                    tmem_ld32(o, to);
                    tmem_wait_ld(o);
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * keep);
                    tmem_st32(to, o);
                }
                tmem_st32(tp, p);
                sum[0] = add2(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
                tmem_wait_st();
                tc_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_p[t]);
            }
            if (n > 0) {
                sum_of[half][at] = l;
                named_sync(pair_bar, 64);
                l += sum_of[half ^ 1][at];
                pipe_wait(&bar_o[t], (it - 1) & 1, abort);
                tc_after_sync();
                tmem_ld32(o, to);
                tmem_wait_ld(o);
                tc_before_sync();
            } else {
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = 0u;
            }
            if (CS == 1) {
                int g, q;
                if (!a.qt.at(u.t0 + t, r, g, q)) return;
                const int h = u.hk * a.qt.G + g;
                if (!FIBATT_CHECKED(h < a.Hq && u.b >= 0 && (int64_t)u.b * a.Hkv * a.pairs < a.units)) return;
                const float inv = l == 0.f ? 0.f : 1.f / l;
                uint4 *out = reinterpret_cast<uint4 *>(a.O.row(u.b, h, q) + 32 * half);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * k]) * inv, __uint_as_float(o[8 * i + 2 * k + 1]) * inv);
                    out[i] = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (half == 0) a.LSE[((int64_t)u.b * a.Hq + h) * a.qt.Nq + q] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
            } else {
                // every copy and product of this tile has completed (bar_o); the other
                // tile's may still read the ring, so a barrier of both comes first
                named_sync(2, 32 * 8 * u.nt);
                float4 *out =
                    reinterpret_cast<float4 *>(reinterpret_cast<float *>(smem) + (t * kTileRows + r) * kJoinLd + 32 * half);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    out[i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                         __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                if (half == 0) {
                    join_m[t * kTileRows + r] = m;
                    join_l[t * kTileRows + r] = l;
                }
            }
        });
    } else {
        give_registers<C::kRegsFew>();
        if (warp == C::kCopyWarp) {
            // ---- copies: they run ahead into the next unit ------------------------------
            int ring = 0, loaded = 0;      // issued: key tiles, units' queries
            bool ok = true;
            const auto queries = [&](const Unit<NT> &u) {
                if (elect_one()) {
                    mbar_expect_tx(&bar_q, u.nt * a.qt.bytes());
                    for (int t = 0; t < u.nt; ++t)
                        load_tile(sq + t * kTileBytes, a.q, a.qt.first_row(u.t0 + t), u.hk * a.qt.G + a.qt.first_head(u.t0 + t),
                                  u.b, &bar_q);
                }
                __syncwarp();
                ++loaded;
            };
            const auto copies = [&](const Unit<NT> &u) {
                const bool later = C::kWalks && loaded > 0;
                for (int j = 0; ok && j < u.n; ++j) {
                    if (j == 0 && !later) queries(u);
                    const int s = ring % C::kStages;
                    ok = ring < C::kStages || pipe_wait(&bar_empty[s], (ring / C::kStages - 1) & 1, abort);
                    if (!ok) break;
                    if (elect_one()) {
                        mbar_expect_tx(&bar_full[s], 2 * kTileBytes);
                        load_tile(skv + (2 * s) * kTileBytes, a.k, (u.lo + j) * kTileRows, u.hk, u.b, &bar_full[s]);
                        load_tile(skv + (2 * s + 1) * kTileBytes, a.v, (u.lo + j) * kTileRows, u.hk, u.b, &bar_full[s]);
                    }
                    __syncwarp();
                    ++ring;
                    if (j == 0 && later) {      // once the scores have read the last queries
                        ok = pipe_wait(&bar_qfree, (loaded - 1) & 1, abort);
                        if (ok) queries(u);
                    }
                }
            };
            if constexpr (C::kWalks) {
#pragma unroll 1
                for (int k = 0, unit = first; ok; ++k, unit += step) {
                    Unit<NT> u;
                    if (unit < a.units) u = Unit<NT>(a, k ? Place<NT>(a, unit) : first_place);
                    else u.n = -1;
                    ok = k < 2 || pipe_wait(&bar_unitfree[k & 1], ((k >> 1) - 1) & 1, abort);
                    if (!ok) break;
                    if (lane == 0) {
                        units[k & 1] = u;
                        mbar_arrive(&bar_unit[k & 1]);
                    }
                    __syncwarp();
                    if (u.n < 0) break;
                    copies(u);
                }
            } else {
                copies(Unit<NT>(a, first_place));
            }
            // leave no copy in flight
            if (lane == 0) {
                if (loaded > 0) mbar_drain(&bar_q, (loaded - 1) & 1);
                for (int i = max(0, ring - C::kStages); i < ring; ++i)
                    mbar_drain(&bar_full[i % C::kStages], (i / C::kStages) & 1);
            }
        } else if (warp == C::kKeysWarp) {
            // ---- which keys of each tile are attended; the others' value rows cleared ----
            int ring = 0;
            bool ok = true;
            each([&](const Unit<NT> &u) {
                const int n = u.n;
                for (int j = 0; ok && j < n; ++j, ++ring) {
                    const int s = ring % C::kStages;
                    const uint4 w = tile_keys(a.ks, u.b, (u.lo + j) * kTileRows, u.bound);
                    ok = pipe_wait(&bar_full[s], (ring / C::kStages) & 1, abort);
                    if (!ok) break;
                    if (!all_keys(w)) {
                        clear_rows(skv + (2 * s + 1) * kTileBytes, w);
                        fence_smem_async();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        keys[s] = w;
                        mbar_arrive(&bar_ready[s]);
                    }
                }
            });
        } else {
            // ---- matrix instructions: the scores by one warp, the values by another, so that
            // neither waits for what the other needs.  The loops' course depends on uniform values
            // only, which keeps descriptors and counters in uniform registers.
            int s = 0, pass = 0;                    // stage of the key tile and its pass through the ring
            int it[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) it[t] = 0;
            if (warp == C::kScoreWarp) {
                const uint32_t id = mma_desc(128, 128, false, a.negative);
                const uint64_t dq = tile_desc(sq), dk = tile_desc(skv);
                int loaded = 0;
                each([&](const Unit<NT> &u) {
                    const int n = __shfl_sync(kFullMask, u.n, 0), nt = __shfl_sync(kFullMask, u.nt, 0);
                    if (n > 0) pipe_wait(&bar_q, loaded++ & 1, abort);
                    for (int j = 0; j < n; ++j) {
                        pipe_wait(&bar_full[s], pass, abort);      // masked keys' scores are not looked at
                        const uint64_t dks = dk + (uint64_t)(s * (2 * kTileBytes >> 4));
#pragma unroll
                        for (int t = 0; t < NT; ++t) {   // S_t = Q_t K_j^T
                            if (t >= nt) break;
                            if (it[t] > 0) pipe_wait(&bar_sfree[t], (it[t] - 1) & 1, abort);
                            ++it[t];
                            tc_after_sync();
                            const uint64_t dqt = dq + (uint64_t)(t * (kTileBytes >> 4));
                            if (elect_one()) {
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    mma_ss(col_s + t * 128, dqt + i * kStepRowwise, dks + i * kStepRowwise, id, i > 0);
                                mma_commit(&bar_s[t]);
                                if (j == n - 1 && t == nt - 1) mma_commit(&bar_qfree);
                            }
                            __syncwarp();
                        }
                        if (++s == C::kStages) {
                            s = 0;
                            pass ^= 1;
                        }
                    }
                });
            } else {
                const uint32_t id = mma_desc(128, 64, true);
                const uint64_t dv = tile_desc(skv + kTileBytes);
                each([&](const Unit<NT> &u) {
                    const int n = __shfl_sync(kFullMask, u.n, 0), nt = __shfl_sync(kFullMask, u.nt, 0);
                    for (int j = 0; j < n; ++j) {
                        pipe_wait(&bar_ready[s], pass, abort);
                        const uint64_t dvs = dv + (uint64_t)(s * (2 * kTileBytes >> 4));
#pragma unroll
                        for (int t = 0; t < NT; ++t) {   // O_t += P_t V_j
                            if (t >= nt) break;
                            pipe_wait(&bar_p[t], it[t] & 1, abort);
                            ++it[t];
                            tc_after_sync();
                            if (elect_one()) {
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    mma_ts(col_o + t * 64, col_p + t * 64 + i * 8, dvs + i * kStepAcross, id, j > 0 || i > 0);
                                mma_commit(&bar_o[t]);
                                if (t == nt - 1) mma_commit(&bar_empty[s]);
                            }
                            __syncwarp();
                        }
                        if (++s == C::kStages) {
                            s = 0;
                            pass ^= 1;
                        }
                    }
                });
            }
            // no matrix instruction in flight when the tensor memory is freed
            uint64_t *end = &bar_end[warp == C::kValueWarp];
            if (elect_one()) mma_commit(end);
            __syncwarp();
            mbar_drain(end, 0);
        }
    }
    __syncwarp();
    tc_before_sync();
    __syncthreads();
    if (warp == C::kValueWarp) tmem_free(tmem, C::kCols);
    if (CS == 1) return;

    // ---- join: CTA r of the cluster finishes every CS-th row ------------------------
    cluster_sync();
    const Unit<NT> u(a, first_place);
    const float *part = reinterpret_cast<const float *>(smem);
    const int groups = C::kThreads / 16, c4 = (threadIdx.x & 15) * 4;
    for (int i = rank + CS * (int)(threadIdx.x >> 4); i < u.nt * kTileRows; i += CS * groups) {
        int g, q;
        if (!a.qt.at(u.t0 + i / kTileRows, i % kTileRows, g, q)) continue;
        float top = kNegInf;
        for (int k = 0; k < CS; ++k) top = fmaxf(top, ld_cluster(cluster_addr(join_m + i, k)));
        const float base = top == kNegInf ? 0.f : top;
        float sum = 0.f;
        float2 x = make_float2(0.f, 0.f), y = x;
        for (int k = 0; k < CS; ++k) {
            const float w = fast_exp2(ld_cluster(cluster_addr(join_m + i, k)) - base);
            sum = fmaf(w, ld_cluster(cluster_addr(join_l + i, k)), sum);
            const uint32_t at = cluster_addr(part + i * kJoinLd + c4, k);
            x = fma2(make_float2(w, w), ld_cluster2(at), x);
            y = fma2(make_float2(w, w), ld_cluster2(at + 8), y);
        }
        const int h = u.hk * a.qt.G + g;
        if (!FIBATT_CHECKED(h < a.Hq && u.b >= 0 && (int64_t)u.b * a.Hkv * a.pairs < a.units)) continue;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<uint2 *>(a.O.row(u.b, h, q) + c4) =
            make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(y.x * inv, y.y * inv));
        if (c4 == 0) a.LSE[((int64_t)u.b * a.Hq + h) * a.qt.Nq + q] = sum == 0.f ? kNegInf : (top + log2f(sum)) * kLn2;
    }
    cluster_sync();   // the others may still read this CTA's part
}

// How many clusters of 2^i CTAs device `dev`, the current one, holds at once.
template <int NT>
int held_clusters(int dev, int i) {
    using C = Cfg<NT>;
    static PerDevice known[5];
    return known[i].get(dev, [=] {
        return i == 0 ? C::kMinBlocks * sm_count()
                      : clusters_held<cross_fwd_mma_kernel<NT>>(1 << i, C::kThreads, C::kSmem);
    });
}

// Query tiles of a CTA and CTAs of a cluster: those with the shortest estimate
//   rounds (key tiles of a CTA x time of one + start, end and join)
// in us, from what was measured: a key tile takes a CTA with both of its query
// tiles 1.0, with one 0.78, a CTA of one tile 0.83, or 1.28 with another on its SM; a
// round's other time is 5, of a cluster 9.5, of CTAs that walk over their units 3.
// (2 sequences, 16 heads, 1569 x 16385, 224 units of 152: clusters of one 266 us, of
// two 229, of four 289; 8 sequences, 12 heads, 197 x 1569, 96 units: 20, 35, 48; one
// sequence, 16 heads, 197 x 4096: one-tile CTAs, clusters of one 31, of four 16.5, of
// eight 18, two-tile CTAs 37, 19 and 31; 768 units of one tile by two: one-tile CTAs
// 16.5, two-tile ones 23; one head, 100 x 16385: clusters of eight 21.7, of sixteen 17.3.)
struct Plan {
    int nt = 0, c = 1;
    float cost = 0.f;
};
template <int NT>
cudaError_t consider(const CrossArgs &a, const QueryTiles &qt, Plan *best) {
    using C = Cfg<NT>;
    const cudaError_t e = prepare_kernel<cross_fwd_mma_kernel<NT>>(C::kSmem, C::kRegs);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)a.B * a.Hkv * ((qt.tiles + NT - 1) / NT);
    const int tiles = (a.Nk + kTileRows - 1) / kTileRows, dev = current_device();
    for (int i = 0; i < 5 && (i == 0 || tiles >= 1 << i); ++i) {
        const int c = 1 << i, held = held_clusters<NT>(dev, i);
        if (held < 1) break;
        const float tile = NT == 2 ? (qt.tiles > 1 ? 1.f : 0.78f) : units * c > sm_count() ? 1.28f : 0.83f;
        const float rounds = (float)((units + held - 1) / held), mine = (float)((tiles + c - 1) / c) * tile;
        const float cost = i > 0          ? rounds * (mine + 9.5f)
                           : C::kWalks ? rounds * (mine + 3.f) + 2.f
                                       : rounds * (mine + 5.f);
        if (!best->nt || cost < best->cost) *best = Plan{NT, c, cost};
    }
    return cudaSuccess;
}

template <int NT>
cudaError_t fwd(const CrossArgs &a, const QueryTiles &qt, int c) {
    using C = Cfg<NT>;
    FwdMmaArgs f;
    f.qt = qt;
    if (!make_tensor(&f.q, a.Q, a.B, a.Hq, a.Nq, qt.nb, qt.gb) || !make_tensor(&f.k, a.K, a.B, a.Hkv, a.Nk, kTileRows, 1) ||
        !make_tensor(&f.v, a.V, a.B, a.Hkv, a.Nk, kTileRows, 1))
        return cudaErrorInvalidValue;
    f.ks = a.keys;
    f.O = rows_of<__nv_bfloat16>(a.O);
    f.LSE = a.LSE;
    f.Hq = a.Hq, f.Hkv = a.Hkv;
    f.pairs = (qt.tiles + NT - 1) / NT;
    // a scale of 0: any c this small leaves every finite score's weight at 1,
    // and -inf of a masked key times c is still -inf
    f.c = std::max(std::fabs(a.scale) * kLog2e, 1e-36f);
    f.negative = a.scale < 0.f;
    const int64_t units = (int64_t)a.B * a.Hkv * f.pairs;
    f.units = (int)units;
    const int64_t grid = c > 1 || !C::kWalks ? units * c : std::min<int64_t>(units, C::kMinBlocks * sm_count());
    return launch_clusters(cross_fwd_mma_kernel<NT>, (unsigned)grid, c, C::kThreads, C::kSmem, a.stream, f);
}

}  // namespace

cudaError_t launch_cross_fwd_mma(const CrossArgs &a) {
    const QueryTiles qt(a.Hq / a.Hkv, a.Nq, a.Hq > 1 && a.Q.stride_h == 0);
    Plan plan;
    cudaError_t e = consider<1>(a, qt, &plan);
    if (e == cudaSuccess) e = consider<2>(a, qt, &plan);
    if (e != cudaSuccess) return e;
    return plan.nt == 2 ? fwd<2>(a, qt, plan.c) : fwd<1>(a, qt, plan.c);
}

FIBATT_DEFINE_ERROR_READER(read_error_cross_mma_fwd, "cross_mma_fwd.cu")

}  // namespace fibatt
