// Cross attention forward on the tensor cores (bf16).
//
// A CTA holds NT tiles of 128 query rows of one key/value head and walks over
// the 128-key tiles of its sequence:
//   S = Q K^T          128 x 128, fp32 in tensor memory (2 x 128 x 128 x 64 flops)
//   P = exp2(c S - m)  two threads own a row, 64 columns each, and exchange their
//                      maxima through shared memory
//   O += P V           P back to tensor memory as bf16, V across its rows
// Warps: 8 per tile for the softmax (four on every scheduler: with one thread a row,
// two, a tile pair took 2090 cycles, most of them waits), one that copies (tensor copies into a ring of
// K/V stages), one that finds each tile's attended keys and clears the other value
// rows, two that issue the matrix instructions.  S of the next key tile is formed while the softmax works on
// this one (S and P have columns of their own), so the tensor cores and the
// exponentials, which take about as long at a head dim of 64, overlap.
//
// The running maximum is raised only when a score exceeds it by more than
// 2^8 (P stays below 256, exact enough in fp32 sums and as relative bf16), so
// O is almost never rescaled; a rescaling reads and rewrites O in tensor memory
// between two products.  P is rounded to bf16 for its product (relative
// 2^-8 a weight, averaging out over the keys); l adds the unrounded weights.
//
// With few units the keys are cut over a cluster, whose CTAs join their (m,
// l, O) through distributed shared memory in rank order.
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
    float c;                 // |scale| log2 e (> 0)
    int negative;            // scale < 0
    FwdMmaArgs() : qt(1, 1, false) {}
};

template <int NT>
__global__ void __launch_bounds__(Cfg<NT>::kThreads, Cfg<NT>::kMinBlocks)
cross_fwd_mma_kernel(const __grid_constant__ FwdMmaArgs a) {
    using C = Cfg<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *sq = smem, *skv = smem + NT * kTileBytes;   // stage s: K at skv + 2 s tiles, V behind it
    __shared__ uint64_t bar_q, bar_full[C::kStages], bar_ready[C::kStages], bar_empty[C::kStages];
    __shared__ uint64_t bar_s[NT], bar_sfree[NT], bar_p[NT], bar_o[NT], bar_end[2];
    __shared__ uint4 keys[C::kStages];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    __shared__ float join_m[NT * kTileRows], join_l[NT * kTileRows];
    __shared__ float half_of[2][2][NT * kTileRows];    // [turn][half]: what the halves of a row exchange
    volatile int *abort = &abort_flag;

    const int warp = warp_number(), lane = threadIdx.x & 31;
    const int CS = (int)cluster_size(), rank = (int)cluster_rank();
    const int64_t unit = blockIdx.x / CS;
    const int pair = (int)(unit % a.pairs), hk = (int)(unit / a.pairs % a.Hkv), b = (int)(unit / a.pairs / a.Hkv);
    const int t0 = pair * NT, nt = min(NT, a.qt.tiles - t0);   // tiles of this unit

    if (threadIdx.x == 0) {
        mbar_init(&bar_q, 1);
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
        mbar_init(&bar_end[0], 1);
        mbar_init(&bar_end[1], 1);
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
    const int bound = a.ks.bound(b), ktiles = (bound + kTileRows - 1) / kTileRows;
    const int lo = (int)((int64_t)ktiles * rank / CS), n = (int)((int64_t)ktiles * (rank + 1) / CS) - lo;

    if (warp < C::kSoftmaxWarps) {
        take_registers<C::kRegsMany>();
        // ---- softmax: two threads a row, in warps four apart, 64 columns each ----------------------
        // (No wait's failure ends the loop: a warp's partner at the named barriers must find it
        // there; what follows is not trusted, since the error word is set.)
        const int t = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3, r = quarter * 32 + lane;
        const int at = t * kTileRows + r, pair_bar = 3 + 4 * t + quarter;
        const uint32_t lanes = (uint32_t)quarter << 21;   // 32 lanes, in the upper 16 bits
        const uint32_t ts = col_s + t * 128 + 64 * half + lanes, tp = col_p + t * 64 + 32 * half + lanes;
        const uint32_t to = col_o + t * 64 + 32 * half + lanes;
        float m = kNegInf, l = 0.f;
        uint32_t o[32];
        if (t < nt) {
            for (int j = 0; j < n; ++j) {
                pipe_wait(&bar_s[t], j & 1, abort);
                tc_after_sync();
                uint32_t s[2][32];
                tmem_ld32(s[0], ts);
                tmem_ld32(s[1], ts + 32);
                tmem_wait_ld(s[0]);
                tmem_pin(s[1]);
                tc_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_sfree[t]);
                if (a.ks.mask || (lo + j + 1) * kTileRows > bound) {
                    const int st = j % C::kStages;
                    pipe_wait(&bar_ready[st], (j / C::kStages) & 1, abort);   // keys[st] is written
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
                half_of[j & 1][half][at] = mine;
                named_sync(pair_bar, 64);
                const float next = fmaxf(mine, half_of[j & 1][half ^ 1][at]) * a.c;
                const bool free = j == 0 || pipe_ready(&bar_o[t], (j - 1) & 1);
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
                if (!free) pipe_wait(&bar_o[t], (j - 1) & 1, abort);
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
            half_of[n & 1][half][at] = l;
            named_sync(pair_bar, 64);
            l += half_of[n & 1][half ^ 1][at];
            if (n > 0) {
                pipe_wait(&bar_o[t], (n - 1) & 1, abort);
                tc_after_sync();
                tmem_ld32(o, to);
                tmem_wait_ld(o);
            } else {
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = 0u;
            }
        }
        int g, q;
        const bool row = t < nt && a.qt.at(t0 + t, r, g, q);
        if (CS == 1) {
            if (row) {
                const int h = hk * a.qt.G + g;
                const float inv = l == 0.f ? 0.f : 1.f / l;
                uint4 *out = reinterpret_cast<uint4 *>(a.O.row(b, h, q) + 32 * half);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * k]) * inv, __uint_as_float(o[8 * i + 2 * k + 1]) * inv);
                    out[i] = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (half == 0) a.LSE[((int64_t)b * a.Hq + h) * a.qt.Nq + q] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
            }
        } else if (t < nt) {
            // every copy and product of this tile has completed (bar_o); the other
            // tile's may still read the ring, so a barrier of both comes first
            named_sync(2, 32 * 8 * nt);
            float4 *out =
                reinterpret_cast<float4 *>(reinterpret_cast<float *>(smem) + (t * kTileRows + r) * kJoinLd + 32 * half);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                out[i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]), __uint_as_float(o[4 * i + 2]),
                                     __uint_as_float(o[4 * i + 3]));
            if (half == 0) {
                join_m[t * kTileRows + r] = m;
                join_l[t * kTileRows + r] = l;
            }
        }
    } else {
        give_registers<C::kRegsFew>();
        if (warp == C::kCopyWarp) {
            // ---- copies -----------------------------------------------------------
            if (n > 0) {
                int issued = 0;
                const auto issue = [&](int j) {   // key tile j into its stage
                    const int s = j % C::kStages;
                    if (elect_one()) {
                        mbar_expect_tx(&bar_full[s], 2 * kTileBytes);
                        load_tile(skv + (2 * s) * kTileBytes, a.k, (lo + j) * kTileRows, hk, b, &bar_full[s]);
                        load_tile(skv + (2 * s + 1) * kTileBytes, a.v, (lo + j) * kTileRows, hk, b, &bar_full[s]);
                    }
                    __syncwarp();
                };
                if (elect_one()) {
                    mbar_expect_tx(&bar_q, nt * a.qt.bytes());
                    for (int t = 0; t < nt; ++t)
                        load_tile(sq + t * kTileBytes, a.q, a.qt.first_row(t0 + t), hk * a.qt.G + a.qt.first_head(t0 + t), b,
                                  &bar_q);
                }
                __syncwarp();
                for (; issued < n; ++issued) {
                    const int last = issued - C::kStages;     // the stage's tile before
                    if (last >= 0 && !pipe_wait(&bar_empty[last % C::kStages], (last / C::kStages) & 1, abort)) break;
                    issue(issued);
                }
                // leave no copy in flight
                if (lane == 0) {
                    mbar_drain(&bar_q, 0);
                    for (int j = max(0, issued - C::kStages); j < issued; ++j)
                        mbar_drain(&bar_full[j % C::kStages], (j / C::kStages) & 1);
                }
            }
        } else if (warp == C::kKeysWarp) {
            // ---- which keys of each tile are attended; the others' value rows cleared ----
            for (int j = 0; j < n; ++j) {
                const int s = j % C::kStages;
                const uint4 w = tile_keys(a.ks, b, (lo + j) * kTileRows, bound);
                if (!pipe_wait(&bar_full[s], (j / C::kStages) & 1, abort)) break;
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
        } else {
            // ---- matrix instructions: the scores by one warp, the values by another, so that
            // neither waits for what the other needs.  The loops' course depends on uniform values
            // only, which keeps descriptors and counters in uniform registers.
            const int nu = __shfl_sync(kFullMask, n, 0), ntu = __shfl_sync(kFullMask, nt, 0);
            int s = 0, ring = 0;                    // stage of tile j and its pass through the ring
            if (warp == C::kScoreWarp) {
                const uint32_t id = mma_desc(128, 128, false, a.negative);
                const uint64_t dq = tile_desc(sq), dk = tile_desc(skv);
                if (nu > 0) pipe_wait(&bar_q, 0, abort);
                for (int j = 0; j < nu; ++j) {
                    pipe_wait(&bar_ready[s], ring, abort);
                    const uint64_t dks = dk + (uint64_t)(s * (2 * kTileBytes >> 4));
                    for (int t = 0; t < ntu; ++t) {   // S_t = Q_t K_j^T
                        if (j > 0) pipe_wait(&bar_sfree[t], (j - 1) & 1, abort);
                        tc_after_sync();
                        const uint64_t dqt = dq + (uint64_t)(t * (kTileBytes >> 4));
                        if (elect_one()) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mma_ss(col_s + t * 128, dqt + i * kStepRowwise, dks + i * kStepRowwise, id, i > 0);
                            mma_commit(&bar_s[t]);
                        }
                        __syncwarp();
                    }
                    if (++s == C::kStages) {
                        s = 0;
                        ring ^= 1;
                    }
                }
            } else {
                const uint32_t id = mma_desc(128, 64, true);
                const uint64_t dv = tile_desc(skv + kTileBytes);
                for (int j = 0; j < nu; ++j) {
                    const uint64_t dvs = dv + (uint64_t)(s * (2 * kTileBytes >> 4));
                    for (int t = 0; t < ntu; ++t) {   // O_t += P_t V_j
                        pipe_wait(&bar_p[t], j & 1, abort);
                        tc_after_sync();
                        if (elect_one()) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                mma_ts(col_o + t * 64, col_p + t * 64 + i * 8, dvs + i * kStepAcross, id, j > 0 || i > 0);
                            mma_commit(&bar_o[t]);
                            if (t == ntu - 1) mma_commit(&bar_empty[s]);
                        }
                        __syncwarp();
                    }
                    if (++s == C::kStages) s = 0;
                }
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
    const float *part = reinterpret_cast<const float *>(smem);
    const int groups = C::kThreads / 16, c4 = (threadIdx.x & 15) * 4;
    for (int i = rank + CS * (int)(threadIdx.x >> 4); i < nt * kTileRows; i += CS * groups) {
        int g, q;
        if (!a.qt.at(t0 + i / kTileRows, i % kTileRows, g, q)) continue;
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
        const int h = hk * a.qt.G + g;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        *reinterpret_cast<uint2 *>(a.O.row(b, h, q) + c4) =
            make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(y.x * inv, y.y * inv));
        if (c4 == 0) a.LSE[((int64_t)b * a.Hq + h) * a.qt.Nq + q] = sum == 0.f ? kNegInf : (top + log2f(sum)) * kLn2;
    }
    cluster_sync();   // the others may still read this CTA's part
}

template <int NT>
cudaError_t fwd(const CrossArgs &a, const QueryTiles &qt) {
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
    const cudaError_t e = prepare_kernel<cross_fwd_mma_kernel<NT>>(C::kSmem, C::kRegs);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)a.B * a.Hkv * f.pairs;
    const int tiles = (a.Nk + kTileRows - 1) / kTileRows;
    int c = 1;
    while (c < 8 && units * c * 2 <= (int64_t)C::kMinBlocks * sm_count() && tiles >= 2 * c) c *= 2;
    return launch_clusters(cross_fwd_mma_kernel<NT>, (unsigned)(units * c), c, C::kThreads, C::kSmem, a.stream, f);
}

}  // namespace

cudaError_t launch_cross_fwd_mma(const CrossArgs &a) {
    const QueryTiles qt(a.Hq / a.Hkv, a.Nq, a.Hq > 1 && a.Q.stride_h == 0);
    return qt.tiles > 1 ? fwd<2>(a, qt) : fwd<1>(a, qt);
}

FIBATT_DEFINE_ERROR_READER(read_error_cross_mma_fwd, "cross_mma_fwd.cu")

}  // namespace fibatt
