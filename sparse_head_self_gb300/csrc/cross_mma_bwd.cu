// Cross attention backward on the tensor cores (bf16): dQ, and dK with dV, from
//   S = scale log2 e Q K^T,  P = exp2(S - LSE log2 e),  dP = dO V^T,
//   dS = P (dP - D),  D = <dO, O>
//   dQ = scale dS K,   dK = scale dS^T Q,   dV = P^T dO.
// Every CTA holds 128 rows of one side and walks over the 128-row tiles of the
// other:
//   queries held (Q, dO):  S, dP are queries x keys;  dQ += dS K_j
//   keys held (K, V):      S^T, dP^T are keys x queries, over the queries of every
//                          head that shares the key head;  dV += P^T dO_i,
//                          dK += dS^T Q_i
// With keys held, a query's LSE and D belong to a column, and every thread needs
// them all: read from shared memory they would take as much of its bandwidth as
// the products do (1024 cycles a tile pair).  They come with the
// products instead: one more k-step, in which the keys' side is ones and the queries'
// side the value in three bf16 parts (24 bits), so S and dP arrive as
// S - LSE / scale and dP - D.  A small kernel before this one computes D and writes
// the parts as that k-step's tile reads them, so that a plain copy brings them.
// Each gradient row is thus summed by one CTA (or one cluster, joined in rank
// order): no atomics, a fixed order.  S and dP are formed twice (7 products of
// 128 x 128 x 64 a tile pair instead of 5); the alternative, one pass that adds
// dQ to memory with atomics, depends on scheduling.
//
// Both kinds of CTA are blocks of one launch.  Warps: 16 that turn S and dP into
// P and dS (a warp has 32 rows and 32 columns of the tile; four warps on every
// scheduler hide each other's waits), one that copies, one that prepares what
// goes with a key tile (the keys attended, the clearing of the others), two that issue the matrix instructions.  The next tile's S and
// dP are formed while this one's P and dS are made.  The weights' side of every
// product over rows is read from tensor memory, as bf16 (relative rounding 2^-8
// a weight, averaging out over the sum).
#include <algorithm>

#include "cluster.cuh"
#include "cross_tiles.cuh"

namespace fibatt {
namespace {

constexpr float kInf = __builtin_inff();
constexpr int kGroups = 4;                        // column groups of a tile, 32 columns each
constexpr int kWeightWarps = 4 * kGroups;
constexpr int kCopyWarp = kWeightWarps, kPrepWarp = kWeightWarps + 1, kScoreWarp = kWeightWarps + 2, kSumWarp = kWeightWarps + 3;
constexpr int kThreads = 32 * (kWeightWarps + 4);
constexpr int kStages = 4;
constexpr int kNarrow = kTileRows * 32;           // bytes of a tile one k-step wide
constexpr size_t kSmem = 1024 + (2 + 2 * kStages) * kTileBytes + (1 + 2 * kStages) * kNarrow;
constexpr int kJoinLd = 68;                       // floats between rows of a partial sum in shared memory
static_assert(2 * kTileRows * kJoinLd * 4 <= 2 * kStages * kTileBytes, "partial sums fit");
// registers a thread: at launch, and after the weight warps took what the others gave
constexpr int kRegs = 96, kRegsFew = 32, kRegsMany = 112;
static_assert(4 * kRegsMany + kRegsFew == 5 * kRegs, "the shares add up");

// columns of tensor memory
constexpr uint32_t kColS = 0, kColDp = 128, kColP = 256, kColDs = 320, kColAcc0 = 384, kColAcc1 = 448, kCols = 512;

struct BwdMmaArgs {
    TensorArg q, g, k, v;       // boxes of query tiles (Q, dO) and of key tiles (K, V)
    QueryTiles qt;
    KeySet ks;
    const float2 *stats;        // (LSE log2 e, D) of every query row
    const uint4 *lse_parts, *d_parts;   // of every query row of whole tiles, then 128 rows of no query
    int npad;                   // rows of a head there
    Rows<__nv_bfloat16> dQ, dK, dV;
    int B, Hq, Hkv, ktiles;
    int key_blocks;             // clusters that hold keys; the others hold queries
    float scale;
    float c;                    // scale log2 e, not 0
    BwdMmaArgs() : qt(1, 1, false) {}
};

struct Shared {
    uint64_t held, full[kStages], ready[kStages], empty[kStages], s, sfree, p, done, end[2];
    uint4 keys[kStages];
    uint32_t tmem;
    int abort;
};

// x as the sum of three bf16 values, the first of eight elements of a row (cut to
// what a bf16 holds: at a scale of 0, 1000 / c is beyond it).
__device__ __forceinline__ uint4 three_parts(float x) {
    x = fminf(fmaxf(x, -3.0e38f), 3.0e38f);
    const float hi = __bfloat162float(__float2bfloat16_rn(x)), rest = x - hi;
    const float mid = __bfloat162float(__float2bfloat16_rn(rest));
    return make_uint4(pack_bf16x2(hi, mid), pack_bf16x2(rest - mid, 0.f), 0u, 0u);
}

// What stands for a query that does not exist: a weight of exp2(-1000) = 0.
__device__ __forceinline__ uint4 no_query(float c) { return three_parts(-1000.f / c); }

// (LSE log2 e, D = <dO, O>) of every query row, and -LSE log2 e / c and -D in
// parts, rows padded to `npad` a head and 128 rows of no query at the end.  16
// threads a row.
__global__ void __launch_bounds__(256)
cross_parts_kernel(int Hq, int Nq, int npad, int64_t rows, Rows<const __nv_bfloat16> O, Rows<const __nv_bfloat16> dO,
                   const float *__restrict__ LSE, float c, float2 *__restrict__ stats, uint4 *__restrict__ lse_parts,
                   uint4 *__restrict__ d_parts) {
    grid_dep_wait();
    grid_dep_launch();
    const int64_t row = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
    const int i = threadIdx.x & 15;
    if (row >= rows + kTileRows) return;   // whole half warps: the shuffles below stay within 16 lanes
    const int64_t bh = row / npad, n = row - bh * npad;
    if (row >= rows || n >= Nq) {
        if (i == 0) lse_parts[row] = no_query(c);
        if (i == 1) d_parts[row] = make_uint4(0, 0, 0, 0);
        return;
    }
    const int64_t b = bh / Hq, h = bh - b * Hq;
    const uint2 o = __ldg(reinterpret_cast<const uint2 *>(O.row(b, h, n)) + i);
    const uint2 g = __ldg(reinterpret_cast<const uint2 *>(dO.row(b, h, n)) + i);
    float d = dot2_bf16(o.x, g.x, dot2_bf16(o.y, g.y, 0.f));
    const unsigned half = 0xffffu << (threadIdx.x & 16);
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) d += __shfl_xor_sync(half, d, m);
    const float lse = __ldg(LSE + bh * Nq + n);
    // a row without keys: its weights are exp2(s - inf) = 0 (and no block meets it)
    const bool none = lse == -kInf;
    const float lse2 = none ? kInf : lse * kLog2e;
    if (i == 0) lse_parts[row] = none ? no_query(c) : three_parts(-lse2 / c);
    if (i == 1) d_parts[row] = three_parts(-d);
    if (i == 2) stats[bh * Nq + n] = make_float2(lse2, d);
}

template <bool KEYS>
__device__ __forceinline__ void run(const BwdMmaArgs &a, Shared &sh, uint8_t *smem, int64_t unit) {
    uint8_t *held = smem, *ring = smem + 2 * kTileBytes;    // stage s: K or Q at ring + 2 s tiles, V or dO behind it
    uint8_t *ones = ring + 2 * kStages * kTileBytes, *parts = ones + kNarrow;   // stage s: LSE at parts + 2 s, D behind it
    volatile int *abort = &sh.abort;
    const int warp = warp_number(), lane = threadIdx.x & 31;
    const int CS = (int)cluster_size(), rank = (int)cluster_rank();
    const int tiles_held = KEYS ? a.ktiles : a.qt.tiles;
    const int mine = (int)(unit % tiles_held), hk = (int)(unit / tiles_held % a.Hkv),
              b = (int)(unit / tiles_held / a.Hkv);
    const uint32_t tmem = sh.tmem;
    const int bound = a.ks.bound(b);
    // the tiles streamed: none for a key tile without keys, or for queries without any
    int64_t tiles;
    uint4 mykeys = make_uint4(0, 0, 0, 0);
    if (KEYS) {
        mykeys = tile_keys(a.ks, b, mine * kTileRows, bound);
        tiles = no_keys(mykeys) ? 0 : a.qt.tiles;
    } else {
        tiles = (bound + kTileRows - 1) / kTileRows;
    }
    const int lo = (int)(tiles * rank / CS), n = (int)(tiles * (rank + 1) / CS) - lo;
    const uint32_t held_bytes = 2 * (KEYS ? (uint32_t)kTileBytes : a.qt.bytes());
    const uint32_t tile_bytes = 2 * (KEYS ? a.qt.bytes() + a.qt.bytes() / 8 : (uint32_t)kTileBytes);

    if (warp < kWeightWarps) {
        take_registers<kRegsMany>();
        // ---- P and dS: row = lane of the quarter, 32 columns ---------------------------------
        const int cg = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        float row_lse = -kInf, row_d = 0.f;     // of a held query: -LSE log2 e, -D
        int g = 0, q = 0;
        const bool row = KEYS ? mine * kTileRows + r < a.ks.Nk : a.qt.at(mine, r, g, q);
        if (!KEYS && row) {
            const float2 st = a.stats[((int64_t)b * a.Hq + hk * a.qt.G + g) * a.qt.Nq + q];
            row_lse = -st.x;
            row_d = -st.y;
        }
        const float c = a.c;
        const float2 cc = make_float2(c, c);
        for (int j = 0; j < n; ++j) {
            const int s = j % kStages;
            pipe_wait(&sh.s, j & 1, abort);
            tc_after_sync();
            uint32_t x[32], y[32];
            tmem_ld32(x, tmem + kColS + 32 * cg + lanes);
            tmem_ld32(y, tmem + kColDp + 32 * cg + lanes);
            tmem_wait_ld(x);
            tmem_pin(y);
            tc_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.sfree);
            uint32_t keep = 0xffffffffu;
            if (!KEYS && (a.ks.mask || (lo + j + 1) * kTileRows > bound)) {
                const uint4 w = sh.keys[s];
                keep = cg == 0 ? w.x : cg == 1 ? w.y : cg == 2 ? w.z : w.w;
            }
            const bool free = j == 0 || pipe_ready(&sh.done, (j - 1) & 1);
            uint32_t p[16], ds[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 sx = make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
                const float2 dp = make_float2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1]));
                const float2 z = KEYS ? mul2(sx, cc) : fma2(sx, cc, make_float2(row_lse, row_lse));
                const float2 w = make_float2(fast_exp2(z.x), fast_exp2(z.y));
                const float2 t = mul2(w, KEYS ? dp : add2(dp, make_float2(row_d, row_d)));
                if (KEYS) p[i] = pack_bf16x2(w.x, w.y);
                ds[i] = pack_bf16x2(t.x, t.y);
            }
            if (!KEYS && keep != 0xffffffffu) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (!((keep >> (2 * i)) & 1)) ds[i] &= 0xffff0000u;
                    if (!((keep >> (2 * i + 1)) & 1)) ds[i] &= 0x0000ffffu;
                }
            }
            // the products have read the last P and dS
            if (!free) pipe_wait(&sh.done, (j - 1) & 1, abort);
            tc_after_sync();
            if (KEYS) tmem_st16(tmem + kColP + 16 * cg + lanes, p);
            tmem_st16(tmem + kColDs + 16 * cg + lanes, ds);
            tmem_wait_st();
            tc_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p);
        }
        if (n > 0) pipe_wait(&sh.done, (n - 1) & 1, abort);
        tc_after_sync();
        // groups 0, 1: the halves of the first sum (dQ or dK); 2, 3: of the second (dV)
        const int acc = cg >> 1, half = cg & 1;
        if (acc == 0 || KEYS) {
            uint32_t o[32];
            if (n > 0) {
                tmem_ld32(o, tmem + (acc ? kColAcc1 : kColAcc0) + 32 * half + lanes);
                tmem_wait_ld(o);
            }
            const float f = acc ? 1.f : a.scale;
            // keys that are not attended have no gradient, whatever their rows hold
            const uint32_t word = (warp & 3) == 0 ? mykeys.x : (warp & 3) == 1 ? mykeys.y : (warp & 3) == 2 ? mykeys.z : mykeys.w;
            const bool zero = n == 0 || (KEYS && !((word >> lane) & 1));
            if (CS == 1) {
                if (row) {
                    __nv_bfloat16 *out = KEYS ? (acc ? a.dV : a.dK).row(b, hk, mine * kTileRows + r)
                                              : a.dQ.row(b, hk * a.qt.G + g, q);
                    uint4 *o4 = reinterpret_cast<uint4 *>(out + 32 * half);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = zero ? 0u
                                        : pack_bf16x2(__uint_as_float(o[8 * i + 2 * k]) * f,
                                                      __uint_as_float(o[8 * i + 2 * k + 1]) * f);
                        o4[i] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            } else {
                // every copy and product has completed: the ring holds the partial sums
                float4 *out = reinterpret_cast<float4 *>(reinterpret_cast<float *>(ring) +
                                                         (acc * kTileRows + r) * kJoinLd + 32 * half);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) w[k] = zero ? 0.f : __uint_as_float(o[4 * i + k]) * f;
                    out[i] = make_float4(w[0], w[1], w[2], w[3]);
                }
            }
        }
    } else {
        give_registers<kRegsFew>();
        if (warp == kCopyWarp) {
            // ---- copies -----------------------------------------------------------------
            if (n > 0) {
                const auto query_tile = [&](uint8_t *dst, int t, uint64_t *bar) {
                    load_tile(dst, a.q, a.qt.first_row(t), hk * a.qt.G + a.qt.first_head(t), b, bar);
                    load_tile(dst + kTileBytes, a.g, a.qt.first_row(t), hk * a.qt.G + a.qt.first_head(t), b, bar);
                };
                const auto key_tile = [&](uint8_t *dst, int t, uint64_t *bar) {
                    load_tile(dst, a.k, t * kTileRows, hk, b, bar);
                    load_tile(dst + kTileBytes, a.v, t * kTileRows, hk, b, bar);
                };
                if (elect_one()) {
                    mbar_expect_tx(&sh.held, held_bytes);
                    if (KEYS) key_tile(held, mine, &sh.held);
                    else query_tile(held, mine, &sh.held);
                }
                __syncwarp();
                int issued = 0;
                for (; issued < n; ++issued) {
                    const int last = issued - kStages, s = issued % kStages;   // the stage's tile before
                    if (last >= 0 && !pipe_wait(&sh.empty[s], (last / kStages) & 1, abort)) break;
                    if (elect_one()) {
                        mbar_expect_tx(&sh.full[s], tile_bytes);
                        if (KEYS) {
                            const int t = lo + issued, rows = a.qt.nb;
                            query_tile(ring + 2 * s * kTileBytes, t, &sh.full[s]);
                            for (int i = 0; i < a.qt.gb; ++i) {
                                const int g = a.qt.first_head(t) + i;
                                const int64_t from = g < a.qt.G ? ((int64_t)b * a.Hq + hk * a.qt.G + g) * a.npad +
                                                                      a.qt.first_row(t)
                                                                : (int64_t)a.B * a.Hq * a.npad;   // no such head
                                uint8_t *to = parts + 2 * s * kNarrow + i * rows * 16;
                                bulk_g2s(to, a.lse_parts + from, rows * 16, &sh.full[s]);
                                bulk_g2s(to + kNarrow, a.d_parts + from, rows * 16, &sh.full[s]);
                            }
                        } else key_tile(ring + 2 * s * kTileBytes, lo + issued, &sh.full[s]);
                    }
                    __syncwarp();
                }
                // leave no copy in flight
                if (lane == 0) {
                    mbar_drain(&sh.held, 0);
                    for (int j = max(0, issued - kStages); j < issued; ++j)
                        mbar_drain(&sh.full[j % kStages], (j / kStages) & 1);
                }
            }
        } else if (warp == kPrepWarp) {
            // ---- which keys of a streamed tile are attended -----------------------------------
            for (int j = 0; !KEYS && j < n; ++j) {
                const int s = j % kStages;
                const uint4 w = tile_keys(a.ks, b, (lo + j) * kTileRows, bound);
                if (!pipe_wait(&sh.full[s], (j / kStages) & 1, abort)) break;
                if (!all_keys(w)) {
                    clear_rows(ring + 2 * s * kTileBytes, w);      // K: read across its rows with weights of 0
                    fence_smem_async();
                }
                if (lane == 0) sh.keys[s] = w;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.ready[s]);
                // once a tile beside the products: who sees S and dP also sees keys[s]
                if (j > 0 && !pipe_wait(&sh.s, (j - 1) & 1, abort)) break;
                if (lane == 0) mbar_arrive(&sh.s);
            }
        } else {
            // ---- matrix instructions, by two warps so that neither kind waits for what the other
            // needs.  The loops' course depends on uniform values only (a wait that gives up is not
            // looked at: what follows is not trusted, since the error word is set).
            const int nu = __shfl_sync(kFullMask, n, 0);
            int s = 0, pass = 0;
            const auto next_stage = [&]() {
                if (++s == kStages) {
                    s = 0;
                    pass ^= 1;
                }
            };
            if (nu > 0 && warp == kScoreWarp) {
                const uint32_t id = mma_desc(128, 128, false);
                const uint64_t h0 = tile_desc(held), h1 = tile_desc(held + kTileBytes);
                const uint64_t r0 = tile_desc(ring), r1 = tile_desc(ring + kTileBytes);
                const uint64_t one = narrow_desc(ones), p0 = narrow_desc(parts);
                pipe_wait(&sh.held, 0, abort);
                for (int j = 0; j < nu; ++j) {
                    const uint64_t at = (uint64_t)(s * (2 * kTileBytes >> 4));
                    pipe_wait(KEYS ? &sh.full[s] : &sh.ready[s], pass, abort);
                    if (j > 0) pipe_wait(&sh.sfree, (j - 1) & 1, abort);
                    tc_after_sync();
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_ss(tmem + kColS, h0 + i * kStepRowwise, r0 + at + i * kStepRowwise, id, i > 0);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_ss(tmem + kColDp, h1 + i * kStepRowwise, r1 + at + i * kStepRowwise, id, i > 0);
                        if (KEYS) {
                            const uint64_t part = p0 + (uint64_t)(s * (2 * kNarrow >> 4));
                            mma_ss(tmem + kColS, one, part, id, true);
                            mma_ss(tmem + kColDp, one, part + (kNarrow >> 4), id, true);
                        }
                        mma_commit(&sh.s);
                    }
                    __syncwarp();
                    next_stage();
                }
            } else if (nu > 0 && warp == kSumWarp) {
                const uint32_t id = mma_desc(128, 64, true);
                const uint64_t r0 = tile_desc(ring), r1 = tile_desc(ring + kTileBytes);
                for (int j = 0; j < nu; ++j) {
                    const uint64_t at = (uint64_t)(s * (2 * kTileBytes >> 4));
                    pipe_wait(&sh.p, j & 1, abort);
                    tc_after_sync();
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            mma_ts(tmem + kColAcc0, tmem + kColDs + i * 8, r0 + at + i * kStepAcross, id, j > 0 || i > 0);
                        if (KEYS) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                mma_ts(tmem + kColAcc1, tmem + kColP + i * 8, r1 + at + i * kStepAcross, id, j > 0 || i > 0);
                        }
                        mma_commit(&sh.done);
                        mma_commit(&sh.empty[s]);
                    }
                    __syncwarp();
                    next_stage();
                }
            }
            if (nu > 0) {   // no matrix instruction in flight when the tensor memory is freed
                uint64_t *end = &sh.end[warp == kSumWarp];
                if (elect_one()) mma_commit(end);
                __syncwarp();
                mbar_drain(end, 0);
            }
        }
    }
    __syncwarp();
    tc_before_sync();
    __syncthreads();
    if (warp == kSumWarp) tmem_free(tmem, kCols);
    if (CS == 1) return;

    // ---- join: CTA r of the cluster finishes every CS-th row -------------------------------
    cluster_sync();
    const float *part = reinterpret_cast<const float *>(ring);
    const int c4 = (threadIdx.x & 15) * 4;
    for (int i = rank + CS * (int)(threadIdx.x >> 4); i < (KEYS ? 2 : 1) * kTileRows; i += CS * (kThreads / 16)) {
        const int acc = i / kTileRows, r = i % kTileRows;
        int g = 0, q = 0;
        if (KEYS ? mine * kTileRows + r >= a.ks.Nk : !a.qt.at(mine, r, g, q)) continue;
        float2 x = make_float2(0.f, 0.f), y = x;
        for (int k = 0; k < CS; ++k) {
            const uint32_t at = cluster_addr(part + i * kJoinLd + c4, k);
            x = add2(x, ld_cluster2(at));
            y = add2(y, ld_cluster2(at + 8));
        }
        __nv_bfloat16 *out = KEYS ? (acc ? a.dV : a.dK).row(b, hk, mine * kTileRows + r)
                                  : a.dQ.row(b, hk * a.qt.G + g, q);
        *reinterpret_cast<uint2 *>(out + c4) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(y.x, y.y));
    }
    cluster_sync();   // the others may still read this CTA's part
}

__global__ void __launch_bounds__(kThreads, 1) cross_bwd_mma_kernel(const __grid_constant__ BwdMmaArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    __shared__ Shared sh;
    const int64_t unit = blockIdx.x / cluster_size();
    const bool holds_keys = unit < a.key_blocks;
    if (threadIdx.x == 0) {
        mbar_init(&sh.held, 1);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.ready[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        mbar_init(&sh.s, holds_keys ? 1 : 2);
        mbar_init(&sh.sfree, kWeightWarps);
        mbar_init(&sh.p, kWeightWarps);
        mbar_init(&sh.done, 1);
        mbar_init(&sh.end[0], 1);
        mbar_init(&sh.end[1], 1);
        sh.abort = 0;
        prefetch_map(&a.q.map);
        prefetch_map(&a.g.map);
        prefetch_map(&a.k.map);
        prefetch_map(&a.v.map);
    }
    if (warp_number() == kSumWarp) tmem_alloc(&sh.tmem, kCols);
    // a query tile of fewer than 128 rows leaves the end of its stage as it is:
    // zeros there, so that weights of 0 meet no NaN
    if (a.qt.nb * a.qt.gb < kTileRows) {
        for (int i = threadIdx.x; i < (2 + 2 * kStages) * kTileBytes / 16; i += kThreads)
            reinterpret_cast<uint4 *>(smem)[i] = make_uint4(0, 0, 0, 0);
        fence_smem_async();
    }
    if (holds_keys) {   // ones in the first three elements of a row; rows of no query until copies bring some
        uint8_t *ones = smem + (2 + 2 * kStages) * kTileBytes;
        const uint4 none = no_query(a.c);
        for (int i = threadIdx.x; i < (1 + 2 * kStages) * kNarrow / 16; i += kThreads) {
            const int tile = i / (kNarrow / 16), r = i % (kNarrow / 16);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < kTileRows && tile == 0) v = make_uint4(0x3f803f80u, 0x3f80u, 0u, 0u);
            else if (r < kTileRows && (tile & 1)) v = none;
            reinterpret_cast<uint4 *>(ones)[i] = v;
        }
        fence_smem_async();
    }
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    grid_dep_wait();
    grid_dep_launch();
    if (holds_keys) run<true>(a, sh, smem, unit);
    else run<false>(a, sh, smem, unit - a.key_blocks);
}

// Rows of a head with the last of its query tiles whole.
int padded_rows(int Nq) { return Nq < kTileRows ? Nq : (Nq + kTileRows - 1) / kTileRows * kTileRows; }

}  // namespace

size_t cross_bwd_mma_workspace(int B, int Hq, int Nq) {
    const size_t rows = (size_t)B * Hq * padded_rows(Nq);
    return 2 * (rows + kTileRows) * sizeof(uint4) + (size_t)B * Hq * Nq * sizeof(float2);
}

cudaError_t launch_cross_bwd_mma(const CrossArgs &a) {
    BwdMmaArgs f;
    f.qt = QueryTiles(a.Hq / a.Hkv, a.Nq, a.Hq > 1 && (a.Q.stride_h == 0 || a.dO.stride_h == 0));
    if (!make_tensor(&f.q, a.Q, a.B, a.Hq, a.Nq, f.qt.nb, f.qt.gb) ||
        !make_tensor(&f.g, a.dO, a.B, a.Hq, a.Nq, f.qt.nb, f.qt.gb) ||
        !make_tensor(&f.k, a.K, a.B, a.Hkv, a.Nk, kTileRows, 1) ||
        !make_tensor(&f.v, a.V, a.B, a.Hkv, a.Nk, kTileRows, 1))
        return cudaErrorInvalidValue;
    f.ks = a.keys;
    f.npad = padded_rows(a.Nq);
    const int64_t rows = (int64_t)a.B * a.Hq * f.npad;
    uint4 *lse_parts = reinterpret_cast<uint4 *>(a.stats), *d_parts = lse_parts + rows + kTileRows;
    float2 *stats = reinterpret_cast<float2 *>(d_parts + rows + kTileRows);
    f.stats = stats;
    f.lse_parts = lse_parts, f.d_parts = d_parts;
    f.dQ = rows_of<__nv_bfloat16>(a.dQ), f.dK = rows_of<__nv_bfloat16>(a.dK), f.dV = rows_of<__nv_bfloat16>(a.dV);
    f.B = a.B, f.Hq = a.Hq, f.Hkv = a.Hkv;
    f.ktiles = (a.Nk + kTileRows - 1) / kTileRows;
    f.scale = a.scale;
    // a scale of 0: any c this small leaves every finite score's weight at exp2(-LSE log2 e)
    f.c = std::copysign(std::max(std::fabs(a.scale) * kLog2e, 1e-36f), a.scale);
    cudaError_t e = prepare_kernel<cross_bwd_mma_kernel>(kSmem, kRegs);
    if (e != cudaSuccess) return e;
    e = launch_clusters(cross_parts_kernel, (unsigned)((rows + kTileRows + 15) / 16), 1, 256, 0, a.stream, a.Hq, a.Nq,
                        f.npad, rows, rows_of<const __nv_bfloat16>(a.O), rows_of<const __nv_bfloat16>(a.dO),
                        static_cast<const float *>(a.LSE), f.c, stats, lse_parts, d_parts);
    if (e != cudaSuccess) return e;
    const int64_t key_units = (int64_t)a.B * a.Hkv * f.ktiles, units = key_units + (int64_t)a.B * a.Hkv * f.qt.tiles;
    f.key_blocks = (int)key_units;
    int c = 1;
    while (c < 8 && units * c * 2 <= sm_count() && std::max(f.ktiles, f.qt.tiles) >= 2 * c) c *= 2;
    return launch_clusters(cross_bwd_mma_kernel, (unsigned)(units * c), c, kThreads, kSmem, a.stream, f);
}

FIBATT_DEFINE_ERROR_READER(read_error_cross_mma_bwd, "cross_mma_bwd.cu")

}  // namespace fibatt
