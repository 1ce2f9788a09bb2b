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
// so each gradient row is summed by one CTA (or one cluster, joined in rank
// order): no atomics, a fixed order.  S and dP are formed twice (7 products of
// 128 x 128 x 64 a tile pair instead of 5); the alternative, one pass that adds
// dQ to memory with atomics, depends on scheduling.
//
// Both kinds of CTA are blocks of one launch.  Warps: 16 that turn S and dP into
// P and dS (a warp has 32 rows and 32 columns of the tile; four warps on every
// scheduler hide each other's waits), one that copies, one that prepares what
// goes with a tile (row statistics, or the keys attended and the clearing of
// the others), one that issues the matrix instructions.  The next tile's S and
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
constexpr int kCopyWarp = kWeightWarps, kPrepWarp = kWeightWarps + 1, kMmaWarp = kWeightWarps + 2;
constexpr int kThreads = 32 * (kWeightWarps + 4);
constexpr int kStages = 4;
constexpr size_t kSmem = 1024 + (2 + 2 * kStages) * kTileBytes;
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
    Rows<__nv_bfloat16> dQ, dK, dV;
    int Hq, Hkv, ktiles;
    int key_blocks;             // clusters that hold keys; the others hold queries
    float scale;
    BwdMmaArgs() : qt(1, 1, false) {}
};

struct Shared {
    uint64_t held, full[kStages], ready[kStages], empty[kStages], s, sfree, p, done, end;
    uint4 keys[kStages];
    float lse[kStages][kTileRows], d[kStages][kTileRows];   // of the streamed queries: -LSE log2 e, -D
    uint32_t tmem;
    int abort;
};

template <bool KEYS>
__device__ __forceinline__ void run(const BwdMmaArgs &a, Shared &sh, uint8_t *smem, int64_t unit) {
    uint8_t *held = smem, *ring = smem + 2 * kTileBytes;    // stage s: K or Q at ring + 2 s tiles, V or dO behind it
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
    const uint32_t tile_bytes = 2 * (KEYS ? a.qt.bytes() : (uint32_t)kTileBytes);

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
        const float c = a.scale * kLog2e;
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
                pipe_wait(&sh.ready[s], (j / kStages) & 1, abort);     // keys[s] is written
                const uint4 w = sh.keys[s];
                keep = cg == 0 ? w.x : cg == 1 ? w.y : cg == 2 ? w.z : w.w;
            }
            if (KEYS) pipe_wait(&sh.ready[s], (j / kStages) & 1, abort);   // the statistics are written
            uint32_t p[16], ds[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float4 l4, d4;
                if (KEYS) {
                    l4 = *reinterpret_cast<const float4 *>(&sh.lse[s][32 * cg + 4 * i]);
                    d4 = *reinterpret_cast<const float4 *>(&sh.d[s][32 * cg + 4 * i]);
                } else {
                    l4 = make_float4(row_lse, row_lse, row_lse, row_lse);
                    d4 = make_float4(row_d, row_d, row_d, row_d);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int e = 4 * i + 2 * k;
                    const float2 l2 = k ? make_float2(l4.z, l4.w) : make_float2(l4.x, l4.y);
                    const float2 d2 = k ? make_float2(d4.z, d4.w) : make_float2(d4.x, d4.y);
                    const float2 z = fma2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), cc, l2);
                    const float2 w = make_float2(fast_exp2(z.x), fast_exp2(z.y));
                    const float2 t = mul2(
                        w, add2(make_float2(__uint_as_float(y[e]), __uint_as_float(y[e + 1])), d2));
                    if (KEYS) p[2 * i + k] = pack_bf16x2(w.x, w.y);
                    ds[2 * i + k] = pack_bf16x2(t.x, t.y);
                }
            }
            if (!KEYS && keep != 0xffffffffu) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (!((keep >> (2 * i)) & 1)) ds[i] &= 0xffff0000u;
                    if (!((keep >> (2 * i + 1)) & 1)) ds[i] &= 0x0000ffffu;
                }
            }
            if (j > 0) {
                pipe_wait(&sh.done, (j - 1) & 1, abort);    // the products have read the last P and dS
                tc_after_sync();
            }
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
                        if (KEYS) query_tile(ring + 2 * s * kTileBytes, lo + issued, &sh.full[s]);
                        else key_tile(ring + 2 * s * kTileBytes, lo + issued, &sh.full[s]);
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
            // ---- what goes with a tile ------------------------------------------------------
            for (int j = 0; j < n; ++j) {
                const int s = j % kStages;
                if (KEYS) {
                    float2 st[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        int g, q;
                        st[i] = a.qt.at(lo + j, 32 * i + lane, g, q)
                                    ? __ldg(a.stats + ((int64_t)b * a.Hq + hk * a.qt.G + g) * a.qt.Nq + q)
                                    : make_float2(kInf, 0.f);      // no such query: its weights are exp2(0 - inf)
                    }
                    if (!pipe_wait(&sh.full[s], (j / kStages) & 1, abort)) break;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        sh.lse[s][32 * i + lane] = -st[i].x;
                        sh.d[s][32 * i + lane] = -st[i].y;
                    }
                } else {
                    const uint4 w = tile_keys(a.ks, b, (lo + j) * kTileRows, bound);
                    if (!pipe_wait(&sh.full[s], (j / kStages) & 1, abort)) break;
                    if (!all_keys(w)) {
                        clear_rows(ring + 2 * s * kTileBytes, w);      // K: read across its rows with weights of 0
                        fence_smem_async();
                    }
                    if (lane == 0) sh.keys[s] = w;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.ready[s]);
            }
        } else if (warp == kMmaWarp) {
            // ---- matrix instructions: the loop's course depends on uniform values only (a wait that
            // gives up is not looked at: what follows is not trusted, since the error word is set)
            const int nu = __shfl_sync(kFullMask, n, 0);
            if (nu > 0) {
                const uint32_t id_s = mma_desc(128, 128, false), id_o = mma_desc(128, 64, true);
                const uint64_t h0 = tile_desc(held), h1 = tile_desc(held + kTileBytes);
                const uint64_t r0 = tile_desc(ring), r1 = tile_desc(ring + kTileBytes);
                int s = 0, pass = 0, s1 = 0;
                pipe_wait(&sh.held, 0, abort);
                for (int j = 0; j <= nu; ++j) {
                    if (j < nu) {
                        const uint64_t at = (uint64_t)(s * (2 * kTileBytes >> 4));
                        pipe_wait(&sh.ready[s], pass, abort);
                        if (j > 0) pipe_wait(&sh.sfree, (j - 1) & 1, abort);
                        tc_after_sync();
                        if (elect_one()) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mma_ss(tmem + kColS, h0 + i * kStepRowwise, r0 + at + i * kStepRowwise, id_s, i > 0);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mma_ss(tmem + kColDp, h1 + i * kStepRowwise, r1 + at + i * kStepRowwise, id_s, i > 0);
                            mma_commit(&sh.s);
                        }
                        __syncwarp();
                    }
                    if (j > 0) {
                        const uint64_t at = (uint64_t)(s1 * (2 * kTileBytes >> 4));
                        pipe_wait(&sh.p, (j - 1) & 1, abort);
                        tc_after_sync();
                        if (elect_one()) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                mma_ts(tmem + kColAcc0, tmem + kColDs + i * 8, r0 + at + i * kStepAcross, id_o,
                                       j > 1 || i > 0);
                            if (KEYS) {
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    mma_ts(tmem + kColAcc1, tmem + kColP + i * 8, r1 + at + i * kStepAcross, id_o,
                                           j > 1 || i > 0);
                            }
                            mma_commit(&sh.done);
                            mma_commit(&sh.empty[s1]);
                        }
                        __syncwarp();
                    }
                    s1 = s;
                    if (++s == kStages) {
                        s = 0;
                        pass ^= 1;
                    }
                }
                if (elect_one()) mma_commit(&sh.end);
                __syncwarp();
                mbar_drain(&sh.end, 0);   // no matrix instruction in flight when the tensor memory is freed
            }
        }
    }
    __syncwarp();
    tc_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) tmem_free(tmem, kCols);
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
    if (threadIdx.x == 0) {
        mbar_init(&sh.held, 1);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.ready[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        mbar_init(&sh.s, 1);
        mbar_init(&sh.sfree, kWeightWarps);
        mbar_init(&sh.p, kWeightWarps);
        mbar_init(&sh.done, 1);
        mbar_init(&sh.end, 1);
        sh.abort = 0;
        prefetch_map(&a.q.map);
        prefetch_map(&a.g.map);
        prefetch_map(&a.k.map);
        prefetch_map(&a.v.map);
    }
    if (warp_number() == kMmaWarp) tmem_alloc(&sh.tmem, kCols);
    // a query tile of fewer than 128 rows leaves the end of its stage as it is:
    // zeros there, so that weights of 0 meet no NaN
    if (a.qt.nb * a.qt.gb < kTileRows) {
        for (int i = threadIdx.x; i < (2 + 2 * kStages) * kTileBytes / 16; i += kThreads)
            reinterpret_cast<uint4 *>(smem)[i] = make_uint4(0, 0, 0, 0);
        fence_smem_async();
    }
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    grid_dep_wait();
    grid_dep_launch();
    const int64_t unit = blockIdx.x / cluster_size();
    if (unit < a.key_blocks) run<true>(a, sh, smem, unit);
    else run<false>(a, sh, smem, unit - a.key_blocks);
}

}  // namespace

cudaError_t launch_cross_bwd_mma(const CrossArgs &a) {
    cudaError_t e = launch_cross_stats(a);
    if (e != cudaSuccess) return e;
    BwdMmaArgs f;
    f.qt = QueryTiles(a.Hq / a.Hkv, a.Nq, a.Hq > 1 && (a.Q.stride_h == 0 || a.dO.stride_h == 0));
    if (!make_tensor(&f.q, a.Q, a.B, a.Hq, a.Nq, f.qt.nb, f.qt.gb) ||
        !make_tensor(&f.g, a.dO, a.B, a.Hq, a.Nq, f.qt.nb, f.qt.gb) ||
        !make_tensor(&f.k, a.K, a.B, a.Hkv, a.Nk, kTileRows, 1) ||
        !make_tensor(&f.v, a.V, a.B, a.Hkv, a.Nk, kTileRows, 1))
        return cudaErrorInvalidValue;
    f.ks = a.keys;
    f.stats = a.stats;
    f.dQ = rows_of<__nv_bfloat16>(a.dQ), f.dK = rows_of<__nv_bfloat16>(a.dK), f.dV = rows_of<__nv_bfloat16>(a.dV);
    f.Hq = a.Hq, f.Hkv = a.Hkv;
    f.ktiles = (a.Nk + kTileRows - 1) / kTileRows;
    f.scale = a.scale;
    e = prepare_kernel<cross_bwd_mma_kernel>(kSmem, kRegs);
    if (e != cudaSuccess) return e;
    const int64_t key_units = (int64_t)a.B * a.Hkv * f.ktiles, units = key_units + (int64_t)a.B * a.Hkv * f.qt.tiles;
    f.key_blocks = (int)key_units;
    int c = 1;
    while (c < 8 && units * c * 2 <= sm_count() && std::max(f.ktiles, f.qt.tiles) >= 2 * c) c *= 2;
    return launch_clusters(cross_bwd_mma_kernel, (unsigned)(units * c), c, kThreads, kSmem, a.stream, f);
}

FIBATT_DEFINE_ERROR_READER(read_error_cross_mma_bwd, "cross_mma_bwd.cu")

}  // namespace fibatt
