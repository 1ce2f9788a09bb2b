// Cross attention backward on the tensor cores (bf16): dQ, and dK with dV, from
//   S = scale log2 e Q K^T,  P = exp2(S - LSE log2 e),  dP = dO V^T,
//   dS = P (dP - D),  D = <dO, O>
//   dQ = scale dS K,   dK = scale dS^T Q,   dV = P^T dO.
// A unit of work holds 128 rows of one side and walks over the 128-row tiles of the
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
// Both kinds are units of one launch, one wave of CTAs that draw them from a
// counter, queries first (each CTA every 152nd unit instead: 613 us where this
// took 595), or two, one of each kind, where their walks differ much; the copies
// run ahead into the next unit.  Warps: 16 that turn
// S and dP into P and dS (a warp has 32 rows and 32 columns of the tile; four warps
// on every scheduler hide each other's waits), one that copies and draws, one that
// prepares what goes with a streamed tile (the keys attended, the clearing of the
// other rows), two that issue the matrix instructions.  The next tile's S and dP
// are formed while this one's P and dS are made.  The weights' side of every
// product over rows is read from tensor memory, as bf16 (relative rounding 2^-8
// a weight, averaging out over the sum).
//
// Measured, back to back in a graph: 2 sequences, 16 heads, 1569 x 16385: 583 to 602 us,
// 903 TFLOP/s of the 5 products at best (1264 of the 7), the small kernel 6 of them (called
// from Python 602 to 617); 8 sequences, 12 heads on 4, 197 x 1569 of several lengths: 38.5 us,
// the small kernel 4.5.  A tile takes about 1490
// cycles, its 3 or 4 products 800 or 1090 of them; the tensor cores are 61% busy, the
// issue slots 49%: what is left are the waits from S to dS to the products, which need
// each other within a tile.
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
constexpr int kNarrow = kTileRows * 16;           // bytes of half a k-step of a tile (the other half: zeros for all)
constexpr size_t kSmem = 1024 + (4 + 2 * kStages) * kTileBytes + (2 + 2 * kStages) * kNarrow;
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
    int query_units, units;     // units that hold queries, which come first, and all of them
    int first_unit;             // of the launch, which has those up to `units`
    int *next_unit;             // units given out behind every CTA's first
    float scale;
    float c;                    // scale log2 e, not 0
    BwdMmaArgs() : qt(1, 1, false) {}
};

// x as the sum of three bf16 values, the first of eight elements of a row (cut to
// what a bf16 holds: at a scale of 0, 1000 / c is beyond it; NaN stays).
__device__ __forceinline__ uint4 three_parts(float x) {
    if (x == x) x = fminf(fmaxf(x, -3.0e38f), 3.0e38f);
    const float hi = __bfloat162float(__float2bfloat16_rn(x)), rest = x - hi;
    const float mid = __bfloat162float(__float2bfloat16_rn(rest));
    return make_uint4(pack_bf16x2(hi, mid), pack_bf16x2(rest - mid, 0.f), 0u, 0u);
}

// What stands for a query that does not exist: a weight of exp2(-1000) = 0.
__device__ __forceinline__ uint4 no_query(float c) { return three_parts(-1000.f / c); }

// D of sequences with few keys is summed from the weights themselves,
// D = sum_k P_k dP_k: O's rounding to bf16 is one of the larger errors of dS when a
// row has few keys.  Against 64 bits, dQ and dK with <dO, O>: 3 keys 0.0032, 8 keys 0.0026,
// from 64 keys on 0.0025; with the sum 0.0024.  Tensors of at most kFewKeys keys have a kernel
// for it.  In longer ones (a padded batch) the first kernel sums a key at a time for the
// sequences of at most kShort, where it matters most: 8 sequences of 393 to 1569 keys take
// 39.7 us with it and without; 64 x 12 heads, 197 queries, with 3 or 8 of 197 keys each, 103
// (<dO, O> 79; up to 16 keys a sequence 127; the other kernel, which takes 16 rows a warp, 99 for
// 3 or 64 keys, but 41.6 for the long sequences).  Keys that a mask leaves are not counted: that
// took 64 x 12 heads of 65 x 197 from 62 to 65 us.
constexpr int kFewKeys = 64, kShort = 8;

// (LSE log2 e, D) of every query row, and -LSE log2 e / c and -D in parts, rows
// padded to `npad` a head and 128 rows of no query at the end.  Eight threads a row.
// D is <dO, O>, but with LENGTHS the sum above for the sequences that are that short.
template <bool LENGTHS>
__global__ void __launch_bounds__(256)
cross_parts_kernel(int Hq, int Hkv, int Nq, int npad, unsigned rows, KeySet ks, Rows<const __nv_bfloat16> Q,
                   Rows<const __nv_bfloat16> K, Rows<const __nv_bfloat16> V, Rows<const __nv_bfloat16> O,
                   Rows<const __nv_bfloat16> dO, const float *__restrict__ LSE, float c, float2 *__restrict__ stats,
                   uint4 *__restrict__ lse_parts, uint4 *__restrict__ d_parts, int *__restrict__ next_unit) {
    grid_dep_wait();
    grid_dep_launch();
    const unsigned row = blockIdx.x * 32 + (threadIdx.x >> 3);
    const int i = threadIdx.x & 7;
    if (blockIdx.x == 0 && threadIdx.x < 2) next_unit[threadIdx.x] = 0;
    if (row >= rows + kTileRows) return;   // whole groups of eight: the shuffles below stay within them
    const unsigned bh = row / (unsigned)npad, n = row - bh * npad;
    if (row >= rows || n >= (unsigned)Nq) {
        if (i == 0) lse_parts[row] = no_query(c);
        if (i == 1) d_parts[row] = make_uint4(0, 0, 0, 0);
        return;
    }
    const unsigned b = bh / (unsigned)Hq, h = bh - b * Hq;
    const uint4 o = __ldg(reinterpret_cast<const uint4 *>(O.row(b, h, n)) + i);
    const uint4 g = __ldg(reinterpret_cast<const uint4 *>(dO.row(b, h, n)) + i);
    const int64_t at = (int64_t)bh * Nq + n;
    const float lse = __ldg(LSE + at);
    // a row without keys: its weights are exp2(s - inf) = 0 (and no block meets it)
    const bool none = lse == -kInf;
    const float lse2 = none ? kInf : lse * kLog2e;
    const unsigned eight = 0xffu << (threadIdx.x & 24);
    const auto share = [](const uint4 &x, const uint4 &y) {      // of <x, y>, this thread's
        return dot2_bf16(x.x, y.x, dot2_bf16(x.y, y.y, 0.f)) + dot2_bf16(x.z, y.z, dot2_bf16(x.w, y.w, 0.f));
    };
    const auto sum = [&](float x) {
#pragma unroll
        for (int m = 1; m < 8; m <<= 1) x += __shfl_xor_sync(eight, x, m);
        return x;
    };
    float d = share(o, g);
    if (LENGTHS) {
        const int bound = ks.bound((int)b), hk = (int)h / (Hq / Hkv);
        if (bound <= kShort) {
            const uint4 q = __ldg(reinterpret_cast<const uint4 *>(Q.row(b, h, n)) + i);
            d = 0.f;
#pragma unroll 1
            for (int j = 0; j < bound; ++j) {
                const uint4 k = __ldg(reinterpret_cast<const uint4 *>(K.row(b, hk, j)) + i);
                const uint4 v = __ldg(reinterpret_cast<const uint4 *>(V.row(b, hk, j)) + i);
                const float p = fast_exp2(fmaf(sum(share(q, k)), c, -lse2));
                if (ks.has((int)b, j)) d = fmaf(p, share(g, v), d);
            }
        }
    }
    d = sum(d);
    if (i == 0) lse_parts[row] = none ? no_query(c) : three_parts(-lse2 / c);
    if (i == 1) d_parts[row] = three_parts(-d);
    if (i == 2) stats[at] = make_float2(lse2, d);
}

// A lane's 16 dims of a row: 32 bytes.
struct Dims {
    uint32_t x[8];
    __device__ __forceinline__ void load(const __nv_bfloat16 *row, int t) {
        const uint4 *p = reinterpret_cast<const uint4 *>(row) + 2 * t;
        const uint4 u = __ldg(p), v = __ldg(p + 1);
        x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0u;
    }
};

// The same for tensors of at most kFewKeys keys (of 128, 192 heads of 1000 queries, it
// would cost 17 of 92 us).  A warp takes 16 queries of a head,
// its eight keys at a time by warp-wide products; lane (g, t) gives them dims 16 t
// to 16 t + 15 of rows g and g + 8 and of key g, four at a time in both operands
// (the order of a sum does not matter), so that it loads 16 bytes at once.
constexpr int kFewWarps = 4;
__global__ void __launch_bounds__(32 * kFewWarps)
cross_parts_few_kernel(int Hq, int Hkv, int Nq, int npad, unsigned heads, KeySet ks, Rows<const __nv_bfloat16> Q,
                       Rows<const __nv_bfloat16> K, Rows<const __nv_bfloat16> V, Rows<const __nv_bfloat16> dO,
                       const float *__restrict__ LSE, float c, float2 *__restrict__ stats, uint4 *__restrict__ lse_parts,
                       uint4 *__restrict__ d_parts, int *__restrict__ next_unit) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const unsigned groups = (unsigned)(npad + 15) / 16, at = blockIdx.x * kFewWarps + warp_number();
    const unsigned bh = at / groups, b = bh / (unsigned)Hq, h = bh - b * Hq;
    const int n0 = 16 * (int)(at - bh * groups);
    grid_dep_wait();
    grid_dep_launch();
    if (at == 0 && lane < 2) next_unit[lane] = 0;
    if (bh >= heads) {      // rows of no query, behind the heads'
        const unsigned i = (at - heads * groups) * 16 + (lane >> 1);
        if (i >= (unsigned)kTileRows) return;
        const int64_t row = (int64_t)heads * npad + i;
        if (lane & 1) d_parts[row] = make_uint4(0, 0, 0, 0);
        else lse_parts[row] = no_query(c);
        return;
    }
    const int hk = (int)h / (Hq / Hkv);
    Dims q[2], w[2];
    float lse2[2], d[2] = {0.f, 0.f};
    bool none[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int n = n0 + g + 8 * i;
        q[i].zero();
        w[i].zero();
        float lse = -kInf;
        if (n < Nq) {
            q[i].load(Q.row(b, h, n), t);
            w[i].load(dO.row(b, h, n), t);
            lse = __ldg(LSE + (int64_t)bh * Nq + n);
        }
        none[i] = lse == -kInf;        // a row without keys: weights of exp2(s - inf) = 0
        lse2[i] = none[i] ? kInf : lse * kLog2e;
    }
    const int bound = ks.bound((int)b);
    for (int k0 = 0; k0 < bound; k0 += 8) {
        const int mine = k0 + (lane & 7);
        const uint32_t in = __ballot_sync(kFullMask, mine < bound && ks.has((int)b, min(mine, bound - 1)));
        Dims k, v;
        k.load(K.row(b, hk, min(k0 + g, bound - 1)), t);
        v.load(V.row(b, hk, min(k0 + g, bound - 1)), t);
        float s[4] = {0.f, 0.f, 0.f, 0.f}, dp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t aq[4] = {q[0].x[2 * i], q[1].x[2 * i], q[0].x[2 * i + 1], q[1].x[2 * i + 1]};
            const uint32_t aw[4] = {w[0].x[2 * i], w[1].x[2 * i], w[0].x[2 * i + 1], w[1].x[2 * i + 1]};
            warp_mma(s, aq, k.x[2 * i], k.x[2 * i + 1]);
            warp_mma(dp, aw, v.x[2 * i], v.x[2 * i + 1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float p = fast_exp2(fmaf(s[i], c, -lse2[i >> 1]));
            if ((in >> (2 * t + (i & 1))) & 1) d[i >> 1] = fmaf(p, dp[i], d[i >> 1]);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        d[i] += __shfl_xor_sync(kFullMask, d[i], 1);
        d[i] += __shfl_xor_sync(kFullMask, d[i], 2);
        const int n = n0 + g + 8 * i;
        if (n >= npad) continue;
        const int64_t row = (int64_t)bh * npad + n;
        const bool query = n < Nq;
        if (t == 0) lse_parts[row] = none[i] ? no_query(c) : three_parts(-lse2[i] / c);
        if (t == 1) d_parts[row] = query ? three_parts(-d[i]) : make_uint4(0, 0, 0, 0);
        if (t == 2 && query) stats[(int64_t)bh * Nq + n] = make_float2(lse2[i], d[i]);
    }
}

// One unit of work: 128 rows of one side of one key/value head, and the part of
// the other side's tiles that this CTA of the cluster streams.  The copying warp works
// it out and passes it on: its divisions and loads would otherwise stand at the start
// of every unit in every warp.
struct Unit {
    int index;               // queries held first, then keys held
    int mine, hk, b, bound, lo, n;
    uint4 keys;              // keys held: which rows are attended
    template <bool KEYS>
    __device__ __forceinline__ void set(const BwdMmaArgs &a, int i) {
        index = i;
        const int unit = KEYS ? i - a.query_units : i, held = KEYS ? a.ktiles : a.qt.tiles;
        mine = unit % held;
        hk = unit / held % a.Hkv;
        b = unit / held / a.Hkv;
        bound = a.ks.bound(b);
        // none for a key tile without keys, or for queries without any
        int64_t tiles;
        keys = make_uint4(0, 0, 0, 0);
        if (KEYS) {
            keys = tile_keys(a.ks, b, mine * kTileRows, bound);
            tiles = no_keys(keys) ? 0 : a.qt.tiles;
        } else {
            tiles = (bound + kTileRows - 1) / kTileRows;
        }
        const int CS = (int)cluster_size(), rank = (int)cluster_rank();
        lo = (int)(tiles * rank / CS);
        n = (int)(tiles * (rank + 1) / CS) - lo;
    }
    // the whole warp calls it; an index behind the last unit stands for the end
    __device__ __forceinline__ void enter(const BwdMmaArgs &a, int i) {
        if (i < a.query_units) set<false>(a, i);
        else if (i < a.units) set<true>(a, i);
        else index = i, mine = hk = b = bound = lo = n = 0, keys = make_uint4(0, 0, 0, 0);
    }
};

struct Shared {
    uint64_t held[2], held_free[2], full[kStages], ready[kStages], empty[kStages], s, sfree, p, done, end[2];
    uint64_t unit_full[2], unit_empty[2];
    uint4 keys[kStages];
    Unit unit[2];               // the CTA's, in turn
    uint32_t tmem;
    int abort;
};

// The CTA's shared memory.
struct Tiles {
    uint8_t *held, *ring, *ones, *parts, *zeros;
    __device__ __forceinline__ explicit Tiles(uint8_t *smem)
        : held(smem), ring(smem + 4 * kTileBytes), ones(ring + 2 * kStages * kTileBytes), parts(ones + kNarrow),
          zeros(parts + 2 * kStages * kNarrow) {}
    // pair i of the held tiles (Q, dO or K, V); stage s: K or Q, V or dO behind it; LSE parts, D parts behind them
    __device__ __forceinline__ uint8_t *pair(int i) const { return held + 2 * i * kTileBytes; }
    __device__ __forceinline__ uint8_t *stage(int s) const { return ring + 2 * s * kTileBytes; }
    __device__ __forceinline__ uint8_t *part(int s) const { return parts + 2 * s * kNarrow; }
};

// The roles of the warps over one unit.  `it` counts the streamed tiles over all
// units of the CTA: tile it is in stage it mod kStages, and each barrier of the
// pipeline completes a phase per tile.

// P and dS: row = lane of the quarter, 32 columns
template <bool KEYS>
__device__ __forceinline__ int weights(const BwdMmaArgs &a, Shared &sh, uint8_t *ring, const Unit &u, int it) {
    volatile int *abort = &sh.abort;
    const int warp = warp_number(), lane = threadIdx.x & 31;
    const int cg = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21, tmem = sh.tmem;
    float row_lse = -kInf, row_d = 0.f;     // of a held query: -LSE log2 e, -D
    int g = 0, q = 0;
    const bool row = (KEYS ? u.mine * kTileRows + r < a.ks.Nk : a.qt.at(u.mine, r, g, q)) &&
                     FIBATT_CHECKED(u.b >= 0 && u.b < a.B && u.hk < a.Hkv);
    if (!KEYS && row) {
        const float2 st = __ldg(a.stats + ((int64_t)u.b * a.Hq + u.hk * a.qt.G + g) * a.qt.Nq + q);
        row_lse = -st.x;
        row_d = -st.y;
    }
    // keys that are not attended have no gradient, whatever their rows hold
    const uint32_t word = (warp & 3) == 0 ? u.keys.x : (warp & 3) == 1 ? u.keys.y : (warp & 3) == 2 ? u.keys.z : u.keys.w;
    const bool zero = u.n == 0 || (KEYS && !((word >> lane) & 1));
    const float2 cc = make_float2(a.c, a.c);
    for (int j = 0; j < u.n; ++j, ++it) {
        pipe_wait(&sh.s, it & 1, abort);
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
        if (!KEYS && (a.ks.mask || (u.lo + j + 1) * kTileRows > u.bound)) {
            const int s = it % kStages;
            pipe_wait(&sh.ready[s], (it / kStages) & 1, abort);     // keys[s] is written
            const uint4 w = sh.keys[s];
            keep = cg == 0 ? w.x : cg == 1 ? w.y : cg == 2 ? w.z : w.w;
        }
        const bool free = it == 0 || pipe_ready(&sh.done, (it - 1) & 1);
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
        if (!free) pipe_wait(&sh.done, (it - 1) & 1, abort);
        tc_after_sync();
        if (KEYS) tmem_st16(tmem + kColP + 16 * cg + lanes, p);
        tmem_st16(tmem + kColDs + 16 * cg + lanes, ds);
        tmem_wait_st();
        tc_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p);
    }
    if (u.n > 0) pipe_wait(&sh.done, (it - 1) & 1, abort);
    tc_after_sync();
    // groups 0, 1: the halves of the first sum (dQ or dK); 2, 3: of the second (dV)
    const int acc = cg >> 1, half = cg & 1;
    if (acc && !KEYS) return it;
    uint32_t o[32];
    if (u.n > 0) {
        tmem_ld32(o, tmem + (acc ? kColAcc1 : kColAcc0) + 32 * half + lanes);
        tmem_wait_ld(o);
        tc_before_sync();
    }
    const float f = acc ? 1.f : a.scale;
    if (cluster_size() == 1) {
        if (!row) return it;
        __nv_bfloat16 *out = KEYS ? (acc ? a.dV : a.dK).row(u.b, u.hk, u.mine * kTileRows + r)
                                  : a.dQ.row(u.b, u.hk * a.qt.G + g, q);
        uint4 *o4 = reinterpret_cast<uint4 *>(out + 32 * half);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = zero ? 0u
                            : pack_bf16x2(__uint_as_float(o[8 * i + 2 * k]) * f, __uint_as_float(o[8 * i + 2 * k + 1]) * f);
            o4[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
        // a cluster has one unit: every copy and product has completed, the ring takes the partial sums
        float4 *out = reinterpret_cast<float4 *>(reinterpret_cast<float *>(ring) + (acc * kTileRows + r) * kJoinLd + 32 * half);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = zero ? 0.f : __uint_as_float(o[4 * i + k]) * f;
            out[i] = make_float4(w[0], w[1], w[2], w[3]);
        }
    }
    return it;
}

// Copies; false: a wait gave up.  `units` counts the units with tiles, whose held
// rows are in pairs of tiles in turn.
template <bool KEYS>
__device__ __forceinline__ bool copies(const BwdMmaArgs &a, Shared &sh, const Tiles &tl, const Unit &u, int &it, int &units) {
    volatile int *abort = &sh.abort;
    if (u.n == 0) return true;
    const auto query_tile = [&](uint8_t *dst, int t, uint64_t *bar) {
        load_tile(dst, a.q, a.qt.first_row(t), u.hk * a.qt.G + a.qt.first_head(t), u.b, bar);
        load_tile(dst + kTileBytes, a.g, a.qt.first_row(t), u.hk * a.qt.G + a.qt.first_head(t), u.b, bar);
    };
    const auto key_tile = [&](uint8_t *dst, int t, uint64_t *bar) {
        load_tile(dst, a.k, t * kTileRows, u.hk, u.b, bar);
        load_tile(dst + kTileBytes, a.v, t * kTileRows, u.hk, u.b, bar);
    };
    const int pair = units & 1;
    if (units >= 2 && !pipe_wait(&sh.held_free[pair], ((units >> 1) - 1) & 1, abort)) return false;
    if (elect_one()) {
        mbar_expect_tx(&sh.held[pair], 2 * (KEYS ? (uint32_t)kTileBytes : a.qt.bytes()));
        if (KEYS) key_tile(tl.pair(pair), u.mine, &sh.held[pair]);
        else query_tile(tl.pair(pair), u.mine, &sh.held[pair]);
    }
    __syncwarp();
    ++units;
    const uint32_t bytes = 2 * (KEYS ? a.qt.bytes() + a.qt.bytes() / 8 : (uint32_t)kTileBytes);
    for (int j = 0; j < u.n; ++j) {
        const int s = it % kStages, t = u.lo + j;
        if (it >= kStages && !pipe_wait(&sh.empty[s], (it / kStages - 1) & 1, abort)) return false;
        if (elect_one()) {
            mbar_expect_tx(&sh.full[s], bytes);
            if (KEYS) {
                const int rows = a.qt.nb;
                query_tile(tl.stage(s), t, &sh.full[s]);
                for (int i = 0; i < a.qt.gb; ++i) {
                    const int g = a.qt.first_head(t) + i;
                    const int64_t none = (int64_t)a.B * a.Hq * a.npad;      // rows of no query
                    int64_t from = g < a.qt.G ? ((int64_t)u.b * a.Hq + u.hk * a.qt.G + g) * a.npad + a.qt.first_row(t)
                                              : none;   // no such head
                    if (!FIBATT_CHECKED(from >= 0 && from + rows <= none + kTileRows)) from = none;   // the workspace's rows
                    uint8_t *to = tl.part(s) + i * rows * 16;
                    bulk_g2s(to, a.lse_parts + from, rows * 16, &sh.full[s]);
                    bulk_g2s(to + kNarrow, a.d_parts + from, rows * 16, &sh.full[s]);
                }
            } else {
                key_tile(tl.stage(s), t, &sh.full[s]);
            }
        }
        __syncwarp();
        ++it;
    }
    return true;
}

// Which keys of a streamed tile are attended; K's other rows, which are read across
// with weights of 0, cleared.  Of streamed queries, the rows behind the tile's last,
// which hold what was there before or the next group's.  false: a wait gave up.
template <bool KEYS>
__device__ __forceinline__ bool prepare(const BwdMmaArgs &a, Shared &sh, const Tiles &tl, const Unit &u, int &it) {
    volatile int *abort = &sh.abort;
    for (int j = 0; j < u.n; ++j, ++it) {
        const int s = it % kStages;
        uint4 w = make_uint4(0, 0, 0, 0);
        int rows = kTileRows;
        if (!KEYS) w = tile_keys(a.ks, u.b, (u.lo + j) * kTileRows, u.bound);
        else rows = min(a.qt.gb, a.qt.G - a.qt.first_head(u.lo + j)) * a.qt.nb;
        if (!pipe_wait(&sh.full[s], (it / kStages) & 1, abort)) return false;
        if (KEYS) {
            if (rows < kTileRows) {
                uint4 *q = reinterpret_cast<uint4 *>(tl.stage(s));       // 8 a row; dO's behind Q's
                for (int i = 8 * rows + (int)(threadIdx.x & 31); i < 8 * kTileRows; i += 32)
                    q[i] = q[i + kTileBytes / 16] = make_uint4(0, 0, 0, 0);
                fence_smem_async();
                __syncwarp();
            }
        } else {
            if (!all_keys(w)) {
                clear_rows(tl.stage(s), w);
                fence_smem_async();
            }
            if ((threadIdx.x & 31) == 0) sh.keys[s] = w;
            __syncwarp();
        }
        if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.ready[s]);
    }
    return true;
}

// Matrix instructions, by two warps so that neither kind waits for what the other
// needs.  The loops' course depends on uniform values only (a wait that gives up
// is not looked at: what follows is not trusted, since the error word is set).
struct Turn {   // a place in the ring
    int s = 0, pass = 0;
    __device__ __forceinline__ void next() {
        if (++s == kStages) {
            s = 0;
            pass ^= 1;
        }
    }
};

// S and dP
template <bool KEYS>
__device__ __forceinline__ void scores(const BwdMmaArgs &a, Shared &sh, const Tiles &tl, const Unit &u, int &it, int &units,
                                       Turn &at) {
    volatile int *abort = &sh.abort;
    if (u.n == 0) return;
    const uint32_t id = mma_desc(128, 128, false), tmem = sh.tmem;
    const int pair = units & 1;
    const uint64_t h0 = tile_desc(tl.pair(pair)), h1 = h0 + (kTileBytes >> 4);
    const uint64_t one = narrow_desc(tl.ones, tl.zeros);
    pipe_wait(&sh.held[pair], (units >> 1) & 1, abort);
    ++units;
    for (int j = 0; j < u.n; ++j, ++it, at.next()) {
        const uint64_t r0 = tile_desc(tl.ring) + (uint64_t)(at.s * (2 * kTileBytes >> 4)), r1 = r0 + (kTileBytes >> 4);
        const uint64_t lse = narrow_desc(tl.part(at.s), tl.zeros), d = narrow_desc(tl.part(at.s) + kNarrow, tl.zeros);
        pipe_wait(&sh.ready[at.s], at.pass, abort);
        if (it > 0) pipe_wait(&sh.sfree, (it - 1) & 1, abort);
        tc_after_sync();
        if (elect_one()) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mma_ss(tmem + kColS, h0 + i * kStepRowwise, r0 + i * kStepRowwise, id, i > 0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mma_ss(tmem + kColDp, h1 + i * kStepRowwise, r1 + i * kStepRowwise, id, i > 0);
            if (KEYS) {
                mma_ss(tmem + kColS, one, lse, id, true);
                mma_ss(tmem + kColDp, one, d, id, true);
            }
            mma_commit(&sh.s);
            if (j == u.n - 1) mma_commit(&sh.held_free[pair]);
        }
        __syncwarp();
    }
}

// dQ, or dK and dV
template <bool KEYS>
__device__ __forceinline__ void sums(const BwdMmaArgs &a, Shared &sh, const Tiles &tl, const Unit &u, int &it, Turn &at) {
    volatile int *abort = &sh.abort;
    const uint32_t id = mma_desc(128, 64, true), tmem = sh.tmem;
    for (int j = 0; j < u.n; ++j, ++it, at.next()) {
        const uint64_t r0 = tile_desc(tl.ring) + (uint64_t)(at.s * (2 * kTileBytes >> 4)), r1 = r0 + (kTileBytes >> 4);
        pipe_wait(&sh.p, it & 1, abort);
        tc_after_sync();
        if (elect_one()) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                mma_ts(tmem + kColAcc0, tmem + kColDs + i * 8, r0 + i * kStepAcross, id, j > 0 || i > 0);
            if (KEYS) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    mma_ts(tmem + kColAcc1, tmem + kColP + i * 8, r1 + i * kStepAcross, id, j > 0 || i > 0);
            }
            mma_commit(&sh.done);
            mma_commit(&sh.empty[at.s]);
        }
        __syncwarp();
    }
}

// Join of a cluster's partial sums: CTA r finishes every CS-th row.
template <bool KEYS>
__device__ __forceinline__ void join(const BwdMmaArgs &a, const Tiles &tl, const Unit &u) {
    const int CS = (int)cluster_size(), rank = (int)cluster_rank();
    const float *part = reinterpret_cast<const float *>(tl.ring);
    const int c4 = (threadIdx.x & 15) * 4;
    for (int i = rank + CS * (int)(threadIdx.x >> 4); i < (KEYS ? 2 : 1) * kTileRows; i += CS * (kThreads / 16)) {
        const int acc = i / kTileRows, r = i % kTileRows;
        int g = 0, q = 0;
        if (KEYS ? u.mine * kTileRows + r >= a.ks.Nk : !a.qt.at(u.mine, r, g, q)) continue;
        if (!FIBATT_CHECKED(u.b >= 0 && u.b < a.B && u.hk < a.Hkv)) continue;
        float2 x = make_float2(0.f, 0.f), y = x;
        for (int k = 0; k < CS; ++k) {
            const uint32_t at = cluster_addr(part + i * kJoinLd + c4, k);
            x = add2(x, ld_cluster2(at));
            y = add2(y, ld_cluster2(at + 8));
        }
        __nv_bfloat16 *out = KEYS ? (acc ? a.dV : a.dK).row(u.b, u.hk, u.mine * kTileRows + r)
                                  : a.dQ.row(u.b, u.hk * a.qt.G + g, q);
        *reinterpret_cast<uint2 *>(out + c4) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(y.x, y.y));
    }
}

__global__ void __launch_bounds__(kThreads, 1) cross_bwd_mma_kernel(const __grid_constant__ BwdMmaArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    __shared__ Shared sh;
    const Tiles tl(smem);
    const int warp = warp_number(), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.held[i], 1);
            mbar_init(&sh.held_free[i], 1);
            mbar_init(&sh.end[i], 1);
            mbar_init(&sh.unit_full[i], 1);
            mbar_init(&sh.unit_empty[i], kWeightWarps + 3);
        }
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.ready[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        mbar_init(&sh.s, 1);
        mbar_init(&sh.sfree, kWeightWarps);
        mbar_init(&sh.p, kWeightWarps);
        mbar_init(&sh.done, 1);
        sh.abort = 0;
        prefetch_map(&a.q.map);
        prefetch_map(&a.g.map);
        prefetch_map(&a.k.map);
        prefetch_map(&a.v.map);
    }
    if (warp == kSumWarp) tmem_alloc(&sh.tmem, kCols);
    // ones in the first three elements of a row; rows of no query until copies bring some
    const uint4 none = no_query(a.c);
    for (int i = threadIdx.x; i < (2 + 2 * kStages) * kTileRows; i += kThreads) {
        const int tile = i / kTileRows;    // ones, then LSE and D of each stage, then zeros
        uint4 v = make_uint4(0, 0, 0, 0);
        if (tile == 0) v = make_uint4(0x3f803f80u, 0x3f80u, 0u, 0u);
        else if ((tile & 1) && tile < 1 + 2 * kStages) v = none;
        reinterpret_cast<uint4 *>(tl.ones)[i] = v;
    }
    fence_smem_async();
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    grid_dep_wait();
    grid_dep_launch();

    // The CTA's units: its first, then what it draws from a counter, which the copying
    // warp does and passes on (CTAs that finish early take more; a unit's results do
    // not depend on who works on it).  A cluster has one unit.
    const int CS = (int)cluster_size(), first = a.first_unit + (int)(blockIdx.x / CS);
    const auto each = [&](auto next, auto queries, auto keys) {
        Unit u = next();
#pragma unroll 1
        for (; u.index < a.query_units; u = next()) queries(u);
#pragma unroll 1
        for (; u.index < a.units; u = next()) keys(u);
    };
    int passed = 0;         // units handed over
    const auto take = [&] {
        const int i = passed & 1;
        Unit u;
        const bool ok = pipe_wait(&sh.unit_full[i], (passed >> 1) & 1, &sh.abort);
        u = sh.unit[i];
        u.index = __shfl_sync(kFullMask, ok ? u.index : a.units, 0);
        u.n = __shfl_sync(kFullMask, u.n, 0);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.unit_empty[i]);
        ++passed;
        return u;
    };
    int it = 0, units = 0;
    if (warp < kWeightWarps) {
        take_registers<kRegsMany>();
        each(take, [&](const Unit &u) { it = weights<false>(a, sh, tl.ring, u, it); },
             [&](const Unit &u) { it = weights<true>(a, sh, tl.ring, u, it); });
    } else {
        give_registers<kRegsFew>();
        if (warp == kCopyWarp) {
            bool ok = true;
            int drawn = first;
            const auto pass = [&] {      // (its copies being out, the next unit's number has come meanwhile)
                const int i = passed & 1;
                Unit u;
                u.enter(a, __shfl_sync(kFullMask, drawn, 0));
                drawn = a.units;
                if (CS == 1 && lane == 0 && u.index < a.units) drawn = a.first_unit + (int)gridDim.x + atomicAdd(a.next_unit, 1);
                ok = ok && (passed < 2 || pipe_wait(&sh.unit_empty[i], ((passed >> 1) - 1) & 1, &sh.abort));
                if (!ok) u.index = a.units;
                else if (lane == 0) {
                    sh.unit[i] = u;
                    mbar_arrive(&sh.unit_full[i]);
                }
                __syncwarp();
                ++passed;
                return u;
            };
            each(pass, [&](const Unit &u) { ok = ok && copies<false>(a, sh, tl, u, it, units); },
                 [&](const Unit &u) { ok = ok && copies<true>(a, sh, tl, u, it, units); });
            if (lane == 0) {   // leave no copy in flight
                for (int i = max(0, units - 2); i < units; ++i) mbar_drain(&sh.held[i & 1], (i >> 1) & 1);
                for (int i = max(0, it - kStages); i < it; ++i) mbar_drain(&sh.full[i % kStages], (i / kStages) & 1);
            }
        } else if (warp == kPrepWarp) {
            bool ok = true;
            each(take, [&](const Unit &u) { ok = ok && prepare<false>(a, sh, tl, u, it); },
                 [&](const Unit &u) { ok = ok && prepare<true>(a, sh, tl, u, it); });
        } else {
            Turn at;
            if (warp == kScoreWarp)
                each(take, [&](const Unit &u) { scores<false>(a, sh, tl, u, it, units, at); },
                     [&](const Unit &u) { scores<true>(a, sh, tl, u, it, units, at); });
            else
                each(take, [&](const Unit &u) { sums<false>(a, sh, tl, u, it, at); }, [&](const Unit &u) { sums<true>(a, sh, tl, u, it, at); });
            // no matrix instruction in flight when the tensor memory is freed
            uint64_t *end = &sh.end[warp == kSumWarp];
            if (elect_one()) mma_commit(end);
            __syncwarp();
            mbar_drain(end, 0);
        }
    }
    __syncwarp();
    tc_before_sync();
    __syncthreads();
    if (warp == kSumWarp) tmem_free(sh.tmem, kCols);
    if (CS == 1) return;
    cluster_sync();
    Unit u;
    u.enter(a, first);
    if (first < a.query_units) join<false>(a, tl, u);
    else join<true>(a, tl, u);
    cluster_sync();   // the others may still read this CTA's part
}

// Rows of a head with the last of its query tiles whole.
int padded_rows(int Nq) { return Nq < kTileRows ? Nq : (Nq + kTileRows - 1) / kTileRows * kTileRows; }

}  // namespace

size_t cross_bwd_mma_workspace(int B, int Hq, int Nq) {
    const size_t rows = (size_t)B * Hq * padded_rows(Nq);
    return 2 * (rows + kTileRows) * sizeof(uint4) + (size_t)B * Hq * Nq * sizeof(float2) + 2 * sizeof(int);
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
    f.next_unit = reinterpret_cast<int *>(stats + (int64_t)a.B * a.Hq * a.Nq);
    f.lse_parts = lse_parts, f.d_parts = d_parts;
    f.dQ = rows_of<__nv_bfloat16>(a.dQ), f.dK = rows_of<__nv_bfloat16>(a.dK), f.dV = rows_of<__nv_bfloat16>(a.dV);
    f.B = a.B, f.Hq = a.Hq, f.Hkv = a.Hkv;
    f.ktiles = (a.Nk + kTileRows - 1) / kTileRows;
    f.scale = a.scale;
    // a scale of 0: any c this small leaves every finite score's weight at exp2(-LSE log2 e)
    f.c = std::copysign(std::max(std::fabs(a.scale) * kLog2e, 1e-36f), a.scale);
    cudaError_t e = prepare_kernel<cross_bwd_mma_kernel>(kSmem, kRegs);
    if (e != cudaSuccess) return e;
    if (a.Nk <= kFewKeys) {
        const int64_t warps = (int64_t)a.B * a.Hq * ((f.npad + 15) / 16) + kTileRows / 16;
        e = launch_clusters(cross_parts_few_kernel, (unsigned)((warps + kFewWarps - 1) / kFewWarps), 1, 32 * kFewWarps, 0,
                            a.stream, a.Hq, a.Hkv, a.Nq, f.npad, (unsigned)(a.B * a.Hq), a.keys,
                            rows_of<const __nv_bfloat16>(a.Q), rows_of<const __nv_bfloat16>(a.K),
                            rows_of<const __nv_bfloat16>(a.V), rows_of<const __nv_bfloat16>(a.dO),
                            static_cast<const float *>(a.LSE), f.c, stats, lse_parts, d_parts, f.next_unit);
    } else {
        const auto kernel = a.keys.len ? cross_parts_kernel<true> : cross_parts_kernel<false>;
        e = launch_clusters(kernel, (unsigned)((rows + kTileRows + 31) / 32), 1, 256, 0, a.stream, a.Hq, a.Hkv, a.Nq, f.npad,
                            (unsigned)rows, a.keys, rows_of<const __nv_bfloat16>(a.Q), rows_of<const __nv_bfloat16>(a.K),
                            rows_of<const __nv_bfloat16>(a.V), rows_of<const __nv_bfloat16>(a.O),
                            rows_of<const __nv_bfloat16>(a.dO), static_cast<const float *>(a.LSE), f.c, stats, lse_parts,
                            d_parts, f.next_unit);
    }
    if (e != cudaSuccess) return e;
    const int64_t query_units = (int64_t)a.B * a.Hkv * f.qt.tiles, key_units = (int64_t)a.B * a.Hkv * f.ktiles;
    f.query_units = (int)query_units;
    // clusters, one unit each, while they all find a place; else one wave of CTAs that walk over the units
    const auto launch = [&](int64_t from, int64_t units, int c) {
        f.first_unit = (int)from;
        f.units = (int)(from + units);
        const int64_t grid = c > 1 ? units * c : std::min<int64_t>(units, sm_count());
        return launch_clusters(cross_bwd_mma_kernel, (unsigned)grid, c, kThreads, kSmem, a.stream, f);
    };
    // (one head, 100 queries on 16385 keys: 27 us in two launches, 82 in one; 16 heads, 100 on 5000:
    // 44 and 36)
    const Launches l(query_units, f.ktiles, key_units, f.qt.tiles, sm_count(), 5, 12);
    if (!l.two) return launch(0, query_units + key_units, l.c);
    e = launch(0, query_units, l.c_query);
    if (e != cudaSuccess) return e;
    ++f.next_unit;
    return launch(query_units, key_units, l.c_key);
}

FIBATT_DEFINE_ERROR_READER(read_error_cross_mma_bwd, "cross_mma_bwd.cu")

}  // namespace fibatt
