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
//
// Attention over a window with sinks (BAND): walks over the tiles that the held rows' windows meet, masked at
// their ends from the positions.  Key tiles first, whose walks are longer (a head group's queries: 36
// tiles next to 9, at window 1024 and 4 heads a key head; queries first: 96 us for 89 on eight clips).  The
// keys of a tile with sinks meet every later query: such walks are cut into parts (SinkParts), whose sums
// a small kernel adds in their order.  Walks being short, what lies between units counts: a unit's
// results are put where its held rows were and leave by tensor copies that the copying warp sends, and
// its rows' statistics are asked for one unit ahead; no thread divides (Div: 261 -> 251 us, and 82.8 -> 78.5 below, where
// a tile of keys took 2140 cycles for 1600).
// Measured (4 sinks): 16 heads on 4, 16385 tokens, window 1024: 249 us, 670 TFLOP/s of the 5 products (about 1600
// cycles a tile of either kind, 2150 between units of 9 or 10 tiles; the small kernels about 20 us of it); 8 sequences,
// 12 heads on 4, up to 1569 tokens, window 512: 74.7, 362 (the first small kernel about 9; units of 5 or 6 tiles of
// keys, 16 of queries).
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
constexpr int kPartSums = 8 * 32 * kWeightWarps;  // float4s of a part's sums, of dK and dV
constexpr int kJoinLd = 68;                       // floats between rows of a partial sum in shared memory
static_assert(2 * kTileRows * kJoinLd * 4 <= 2 * kStages * kTileBytes, "partial sums fit");
// registers a thread: at launch, and after the weight warps took what the others gave
constexpr int kRegs = 96, kRegsFew = 32, kRegsMany = 112;
static_assert(4 * kRegsMany + kRegsFew == 5 * kRegs, "the shares add up");

// columns of tensor memory
constexpr uint32_t kColS = 0, kColDp = 128, kColP = 256, kColDs = 320, kColAcc0 = 384, kColAcc1 = 448, kCols = 512;

// What only a window's calls have.  (Other launches do not carry it.)
template <bool BAND>
struct BwdBandArgs {};
template <>
struct BwdBandArgs<true> {
    Band band;
    Div by_heads, by_hkv, by_sinks;     // heads of keys of all sequences, of one, and the sinks' tiles of all
    int chunks, chunk_tiles;    // parts of a sinks' walk and the query tiles of each, ...
    int sink_tiles, sink_units; // ... key tiles that have such walks, units of those parts
    float4 *parts;              // their partial sums, one after another
    int cleared;                // dQ of queries outside their sequence is, and units of such alone are left out
    TensorArg dq, dk, dv;       // the gradients as tensor copies write them (dQ: tiles of 128 queries)
};

template <bool BAND>
struct BwdMmaArgs : BwdBandArgs<BAND> {
    TensorArg q, g, k, v;       // boxes of query tiles (Q, dO) and of key tiles (K, V)
    TilesOf<BAND> qt;
    KeySet ks;
    const float2 *stats;        // (LSE log2 e, D) of every query row
    const uint4 *lse_parts, *d_parts;   // of every query row of whole tiles, then 128 rows of no query
    int npad;                   // rows of a head there
    Rows<__nv_bfloat16> dQ, dK, dV;
    int B, Hq, Hkv, ktiles;
    int first_kind, units;      // units of the kind that comes first (queries held; BAND: keys held), and all of them
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
    if (none) d = 0.f;      // (dO may hold anything)
    if (i == 0) lse_parts[row] = none ? no_query(c) : three_parts(-lse2 / c);
    if (i == 1) d_parts[row] = three_parts(-d);
    if (i == 2) stats[at] = make_float2(lse2, d);
}

// The same for a window's queries where a head has rows enough: a block has 64 rows of one head,
// four threads each, and rows outside their sequence are not read; their dQ is cleared, which
// leaves the next kernel no units of queries without tiles.  (The gradient of 16 heads of
// 16385 tokens 268 us, 270 with the kernel above; of eight clips of several lengths 86.7 and 89.2.)
constexpr int kPartRows = 64;
__global__ void __launch_bounds__(4 * kPartRows)
window_parts_kernel(int Hq, int Nq, int npad, unsigned heads, KeySet ks, Band band, Rows<const __nv_bfloat16> O,
                    Rows<const __nv_bfloat16> dO, const float *__restrict__ LSE, float c, float2 *__restrict__ stats,
                    uint4 *__restrict__ lse_parts, uint4 *__restrict__ d_parts, int *__restrict__ next_unit,
                    Rows<__nv_bfloat16> dQ) {
    grid_dep_wait();
    grid_dep_launch();
    if (blockIdx.x == 0 && threadIdx.x < 2) next_unit[threadIdx.x] = 0;
    const unsigned steps = (unsigned)(npad + kPartRows - 1) / kPartRows, bh = blockIdx.x / steps;
    const int n = (int)(blockIdx.x - bh * steps) * kPartRows + (int)(threadIdx.x >> 2), i = threadIdx.x & 3;
    if (bh >= heads) {      // 128 rows of no query, behind the heads'
        const unsigned row = (blockIdx.x - heads * steps) * kPartRows + (threadIdx.x >> 2);
        if (i == 0) lse_parts[(int64_t)heads * npad + row] = no_query(c);
        if (i == 1) d_parts[(int64_t)heads * npad + row] = make_uint4(0, 0, 0, 0);
        return;
    }
    if (n >= npad) return;  // whole groups of four
    const int b = (int)(bh / (unsigned)Hq), h = (int)(bh - (unsigned)b * Hq), p = band.first(b) + n;
    float lse2 = kInf, d = 0.f;
    bool none = true;
    if (n < Nq && p >= 0 && p < ks.bound(b)) {
        const uint4 *o = reinterpret_cast<const uint4 *>(O.row(b, h, n)) + 2 * i, *g = reinterpret_cast<const uint4 *>(dO.row(b, h, n)) + 2 * i;
        const uint4 o0 = __ldg(o), o1 = __ldg(o + 1), g0 = __ldg(g), g1 = __ldg(g + 1);
        const float lse = __ldg(LSE + (int64_t)bh * Nq + n);
        none = lse == -kInf;
        if (!none) {
            lse2 = lse * kLog2e;
            d = dot2_bf16(o0.x, g0.x, dot2_bf16(o0.y, g0.y, 0.f)) + dot2_bf16(o0.z, g0.z, dot2_bf16(o0.w, g0.w, 0.f)) +
                (dot2_bf16(o1.x, g1.x, dot2_bf16(o1.y, g1.y, 0.f)) + dot2_bf16(o1.z, g1.z, dot2_bf16(o1.w, g1.w, 0.f)));
        }
    } else if (n < Nq) {
        uint4 *to = reinterpret_cast<uint4 *>(dQ.row(b, h, n)) + 2 * i;
        to[0] = to[1] = make_uint4(0, 0, 0, 0);
    }
    const unsigned four = 0xfu << (threadIdx.x & 28);
    d += __shfl_xor_sync(four, d, 1);
    d += __shfl_xor_sync(four, d, 2);
    const int64_t row = (int64_t)bh * npad + n;
    if (i == 0) lse_parts[row] = none ? no_query(c) : three_parts(-lse2 / c);
    if (i == 1) d_parts[row] = n < Nq ? three_parts(-d) : make_uint4(0, 0, 0, 0);
    if (i == 2 && n < Nq) stats[(int64_t)bh * Nq + n] = make_float2(lse2, d);
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
// BAND: also for windows of so few keys, sinks among them (a long sequence's first rows, of few keys too,
// have <dO, O>: with the sum for those of up to 8 keys the first kernel took 4 us more, whose rows it all slows).
constexpr int kFewWarps = 4;
template <bool BAND>
__global__ void __launch_bounds__(32 * kFewWarps)
cross_parts_few_kernel(int Hq, int Hkv, int Nq, int npad, unsigned heads, KeySet ks, Band band, Rows<const __nv_bfloat16> Q,
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
    int bound = ks.bound((int)b), front = 0, oldest = 0, at_p[2] = {-1, -1};
    if constexpr (BAND) {      // the eights with keys of the 16 queries: those of the sinks, and from the oldest on
        const int p = band.first((int)b) + n0, last = min(bound, p + min(16, Nq - n0)) - 1;
        bound = last >= max(0, p) ? last + 1 : 0;
        oldest = max(0, p - band.window + 1) & ~7;
        front = min(band.sinks, oldest);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (p + g + 8 * i <= last) at_p[i] = p + g + 8 * i;
    }
    for (int k0 = 0; k0 < bound; k0 += 8) {
        if (BAND && k0 >= front) k0 = max(k0, oldest);
        const int mine = k0 + (lane & 7);
        const uint32_t in = __ballot_sync(kFullMask, mine < bound && (BAND || ks.has((int)b, min(mine, bound - 1))));
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
            const bool on = BAND ? band.sees(at_p[i >> 1], k0 + 2 * t + (i & 1)) : (in >> (2 * t + (i & 1))) & 1;
            if (on) d[i >> 1] = fmaf(p, dp[i], d[i >> 1]);
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
template <bool BAND>
struct UnitBand {};
template <>
struct UnitBand<true> {
    int p0, first, last;     // position of query 0; of the unit's queries, held or streamed, that attend keys of it
    int chunk;               // keys held: the part of the walk that this unit has, -1: all of it
    int leaves;              // the pair of places for held rows from where its gradients leave by tensor copies, -1: none
    KeyWalk<kTileRows> walk;    // held queries
    __device__ __forceinline__ UnitBand() {}
};
template <bool BAND>
struct Unit : UnitBand<BAND> {
    int index;               // queries held first, then keys held (BAND: keys first, whose walks are longer)
    int mine, hk, b, bound, lo, n;
    uint4 keys;              // keys held: which rows are attended
    template <bool KEYS>
    __device__ __forceinline__ void set(const BwdMmaArgs<BAND> &a, int i) {
        index = i;
        if constexpr (BAND) set_band<KEYS>(a, KEYS ? i : i - a.first_kind);
        else set_all<KEYS>(a, i);
    }
    template <bool KEYS>
    __device__ __forceinline__ void set_all(const BwdMmaArgs<BAND> &a, int i) {
        const int unit = KEYS ? i - a.first_kind : i, held = KEYS ? a.ktiles : a.qt.tiles;
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
    // The units with the longest walks first: the last queries, the first keys.
    // Tiles with sinks, whose keys all later queries attend, have their walks cut into parts
    // about as long as the others' walks.
    template <bool KEYS>
    __device__ __forceinline__ void set_band(const BwdMmaArgs<BAND> &a, int unit) {
        const int heads = a.Hkv * a.B;
        this->chunk = -1;
        if (KEYS) {
            const int tiles = a.sink_tiles * heads;
            if (unit < a.sink_units) this->chunk = a.by_sinks.of(unit), unit = a.by_sinks.rest(unit);
            else unit += tiles - a.sink_units;
        }
        mine = a.by_heads.of(unit);
        unit -= mine * heads;
        if (!KEYS) mine = a.qt.tiles - 1 - mine;
        b = a.by_hkv.of(unit);
        hk = unit - b * a.Hkv;
        bound = a.ks.bound(b);
        this->p0 = a.band.first(b);
        keys = make_uint4(0, 0, 0, 0);
        const int end = min(bound, this->p0 + a.qt.Nq);       // behind the last position of a query
        int tiles, from = 0;
        if (KEYS) {
            const int k0 = mine * kTileRows, k1 = min(k0 + kTileRows, bound) - 1;
            this->first = max(this->p0, k0);        // (k0 >= 0)
            this->last = (k0 < a.band.sinks ? end : min(end, k1 + a.band.window)) - 1;
            const bool some = k0 <= k1 && this->first <= this->last;
            if (!some) this->last = this->first - 1;
            from = some ? a.qt.by_rows.of(this->first - this->p0) * a.qt.groups : 0;
            tiles = some ? (a.qt.by_rows.of(this->last - this->p0) + 1) * a.qt.groups - from : 0;
            keys = band_keys(a.band, this->first, this->last, k0);
        } else {
            this->first = max(0, this->p0 + a.qt.first_row(mine));
            this->last = min(end, this->p0 + a.qt.first_row(mine) + a.qt.nb) - 1;
            this->walk = KeyWalk<kTileRows>(a.band, this->first, this->last);
            tiles = this->walk.n;
        }
        if (KEYS && this->chunk >= 0) {      // (a walk may be shorter than its parts)
            const int at = this->chunk * a.chunk_tiles;
            lo = from + at;
            n = max(0, min(a.chunk_tiles, tiles - at));
            return;
        }
        const int CS = (int)cluster_size(), rank = (int)cluster_rank();
        lo = 0, n = tiles;
        if (CS > 1) {
            lo = (int)((int64_t)tiles * rank / CS);
            n = (int)((int64_t)tiles * (rank + 1) / CS) - lo;
        }
        lo += from;
    }
    // first key of tile j of held queries' walk
    __device__ __forceinline__ int key(int j) const {
        if constexpr (BAND) return this->walk.key(lo + j);
        else return (lo + j) * kTileRows;
    }
    // the whole warp calls it; an index behind the last unit stands for the end
    __device__ __forceinline__ void enter(const BwdMmaArgs<BAND> &a, int i) {
        if (i < a.first_kind) set<BAND>(a, i);
        else if (i < a.units) set<!BAND>(a, i);
        else index = i, mine = hk = b = bound = lo = n = 0, keys = make_uint4(0, 0, 0, 0);
    }
};

template <bool BAND>
struct Shared {
    uint64_t held[2], held_free[2], full[kStages], ready[kStages], empty[kStages], s, sfree, p, done, end[2];
    uint64_t unit_full[2], unit_empty[2];
    uint4 keys[kStages];
    uint64_t out[2];            // BAND: a unit is over, in turn; ...
    Unit<BAND> unit[2];         // the CTA's, in turn
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

// (LSE log2 e, D) of a thread's row of held queries; anything where it has none.  (No branch, at whose end the
// value would be waited for.)
__device__ __forceinline__ float2 row_stats(const BwdMmaArgs<true> &a, const Unit<true> &u) {
    const int r = (int)(warp_number() & 3) * 32 + (int)(threadIdx.x & 31);
    int g, q;
    const bool row = u.index >= a.first_kind && u.index < a.units && a.qt.at(u.mine, r, g, q);
    return __ldg(a.stats + (row ? ((int64_t)u.b * a.Hq + u.hk * a.qt.G + g) * a.qt.Nq + q : 0));
}

// P and dS: row = lane of the quarter, 32 columns.  BAND: `stats` of the unit's rows; `ahead` before the
// unit's end, which hides what the next one has to wait for.
template <bool KEYS, bool BAND, typename Ahead>
__device__ __forceinline__ int weights(const BwdMmaArgs<BAND> &a, Shared<BAND> &sh, const Tiles &tl, const Unit<BAND> &u, int it,
                                       float2 &stats, Ahead ahead) {
    uint8_t *const ring = tl.ring;
    volatile int *abort = &sh.abort;
    const int warp = warp_number(), lane = threadIdx.x & 31;
    const int cg = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21, tmem = sh.tmem;
    float row_lse = -kInf, row_d = 0.f;     // of a held query: -LSE log2 e, -D
    int g = 0, q = 0;
    const bool row = (KEYS ? u.mine * kTileRows + r < a.ks.Nk : a.qt.at(u.mine, r, g, q)) &&
                     FIBATT_CHECKED(u.b >= 0 && u.b < a.B && u.hk < a.Hkv);
    if (!KEYS && row) {
        if (!BAND) stats = __ldg(a.stats + ((int64_t)u.b * a.Hq + u.hk * a.qt.G + g) * a.qt.Nq + q);
        row_lse = -stats.x;
        row_d = -stats.y;
    }
    // keys that are not attended have no gradient, whatever their rows hold
    const uint32_t word = (warp & 3) == 0 ? u.keys.x : (warp & 3) == 1 ? u.keys.y : (warp & 3) == 2 ? u.keys.z : u.keys.w;
    const bool zero = u.n == 0 || (KEYS && !((word >> lane) & 1));
    // BAND: the row's position, -1 for none (held queries); the tile's; held keys and tiles
    // of several heads: which columns attend the row's key, the same for all of the walk
    int p = -1, lowest = 0, highest = 0;
    uint32_t same = 0;
    if constexpr (BAND) {
        if (!KEYS) {
            lowest = u.p0 + a.qt.first_row(u.mine);
            highest = u.p0 + min(a.qt.Nq, a.qt.first_row(u.mine) + a.qt.nb) - 1;
            p = lowest + a.qt.by_rows.rest(r);
            if (p >= u.bound) p = -1;
        } else if (a.qt.nb < kTileRows) {
            const int k = u.mine * kTileRows + r;
            for (int i = 0, n = a.qt.by_rows.rest(32 * cg); i < 32; ++i) {
                const int at = u.p0 + n;
                if (at >= u.first && at <= u.last && a.band.sees(at, k)) same |= 1u << i;
                if (++n == a.qt.nb) n = 0;
            }
        }
    }
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
        if constexpr (BAND) {
            if (KEYS) {
                const int k0 = u.mine * kTileRows, k = k0 + r, q = a.qt.first_row(u.lo + j), at = u.p0 + q;
                if (a.qt.nb < kTileRows) keep = same;
                else if (!(at >= k0 + kTileRows - 1 && at + kTileRows <= min(u.bound, u.p0 + a.qt.Nq) &&
                           (at + kTileRows - 1 < k0 + a.band.window || k0 + kTileRows <= a.band.sinks)))
                    keep = queries_of(a.band, k, at + 32 * cg, u.last + 1);
            } else {
                const Band w = u.walk.band(a.band, u.lo + j);
                const int k0 = u.key(j), k1 = k0 + kTileRows - 1;
                if (!(k1 <= lowest && highest < u.bound && (k0 > highest - w.window || k1 < w.sinks)))
                    keep = keys_of(w, p, k0 + 32 * cg);
            }
        } else if (!KEYS && (a.ks.mask || (u.lo + j + 1) * kTileRows > u.bound)) {
            const int s = it % kStages;
            pipe_wait(&sh.ready[s], (it / kStages) & 1, abort);     // keys[s] is written
            const uint4 w = sh.keys[s];
            keep = cg == 0 ? w.x : cg == 1 ? w.y : cg == 2 ? w.z : w.w;
        }
        const bool free = it == 0 || pipe_ready(&sh.done, (it - 1) & 1);
        uint32_t p16[16], ds[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 sx = make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
            const float2 dp = make_float2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1]));
            const float2 z = KEYS ? mul2(sx, cc) : fma2(sx, cc, make_float2(row_lse, row_lse));
            const float2 w = make_float2(fast_exp2(z.x), fast_exp2(z.y));
            const float2 t = mul2(w, KEYS ? dp : add2(dp, make_float2(row_d, row_d)));
            if (KEYS) p16[i] = pack_bf16x2(w.x, w.y);
            ds[i] = pack_bf16x2(t.x, t.y);
        }
        if ((BAND || !KEYS) && keep != 0xffffffffu) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                uint32_t in = 0xffffffffu;
                if (!((keep >> (2 * i)) & 1)) in &= 0xffff0000u;
                if (!((keep >> (2 * i + 1)) & 1)) in &= 0x0000ffffu;
                ds[i] &= in;
                if (KEYS) p16[i] &= in;
            }
        }
        // the products have read the last P and dS
        if (!free) pipe_wait(&sh.done, (it - 1) & 1, abort);
        tc_after_sync();
        if (KEYS) tmem_st16(tmem + kColP + 16 * cg + lanes, p16);
        tmem_st16(tmem + kColDs + 16 * cg + lanes, ds);
        tmem_wait_st();
        tc_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p);
    }
    ahead();
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
    if constexpr (BAND) {
        if (KEYS && u.chunk >= 0 && FIBATT_CHECKED(u.mine < a.sink_tiles && u.chunk < a.chunks)) {       // (see window_sum_kernel)
            const int tile = (u.mine * a.B + u.b) * a.Hkv + u.hk;
            float4 *mine = a.parts + ((int64_t)tile * a.chunks + u.chunk) * kPartSums + threadIdx.x;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                __stcg(mine + i * 32 * kWeightWarps,
                       zero ? make_float4(0.f, 0.f, 0.f, 0.f)
                            : make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                          __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3])));
            return it;
        }
        if (u.leaves >= 0) {
            uint8_t *const tile = tl.pair(u.leaves) + acc * kTileBytes;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = zero ? 0u
                                : pack_bf16x2(__uint_as_float(o[8 * i + 2 * k]) * f, __uint_as_float(o[8 * i + 2 * k + 1]) * f);
                *reinterpret_cast<uint4 *>(tile + r * 128 + (((4 * half + i) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            fence_smem_async();
            return it;
        }
    }
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

// BAND, one lane: the gradients of a unit that is over leave.
__device__ __forceinline__ void send(const BwdMmaArgs<true> &a, const Tiles &tl, const Unit<true> &u) {
    if (u.leaves < 0 || !FIBATT_CHECKED(u.b >= 0 && u.b < a.B && u.hk < a.Hkv)) return;
    const uint8_t *tile = tl.pair(u.leaves);
    if (u.index >= a.first_kind) {
        tile_store(&a.dq.map, a.qt.first_row(u.mine), (u.hk * a.qt.G + a.qt.first_head(u.mine)) * a.dq.head_step,
                   u.b * a.dq.seq_step, tile);
    } else {
        tile_store(&a.dk.map, u.mine * kTileRows, u.hk * a.dk.head_step, u.b * a.dk.seq_step, tile);
        tile_store(&a.dv.map, u.mine * kTileRows, u.hk * a.dv.head_step, u.b * a.dv.seq_step, tile + kTileBytes);
    }
    stores_read();
}

// Copies; false: a wait gave up.  `units` counts the units with tiles, whose held
// rows are in pairs of tiles in turn.
template <bool KEYS, bool BAND>
__device__ __forceinline__ bool copies(const BwdMmaArgs<BAND> &a, Shared<BAND> &sh, const Tiles &tl, const Unit<BAND> &u, int &it, int &units) {
    volatile int *abort = &sh.abort;
    if (u.n == 0) return true;
    const auto query_tile = [&](uint8_t *dst, int t, uint64_t *bar) {
        load_tile(dst, a.q, a.qt.first_row(t), u.hk * a.qt.G + a.qt.first_head(t), u.b, bar);
        load_tile(dst + kTileBytes, a.g, a.qt.first_row(t), u.hk * a.qt.G + a.qt.first_head(t), u.b, bar);
    };
    const auto key_tile = [&](uint8_t *dst, int k0, uint64_t *bar) {
        load_tile(dst, a.k, k0, u.hk, u.b, bar);
        load_tile(dst + kTileBytes, a.v, k0, u.hk, u.b, bar);
    };
    const int pair = units & 1;
    if (units >= 2 && !pipe_wait(&sh.held_free[pair], ((units >> 1) - 1) & 1, abort)) return false;
    if (elect_one()) {
        mbar_expect_tx(&sh.held[pair], 2 * (KEYS ? (uint32_t)kTileBytes : a.qt.bytes()));
        if (KEYS) key_tile(tl.pair(pair), u.mine * kTileRows, &sh.held[pair]);
        else query_tile(tl.pair(pair), u.mine, &sh.held[pair]);
    }
    __syncwarp();
    ++units;
    const uint32_t bytes = 2 * (KEYS ? a.qt.bytes() + a.qt.bytes() / 8 : (uint32_t)kTileBytes);
    for (int j = 0; j < u.n; ++j) {
        const int s = it % kStages, t = u.lo + j;     // of streamed queries
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
                key_tile(tl.stage(s), u.key(j), &sh.full[s]);
            }
        }
        __syncwarp();
        ++it;
    }
    return true;
}

// Bit r: row r of query tile t is a query of the sequence.  The same in every lane.
__device__ __forceinline__ uint4 tile_queries(const BwdMmaArgs<true> &a, const Unit<true> &u, int t) {
    if (a.qt.nb == kTileRows && u.p0 + a.qt.first_row(t) >= 0 &&
        a.qt.first_row(t) + kTileRows <= min(a.qt.Nq, u.bound - u.p0))
        return make_uint4(~0u, ~0u, ~0u, ~0u);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int g, n;
        const bool in = a.qt.at(t, 32 * i + (int)(threadIdx.x & 31), g, n);
        w[i] = __ballot_sync(kFullMask, in && u.p0 + n >= 0 && u.p0 + n < u.bound);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Which keys of a streamed tile are attended; K's other rows, which are read across
// with weights of 0, cleared.  Of streamed queries, the rows behind the tile's last,
// which hold what was there before or the next group's.  false: a wait gave up.
template <bool KEYS, bool BAND>
__device__ __forceinline__ bool prepare(const BwdMmaArgs<BAND> &a, Shared<BAND> &sh, const Tiles &tl, const Unit<BAND> &u, int &it) {
    volatile int *abort = &sh.abort;
    for (int j = 0; j < u.n; ++j, ++it) {
        const int s = it % kStages;
        uint4 w = make_uint4(0, 0, 0, 0);
        int rows = kTileRows;
        if constexpr (BAND) w = KEYS ? tile_queries(a, u, u.lo + j) : band_keys(u.walk.band(a.band, u.lo + j), u.first, u.last, u.key(j));
        else if (!KEYS) w = tile_keys(a.ks, u.b, u.key(j), u.bound);
        else rows = min(a.qt.gb, a.qt.G - a.qt.first_head(u.lo + j)) * a.qt.nb;
        if (!pipe_wait(&sh.full[s], (it / kStages) & 1, abort)) return false;
        if (BAND && KEYS) {
            if (!all_keys(w)) {     // queries outside their sequence: a weight of 0 meets no NaN
                clear_rows(tl.stage(s), w);
                clear_rows(tl.stage(s) + kTileBytes, w);
                fence_smem_async();
                __syncwarp();
            }
        } else if (KEYS) {
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
template <bool KEYS, bool BAND>
__device__ __forceinline__ void scores(const BwdMmaArgs<BAND> &a, Shared<BAND> &sh, const Tiles &tl, const Unit<BAND> &u, int &it, int &units,
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
template <bool KEYS, bool BAND>
__device__ __forceinline__ void sums(const BwdMmaArgs<BAND> &a, Shared<BAND> &sh, const Tiles &tl, const Unit<BAND> &u, int &it, Turn &at) {
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
template <bool KEYS, bool BAND>
__device__ __forceinline__ void join(const BwdMmaArgs<BAND> &a, const Tiles &tl, const Unit<BAND> &u) {
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

template <bool BAND>
__global__ void __launch_bounds__(kThreads, 1) cross_bwd_mma_kernel(const __grid_constant__ BwdMmaArgs<BAND> a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    __shared__ Shared<BAND> sh;
    const Tiles tl(smem);
    const int warp = warp_number(), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.held[i], 1);
            mbar_init(&sh.held_free[i], 1);
            mbar_init(&sh.out[i], kWeightWarps);
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
        Unit<BAND> u = next();
#pragma unroll 1
        for (; u.index < a.first_kind; u = next()) {
            if constexpr (BAND) keys(u);
            else queries(u);
        }
#pragma unroll 1
        for (; u.index < a.units; u = next()) {
            if constexpr (BAND) queries(u);
            else keys(u);
        }
    };
    int passed = 0;         // units handed over
    const auto take = [&] {
        const int i = passed & 1;
        Unit<BAND> u;
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
        float2 stats = make_float2(kInf, 0.f);       // BAND: of the next unit's rows
        const auto ahead = [&] {
            if constexpr (BAND) {
                if (pipe_wait(&sh.unit_full[passed & 1], (passed >> 1) & 1, &sh.abort)) stats = row_stats(a, sh.unit[passed & 1]);
                __syncwarp();
            }
        };
        ahead();
        const auto over = [&] {
            if constexpr (BAND) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.out[(passed - 1) & 1]);
            }
        };
        each(take,
             [&](const Unit<BAND> &u) {
                 it = weights<false, BAND>(a, sh, tl, u, it, stats, ahead);
                 over();
             },
             [&](const Unit<BAND> &u) {
                 it = weights<true, BAND>(a, sh, tl, u, it, stats, ahead);
                 over();
             });
    } else {
        give_registers<kRegsFew>();
        if (warp == kCopyWarp) {
            bool ok = true;
            int drawn = first;
            // BAND: a unit of queries outside their sequence alone, whose dQ is cleared already
            const auto outside = [&](const Unit<BAND> &u) {
                if constexpr (BAND) return a.cleared && CS == 1 && u.n == 0 && u.index >= a.first_kind && u.index < a.units;
                else return false;
            };
            const auto pass = [&] {      // (its copies being out, the next unit's number has come meanwhile)
                const int i = passed & 1;
                Unit<BAND> u;
                do {
                    u.enter(a, __shfl_sync(kFullMask, drawn, 0));
                    drawn = a.units;
                    if (CS == 1 && lane == 0 && u.index < a.units) drawn = a.first_unit + (int)gridDim.x + atomicAdd(a.next_unit, 1);
                } while (outside(u));
                ok = ok && (passed < 2 || pipe_wait(&sh.unit_empty[i], ((passed >> 1) - 1) & 1, &sh.abort));
                if constexpr (BAND) {      // (the unit before last is over by now, or nearly)
                    ok = ok && (passed < 2 || pipe_wait(&sh.out[i], ((passed >> 1) - 1) & 1, &sh.abort));
                    if (ok && passed >= 2 && lane == 0) send(a, tl, sh.unit[i]);
                    const bool rows = u.index < a.first_kind ? u.chunk < 0 : a.qt.nb == kTileRows;
                    u.leaves = u.index < a.units && u.n > 0 && CS == 1 && rows ? units & 1 : -1;
                }
                if (!ok) u.index = a.units;
                else if (lane == 0) {
                    sh.unit[i] = u;
                    mbar_arrive(&sh.unit_full[i]);
                }
                __syncwarp();
                ++passed;
                return u;
            };
            each(pass, [&](const Unit<BAND> &u) { ok = ok && copies<false, BAND>(a, sh, tl, u, it, units); },
                 [&](const Unit<BAND> &u) { ok = ok && copies<true, BAND>(a, sh, tl, u, it, units); });
            if constexpr (BAND) {      // the last units' gradients
                for (int i = max(0, passed - 2); ok && i < passed - 1; ++i) {      // (the last one passed is the end)
                    ok = pipe_wait(&sh.out[i & 1], (i >> 1) & 1, &sh.abort);
                    if (ok && lane == 0) send(a, tl, sh.unit[i & 1]);
                }
                if (lane == 0) stores_done();
                __syncwarp();
            }
            if (lane == 0) {   // leave no copy in flight
                for (int i = max(0, units - 2); i < units; ++i) mbar_drain(&sh.held[i & 1], (i >> 1) & 1);
                for (int i = max(0, it - kStages); i < it; ++i) mbar_drain(&sh.full[i % kStages], (i / kStages) & 1);
            }
        } else if (warp == kPrepWarp) {
            bool ok = true;
            each(take, [&](const Unit<BAND> &u) { ok = ok && prepare<false, BAND>(a, sh, tl, u, it); },
                 [&](const Unit<BAND> &u) { ok = ok && prepare<true, BAND>(a, sh, tl, u, it); });
        } else {
            Turn at;
            if (warp == kScoreWarp)
                each(take, [&](const Unit<BAND> &u) { scores<false, BAND>(a, sh, tl, u, it, units, at); },
                     [&](const Unit<BAND> &u) { scores<true, BAND>(a, sh, tl, u, it, units, at); });
            else
                each(take, [&](const Unit<BAND> &u) { sums<false, BAND>(a, sh, tl, u, it, at); }, [&](const Unit<BAND> &u) { sums<true, BAND>(a, sh, tl, u, it, at); });
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
    Unit<BAND> u;
    u.enter(a, first);
    if (first < a.first_kind) join<BAND, BAND>(a, tl, u);
    else join<!BAND, BAND>(a, tl, u);
    cluster_sync();   // the others may still read this CTA's part
}

// dK and dV of the key tiles whose walks were cut: the parts' sums, in their order.  A thread
// adds the four values that thread t of the weight warps left at i.
__global__ void __launch_bounds__(256)
window_sum_kernel(const __grid_constant__ BwdMmaArgs<true> a) {
    grid_dep_wait();
    grid_dep_launch();
    const int tile = blockIdx.x / (kPartSums / 256), e = blockIdx.x % (kPartSums / 256) * 256 + threadIdx.x;
    const int i = e / (32 * kWeightWarps), t = e % (32 * kWeightWarps), warp = t >> 5, acc = warp >> 3;
    const int hk = tile % a.Hkv, b = tile / a.Hkv % a.B, k = tile / a.Hkv / a.B * kTileRows + (warp & 3) * 32 + (t & 31);
    if (k >= a.ks.Nk) return;
    const float4 *from = a.parts + (int64_t)tile * a.chunks * kPartSums + e;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int c = 0; c < a.chunks; ++c) {
        const float4 y = __ldg(from + (int64_t)c * kPartSums);
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
    }
    const float f = acc ? 1.f : a.scale;
    *reinterpret_cast<uint2 *>((acc ? a.dV : a.dK).row(b, hk, k) + 32 * ((warp >> 2) & 1) + 4 * i) =
        make_uint2(pack_bf16x2(x.x * f, x.y * f), pack_bf16x2(x.z * f, x.w * f));
}

// Rows of a head with the last of its query tiles whole.
int padded_rows(int Nq) { return Nq < kTileRows ? Nq : (Nq + kTileRows - 1) / kTileRows * kTileRows; }

}  // namespace

namespace {

// How the walks of key tiles with sinks are cut: into parts as long as the other tiles' walks, or as half of
// what an SM has in all where that is more (they come first, so that the rest evens them out), as
// long as there are no more than kParts of them in all (two a SM, each with 64 KB of partial sums; a number of its
// own, so that the workspace that a call asks for and the one it uses agree whatever device is current).  (One
// sequence of 16385 tokens, 16 heads on 4, window 1024, 4 sinks: walks of 516 tiles next to others of
// 36; in one part 673 us, in parts of 36 266, as here 261; window 128: 151 and 129; eight sequences of
// 1569, 12 heads on 4, window 512, in one part here: 107 and 101.6.)
struct SinkParts {
    static constexpr int64_t kParts = 304;
    int64_t tiles = 0, chunks = 1, length = 0;       // key tiles of a head; parts of each, query tiles of a part
    SinkParts(int B, int Hkv, int Nk, const Band &w, const BandTiles &qt) {
        const int64_t ktiles = (Nk + kTileRows - 1) / kTileRows;
        tiles = std::min<int64_t>((w.sinks + kTileRows - 1) / kTileRows, ktiles);
        if (tiles == 0) return;
        const int64_t other = ((int64_t)(w.window + kTileRows) / qt.nb + 1) * qt.groups, heads = (int64_t)B * Hkv * tiles;
        // tiles that all walks have, of keys that the windows meet and of queries
        const int64_t met = std::min<int64_t>(ktiles, ((int64_t)qt.Nq + w.window) / kTileRows + 1);
        const int64_t all = (int64_t)B * Hkv * (met * std::min<int64_t>(other, qt.tiles) +
                                                qt.tiles * std::min<int64_t>(ktiles, w.window / kTileRows + 2));
        length = std::max({other, all / kParts, (heads * qt.tiles + kParts - 1) / kParts, (qt.tiles + 255) / (int64_t)256});
        chunks = (qt.tiles + length - 1) / length;
    }
    size_t bytes(int B, int Hkv) const {
        return chunks > 1 ? (size_t)B * Hkv * tiles * chunks * kPartSums * sizeof(float4) : 0;
    }
};

size_t round_16(size_t x) { return (x + 15) / 16 * 16; }

}  // namespace

size_t cross_bwd_mma_workspace(int B, int Hq, int Nq) {
    const size_t rows = (size_t)B * Hq * padded_rows(Nq);
    return 2 * (rows + kTileRows) * sizeof(uint4) + (size_t)B * Hq * Nq * sizeof(float2) + 2 * sizeof(int);
}

size_t window_bwd_mma_workspace(int B, int Hq, int Hkv, int Nq, int Nk, int window, int sinks) {
    // (heads with rows of their own or broadcast ones, whose tiles are others)
    const Band w{nullptr, Nq, Nk, window, sinks};
    size_t most = 0;
    for (const bool shared : {false, true}) most = std::max(most, SinkParts(B, Hkv, Nk, w, BandTiles(Hq / Hkv, Nq, shared)).bytes(B, Hkv));
    return round_16(cross_bwd_mma_workspace(B, Hq, Nq)) + most;
}

namespace {

template <bool BAND>
cudaError_t bwd(const CrossArgs &a) {
    BwdMmaArgs<BAND> f;
    f.qt = TilesOf<BAND>(a.Hq / a.Hkv, a.Nq, a.Hq > 1 && (a.Q.stride_h == 0 || a.dO.stride_h == 0));
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
    if constexpr (BAND) {
        f.band = a.band;
        f.chunks = 1, f.chunk_tiles = f.sink_tiles = f.sink_units = f.cleared = 0;
        f.parts = nullptr;
        if ((f.qt.nb == kTileRows && !make_tensor(&f.dq, a.dQ, a.B, a.Hq, a.Nq, kTileRows, 1)) ||
            !make_tensor(&f.dk, a.dK, a.B, a.Hkv, a.Nk, kTileRows, 1) || !make_tensor(&f.dv, a.dV, a.B, a.Hkv, a.Nk, kTileRows, 1))
            return cudaErrorInvalidValue;
        f.by_heads = Div((uint32_t)(a.B * a.Hkv)), f.by_hkv = Div((uint32_t)a.Hkv);
        const SinkParts p(a.B, a.Hkv, a.Nk, a.band, f.qt);
        if (p.chunks > 1) {
            f.chunks = (int)p.chunks;
            f.chunk_tiles = (int)p.length;
            f.sink_tiles = (int)p.tiles;
            f.sink_units = (int)((int64_t)a.B * a.Hkv * p.tiles * p.chunks);
            f.by_sinks = Div((uint32_t)(a.B * a.Hkv * (int)p.tiles));
            f.parts = reinterpret_cast<float4 *>(reinterpret_cast<char *>(a.stats) +
                                                 round_16(cross_bwd_mma_workspace(a.B, a.Hq, a.Nq)));
        }
    }
    f.dQ = rows_of<__nv_bfloat16>(a.dQ), f.dK = rows_of<__nv_bfloat16>(a.dK), f.dV = rows_of<__nv_bfloat16>(a.dV);
    f.B = a.B, f.Hq = a.Hq, f.Hkv = a.Hkv;
    f.ktiles = (a.Nk + kTileRows - 1) / kTileRows;
    f.scale = a.scale;
    // a scale of 0: any c this small leaves every finite score's weight at exp2(-LSE log2 e)
    f.c = std::copysign(std::max(std::fabs(a.scale) * kLog2e, 1e-36f), a.scale);
    cudaError_t e = prepare_kernel<cross_bwd_mma_kernel<BAND>>(kSmem, kRegs);
    if (e != cudaSuccess) return e;
    if (a.Nk <= kFewKeys || (BAND && (int64_t)a.band.window + a.band.sinks <= kFewKeys)) {
        const int64_t warps = (int64_t)a.B * a.Hq * ((f.npad + 15) / 16) + kTileRows / 16;
        e = launch_clusters(cross_parts_few_kernel<BAND>, (unsigned)((warps + kFewWarps - 1) / kFewWarps), 1, 32 * kFewWarps, 0,
                            a.stream, a.Hq, a.Hkv, a.Nq, f.npad, (unsigned)(a.B * a.Hq), a.keys, a.band,
                            rows_of<const __nv_bfloat16>(a.Q), rows_of<const __nv_bfloat16>(a.K),
                            rows_of<const __nv_bfloat16>(a.V), rows_of<const __nv_bfloat16>(a.dO),
                            static_cast<const float *>(a.LSE), f.c, stats, lse_parts, d_parts, f.next_unit);
    } else if (BAND && f.npad >= kPartRows) {
        const unsigned heads = (unsigned)(a.B * a.Hq), steps = (unsigned)((f.npad + kPartRows - 1) / kPartRows);
        e = launch_clusters(window_parts_kernel, heads * steps + kTileRows / kPartRows, 1, 4 * kPartRows, 0, a.stream, a.Hq, a.Nq,
                            f.npad, heads, a.keys, a.band, rows_of<const __nv_bfloat16>(a.O),
                            rows_of<const __nv_bfloat16>(a.dO), static_cast<const float *>(a.LSE), f.c, stats, lse_parts,
                            d_parts, f.next_unit, f.dQ);
        if constexpr (BAND) f.cleared = 1;
    } else {
        const auto kernel = !BAND && a.keys.len ? cross_parts_kernel<true> : cross_parts_kernel<false>;
        e = launch_clusters(kernel, (unsigned)((rows + kTileRows + 31) / 32), 1, 256, 0, a.stream, a.Hq, a.Hkv, a.Nq, f.npad,
                            (unsigned)rows, a.keys, rows_of<const __nv_bfloat16>(a.Q), rows_of<const __nv_bfloat16>(a.K),
                            rows_of<const __nv_bfloat16>(a.V), rows_of<const __nv_bfloat16>(a.O),
                            rows_of<const __nv_bfloat16>(a.dO), static_cast<const float *>(a.LSE), f.c, stats, lse_parts,
                            d_parts, f.next_unit);
    }
    if (e != cudaSuccess) return e;
    const int64_t query_units = (int64_t)a.B * a.Hkv * f.qt.tiles;
    int64_t key_units = (int64_t)a.B * a.Hkv * f.ktiles;
    if constexpr (BAND) key_units += f.sink_units - (int64_t)a.B * a.Hkv * f.sink_tiles;
    f.first_kind = (int)(BAND ? key_units : query_units);
    // clusters, one unit each, while they all find a place; else one wave of CTAs that walk over the units
    const auto launch = [&](int64_t from, int64_t units, int c) {
        f.first_unit = (int)from;
        f.units = (int)(from + units);
        const int64_t grid = c > 1 ? units * c : std::min<int64_t>(units, sm_count());
        return launch_clusters(cross_bwd_mma_kernel<BAND>, (unsigned)grid, c, kThreads, kSmem, a.stream, f);
    };
    // (one head, 100 queries on 16385 keys: 27 us in two launches, 82 in one; 16 heads, 100 on 5000:
    // 44 and 36)
    int64_t query_walk = f.ktiles, key_walk = f.qt.tiles;
    if constexpr (BAND) {      // tiles that hold the windows of a tile's rows, and the sinks
        query_walk = std::min<int64_t>(query_walk, ((int64_t)a.band.window + f.qt.nb) / kTileRows + 1 + (a.band.sinks + kTileRows - 1) / kTileRows);
        if (a.band.sinks == 0 || f.chunks > 1) key_walk = std::min<int64_t>(key_walk, (((int64_t)a.band.window + kTileRows) / f.qt.nb + 2) * f.qt.groups);
    }
    const Launches l(query_units, query_walk, key_units, key_walk, sm_count(), 5, 12);
    if constexpr (BAND) {
        if (f.chunks > 1) {      // (no clusters: there are units enough)
            e = launch(0, query_units + key_units, 1);
            if (e != cudaSuccess) return e;
            const unsigned blocks = (unsigned)(a.B * a.Hkv * f.sink_tiles * (kPartSums / 256));
            return launch_clusters(window_sum_kernel, blocks, 1, 256, 0, a.stream, f);
        }
    }
    if (!l.two) return launch(0, query_units + key_units, l.c);
    e = BAND ? launch(0, key_units, l.c_key) : launch(0, query_units, l.c_query);
    if (e != cudaSuccess) return e;
    ++f.next_unit;
    return BAND ? launch(key_units, query_units, l.c_query) : launch(query_units, key_units, l.c_key);
}

}  // namespace

cudaError_t launch_cross_bwd_mma(const CrossArgs &a) { return a.banded ? bwd<true>(a) : bwd<false>(a); }

FIBATT_DEFINE_ERROR_READER(read_error_cross_mma_bwd, "cross_mma_bwd.cu")

}  // namespace fibatt
