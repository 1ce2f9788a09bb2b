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
//
// Attention over a window with sinks (BAND): a query tile's walk is over the tiles from the
// oldest key that its queries attend to the newest, and over those of the sinks, so that 128 queries
// with a window of w cost about (w + 127) / 128 rounded up, and one; only the tiles at the
// window's two ends and the sinks' are masked, from the positions, without memory.  Such walks are short
// (2 to 9 tiles), and what a unit costs besides, about 1.8 us of a SM's time, decides.  Hence:
//   one tile of queries a CTA, two CTAs a SM, each of which goes on with the unit of a CTA that has not
//     started, struck off by the hardware (the third shape below 44 -> 35 us, the second 98 -> 78)
//   the next unit's queries are copied to a second place while this one's are in use, and O leaves from
//     its queries' place by a tensor copy that nobody waits for (the third 49 -> 44)
//   walks start at the oldest key, not at a multiple of 128 (the third 34 -> 32)
//   tiles of neighbouring positions and of heads that share keys are neighbours in the grid: L2 serves 81% of the reads
//   few sinks in front of the window's first tile, and 32 columns left out, where that pays (below)
// Measured (4 sinks): 16 heads on 4 key heads, 16385 tokens, window 1024: 95.1 us, 703 TFLOP/s of
// the pairs attended (36% and 37% of the time tensor cores and exponentials work, issue slots 63% taken); 2 times 1569
// queries on 16385 keys, window 4096: 75.2, 701; 8 sequences, 12 heads on 4, up to 1569 tokens, window
// 512: 30.2, 358 (units of 5 or 6 tiles, two or three of them masked); 64 sequences, 12 heads, up
// to 197 tokens, window 64, 1 sink: 23.2, 2.7 TB/s.
#include <algorithm>

#include "cluster.cuh"
#include "cross_tiles.cuh"

namespace fibatt {
namespace {

constexpr float kNegInf = -__builtin_inff();
constexpr float kRaise = 8.f;    // log2 units
constexpr int kJoinLd = 68;      // floats between rows of a partial O in shared memory

template <int NT, bool BAND>
struct Cfg {
    static_assert(NT == 1 || !BAND, "two tiles of a window's queries are two CTAs");
    static constexpr int kSoftmaxWarps = 8 * NT;
    static constexpr int kCopyWarp = kSoftmaxWarps, kKeysWarp = kSoftmaxWarps + 1;
    static constexpr int kScoreWarp = kSoftmaxWarps + 2, kValueWarp = kSoftmaxWarps + 3;
    static constexpr int kThreads = 32 * (kSoftmaxWarps + 4);   // whole warp groups
    static constexpr int kQueries = BAND ? 2 : 1;      // units whose queries are held
    static constexpr int kStages = NT == 2 ? 5 : 2;
    static constexpr uint32_t kCols = NT * 256;        // S 128, P 64, O 64 a tile
    static constexpr size_t kSmem = 1024 + kQueries * NT * kTileBytes + kStages * 2 * kTileBytes;
    static constexpr int kMinBlocks = NT == 2 ? 1 : 2;
    static constexpr bool kWalks = NT == 1;            // one wave of CTAs for all units
    // registers a thread: at launch, and after the softmax warps took what the others gave
    static constexpr int kRegs = NT == 2 ? 96 : 80, kRegsFew = 32, kRegsMany = NT == 2 ? 112 : 104;
    static_assert(2 * NT * kRegsMany + kRegsFew == (2 * NT + 1) * kRegs, "the shares add up");
    static_assert(NT * kTileRows * kJoinLd * 4 <= NT * kTileBytes + kStages * 2 * kTileBytes, "partial O fits");
};

// What only a window's calls have.  (Other launches do not carry it: the tensor maps alone are 0.6 KB.)
template <bool BAND>
struct FwdBandArgs {};
template <>
struct FwdBandArgs<true> {
    Band band;
    Div by_heads, by_hkv;    // heads of keys of all sequences, of one
    TensorArg o;             // tiles of one head: O as tensor copies write it
    // few sinks lie in front of the windows' first tile, in `front` rows of it (0: in tiles of their
    // own); boxes of those and of the other rows
    int front;
    TensorArg kv_front[2], kv_rest[2];
};

template <bool BAND>
struct FwdMmaArgs : FwdBandArgs<BAND> {
    TensorArg q, k, v;
    TilesOf<BAND> qt;
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
template <int NT, bool BAND>
struct Place {
    int t0, nt, hk, b;
    __device__ __forceinline__ Place() {}
    __device__ __forceinline__ Place(const FwdMmaArgs<BAND> &a, int unit) {
        if constexpr (BAND) {      // the last queries, which attend the most keys, first
            const int step = a.by_heads.of(unit), head = unit - step * (int)a.by_heads.d;
            t0 = (a.pairs - 1 - step) * NT;
            b = a.by_hkv.of(head);
            hk = head - b * a.Hkv;
        } else {
            t0 = unit % a.pairs * NT;
            hk = unit / a.pairs % a.Hkv;
            b = unit / a.pairs / a.Hkv;
        }
        nt = min(NT, a.qt.tiles - t0);      // tiles of this unit
    }
};
// ... and the part of its sequence's key tiles that this CTA of the cluster walks
// over.  CTAs that walk over their units have them from the copying warp.
template <int NT, bool BAND>
struct Unit : Place<NT, BAND> {
    int bound, lo, n;
    __device__ __forceinline__ Unit() {}
    __device__ __forceinline__ Unit(const FwdMmaArgs<BAND> &a, const Place<NT, BAND> &p) : Place<NT, BAND>(p) { set(a); }
    __device__ __forceinline__ void set(const FwdMmaArgs<BAND> &a) {
        bound = a.ks.bound(this->b);
        const int ktiles = (bound + kTileRows - 1) / kTileRows, CS = (int)cluster_size(), rank = (int)cluster_rank();
        lo = (int)((int64_t)ktiles * rank / CS);
        n = (int)((int64_t)ktiles * (rank + 1) / CS) - lo;
    }
    // first key of its tile j
    __device__ __forceinline__ int key(int j) const { return (lo + j) * kTileRows; }
};
template <int NT>
struct Unit<NT, true> : Place<NT, true> {
    int bound, lo, n;
    int row, head;                  // of the tile's first query
    int p0, first, last;            // position of that query; of the first and the last of the tile's that attend keys
    int front;                      // rows of the walk's first tile that are the sinks'
    KeyWalk<kTileRows> walk;
    __device__ __forceinline__ Unit() {}
    __device__ __forceinline__ Unit(const FwdMmaArgs<true> &a, const Place<NT, true> &p) : Place<NT, true>(p) { set(a); }
    __device__ __forceinline__ void set(const FwdMmaArgs<true> &a) {
        bound = a.ks.bound(this->b);
        row = a.qt.first_row(this->t0);
        head = this->hk * a.qt.G + a.qt.first_head(this->t0);
        p0 = a.band.first(this->b) + row;
        first = max(0, p0);
        last = min(bound, p0 + min(a.qt.Nq - row, a.qt.nb)) - 1;
        walk = KeyWalk<kTileRows>(a.band, first, last);
        front = 0;
        if (a.front && walk.n > 0) {
            const int from = max(0, first - a.band.window + 1) - a.front, n = (last - from) / kTileRows + 1;
            if (from + a.front > a.band.sinks && n < walk.n) {
                front = a.front;
                walk.sinks = 0, walk.oldest = from, walk.n = n;
            }
        }
        const int CS = (int)cluster_size(), rank = (int)cluster_rank();
        lo = 0, n = walk.n;
        if (CS > 1) {
            lo = (int)((int64_t)walk.n * rank / CS);
            n = (int)((int64_t)walk.n * (rank + 1) / CS) - lo;
        }
    }
    __device__ __forceinline__ int key(int j) const { return walk.key(lo + j); }
    __device__ __forceinline__ Band band(const FwdMmaArgs<true> &a, int j) const { return walk.band(a.band, lo + j); }
    // tile j's first rows are the sinks'
    __device__ __forceinline__ bool fronted(int j) const { return front && lo + j == 0; }
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

// FRONT: sinks lie in front of the windows' first tiles.  NARROW: windows of which many tiles' 32 columns have no key.
template <int NT, bool BAND, bool FRONT = false, bool NARROW = false>
__global__ void __launch_bounds__(Cfg<NT, BAND>::kThreads, Cfg<NT, BAND>::kMinBlocks)
cross_fwd_mma_kernel(const __grid_constant__ FwdMmaArgs<BAND> a) {
    using C = Cfg<NT, BAND>;
    using Work = Unit<NT, BAND>;
    using Where = Place<NT, BAND>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *sq = smem, *skv = smem + C::kQueries * NT * kTileBytes;   // stage s: K at skv + 2 s tiles, V behind it
    __shared__ uint64_t bar_q[C::kQueries], bar_qfree[C::kQueries], bar_full[C::kStages], bar_ready[C::kStages], bar_empty[C::kStages];
    __shared__ uint64_t bar_s[NT], bar_sfree[NT], bar_p[NT], bar_o[NT], bar_end[2];
    __shared__ uint64_t bar_unit[2], bar_unitfree[2];
    __shared__ __align__(16) uint4 drawn[2];    // BAND: the hardware's answers, in turn
    __shared__ uint64_t bar_drawn[2];
    __shared__ Work units[2];       // of a CTA that walks, in turn; n < 0: no more
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
    const Where first_place(a, first);

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kQueries; ++i) {
            mbar_init(&bar_q[i], 1);
            mbar_init(&bar_qfree[i], BAND ? 2 : 1);
        }
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
            mbar_init(&bar_drawn[i], 1);
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
            body(Work(a, first_place));
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
        // BAND: the unit's O leaves by a tensor copy from where its queries were.  `loaded` counts units with queries;
        // one thread stores, and hands the place on when it has been read.
        int loaded = 0, held = -1;
        const auto hand_on = [&] {
            if (held < 0) return;
            stores_read();
            mbar_arrive(&bar_qfree[held]);
            held = -1;
        };
        each([&](const Work &u) {
            if (t >= u.nt) {
                skipped += u.n;
                return;
            }
            const int n = u.n, whole = a.ks.mask ? 0 : u.bound / kTileRows - u.lo;   // the tiles attended wholly come first
            int p = -1, highest = 0;                 // positions: of the row, of the tile's last
            if constexpr (BAND) {
                highest = u.p0 + min(a.qt.Nq - u.row, a.qt.nb) - 1;
                p = u.p0 + (a.qt.gb == 1 ? r : a.qt.by_rows.rest(r));
                if (p > highest || p >= u.bound) p = -1;
            }
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
                bool live[2] = {true, true};        // NARROW: whether the warp's rows attend any of 32 columns
                if constexpr (BAND) {
                    const Band w = u.band(a, j);
                    const int k0 = u.key(j), k1 = k0 + kTileRows - 1;
                    const bool all = k1 <= u.p0 && highest < u.bound && (k0 > highest - w.window || k1 < w.sinks);
                    if (!all) {       // (nor is a fronted one)
                        uint32_t words[2] = {keys_of(w, p, k0 + 64 * half), keys_of(w, p, k0 + 64 * half + 32)};
                        if constexpr (FRONT)
                            if (half == 0 && u.fronted(j)) words[0] = (words[0] & ~bits_below(u.front)) | (p < 0 ? 0u : bits_below(w.sinks));
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if (NARROW) live[i] = __any_sync(kFullMask, words[i] != 0u);
                            if (NARROW && !live[i]) continue;
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!((words[i] >> k) & 1)) s[i][k] = __float_as_uint(kNegInf);
                        }
                    }
                } else if (j >= whole) {
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
                float top[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (NARROW && !live[i >> 1]) continue;
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
                for (int i = 0; i < 2; ++i) {
                    if (NARROW && !live[i]) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) p[16 * i + k] = 0u;
                        continue;
                    }
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float2 x = fma2(make_float2(__uint_as_float(s[i][2 * k]), __uint_as_float(s[i][2 * k + 1])),
                                              make_float2(a.c, a.c), make_float2(base, base));
                        const float2 y = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                        sum[k & 1] = add2(sum[k & 1], y);
                        p[16 * i + k] = pack_bf16x2(y.x, y.y);
                    }
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
                if (BAND && j == 0) {
                    hand_on();
                    __syncwarp();
                }
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
            if constexpr (BAND) if (n > 0 && CS == 1) {
                const int place = loaded++ % C::kQueries;
                if (a.qt.gb == 1) {
                    uint8_t *tile = sq + place * kTileBytes;
                    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * k]) * inv, __uint_as_float(o[8 * i + 2 * k + 1]) * inv);
                        *reinterpret_cast<uint4 *>(tile + r * 128 + (((4 * half + i) ^ (r & 7)) << 4)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    fence_smem_async();
                    named_sync(2, 32 * C::kSoftmaxWarps);
                    const int q = u.row, h = u.head;
                    if (threadIdx.x == 0 && FIBATT_CHECKED(h < a.Hq && u.b >= 0 && q < a.qt.Nq)) {
                        tile_store(&a.o.map, q, h * a.o.head_step, u.b * a.o.seq_step, tile);
                        held = place;
                    }
                    if (half == 0 && r < a.qt.nb && q + r < a.qt.Nq)
                        a.LSE[((int64_t)u.b * a.Hq + h) * a.qt.Nq + q + r] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
                    return;
                }
                if (threadIdx.x == 0) mbar_arrive(&bar_qfree[place]);
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
        if (BAND && held >= 0) stores_done();
    } else {
        give_registers<C::kRegsFew>();
        if (warp == C::kCopyWarp) {
            // ---- copies: they run ahead into the next unit ------------------------------
            int ring = 0, loaded = 0;      // issued: key tiles, units' queries
            bool ok = true;
            const auto queries = [&](const Work &u) {
                uint64_t *bar = &bar_q[loaded % C::kQueries];
                uint8_t *dst = sq + loaded % C::kQueries * NT * kTileBytes;
                if (elect_one()) {
                    mbar_expect_tx(bar, u.nt * a.qt.bytes());
                    if constexpr (BAND)
                        load_tile(dst, a.q, u.row, u.head, u.b, bar);
                    else
                        for (int t = 0; t < u.nt; ++t)
                            load_tile(dst + t * kTileBytes, a.q, a.qt.first_row(u.t0 + t),
                                      u.hk * a.qt.G + a.qt.first_head(u.t0 + t), u.b, bar);
                }
                __syncwarp();
                ++loaded;
            };
            // BAND: the next unit is that of a CTA that has not started, which the hardware strikes off for us.  It
            // is asked for ahead of the last copies of this one.
            int asked = 0;
            const auto ask = [&] {
                if (lane == 0) {
                    fence_smem_async();
                    draw_cta(&drawn[asked & 1], &bar_drawn[asked & 1]);
                }
                ++asked;
                __syncwarp();
            };
            const auto copies = [&](const Work &u) {
                // (with one place for queries: behind the first keys, once the scores have read the last queries)
                const bool later = C::kWalks && !BAND && loaded > 0;
                if (BAND && u.n > 0 && loaded >= C::kQueries)
                    ok = pipe_wait(&bar_qfree[loaded % C::kQueries], (loaded / C::kQueries - 1) & 1, abort);
                if (BAND && CS == 1 && u.n <= 1) ask();
                for (int j = 0; ok && j < u.n; ++j) {
                    if (j == 0 && !later) queries(u);
                    if (BAND && CS == 1 && u.n > 1 && j == u.n - 1) ask();
                    const int s = ring % C::kStages;
                    ok = ring < C::kStages || pipe_wait(&bar_empty[s], (ring / C::kStages - 1) & 1, abort);
                    if (!ok) break;
                    if (elect_one()) {
                        mbar_expect_tx(&bar_full[s], 2 * kTileBytes);
                        bool whole = true;
                        if constexpr (FRONT) whole = !u.fronted(j);
                        if (whole) {
                            load_tile(skv + (2 * s) * kTileBytes, a.k, u.key(j), u.hk, u.b, &bar_full[s]);
                            load_tile(skv + (2 * s + 1) * kTileBytes, a.v, u.key(j), u.hk, u.b, &bar_full[s]);
                        } else if constexpr (FRONT) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                uint8_t *dst = skv + (2 * s + i) * kTileBytes;
                                load_tile(dst, a.kv_front[i], 0, u.hk, u.b, &bar_full[s]);
                                load_tile(dst + u.front * 128, a.kv_rest[i], u.key(j) + u.front, u.hk, u.b, &bar_full[s]);
                            }
                        }
                    }
                    __syncwarp();
                    ++ring;
                    if (j == 0 && later) {
                        ok = pipe_wait(&bar_qfree[0], (loaded - 1) & 1, abort);
                        if (ok) queries(u);
                    }
                }
            };
            if constexpr (C::kWalks) {
#pragma unroll 1
                for (int k = 0, unit = first; ok; ++k, unit += step) {
                    Work u;
                    if (BAND && k > 0) {
                        unit = a.units;
                        if (CS == 1) {
                            ok = pipe_wait(&bar_drawn[(k - 1) & 1], ((k - 1) >> 1) & 1, abort);
                            if (!ok) break;
                            const int next = drawn_cta(&drawn[(k - 1) & 1]);
                            if (next >= 0) unit = next;
                        }
                    }
                    if (unit < a.units) u = Work(a, k ? Where(a, unit) : first_place);
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
                copies(Work(a, first_place));
            }
            // leave no copy in flight
            if (lane == 0) {
                for (int i = max(0, asked - 2); i < asked; ++i) mbar_drain(&bar_drawn[i & 1], (i >> 1) & 1);
                for (int i = max(0, loaded - C::kQueries); i < loaded; ++i)
                    mbar_drain(&bar_q[i % C::kQueries], (i / C::kQueries) & 1);
                for (int i = max(0, ring - C::kStages); i < ring; ++i)
                    mbar_drain(&bar_full[i % C::kStages], (i / C::kStages) & 1);
            }
        } else if (warp == C::kKeysWarp) {
            // ---- which keys of each tile are attended; the others' value rows cleared ----
            int ring = 0;
            bool ok = true;
            each([&](const Work &u) {
                const int n = u.n;
                for (int j = 0; ok && j < n; ++j, ++ring) {
                    const int s = ring % C::kStages;
                    uint4 w;
                    if constexpr (BAND) {
                        w = band_keys(u.band(a, j), u.first, u.last, u.key(j));
                        if (FRONT && u.fronted(j)) w.x = (w.x & ~bits_below(u.front)) | bits_below(a.band.sinks);
                    } else w = tile_keys(a.ks, u.b, u.key(j), u.bound);
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
                each([&](const Work &u) {
                    const int n = __shfl_sync(kFullMask, u.n, 0), nt = __shfl_sync(kFullMask, u.nt, 0);
                    const int place = loaded % C::kQueries;
                    if (n > 0) pipe_wait(&bar_q[place], (loaded++ / C::kQueries) & 1, abort);
                    for (int j = 0; j < n; ++j) {
                        pipe_wait(&bar_full[s], pass, abort);      // masked keys' scores are not looked at
                        const uint64_t dks = dk + (uint64_t)(s * (2 * kTileBytes >> 4));
#pragma unroll
                        for (int t = 0; t < NT; ++t) {   // S_t = Q_t K_j^T
                            if (t >= nt) break;
                            if (it[t] > 0) pipe_wait(&bar_sfree[t], (it[t] - 1) & 1, abort);
                            ++it[t];
                            tc_after_sync();
                            const uint64_t dqt = dq + (uint64_t)((place * NT + t) * (kTileBytes >> 4));
                            if (elect_one()) {
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    mma_ss(col_s + t * 128, dqt + i * kStepRowwise, dks + i * kStepRowwise, id, i > 0);
                                mma_commit(&bar_s[t]);
                                if (j == n - 1 && t == nt - 1) mma_commit(&bar_qfree[place]);
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
                each([&](const Work &u) {
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
    const Work u(a, first_place);
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
template <int NT, bool BAND, bool FRONT, bool NARROW>
int held_clusters(int dev, int i) {
    using C = Cfg<NT, BAND>;
    static PerDevice known[5];
    return known[i].get(dev, [=] {
        return i == 0 ? C::kMinBlocks * sm_count()
                      : clusters_held<cross_fwd_mma_kernel<NT, BAND, FRONT, NARROW>>(1 << i, C::kThreads, C::kSmem);
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
template <int NT, bool BAND, bool FRONT = false, bool NARROW = false>
cudaError_t consider(const CrossArgs &a, const TilesOf<BAND> &qt, Plan *best) {
    using C = Cfg<NT, BAND>;
    const cudaError_t e = prepare_kernel<cross_fwd_mma_kernel<NT, BAND, FRONT, NARROW>>(C::kSmem, C::kRegs);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)a.B * a.Hkv * ((qt.tiles + NT - 1) / NT);
    int tiles = (a.Nk + kTileRows - 1) / kTileRows;
    const int dev = current_device();
    if constexpr (BAND)      // of the windows of a unit's rows, and of the sinks
        tiles = (int)std::min<int64_t>(tiles, ((int64_t)a.band.window + (NT / qt.groups + 1) * qt.nb) / kTileRows + 1 +
                                                  (a.band.sinks + kTileRows - 1) / kTileRows);
    for (int i = 0; i < 5 && (i == 0 || tiles >= 1 << i); ++i) {
        const int c = 1 << i, held = held_clusters<NT, BAND, FRONT, NARROW>(dev, i);
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

// Rows that few sinks take in front of a tile of keys, 0: none (in eights, after which the tiles'
// swizzle repeats).  Query tiles are as many rows shorter, so that their windows and the sinks
// fill whole tiles; taken where all of them then take less, by 1.5%, than with a tile for the sinks: counted
// in key tiles, of which a unit's start and end cost 3, over the windows' mean length (they
// grow up to the first `window` queries, which need no such tile).  (16 heads on 4, 16385 tokens, 4 sinks: window
// 128 45.5 -> 40.6 us, 512 68 -> 64, 1024 97.7 -> 94.4; 8 sequences, 12 heads on 4, window 512:
// 1680 tokens 40.2 -> 37.3, 1569 tokens, 14 units for 13, 37.0 -> 37.2: not taken.)
int front_rows(const CrossArgs &a) {
    const int front = (a.band.sinks + 7) / 8 * 8, rows = kTileRows - front;
    if (front == 0 || front > 32 || a.Nq < 2 * kTileRows) return 0;
    const double first = a.Nk - a.Nq, window = a.band.window, grow = std::min<double>(std::max(window - first, 0.), a.Nq);
    const double mean = (window - grow * grow / (2. * a.Nq)) / kTileRows, late = 1. - grow / a.Nq;
    const auto cost = [&](int rows, double tiles) { return (a.Nq + rows - 1) / rows * (mean + 1. + tiles + 3.); };
    return 1.015 * cost(rows, 0.) < cost(kTileRows, late) ? front : 0;
}

template <int NT, bool BAND, bool FRONT = false, bool NARROW = false>
cudaError_t fwd(const CrossArgs &a, const TilesOf<BAND> &qt, int c) {
    using C = Cfg<NT, BAND>;
    FwdMmaArgs<BAND> f;
    f.qt = qt;
    if (!make_tensor(&f.q, a.Q, a.B, a.Hq, a.Nq, qt.nb, qt.gb) || !make_tensor(&f.k, a.K, a.B, a.Hkv, a.Nk, kTileRows, 1) ||
        !make_tensor(&f.v, a.V, a.B, a.Hkv, a.Nk, kTileRows, 1))
        return cudaErrorInvalidValue;
    if constexpr (BAND) {
        f.band = a.band;
        f.by_heads = Div((uint32_t)(a.B * a.Hkv)), f.by_hkv = Div((uint32_t)a.Hkv);
        f.front = FRONT ? kTileRows - qt.nb : 0;
        if (qt.gb == 1 && !make_tensor(&f.o, a.O, a.B, a.Hq, a.Nq, qt.nb, 1)) return cudaErrorInvalidValue;
        const fibatt_heads *kv[2] = {&a.K, &a.V};
        for (int i = 0; f.front && i < 2; ++i)
            if (!make_tensor(&f.kv_front[i], *kv[i], a.B, a.Hkv, a.Nk, f.front, 1) ||
                !make_tensor(&f.kv_rest[i], *kv[i], a.B, a.Hkv, a.Nk, kTileRows - f.front, 1))
                return cudaErrorInvalidValue;
    }
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
    const int64_t grid = c > 1 || !C::kWalks || BAND ? units * c : std::min<int64_t>(units, C::kMinBlocks * sm_count());
    return launch_clusters(cross_fwd_mma_kernel<NT, BAND, FRONT, NARROW>, (unsigned)grid, c, C::kThreads, C::kSmem, a.stream, f);
}

// Up to such a window the softmax leaves out every 32 columns of which a warp's rows attend none.  (4 sequences of 4096
// tokens, 8 heads: a window of 64 20.3 us without, 18.1 with; of 128, 4 sinks: 23.4 and 22.8; of 512, 4 sinks: 34.8 and
// 35.8, where what some warps leave out is waited for by the others, and every tile pays for the branches.)
constexpr int kNarrow = 128;

template <bool FRONT, bool NARROW>
cudaError_t launch_band(const CrossArgs &a, int front) {
    const BandTiles qt(a.Hq / a.Hkv, a.Nq, a.Hq > 1 && a.Q.stride_h == 0, kTileRows - front);
    Plan plan;
    const cudaError_t e = consider<1, true, FRONT, NARROW>(a, qt, &plan);
    return e == cudaSuccess ? fwd<1, true, FRONT, NARROW>(a, qt, plan.c) : e;
}

cudaError_t launch(const CrossArgs &a) {
    const QueryTiles qt(a.Hq / a.Hkv, a.Nq, a.Hq > 1 && a.Q.stride_h == 0);
    Plan plan;
    cudaError_t e = consider<1, false>(a, qt, &plan);
    if (e == cudaSuccess) e = consider<2, false>(a, qt, &plan);
    if (e != cudaSuccess) return e;
    return plan.nt == 2 ? fwd<2, false>(a, qt, plan.c) : fwd<1, false>(a, qt, plan.c);
}

}  // namespace

cudaError_t launch_cross_fwd_mma(const CrossArgs &a) {
    if (!a.banded) return launch(a);
    const int front = front_rows(a);
    if (a.band.window <= kNarrow) return front ? launch_band<true, true>(a, front) : launch_band<false, true>(a, 0);
    return front ? launch_band<true, false>(a, front) : launch_band<false, false>(a, 0);
}

FIBATT_DEFINE_ERROR_READER(read_error_cross_mma_fwd, "cross_mma_fwd.cu")

}  // namespace fibatt
