// Shared by the tensor-core cross attention kernels: how query rows make
// tiles, which keys of a tile are attended, and the tensor maps.
#pragma once

#include <cuda.h>

#include "cross.h"
#ifdef __CUDACC__
#include "tcgen05.cuh"
#endif

namespace fibatt {

constexpr int kTileRows = 128;
constexpr int kTileBytes = kTileRows * 128;   // 64 bf16 a row

// The query rows of one key/value head in tiles of 128: `gb` of the G query
// heads that share it by `nb` queries each (nb gb <= 128).  Row r of tile t
// is query n of head g:
//   g = gb (t / ntiles) + r / nb,   n = nb (t mod ntiles) + r mod nb
// so short sequences of several heads share a tile, and a tile of a long one
// holds 128 queries of one head.
struct QueryTiles {
    int G, Nq;
    int nb, gb;      // queries and heads of a tile
    int ntiles;      // tiles along the queries
    int tiles;       // of one key/value head
    // shared_rows: the heads' rows are one and the same in memory (a stride of
    // 0), so no copy can bring several of them
    QueryTiles(int G, int Nq, bool shared_rows) : G(G), Nq(Nq) {
        nb = Nq < kTileRows ? Nq : kTileRows;
        gb = shared_rows ? 1 : kTileRows / nb < G ? kTileRows / nb : G;
        ntiles = (Nq + nb - 1) / nb;
        tiles = ntiles * ((G + gb - 1) / gb);
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int first_head(int t) const { return t / ntiles * gb; }
    __device__ __forceinline__ int first_row(int t) const { return t % ntiles * nb; }
    // head (within the group) and query of row r; false: no such row
    __device__ __forceinline__ bool at(int t, int r, int &g, int &n) const {
        g = first_head(t) + r / nb;
        n = first_row(t) + r % nb;
        return r < nb * gb && g < G && n < Nq;
    }
    __device__ __forceinline__ uint32_t bytes() const { return (uint32_t)(nb * gb) * 128u; }
#endif
};

// A head tensor as the copies see it.  Heads or sequences with a stride of 0
// (a broadcast) become a dimension of one element and a coordinate of 0.
struct TensorArg {
    CUtensorMap map;
    int head_step, seq_step;   // 1, or 0 where the dimension is broadcast
};
// Boxes of `rows` rows by `heads` heads, which arrive with the 128-byte swizzle
// (bf16) or as they are; false when the map cannot be made.
bool make_tensor(TensorArg *t, const fibatt_heads &v, int B, int H, int N, int rows, int heads,
                 fibatt_dtype dtype = FIBATT_BF16, bool swizzle = true);

#ifdef __CUDACC__
__device__ __forceinline__ void load_tile(void *dst, const TensorArg &t, int row, int head, int seq, uint64_t *bar) {
    tile_load(dst, &t.map, row, head * t.head_step, seq * t.seq_step, bar);
}

// Bit k of the result's four words: key n0 + k is attended.  The same in every
// lane; the whole warp calls it.
__device__ __forceinline__ uint4 tile_keys(const KeySet &ks, int b, int n0, int bound) {
    const int lane = threadIdx.x & 31;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int k = n0 + 32 * i + lane;
        w[i] = __ballot_sync(kFullMask, k < bound && ks.has(b, k));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ bool all_keys(const uint4 &w) { return (w.x & w.y & w.z & w.w) == 0xffffffffu; }
__device__ __forceinline__ bool no_keys(const uint4 &w) { return (w.x | w.y | w.z | w.w) == 0u; }

// Zeros into the tile's rows whose bit in `w` is 0 (whole rows, so the swizzle
// does not matter); the whole warp calls it.  What stands in memory behind a
// sequence's keys would otherwise meet weights of 0, and 0 x NaN is not 0.
__device__ __forceinline__ void clear_rows(uint8_t *tile, const uint4 &w) {
    const int lane = threadIdx.x & 31;
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((words[i] >> lane) & 1) continue;
        uint4 *row = reinterpret_cast<uint4 *>(tile + (32 * i + lane) * 128);
#pragma unroll
        for (int c = 0; c < 8; ++c) row[(c + lane) & 7] = make_uint4(0, 0, 0, 0);
    }
}

// For a few rows, by the whole warp: c += A (16 x 16) B (16 x 8)
__device__ __forceinline__ void warp_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
#endif

}  // namespace fibatt
