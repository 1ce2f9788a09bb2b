// Internal declarations of the paged cache of keys and values in 8 bits.  The
// operations and every argument rule are documented in include/fibatt.h.
#pragma once

#include "cross.h"

namespace fibatt {

constexpr int kPage = FIBATT_CACHE_PAGE;              // tokens of a page
constexpr int kPageBytes = kPage * kHeadDim;          // of its keys, or of its values

struct CacheArgs {
    int B, Hkv, N;               // N: tokens a sequence of the call
    fibatt_dtype dtype;
    int pages, table_len;
    uint8_t *data;               // [pages, Hkv, 2, 4096]: keys [token][dim], values [dim][token]
    float *scales;               // [pages, Hkv, 2]
    const int32_t *table;        // [B, table_len]
    int64_t table_sb;
    const int32_t *start, *count;    // [B] or null
    fibatt_heads K, V;           // of a store, a load
    // of the attention
    int Hq;
    float scale;
    int window, sinks;
    fibatt_heads Q, O;
    float *LSE;
    cudaStream_t stream;
    // Position of the call's first token.  (One further out leaves no token a place in the table.)
    __host__ __device__ __forceinline__ int first(int b) const {
        return start ? most(-N, least(load_number(start + b), table_len * kPage)) : 0;
    }
    __host__ __device__ __forceinline__ int tokens(int b) const { return count ? most(0, least(load_number(count + b), N)) : N; }
    // A sequence's page number `i`, -1 where the table has none there or one that the cache has not.
    __host__ __device__ __forceinline__ int page(int b, int i) const {
        if ((unsigned)i >= (unsigned)table_len) return -1;
        const int p = load_number(table + b * table_sb + i);
        return (unsigned)p < (unsigned)pages ? p : -1;
    }
    __host__ __device__ __forceinline__ int64_t place(int page, int hk) const { return (int64_t)page * Hkv + hk; }
};

// Pages that N tokens lie in at most.
__host__ __device__ constexpr int64_t pages_of(int64_t N) { return (N + 2 * kPage - 2) / kPage; }

// Where block `i` of a store or a load works: a page's keys or values of one head.
struct Spot {
    int b, hk, kind, page;               // kind 0: keys, 1: values; page -1: none, or none of the call's tokens in it
    int lo, hi;                          // its tokens that the call has: [lo, hi) of 64
    int token;                           // number in the call of the page's first (may be negative)
    bool lost;                           // tokens without a page
    __host__ __device__ __forceinline__ Spot(const CacheArgs &a, unsigned i) {
        kind = i & 1;
        i >>= 1;
        hk = i % (unsigned)a.Hkv;
        i /= (unsigned)a.Hkv;
        const unsigned slots = (unsigned)pages_of(a.N);
        b = i / slots;
        const int start = a.first(b), slot = (start >> 6) + (int)(i % slots);      // (rounded down, also before token 0)
        token = slot * kPage - start;
        lo = most(0, -token);
        hi = least(kPage, a.tokens(b) - token);
        page = lo < hi ? a.page(b, slot) : -1;
        lost = lo < hi && page < 0;
    }
};

cudaError_t launch_cache_store(const CacheArgs &a);
cudaError_t launch_cache_load(const CacheArgs &a);
cudaError_t launch_cache_fwd(const CacheArgs &a);
cudaError_t read_error_cross_cache(unsigned *code, bool clear);

}  // namespace fibatt
