// C ABI of the paged 8-bit cache: argument checks and dispatch.  The operations and
// every argument rule are documented in include/fibatt.h.
#include <cmath>

#include "cross_cache.h"
#include "cross_checks.h"

namespace fibatt {
namespace {

fibatt_status check_cache(const fibatt_cache *d, int heads) {
    if (!d) return invalid("the description is NULL");
    if (fibatt_status st = check_type(d->D, d->dtype)) return st;
    if (d->B < 1 || d->Hkv < 1 || d->N < 1 || d->pages < 1 || d->table_len < 1)
        return invalid(fmt("B=%d, Hkv=%d, N=%d, pages=%d, table_len=%d must be >= 1", d->B, d->Hkv, d->N, d->pages, d->table_len));
    if (d->N >= 1 << 30 || d->table_len >= 1 << 24) return invalid("N must be below 2^30 and table_len below 2^24");
    fibatt_status st;
    if ((st = check_ptr(d->data, "data")) || (st = check_ptr(d->scales, "scales", 8)) || (st = check_ptr(d->table, "table", 4)))
        return st;
    if (d->table_stride_b < 0) return invalid("table_stride_b is negative");
    if (off(d->start, 4) || off(d->count, 4)) return invalid("start or count is not 4-byte aligned");
    // blocks of the kernels: two a page and head at most, or a cluster of eight for every 16 rows of a key head
    const int64_t bh = (int64_t)d->B * d->Hkv, rows = (int64_t)heads / d->Hkv * d->N;
    if (bh > 0x7fffffffLL || 2 * bh * ((d->N + 126LL) / 64) > 0x7fffffffLL || rows > 0x7fffffffLL - 16 ||
        bh * ((rows + 15) / 16) > 0x7fffffffLL / 8)
        return invalid("too many tokens for one call (2^31 - 1 blocks)");
    if (fault("arg")) return invalid("injected argument fault (FIBATT_FAULT=arg)");
    return FIBATT_OK;
}

CacheArgs cache_args(const fibatt_cache *d, cudaStream_t stream) {
    CacheArgs a = {};
    a.B = d->B, a.Hkv = d->Hkv, a.N = d->N;
    a.dtype = d->dtype;
    a.pages = d->pages, a.table_len = d->table_len;
    a.data = static_cast<uint8_t *>(d->data);
    a.scales = d->scales;
    a.table = d->table, a.table_sb = d->table_stride_b;
    a.start = d->start, a.count = d->count;
    a.stream = stream;
    return a;
}

fibatt_status move(const fibatt_cache *d, const fibatt_heads *K, const fibatt_heads *V, bool store, cudaStream_t stream) {
    fibatt_status st = check_cache(d, 0);
    if (st != FIBATT_OK || (st = check_heads(K, "K", d->dtype, d->B, d->Hkv, d->N, !store)) ||
        (st = check_heads(V, "V", d->dtype, d->B, d->Hkv, d->N, !store)))
        return st;
    if (fault("launch")) return set_error(FIBATT_ERR_CUDA, "injected launch failure (FIBATT_FAULT=launch)");
    CacheArgs a = cache_args(d, stream);
    a.K = *K, a.V = *V;
    const cudaError_t e = store ? launch_cache_store(a) : launch_cache_load(a);
    return e == cudaSuccess ? FIBATT_OK : cuda_error(e, store ? "fibatt_cache_store launch" : "fibatt_cache_load launch");
}

}  // namespace
}  // namespace fibatt

using namespace fibatt;

extern "C" {

fibatt_status fibatt_cache_store(const fibatt_cache *d, const fibatt_heads *K, const fibatt_heads *V, cudaStream_t stream) {
    const ProfileReport report("fibatt_cache_store");
    return move(d, K, V, true, stream);
}

fibatt_status fibatt_cache_load(const fibatt_cache *d, const fibatt_heads *K, const fibatt_heads *V, cudaStream_t stream) {
    const ProfileReport report("fibatt_cache_load");
    return move(d, K, V, false, stream);
}

fibatt_status fibatt_cache_fwd(const fibatt_cache *d, int Hq, float scale, int window, int sinks, const fibatt_heads *Q,
                               const fibatt_heads *O, float *LSE, cudaStream_t stream) {
    const ProfileReport report("fibatt_cache_fwd");
    if (Hq < 1) return invalid(fmt("Hq=%d must be >= 1", Hq));
    if (d && d->Hkv > 0 && Hq % d->Hkv) return invalid(fmt("Hkv=%d does not divide Hq=%d", d->Hkv, Hq));
    fibatt_status st = check_cache(d, Hq);
    if (st != FIBATT_OK) return st;
    if (!std::isfinite(scale)) return invalid("scale is not finite");
    if (window < 1) return invalid(fmt("window=%d must be >= 1", window));
    if (sinks < 0) return invalid(fmt("sinks=%d must be >= 0", sinks));
    if ((st = check_heads(Q, "Q", d->dtype, d->B, Hq, d->N, false)) || (st = check_heads(O, "O", d->dtype, d->B, Hq, d->N, true)) ||
        (st = check_ptr(LSE, "LSE", 4)))
        return st;
    if (fault("launch")) return set_error(FIBATT_ERR_CUDA, "injected launch failure (FIBATT_FAULT=launch)");
    CacheArgs a = cache_args(d, stream);
    const int keys = d->table_len * FIBATT_CACHE_PAGE;
    a.Hq = Hq;
    a.scale = scale;
    // (a window that reaches the first key makes sinks of no account)
    a.window = std::min(window, keys);
    a.sinks = a.window == keys ? 0 : std::min(sinks, keys);
    a.Q = *Q, a.O = *O;
    a.LSE = LSE;
    const cudaError_t e = launch_cache_fwd(a);
    return e == cudaSuccess ? FIBATT_OK : cuda_error(e, "fibatt_cache_fwd launch");
}

}  // extern "C"
