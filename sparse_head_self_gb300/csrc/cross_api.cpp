// C ABI of the query/key norm and of the cross attention: argument checks and
// dispatch.  The operations and every argument rule are documented in
// include/fibatt.h.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <string>

#include "cross.h"

namespace fibatt {
namespace {

std::string fmt(const char *f, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, f);
    vsnprintf(buf, sizeof buf, f, ap);
    va_end(ap);
    return buf;
}

fibatt_status invalid(const std::string &m) { return set_error(FIBATT_ERR_INVALID_ARG, m); }
fibatt_status unsupported(const std::string &m) { return set_error(FIBATT_ERR_UNSUPPORTED, m); }
bool off(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

fibatt_status check_type(int D, fibatt_dtype t) {
    if (D != kHeadDim) return unsupported(fmt("head dim %d unsupported (only %d)", D, kHeadDim));
    if (t != FIBATT_F32 && t != FIBATT_BF16) return unsupported(fmt("unknown dtype %d", (int)t));
    return FIBATT_OK;
}

fibatt_status check_ptr(const void *p, const char *name, size_t a = 16) {
    if (!p) return invalid(fmt("%s is NULL", name));
    if (off(p, a)) return invalid(fmt("%s is not %zu-byte aligned", name, a));
    return FIBATT_OK;
}

int64_t size_of(fibatt_dtype t) { return t == FIBATT_F32 ? 4 : 2; }

// A head tensor of B sequences, H heads and N rows; `out`: the call writes it.
fibatt_status check_heads(const fibatt_heads *v, const char *name, fibatt_dtype t, int B, int H, int N, bool out) {
    if (!v) return invalid(fmt("%s is NULL", name));
    if (fibatt_status st = check_ptr(v->ptr, name)) return st;
    const int64_t strides[3] = {v->stride_b, v->stride_h, v->stride_n};
    const int sizes[3] = {B, H, N};
    for (int i = 0; i < 3; ++i) {
        if (strides[i] < 0 || strides[i] > (int64_t)1 << 38 || strides[i] * size_of(t) % 16)
            return invalid(fmt("%s: stride %lld is not a multiple of 16 bytes in [0, 2^38]", name, (long long)strides[i]));
        if (i == 2 && N > 1 && strides[i] == 0) return invalid(fmt("%s: rows with a stride of 0", name));
        if (out && sizes[i] > 1 && strides[i] < kHeadDim)
            return invalid(fmt("%s is written, but a stride of %lld lets its rows overlap", name, (long long)strides[i]));
    }
    return FIBATT_OK;
}

fibatt_status check_cross(const fibatt_cross *d) {
    if (!d) return invalid("the description is NULL");
    if (fibatt_status st = check_type(d->D, d->dtype)) return st;
    if (d->B < 1 || d->Hq < 1 || d->Hkv < 1 || d->Nq < 1 || d->Nk < 1)
        return invalid(fmt("B=%d, Hq=%d, Hkv=%d, Nq=%d, Nk=%d must be >= 1", d->B, d->Hq, d->Hkv, d->Nq, d->Nk));
    if (d->Hq % d->Hkv) return invalid(fmt("Hkv=%d does not divide Hq=%d", d->Hkv, d->Hq));
    if (!std::isfinite(d->scale)) return invalid("scale is not finite");
    if (off(d->kv_len, 4)) return invalid("kv_len is not 4-byte aligned");
    if (d->key_mask && d->key_mask_stride_b < 0) return invalid("key_mask_stride_b is negative");
    // blocks of the kernels: one a 64-row tile and head at most, and an eighth of what a grid may
    // have (clusters, of up to 16, are launched only while all of them find a place at once)
    const int64_t qb = (int64_t)d->B * d->Hq, kb = (int64_t)d->B * d->Hkv;
    if (qb > 0x7fffffffLL || qb * ((d->Nq + 63LL) / 64) > 0x7fffffffLL / 8 || kb * ((d->Nk + 63LL) / 64) > 0x7fffffffLL / 8 ||
        qb * ((d->Nq + 127LL) / 128 * 128) > 0x7fffffffLL - 256)
        return invalid("too many rows for one call (2^31 query rows, 2^31 - 1 blocks)");
    if (d->Nq > 0x7fffff00 || d->Nk > 0x7fffff00) return invalid("Nq and Nk must be below 2^31 - 256");
    if (fault("arg")) return invalid("injected argument fault (FIBATT_FAULT=arg)");
    return FIBATT_OK;
}

CrossArgs cross_args(const fibatt_cross *d, const fibatt_heads *Q, const fibatt_heads *K, const fibatt_heads *V,
                     const fibatt_heads *O, cudaStream_t stream) {
    CrossArgs a = {};
    a.B = d->B, a.Hq = d->Hq, a.Hkv = d->Hkv, a.Nq = d->Nq, a.Nk = d->Nk;
    a.dtype = d->dtype;
    a.scale = d->scale;
    a.keys = KeySet{d->kv_len, d->key_mask, d->key_mask_stride_b, d->Nk};
    a.Q = *Q, a.K = *K, a.V = *V, a.O = *O;
    a.stream = stream;
    return a;
}

fibatt_status check_norm(const fibatt_qk_norm *d, const void *X, int64_t sb, int64_t sn) {
    if (!d) return invalid("the description is NULL");
    if (fibatt_status st = check_type(d->D, d->dtype)) return st;
    if (d->B < 1 || d->N < 1) return invalid(fmt("B=%d and N=%d must be >= 1", d->B, d->N));
    if (d->Hq < 0 || d->Hk < 0 || d->Hv < 0 || (int64_t)d->Hq + d->Hk + d->Hv < 1 ||
        (int64_t)d->Hq + d->Hk + d->Hv > 1 << 20)
        return invalid(fmt("heads %d, %d, %d: each >= 0, one at least", d->Hq, d->Hk, d->Hv));
    if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return invalid("eps must be finite and >= 0");
    if (off(d->q_weight, 16) || off(d->k_weight, 16)) return invalid("a weight is not 16-byte aligned");
    if (d->rot_dims < 0 || d->rot_dims > kHeadDim || d->rot_dims % 16)
        return invalid(fmt("rot_dims %d is not 0, 16, 32, 48 or 64", d->rot_dims));
    if (d->rot_dims) {
        fibatt_status st;
        if ((st = check_ptr(d->cos, "cos")) || (st = check_ptr(d->sin, "sin"))) return st;
        if (d->table_len < 1 || (!d->positions && d->table_len < d->N))
            return invalid(fmt("tables of %d positions for %d tokens", d->table_len, d->N));
        if (off(d->positions, 4)) return invalid("positions is not 4-byte aligned");
        if (d->positions && d->positions_stride_b < 0) return invalid("positions_stride_b is negative");
    }
    if (fibatt_status st = check_ptr(X, "X")) return st;
    for (int64_t s : {sb, sn})
        if (s < 0 || s > (int64_t)1 << 38 || s * size_of(d->dtype) % 16)
            return invalid(fmt("X: stride %lld is not a multiple of 16 bytes in [0, 2^38]", (long long)s));
    if ((int64_t)d->B * d->N > 0x7fffff00LL) return invalid("too many tokens for one call (2^31 - 256)");
    if (fault("arg")) return invalid("injected argument fault (FIBATT_FAULT=arg)");
    return FIBATT_OK;
}

QkNormArgs norm_args(const fibatt_qk_norm *d, const void *X, int64_t sb, int64_t sn, cudaStream_t stream) {
    QkNormArgs q = {};
    q.B = d->B, q.N = d->N, q.Hq = d->Hq, q.Hk = d->Hk, q.Hv = d->Hv;
    q.dtype = d->dtype;
    q.X = X, q.x_sb = sb, q.x_sn = sn;
    q.wq = d->q_weight, q.wk = d->k_weight;
    q.eps = d->eps;
    q.rot = d->rot_dims, q.interleaved = d->interleaved != 0;
    q.cos = d->cos, q.sin = d->sin, q.P = d->table_len;
    q.pos = d->rot_dims ? d->positions : nullptr, q.pos_sb = d->positions_stride_b;
    q.stream = stream;
    return q;
}

}  // namespace

int sm_count() {
    static thread_local int dev_of = -1, count = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 152;
    if (dev != dev_of) {
        if (cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 152;
        dev_of = dev;
    }
    return count;
}

}  // namespace fibatt

using namespace fibatt;

extern "C" {

fibatt_status fibatt_qk_norm_fwd(const fibatt_qk_norm *d, const void *X, int64_t x_stride_b, int64_t x_stride_n,
                                 void *Q, void *K, void *V, cudaStream_t stream) {
    const ProfileReport report("fibatt_qk_norm_fwd");
    fibatt_status st = check_norm(d, X, x_stride_b, x_stride_n);
    if (st != FIBATT_OK) return st;
    if ((d->Hq && (st = check_ptr(Q, "Q"))) || (d->Hk && (st = check_ptr(K, "K"))) ||
        (d->Hv && (st = check_ptr(V, "V"))))
        return st;
    if (fault("launch")) return set_error(FIBATT_ERR_CUDA, "injected launch failure (FIBATT_FAULT=launch)");
    QkNormArgs q = norm_args(d, X, x_stride_b, x_stride_n, stream);
    q.Q = Q, q.K = K, q.V = V;
    const cudaError_t e = launch_qk_norm_fwd(q);
    return e == cudaSuccess ? FIBATT_OK : cuda_error(e, "fibatt_qk_norm_fwd launch");
}

size_t fibatt_qk_norm_bwd_workspace_bytes(void) { return qk_norm_bwd_workspace(); }

fibatt_status fibatt_qk_norm_bwd(const fibatt_qk_norm *d, const void *X, int64_t x_stride_b, int64_t x_stride_n,
                                 const void *dQ, const void *dK, const void *dV, void *dX, int64_t dx_stride_b,
                                 int64_t dx_stride_n, void *dq_weight, void *dk_weight, void *workspace,
                                 size_t ws_bytes, cudaStream_t stream) {
    const ProfileReport report("fibatt_qk_norm_bwd");
    fibatt_status st = check_norm(d, X, x_stride_b, x_stride_n);
    if (st != FIBATT_OK) return st;
    if ((d->Hq && (st = check_ptr(dQ, "dQ"))) || (d->Hk && (st = check_ptr(dK, "dK"))) ||
        (d->Hv && (st = check_ptr(dV, "dV"))) || (st = check_ptr(dX, "dX")) ||
        (st = check_ptr(workspace, "workspace")))
        return st;
    const int64_t row = ((int64_t)d->Hq + d->Hk + d->Hv) * kHeadDim;
    const int64_t strides[2] = {dx_stride_b, dx_stride_n};
    const int sizes[2] = {d->B, d->N};
    for (int i = 0; i < 2; ++i)
        if (strides[i] < 0 || strides[i] > (int64_t)1 << 38 || strides[i] * size_of(d->dtype) % 16 ||
            (sizes[i] > 1 && strides[i] < row))
            return invalid(fmt("dX: stride %lld must be a multiple of 16 bytes that keeps its rows apart",
                               (long long)strides[i]));
    if (off(dq_weight, 4) || off(dk_weight, 4)) return invalid("a weight's gradient is not 4-byte aligned");
    if (ws_bytes < qk_norm_bwd_workspace())
        return invalid(fmt("workspace holds %zu bytes, %zu needed", ws_bytes, qk_norm_bwd_workspace()));
    if (fault("launch")) return set_error(FIBATT_ERR_CUDA, "injected launch failure (FIBATT_FAULT=launch)");
    QkNormArgs q = norm_args(d, X, x_stride_b, x_stride_n, stream);
    q.dQ = dQ, q.dK = dK, q.dV = dV, q.dX = dX, q.dx_sb = dx_stride_b, q.dx_sn = dx_stride_n;
    q.dwq = d->q_weight ? dq_weight : nullptr, q.dwk = d->k_weight ? dk_weight : nullptr;
    q.ws = static_cast<float *>(workspace);
    const cudaError_t e = launch_qk_norm_bwd(q);
    return e == cudaSuccess ? FIBATT_OK : cuda_error(e, "fibatt_qk_norm_bwd launch");
}

fibatt_status fibatt_cross_fwd(const fibatt_cross *d, const fibatt_heads *Q, const fibatt_heads *K,
                               const fibatt_heads *V, const fibatt_heads *O, float *LSE, cudaStream_t stream) {
    const ProfileReport report("fibatt_cross_fwd");
    fibatt_status st = check_cross(d);
    if (st != FIBATT_OK) return st;
    if ((st = check_heads(Q, "Q", d->dtype, d->B, d->Hq, d->Nq, false)) ||
        (st = check_heads(K, "K", d->dtype, d->B, d->Hkv, d->Nk, false)) ||
        (st = check_heads(V, "V", d->dtype, d->B, d->Hkv, d->Nk, false)) ||
        (st = check_heads(O, "O", d->dtype, d->B, d->Hq, d->Nq, true)) || (st = check_ptr(LSE, "LSE", 4)))
        return st;
    if (fault("launch")) return set_error(FIBATT_ERR_CUDA, "injected launch failure (FIBATT_FAULT=launch)");
    CrossArgs a = cross_args(d, Q, K, V, O, stream);
    a.LSE = LSE;
    const cudaError_t e = cross_rows_takes(a)         ? launch_cross_rows(a)
                          : a.dtype == FIBATT_BF16 ? launch_cross_fwd_mma(a)
                                                   : launch_cross_fwd_f32(a);
    return e == cudaSuccess ? FIBATT_OK : cuda_error(e, "fibatt_cross_fwd launch");
}

size_t fibatt_cross_bwd_workspace_bytes(const fibatt_cross *d) {
    if (!d || d->B < 1 || d->Hq < 1 || d->Nq < 1) return 0;
    const size_t bytes = d->dtype == FIBATT_BF16 ? cross_bwd_mma_workspace(d->B, d->Hq, d->Nq)
                                                 : (size_t)d->B * d->Hq * d->Nq * sizeof(float2);
    return (bytes + 255) / 256 * 256;
}

fibatt_status fibatt_cross_bwd(const fibatt_cross *d, const fibatt_heads *Q, const fibatt_heads *K,
                               const fibatt_heads *V, const fibatt_heads *O, const float *LSE, const fibatt_heads *dO,
                               const fibatt_heads *dQ, const fibatt_heads *dK, const fibatt_heads *dV, void *workspace,
                               size_t ws_bytes, cudaStream_t stream) {
    const ProfileReport report("fibatt_cross_bwd");
    fibatt_status st = check_cross(d);
    if (st != FIBATT_OK) return st;
    if ((st = check_heads(Q, "Q", d->dtype, d->B, d->Hq, d->Nq, false)) ||
        (st = check_heads(K, "K", d->dtype, d->B, d->Hkv, d->Nk, false)) ||
        (st = check_heads(V, "V", d->dtype, d->B, d->Hkv, d->Nk, false)) ||
        (st = check_heads(O, "O", d->dtype, d->B, d->Hq, d->Nq, false)) ||
        (st = check_heads(dO, "dO", d->dtype, d->B, d->Hq, d->Nq, false)) ||
        (st = check_heads(dQ, "dQ", d->dtype, d->B, d->Hq, d->Nq, true)) ||
        (st = check_heads(dK, "dK", d->dtype, d->B, d->Hkv, d->Nk, true)) ||
        (st = check_heads(dV, "dV", d->dtype, d->B, d->Hkv, d->Nk, true)) || (st = check_ptr(LSE, "LSE", 4)) ||
        (st = check_ptr(workspace, "workspace")))
        return st;
    if (ws_bytes < fibatt_cross_bwd_workspace_bytes(d))
        return invalid(fmt("workspace holds %zu bytes, %zu needed", ws_bytes, fibatt_cross_bwd_workspace_bytes(d)));
    if (fault("launch")) return set_error(FIBATT_ERR_CUDA, "injected launch failure (FIBATT_FAULT=launch)");
    CrossArgs a = cross_args(d, Q, K, V, O, stream);
    a.LSE = const_cast<float *>(LSE);
    a.dO = *dO, a.dQ = *dQ, a.dK = *dK, a.dV = *dV;
    a.stats = static_cast<float2 *>(workspace);
    const cudaError_t e = a.dtype == FIBATT_BF16 ? launch_cross_bwd_mma(a) : launch_cross_bwd_f32(a);
    return e == cudaSuccess ? FIBATT_OK : cuda_error(e, "fibatt_cross_bwd launch");
}

}  // extern "C"
