/*
 * fibatt.h -- C ABI of libfibatt: Fibottention's per-head sparse
 * self-attention (forward and backward) on NVIDIA GB300 (sm_103a).
 *
 * The operation ("Fibottention: Inceptive Visual Representation Learning
 * with Diverse Attention Across Heads", arXiv 2406.19391, Sec. 3):
 *
 *   head h of H, query j in [0, N) attends exactly the keys k with
 *       |j - k| in Fib(a_h, b_h)  and  |j - k| <= w_h      (support Omega_h)
 *   plus k = j when the main diagonal is included.  Fib(a, b) is the
 *   generalised Fibonacci sequence f_1 = a, f_2 = b, f_{n+2} = f_{n+1} + f_n
 *   (project README, Algorithm 1), and (a_h, b_h) is normally row h of the
 *   Wythoff array (Sec. 3.2).  Scores outside Omega_h are excluded from the
 *   softmax:
 *       s_jk = scale * <Q_j, K_k>                 (j,k) in Omega_h
 *       LSE_j = log sum_{k:(j,k) in Omega_h} exp(s_jk)
 *       O_j  = sum_{k:(j,k) in Omega_h} exp(s_jk - LSE_j) V_k
 *   (README, Algorithm 3: scores, mask, row softmax, weighted sum of V).
 *
 * Beside it, for the layers around it: the norms of queries and keys with the
 * position rotation (fibatt_qk_norm_fwd, _bwd) and the attention to another
 * sequence's states (fibatt_cross_fwd, _bwd).
 *
 * Conventions shared by every call below (the two beside it state their own
 * layouts):
 *   - Tensors are dense, row-major [B, H, N, D] with D = 64 (one row = 64
 *     contiguous elements), in the I/O dtype fibatt_dtype; LSE is fp32
 *     [B, H, N].  All tensor pointers are DEVICE pointers owned by the
 *     caller, 16-byte aligned (LSE: 4-byte aligned), on the current device.
 *   - Arithmetic is fp32 with fp32 accumulation; bf16 outputs are rounded to
 *     nearest-even once, at the end.  LSE is the natural log.  One exception,
 *     for bf16 I/O in the shared-memory forward kernels: each softmax weight
 *     is rounded to bf16 before its P.V update (products exact, sums fp32),
 *     and O is divided by the sum of those rounded weights, so O stays a
 *     convex combination of value rows; the LSE uses the fp32 weights.
 *   - fwd/bwd are asynchronous on `stream` and never synchronise.  They do not
 *     allocate device memory.
 *   - A support handle is host memory only (its tables travel to the GPU as
 *     kernel arguments), so one handle may be used on any device and from
 *     any stream; it must not be destroyed while a call using it is being
 *     made (kernels already launched do not reference it).
 *   - Every call returns a fibatt_status; on failure, fibatt_last_error()
 *     gives a message for the calling thread.  Nothing is ever trapped on the
 *     device.
 */
#ifndef FIBATT_H_
#define FIBATT_H_

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FIBATT_OK = 0,
    FIBATT_ERR_INVALID_ARG = 1,   /* a size, pointer or parameter is out of its range      */
    FIBATT_ERR_UNSUPPORTED = 2,   /* valid, but outside what this build implements          */
    FIBATT_ERR_CUDA = 3,          /* a CUDA launch or runtime call failed (message attached) */
    FIBATT_ERR_OOM = 4            /* host allocation failed                                 */
} fibatt_status;

typedef enum {
    FIBATT_F32 = 0,               /* float32 I/O                          */
    FIBATT_BF16 = 1               /* bfloat16 I/O, fp32 accumulation      */
} fibatt_dtype;

/* Opaque per-layer support: the signed-offset table of every head. */
typedef struct fibatt_support *fibatt_support_t;

/* Limits of this build (UNSUPPORTED beyond them). */
#define FIBATT_HEAD_DIM 64        /* D                                         */
#define FIBATT_CACHE_PAGE 64      /* tokens of a page of the 8-bit cache       */
#define FIBATT_MAX_HEADS 64       /* H                                         */
#define FIBATT_MAX_ENTRIES 1024   /* signed offsets summed over all heads      */

/* ------------------------------------------------------------- helpers --- */

/* Row i (i >= 1) of the Wythoff array (Fibottention Sec. 3.2): writes its
 * first two entries a = floor(floor(i*phi)*phi), b = floor(floor(i*phi)*phi^2),
 * computed in exact integer arithmetic.  Rows are disjoint and together
 * contain every positive integer once.  INVALID_ARG unless 1 <= i <= 1e8. */
fibatt_status fibatt_wythoff_row(int64_t i, int64_t *a, int64_t *b);

/* The "modified" Wythoff row of the project README (Algorithm 2): the two
 * terms that precede row i, (2a - b, b - a).  Same argument rules. */
fibatt_status fibatt_wythoff_row_modified(int64_t i, int64_t *a, int64_t *b);

/* Per-head windows (Fibottention Sec. 3.2):
 *     w[i-1] = w_min + floor((w_max - w_min) * (i - 1) / (h - 1)),  i = 1..h
 * (h = 1 gives w_min).  w has h entries, caller-owned.
 * INVALID_ARG unless h >= 1 and 1 <= w_min <= w_max. */
fibatt_status fibatt_window_schedule(int h, int64_t w_min, int64_t w_max, int64_t *w);

/* ------------------------------------------------------------- support --- */

/* Build the support of H heads over N tokens (Fibottention Sec. 3, support
 * set Omega_w^{Fib(a,b)}; README Algorithm 1 for the sequence).  a, b, w are
 * host arrays of H entries; head h uses Fib(a[h], b[h]) cut at w[h]:
 * the distances kept are the distinct terms f with f <= min(w[h], N - 1), and
 * the head's table is the ascending signed list {-f...} U {0 if include_diag
 * or 0 in Fib} U {+f...}.  A per-layer head permutation is applied by the
 * caller by permuting a, b and w.
 * INVALID_ARG: H < 1, N < 1, a[h] < 0, b[h] < 0, a[h] = b[h] = 0, w[h] < 1 or
 * w[h] > N, out == NULL.  UNSUPPORTED: H > FIBATT_MAX_HEADS or more than
 * FIBATT_MAX_ENTRIES signed entries in total.  *out is owned by the caller
 * and released with fibatt_support_destroy. */
fibatt_status fibatt_support_build(int H, int N, const int64_t *a, const int64_t *b,
                                   const int64_t *w, int include_diag, fibatt_support_t *out);

/* Build a support from explicit unsigned distances (any dilation sequence,
 * Fibottention Sec. 3: constant c*n or exponential dilation, or the full
 * range 0..N-1 for dense attention).  counts[h] distances for head h are
 * concatenated in `distances`; duplicates count once, distances > N - 1 are
 * dropped, 0 means the main diagonal.  INVALID_ARG on a negative count or
 * distance; limits as fibatt_support_build. */
fibatt_status fibatt_support_build_distances(int H, int N, const int32_t *counts,
                                             const int32_t *distances, int include_diag,
                                             fibatt_support_t *out);

/* Make token 0 global in every head of the support, or banded again
 * (enabled = 0): the class token attends every key and every query attends
 * it, on top of the banded Fibonacci support (Fibottention README,
 * Algorithm 2, whose mask keeps row 0 and column 0 all ones).  The signed
 * tables keep describing the banded part; fibatt_support_get's pair counts
 * include the global pairs.  With it enabled, the dense row of token 0 (and
 * for the backward its dense row and the column of key 0) is computed inside
 * the shared-memory-resident kernels when their plan allows it, else by up to
 * three extra small kernels; FIBATT_PATH=generic and fibatt_bwd_noalloc are
 * UNSUPPORTED, and the backward's workspace grows by 2 x N fp32 per (b, h)
 * (used by the extra kernels only).  Not thread-safe against calls using the
 * support. */
fibatt_status fibatt_support_set_global_token(fibatt_support_t s, int enabled);

/* Sizes of a support: heads, tokens, and total signed entries. */
fibatt_status fibatt_support_info(fibatt_support_t s, int *H, int *N, int *total_entries);

/* Copy a support's tables out (host arrays, caller-sized from
 * fibatt_support_info): counts[H] signed entries per head, signed_offsets in
 * CSR order (head 0's ascending list, then head 1's, ...), pairs[H] = |Omega_h|,
 * the number of attended (j,k) pairs of head h.  Any output may be NULL. */
fibatt_status fibatt_support_get(fibatt_support_t s, int32_t *counts, int32_t *signed_offsets,
                                 int64_t *pairs);

void fibatt_support_destroy(fibatt_support_t s);

/* ------------------------------------------------------------ attention --- */

/* Forward pass.  Q, K, V: [B, H, N, D] (dtype); writes O: [B, H, N, D] (dtype)
 * and LSE: [B, H, N] fp32, natural log.  A query row with no support gets
 * O = 0 and LSE = -inf.  scale multiplies every dot product (1/sqrt(D) in
 * ViT; any finite value).  INVALID_ARG: NULL or misaligned pointer, B < 1,
 * B*H > 2^31-1, non-finite scale.  UNSUPPORTED: D != 64, unknown dtype.
 * CUDA: launch failure (the message names the CUDA error). */
fibatt_status fibatt_fwd(fibatt_support_t s, int B, int D, fibatt_dtype dtype,
                         const void *Q, const void *K, const void *V, float scale,
                         void *O, float *LSE, cudaStream_t stream);

/* Device scratch the backward pass may need for B batches of this support,
 * in bytes: the larger of one fp32 per query row (D_j = <dO_j, O_j>, global-
 * memory kernels) and the pair weights P and dS of every attended pair
 * (2 x the largest per-head table x N fp32 per (b, h); kernels for windows
 * too wide for shared memory).  The shared-memory-resident kernels touch
 * none of it. */
size_t fibatt_bwd_workspace_bytes(fibatt_support_t s, int B);

/* Backward pass for the loss whose gradient with respect to O is dO:
 *   P_jk = exp(s_jk - LSE_j),  dP_jk = <dO_j, V_k>,  D_j = <dO_j, O_j>,
 *   dS_jk = P_jk (dP_jk - D_j),
 *   dQ_j = scale sum_k dS_jk K_k,  dK_k = scale sum_j dS_jk Q_j,
 *   dV_k = sum_j P_jk dO_j      (sums over (j,k) in Omega_h)
 * (the exact derivative of the forward pass above; the pages print no
 * backward).  Q, K, V, O, dO: [B, H, N, D] (dtype); LSE from fibatt_fwd;
 * writes dQ, dK, dV: [B, H, N, D] (dtype).  workspace: device memory of at
 * least fibatt_bwd_workspace_bytes(s, B) bytes, 16-byte aligned, caller-owned
 * (contents on entry are ignored); may be NULL when that size is 0.
 * Errors as fibatt_fwd, plus INVALID_ARG when the workspace is too small. */
fibatt_status fibatt_bwd(fibatt_support_t s, int B, int D, fibatt_dtype dtype,
                         const void *Q, const void *K, const void *V, const void *O,
                         const float *LSE, const void *dO, float scale,
                         void *dQ, void *dK, void *dV, void *workspace, size_t ws_bytes,
                         cudaStream_t stream);

/* Scratch rows (fp32 each) built into the library for fibatt_bwd_noalloc. */
#define FIBATT_NOALLOC_MAX_ROWS (1u << 20)

/* Backward pass for callers that cannot allocate device memory (for example
 * code that runs where the allocator is off limits, or a plugin that is
 * handed fixed buffers).  Same arguments, results and errors as fibatt_bwd
 * without the workspace: the scratch (one fp32 per query row) lives in a
 * fixed array of FIBATT_NOALLOC_MAX_ROWS rows that every GPU loading the
 * library holds until the process exits, so this call allocates nothing.
 * INVALID_ARG when B*H*N exceeds FIBATT_NOALLOC_MAX_ROWS.  The first call on
 * a device looks up the array's device address on that device (make it before
 * any stream capture).  All calls on a device share the array: calls that
 * overlap on the GPU race on it.  No counterpart in the paper: this is a
 * library convenience, not part of the method. */
fibatt_status fibatt_bwd_noalloc(fibatt_support_t s, int B, int D, fibatt_dtype dtype,
                                 const void *Q, const void *K, const void *V, const void *O,
                                 const float *LSE, const void *dO, float scale,
                                 void *dQ, void *dK, void *dV, cudaStream_t stream);

/* ------------------------------------------------- query and key norms --- */

/* Norm of every query and key head with the position rotation, from the
 * packed projection of a layer straight to the [B, H, N, 64] tensors that the
 * attention calls read:
 *     X [B, N, (Hq + Hk + Hv) 64]:  Hq query heads, Hk key heads, Hv value
 *     heads of each token side by side (any of the three counts may be 0).
 * One query head's values x, with the weight w = q_weight, and likewise one
 * key head's with k_weight:
 *     y = w x / sqrt(<x, x> / 64 + eps)     (y = x where the weight is NULL)
 * then the first rot_dims values of y in pairs (y1, y2), pair i of a token at
 * position p by the angle whose cosine and sine are c = cos[p, i], s = sin[p, i]:
 *     (y1, y2) -> (y1 c - y2 s, y1 s + y2 c)
 * Pairs are dims (i, i + rot_dims / 2), or neighbours (2 i, 2 i + 1) when
 * interleaved is set.  Value heads are copied, and what is not
 * rotated (dims behind rot_dims, tokens that positions leave out) is left as it is.
 * Arithmetic in fp32, one rounding to the I/O type. */
typedef struct {
    int B, N;                    /* sequences, tokens                               */
    int Hq, Hk, Hv;              /* heads of each kind, >= 0, one at least           */
    int D;                       /* head dim, FIBATT_HEAD_DIM                        */
    fibatt_dtype dtype;          /* of X, the weights, Q, K, V and their gradients   */
    const void *q_weight;        /* [64] or NULL: queries are not normalised         */
    const void *k_weight;        /* [64] or NULL: keys are not normalised            */
    float eps;                   /* finite, >= 0                                     */
    int rot_dims;                /* 0 (no rotation), 16, 32, 48 or 64                */
    int interleaved;             /* pairs are neighbours                             */
    const float *cos, *sin;      /* [table_len, rot_dims / 2] fp32; unused when rot_dims is 0 */
    int table_len;
    const int32_t *positions;    /* [B, N] (rows positions_stride_b apart; 0: one row for
                                    every sequence) or NULL: token n is at position n.
                                    A token at a negative position is not rotated (a class
                                    token, say); one at table_len or behind it is not rotated
                                    either, and sets bit 3 of the device error word.   */
    int64_t positions_stride_b;
} fibatt_qk_norm;

/* X: token rows of (Hq + Hk + Hv) 64 contiguous elements, x_stride_n elements
 * between the tokens and x_stride_b between the sequences of one.  Writes
 * Q [B, Hq, N, 64], K [B, Hk, N, 64] and V [B, Hv, N, 64], dense (a part
 * without heads may be NULL).  INVALID_ARG: B or N < 1, B N above 2^31 - 256, a negative head count
 * or none, a NULL or misaligned pointer (16 bytes; positions 4), a stride
 * that is not a multiple of 16 bytes, eps, rot_dims or table_len out of their range,
 * positions NULL with table_len < N.  UNSUPPORTED: D, dtype. */
fibatt_status fibatt_qk_norm_fwd(const fibatt_qk_norm *d, const void *X, int64_t x_stride_b,
                                 int64_t x_stride_n, void *Q, void *K, void *V, cudaStream_t stream);

/* Device scratch of fibatt_qk_norm_bwd, in bytes (the blocks' sums of the
 * weights' gradients). */
size_t fibatt_qk_norm_bwd_workspace_bytes(void);

/* Gradient of the call above: from dQ, dK, dV (dense, as Q, K, V) to dX
 * (strides as X's; may not overlap X) and to the weights' gradients
 * dq_weight, dk_weight [64] in the I/O type, summed over all tokens and heads
 * in fp32 in a fixed order, in fp32 I/O with what the additions of partial
 * sums round off kept (written only where the weight is not NULL; either
 * may be NULL when its gradient is not wanted).  Heads of a kind without a
 * weight are not read from X, on which their gradient does not depend.  workspace: 16-byte aligned,
 * for one call at a time. */
fibatt_status fibatt_qk_norm_bwd(const fibatt_qk_norm *d, const void *X, int64_t x_stride_b,
                                 int64_t x_stride_n, const void *dQ, const void *dK, const void *dV,
                                 void *dX, int64_t dx_stride_b, int64_t dx_stride_n, void *dq_weight,
                                 void *dk_weight, void *workspace, size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------ cross attention --- */

/* Attention of the queries of one sequence to the states of another (a
 * decoder's to an encoder's): Nq queries, Nk keys and values, every query head
 * h reading key/value head h / (Hq / Hkv).  Sequence b attends the keys
 *     k < kv_len[b] (every key when kv_len is NULL)   and
 *     key_mask[b, k] != 0 (every key when key_mask is NULL),
 * the same for all its queries:
 *     s_jk = scale <Q_j, K_k>,  LSE_j = log sum_k exp(s_jk),
 *     O_j = sum_k exp(s_jk - LSE_j) V_k
 * A sequence that attends no key gets O = 0 and LSE = -inf.  What memory
 * holds in keys and values that are not attended (NaN, infinities) reaches no
 * result, and their gradients are zeros. */
typedef struct {
    int B, Hq, Hkv;              /* >= 1; Hkv divides Hq                             */
    int Nq, Nk;                  /* >= 1                                             */
    int D;                       /* head dim, FIBATT_HEAD_DIM                        */
    fibatt_dtype dtype;
    float scale;                 /* any finite value                                 */
    const int32_t *kv_len;       /* device, [B], or NULL; clamped to [0, Nk]          */
    const uint8_t *key_mask;     /* device, [B, Nk] bytes, or NULL                    */
    int64_t key_mask_stride_b;   /* bytes between the mask's rows (0: one for all)    */
} fibatt_cross;

/* A tensor of heads: element [b, h, n, d] at ptr + b stride_b + h stride_h +
 * n stride_n + d (strides in elements), so that [B, H, N, 64] and
 * [B, N, H, 64] tensors and slices of packed projections are all read and
 * written in place.  ptr 16-byte aligned, strides >= 0 and multiples of 16
 * bytes; a tensor that a call writes has no two rows in one place, one that it
 * reads may be broadcast over sequences and heads (stride_b, stride_h of 0).
 * What a call writes overlaps nothing that it reads. */
typedef struct {
    void *ptr;
    int64_t stride_b, stride_h, stride_n;
} fibatt_heads;

/* Forward pass.  Q, O: Hq heads of Nq rows; K, V: Hkv heads of Nk rows; LSE:
 * [B, Hq, Nq] fp32, dense, natural log.  Arithmetic is fp32 with fp32
 * accumulation; for bf16 the softmax weights are rounded to bf16 before their
 * product with V (the sums and the LSE use the unrounded ones), and O once at
 * the end; for fp32 products keep 22 bits of each operand (with more than eight
 * query rows to a key head), so that a value that is attended and infinite, or within
 * 2^-12 of the type's largest, may give NaN where 24-bit products do not.  INVALID_ARG: a size or stride out of its range, a NULL or
 * misaligned pointer, a scale that is not finite, 2^31 query rows (a head's
 * rounded up to 128) or more.
 * UNSUPPORTED: D, dtype. */
fibatt_status fibatt_cross_fwd(const fibatt_cross *d, const fibatt_heads *Q, const fibatt_heads *K,
                               const fibatt_heads *V, const fibatt_heads *O, float *LSE,
                               cudaStream_t stream);

/* Device scratch of fibatt_cross_bwd, in bytes: two floats a query row, and in
 * 16 bits 32 bytes a row more (rows rounded up to 128 a head) and two counters. */
size_t fibatt_cross_bwd_workspace_bytes(const fibatt_cross *d);

/* Backward pass for the loss whose gradient with respect to O is dO:
 *     P_jk = exp(s_jk - LSE_j),  D_j = <dO_j, O_j>,  dS_jk = P_jk (<dO_j, V_k> - D_j),
 *     dQ_j = scale sum_k dS_jk K_k,   dK_k = scale sum_j dS_jk Q_j,   dV_k = sum_j P_jk dO_j,
 * the last two over the queries of every head that shares the key head.  No
 * atomics: results do not depend on scheduling.  For bf16, P and dS are
 * rounded to bf16 before the products that sum them, and with Nk <= 64, or for
 * a sequence of at most 8 keys by kv_len, D is summed as sum_k P_jk <dO_j, V_k>,
 * which O's rounding does not enter (against 64 bits, 3 keys: dQ and dK 0.0024 off, otherwise
 * 0.0032, as for 3 keys that key_mask leaves of a longer sequence).  O and LSE are
 * fibatt_cross_fwd's.  workspace: 16-byte aligned, for one call at a time.
 * Errors as fibatt_cross_fwd, plus INVALID_ARG for a workspace too small. */
fibatt_status fibatt_cross_bwd(const fibatt_cross *d, const fibatt_heads *Q, const fibatt_heads *K,
                               const fibatt_heads *V, const fibatt_heads *O, const float *LSE,
                               const fibatt_heads *dO, const fibatt_heads *dQ, const fibatt_heads *dK,
                               const fibatt_heads *dV, void *workspace, size_t ws_bytes,
                               cudaStream_t stream);

/* ------------------------------------ attention over a window, with sinks --- */

/* Causal attention of a sequence's tokens to the last `window` of them, with
 * the first `sinks` tokens visible to all (a decoder's self-attention; every
 * query head h reads key/value head h / (Hq / Hkv)).  Query j of sequence b
 * is at position
 *     p = q_start[b] + j   (Nk - Nq + j when q_start is NULL: the last Nq of Nk tokens)
 * and attends the keys k (at positions 0 to kv_len[b] - 1, all Nk when kv_len is NULL) with
 *     k <= p   and   (k > p - window  or  k < sinks);
 * a query at a negative position, or at kv_len[b] or behind it (padding), attends none and
 * gets O = 0, LSE = -inf and dQ = 0.  s, LSE, O and the gradients are otherwise those of the
 * cross attention above, summed over these pairs.  What memory holds in
 * keys and values that no query of its sequence attends, and in queries and rows of dO that
 * attend nothing (NaN, infinities), reaches no result.  A key or value that
 * is not finite and is attended reaches the queries that attend it, and may reach
 * those within 255 rows of them; a query or a row of dO that is not finite
 * reaches the gradients of the keys that it attends, and may reach those of attended keys
 * within 255 of them. */
typedef struct {
    int B, Hq, Hkv;              /* >= 1; Hkv divides Hq                             */
    int Nq, Nk;                  /* >= 1, below 2^30; Nq <= Nk when q_start is NULL   */
    int D;                       /* head dim, FIBATT_HEAD_DIM                        */
    fibatt_dtype dtype;
    float scale;                 /* any finite value                                 */
    int window;                  /* >= 1 keys up to the query's own; Nk or more: all of them */
    int sinks;                   /* >= 0                                             */
    const int32_t *q_start;      /* device, [B], or NULL                              */
    const int32_t *kv_len;       /* device, [B], or NULL; clamped to [0, Nk]          */
} fibatt_window;

/* Forward pass; tensors, arithmetic and errors as fibatt_cross_fwd, with
 * INVALID_ARG for a window, sinks, Nq or Nk out of its range. */
fibatt_status fibatt_window_fwd(const fibatt_window *d, const fibatt_heads *Q, const fibatt_heads *K,
                                const fibatt_heads *V, const fibatt_heads *O, float *LSE,
                                cudaStream_t stream);

/* Device scratch of fibatt_window_bwd, in bytes. */
size_t fibatt_window_bwd_workspace_bytes(const fibatt_window *d);

/* Backward pass, as fibatt_cross_bwd; for bf16, D_j is summed from the weights with Nk
 * <= 64 or window + sinks <= 64, and is <dO_j, O_j> with the O that is given otherwise.
 * Keys that no query attends get gradients of 0. */
fibatt_status fibatt_window_bwd(const fibatt_window *d, const fibatt_heads *Q, const fibatt_heads *K,
                                const fibatt_heads *V, const fibatt_heads *O, const float *LSE,
                                const fibatt_heads *dO, const fibatt_heads *dQ, const fibatt_heads *dK,
                                const fibatt_heads *dV, void *workspace, size_t ws_bytes,
                                cudaStream_t stream);

/* ------------------------------------------------- paged cache in 8 bits --- */

/* Keys and values of tokens in 8 bits, in pages of FIBATT_CACHE_PAGE = 64
 * tokens that a table hands to sequences: token p of sequence b is row p mod 64
 * of page table[b, p / 64].  A key/value head's part of a page is two pieces of 4096
 * e4m3 bytes, the keys as [64 tokens][64 dims] and behind them the values as
 * [64 dims][64 tokens], each with a scale: a byte stands for its e4m3 value
 * times the scale.  Scales are powers of two from 2^-100 to 2^120 (what else stands
 * there is read as the power of two at or below its size, within those bounds, NaN and
 * infinities as the largest).
 *
 * A call has N tokens of every sequence, token n of them at position
 * start[b] + n (n when start is NULL); of sequence b the first count[b] count (all
 * when count is NULL; clamped to [0, N]).  The caller keeps the table, and which pages are free; a
 * page may be in several sequences' tables as long as none of them stores
 * into it.  Table entries that no token of a call needs may hold anything.
 * A token whose position is outside the table, or whose entry there is not a
 * page of the cache, is not stored, loads as zeros, is attended by nobody and
 * sets bit 4 of the device error word.  As a query one outside the table attends
 * nothing; one inside it attends the keys of the pages that are there. */
typedef struct {
    int B, Hkv, N;               /* >= 1; N below 2^30                               */
    int D;                       /* head dim, FIBATT_HEAD_DIM                        */
    fibatt_dtype dtype;          /* of the tensors beside the cache                  */
    int pages;                   /* of the cache, >= 1                               */
    int table_len;               /* entries of a sequence's row of the table, >= 1, below 2^24 */
    void *data;                  /* device, [pages, Hkv, 2, 4096] bytes, 16-byte aligned */
    float *scales;               /* device, [pages, Hkv, 2], 8-byte aligned          */
    const int32_t *table;        /* device, [B, table_len]                           */
    int64_t table_stride_b;      /* entries between the table's rows                 */
    const int32_t *start;        /* device, [B], or NULL                             */
    const int32_t *count;        /* device, [B], or NULL                             */
} fibatt_cache;

/* Stores tokens: K, V Hkv heads of N rows.  A page's scale is the smallest power of two
 * whose 448th multiple reaches the largest finite value stored in that piece of
 * it, and a value becomes the nearest e4m3 multiple of it (ties to
 * even; infinities the largest, NaN stays NaN; at the scale of 2^120 finite values to 240 of
 * it at most, the largest multiple that bf16 and fp32 hold).  A call that begins a page sets its
 * scale anew; one that continues it (a first position that is not a multiple
 * of 64) raises the scale where its tokens need that, and rounds the page's older
 * tokens again, which changes only values below 2^-6 of the new scale; the
 * page's rows behind the call's tokens are left as they were.  No page may be stored
 * into twice in a call, by two sequences or by one whose table names it twice.  INVALID_ARG:
 * a size or stride out of its range, a NULL or misaligned pointer, 2^31 blocks (two a
 * page and head) or more.  UNSUPPORTED: D, dtype. */
fibatt_status fibatt_cache_store(const fibatt_cache *d, const fibatt_heads *K, const fibatt_heads *V,
                                 cudaStream_t stream);

/* Loads tokens into K, V: the values that the bytes stand for (exact in bf16
 * and fp32; infinite at 2^128 and beyond, which finite values are not stored as), zeros from count[b] on.  Errors as above. */
fibatt_status fibatt_cache_load(const fibatt_cache *d, const fibatt_heads *K, const fibatt_heads *V,
                                cudaStream_t stream);

/* Attention of the N tokens' queries (Hq heads, Hkv divides Hq) to the
 * cache, which holds their own keys already: a query at position p attends the
 * keys k <= p with k > p - window or k < sinks (window >= 1: one of 64 table_len or
 * more is all keys), as in fibatt_window_fwd; a query that count leaves out attends
 * none: O = 0, LSE = -inf.  Made for single tokens and a handful (up to 16 query rows
 * of a key head read its pages once, more read them again); a long prompt's own part is
 * fibatt_window_fwd's, on fibatt_cache_load's keys where the cache holds earlier ones.
 * Arithmetic: products of halves with fp32 sums (queries exact in bf16, 22 bits in fp32,
 * relative to their row's largest; weights 11 bits in bf16 I/O, 22 in fp32), O rounded
 * once; weights are held times up to 2^15, so that of n attended keys values above 2^112 / n may
 * give infinities.  What the pages hold behind the last token, or in
 * keys that no query attends, reaches no result (one that is not finite and is
 * attended may reach the other queries of its block of 16 rows).  Errors as above, and
 * INVALID_ARG for Hq, scale, window, sinks out of their range. */
fibatt_status fibatt_cache_fwd(const fibatt_cache *d, int Hq, float scale, int window, int sinks,
                               const fibatt_heads *Q, const fibatt_heads *O, float *LSE,
                               cudaStream_t stream);

/* Message for the last failing call on this thread ("" if none). */
const char *fibatt_last_error(void);

/* Library version string. */
const char *fibatt_version(void);

/* Device-side error word of the current device: bit 0 (1) is set when a
 * kernel gave up waiting for its shared-memory staging copies (a bounded wait
 * of about 2 s; the kernel then returns without writing its outputs); bit 1
 * (2) when a producer left before its last copies had landed (also after
 * about 2 s); bit 2 (4), in the bounds-checked debug build only (built with
 * -DFIBATT_CHECKS), when a kernel's bounds check failed and it skipped the
 * access (the first failing source line is then printed to stderr); bit 3
 * (8) when fibatt_qk_norm_fwd or _bwd met a position behind its tables; bit 4
 * (16) when a call on the 8-bit cache met a token without a page.
 * (fibatt_cross_fwd and _bwd, fibatt_window_fwd and _bwd and fibatt_cache_fwd may write outputs after bit 0 or 1: not to be
 * trusted.)  The word is the OR over every kernel file's copy.  This call synchronises with
 * the device.  With clear != 0 the word is reset.  CUDA on a failed copy. */
fibatt_status fibatt_device_error(int clear, unsigned *code);

/* Number of CUDA kernels this library has launched in this process so far
 * (all devices, all threads); for accounting in benchmarks and tests. */
uint64_t fibatt_launch_count(void);

#ifdef __cplusplus
}
#endif

#endif /* FIBATT_H_ */
