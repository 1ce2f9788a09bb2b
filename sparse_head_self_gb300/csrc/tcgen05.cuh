// The 5th-generation tensor cores in inline PTX (sm_103a): tensor memory,
// matrix instructions, their descriptors, and tiled tensor copies.
//
// Operand tiles are 64-element (128-byte) bf16 rows in shared memory, as the
// tensor copies leave them: rows 128 bytes apart, 16-byte chunks swizzled
// within each group of eight rows (the 128-byte pattern), tiles on 1024-byte
// boundaries.  A tile is read
//   along its rows ("K-major", both operands of Q K^T): a k-step of 16
//   elements starts 32 bytes further on;
//   across its rows ("MN-major", the V of P V: the rows are the summed
//   index): a k-step of 16 rows starts 2048 bytes further on.
// In both the groups of eight rows are 1024 bytes apart.
// The other operand of a product over rows (P, dS) is read from tensor
// memory: lane i, bf16 pair c in column c.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "tma_common.cuh"

namespace fibatt {

// ---- tensor memory ----------------------------------------------------------
// One warp allocates (the base address lands in shared memory) and, when no
// warp uses the columns any more, frees them.  An address: lane in the upper
// 16 bits, 32-bit column in the lower.
__device__ __forceinline__ void tmem_alloc(uint32_t *dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Around the barriers that order tensor-memory accesses of different threads.
__device__ __forceinline__ void tc_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 columns of the warp's 32 lanes (lane = thread): the lanes of warp w are
// 32 (w mod 4) and up.
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// After tmem_ld32: the values may be used.  The registers are operands, so that
// no use of them moves ahead of the wait; a further array of the same
// wait is pinned behind it by tmem_pin.
__device__ __forceinline__ void tmem_pin(uint32_t (&r)[32]) {
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                 "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]),
                 "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
                 "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    tmem_pin(r);
}

// Registers of the calling warp group (all of its warps call it): the blocks
// below are launched with the sum of their groups' shares.
template <int R>
__device__ __forceinline__ void take_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void give_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// mbar_wait (tma_common.cuh) for the short waits between the warps of a
// pipeline: polls without the suspend hint, whose wake-up costs more than such a
// wait.  Bounded in the same way.
__device__ __forceinline__ bool pipe_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    const uint32_t b = smem_u32(bar);
    unsigned long long t0 = 0;
    for (uint32_t i = 1;; ++i) {
        uint32_t done;
        asm volatile(
            "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
            : "=r"(done)
            : "r"(b), "r"(parity)
            : "memory");
        if (done) return true;
        if ((i & 63) != 1) continue;
        if (*abort) return false;
        const unsigned long long now = global_ns();
        if (t0 == 0) {
            t0 = now;
        } else if (now - t0 > kWaitLimitNs) {
            atomicOr(&g_device_error, kErrWaitTimeout);
            *abort = 1;
            return false;
        }
    }
}

// 16 columns.
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Whether the phase has completed, without waiting: asked for ahead of work whose
// end needs it, the answer costs nothing there.
__device__ __forceinline__ bool pipe_ready(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(done)
                 : "r"(smem_u32(bar)), "r"(parity)
                 : "memory");
    return done != 0;
}

// ---- descriptors --------------------------------------------------------------
// A swizzled tile at `p` (shared memory): start address in 16-byte units,
// 1024 bytes between groups of eight rows, version 1, 128-byte swizzle.  The
// leading offset is not used by tiles one swizzle pattern wide.
__device__ __forceinline__ uint64_t tile_desc(const void *p) {
    return (uint64_t)((smem_u32(p) & 0x3ffffu) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}
// A tile of 128 rows of 16 elements, one k-step wide, not swizzled: the rows'
// first eight elements (16 bytes each) one after another at `p`, their last eight
// at `last`, behind it.
__device__ __forceinline__ uint64_t narrow_desc(const void *p, const void *last) {
    return (uint64_t)((smem_u32(p) & 0x3ffffu) >> 4) | ((uint64_t)((smem_u32(last) - smem_u32(p)) >> 4) << 16) |
           ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
}
constexpr uint64_t kStepRowwise = 32 >> 4;     // 16 elements along the rows
constexpr uint64_t kStepAcross = 2048 >> 4;    // 16 rows

// Instruction descriptor: fp32 accumulator, bf16 operands, M x N; `across_b`:
// the second operand is read across its rows; `negate_a`: minus the first.
__host__ __device__ constexpr uint32_t mma_desc(uint32_t M, uint32_t N, bool across_b, bool negate_a = false) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((negate_a ? 1u : 0u) << 13) | ((across_b ? 1u : 0u) << 16) |
           ((N >> 3) << 17) | ((M >> 4) << 24);
}

// One lane of a converged warp.  Matrix instructions and copies are issued
// inside `if (elect_one())` from code that the whole warp runs, so that their
// descriptors are formed in uniform registers: from a branch on the lane number
// each instruction took about 100 cycles to issue.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
    return p != 0;
}
// The warp's number, the same register for the whole warp.
__device__ __forceinline__ int warp_number() { return __shfl_sync(kFullMask, (int)(threadIdx.x >> 5), 0); }

// ---- matrix instructions (one thread issues them) ------------------------------
// D (tensor memory) = A B or += A B, A and B from shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// The same with A from tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// `bar` gets an arrival when every matrix instruction issued so far by this
// thread has completed.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// ---- CTAs that have not started -----------------------------------------------------
// Strikes one of the grid's off, whose work the caller then has; the answer and 16
// bytes of the barrier's phase come when it is decided.  Not to be asked again once
// there was none.
__device__ __forceinline__ void draw_cta(uint4 *answer, uint64_t *bar) {
    mbar_expect_tx(bar, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(answer)),
                 "r"(smem_u32(bar))
                 : "memory");
}
// Its number along x, -1: there was none.
__device__ __forceinline__ int drawn_cta(const uint4 *answer) {
    int x;
    asm volatile(
        "{ .reg .b128 r; .reg .pred p; ld.shared.b128 r, [%1]; clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r; "
        "mov.b32 %0, -1; @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r; }"
        : "=r"(x)
        : "r"(smem_u32(answer))
        : "memory");
    return x;
}

// ---- tiled tensor copies -------------------------------------------------------
// A box of the 4-D tensor (element, row, head, sequence) to shared memory.
// The element coordinate is always 0; rows and heads behind the tensor's end
// arrive as zeros.
__device__ __forceinline__ void tile_load(void *dst, const CUtensorMap *map, int row, int head, int seq, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(0), "r"(row), "r"(head), "r"(seq), "r"(smem_u32(bar))
        : "memory");
}
// The box back to memory (rows behind the tensor's end are left out), as one of the
// thread's bulk operations; waits for its operations: until they have read shared
// memory, until they are complete.
__device__ __forceinline__ void tile_store(const CUtensorMap *map, int row, int head, int seq, const void *src) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(map), "r"(0),
                 "r"(row), "r"(head), "r"(seq), "r"(smem_u32(src))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// Plain writes to shared memory before it are seen by the tensor cores after.
__device__ __forceinline__ void fence_smem_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

}  // namespace fibatt
