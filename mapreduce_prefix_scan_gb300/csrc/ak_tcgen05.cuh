// ak_tcgen05.cuh -- sm_100a+ tensor-core building blocks in inline PTX:
// tensor memory (TMEM), shared-memory matrix descriptors and tcgen05.mma with
// bfloat16 operands and float32 accumulators, for one CTA (cta_group::1).
//
// Layouts used here. All operand tiles in shared memory are rows of 128 bytes
// (64 bfloat16) with the 128-byte swizzle, as TMA writes them:
//   K-major   the row index is M or N, the 64 values run along K: a step of
//             16 along K is 32 bytes; 8-row groups are 1024 bytes apart;
//   MN-major  the row index is K, the 64 values run along M or N: a step of
//             16 along K is 2048 bytes; the next 64 values of M or N are
//             `lbo` bytes away.
#pragma once

#include "ak_tma.cuh"

namespace ak {

// --------------------------------------------------------------------------
// tensor memory
// --------------------------------------------------------------------------

// One warp allocates `cols` columns (a power of two >= 32) and receives the
// address in shared memory; the same warp frees them.
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(cols)
                 : "memory");
    // the SM's next block may allocate
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
// Orders tcgen05 work before / after a thread synchronisation.
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Shared-memory writes of this thread become visible to the tensor core and TMA.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

#define AK_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define AK_W8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])

// 16 consecutive columns of this warp's 32 lanes (warp w of a warpgroup: lanes
// 32 w .. 32 w + 31): thread = lane, register = column. The registers hold
// the values only after tmem_wait_ld(r).
__device__ __forceinline__ void tmem_ld(uint32_t (&r)[16], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : AK_R8(r, 0), AK_R8(r, 8)
        : "r"(addr));
}
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        AK_W8(r, 0), AK_W8(r, 8)
        : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), AK_W8(r, 0) : "memory");
}
// Waits for this thread's TMEM loads; the registers pass through the
// statement so that no use of them moves in front of it.
#define AK_RW8(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : AK_RW8(r, 0), AK_RW8(r, 8)::"memory");
}
#undef AK_RW8
#undef AK_R8
#undef AK_W8

// --------------------------------------------------------------------------
// descriptors and products
// --------------------------------------------------------------------------

// Matrix descriptor of a 128-byte-swizzled tile at shared address `addr`
// (1024-byte aligned tile base plus a step along K). Field units: 16 bytes.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo) {
    return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: bf16 x bf16 -> f32, M x N, operand majors (true: MN).
constexpr uint32_t mma_idesc(int m, int n, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// D (+)= A B over 16 of K, A and B in shared memory. A whole warp executes
// this with equal arguments and the thread with `leader` set issues it: the
// code around stays uniform, so the operands live in uniform registers. (A
// branch around single-thread issue costs about 130 cycles a product in
// register moves, more than the product takes.)
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(leader)
        : "memory");
}
// The same with A in tensor memory: lane = row, two bf16 of K a column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(leader)
        : "memory");
}
// Arrives on `bar` once every product issued so far by the leader is done.
__device__ __forceinline__ void mma_commit(uint64_t* bar, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
        "r"(leader)
        : "memory");
}

}  // namespace ak
