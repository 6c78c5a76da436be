// santa_tcgen05.cuh -- the fifth-generation tensor cores: products with operands in shared
// memory (descriptors) or tensor memory, accumulators in tensor memory.
#pragma once

#include "santa_common.cuh"

namespace santa {

// Shared-memory operand of 16-bit elements in the 128-byte swizzle that TMA writes: groups of
// 8 rows x 128 bytes (1024 bytes, 1024-byte aligned) `group_bytes` apart along the rows, blocks
// of 128 bytes of a row `block_bytes` apart (used where the row is the non-contracted dimension).
// (The address below 256 KB, so its 14 bits need no mask, and a step along the operand is an
// addition of step >> 4.)
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t block_bytes, uint32_t group_bytes) {
    const uint32_t low = (addr >> 4) + ((block_bytes >> 4) << 16);
    const uint32_t high = group_bytes >> 4 | 1u << 14 | 2u << 29;
    return uint64_t(high) << 32 | low;
}
// bf16 x bf16 -> fp32, M x N; b_rows: B's rows are the contracted dimension.
constexpr uint32_t mma_kind(int M, int N, bool b_rows) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (b_rows ? 1u << 16 : 0u) | uint32_t(N >> 3) << 17 | uint32_t(M >> 4) << 24;
}
// One lane of a converged warp, the same each time.  Products are issued by warps that run as one up to
// this choice: their operands are then uniform (in a lane's own branch every product took 110 cycles to
// issue, against 32 to 64 that it takes the tensor cores).
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
// D (tensor memory) = A B, or += with `add`; 16 elements of the contracted dimension.  One thread.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(kind), "r"(uint32_t(add))
        : "memory");
}
// The same with A in tensor memory: a lane per row, two elements per column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t kind, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(kind), "r"(uint32_t(add))
        : "memory");
}
// Arrives on `bar` when the products issued by this thread so far have completed.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
// Tensor memory: all 512 columns, one warp; the address lands in shared memory.
__device__ __forceinline__ void tmem_alloc(uint32_t *addr) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(addr)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void tc_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 16 columns of the warp's 32 lanes.  The values are there after tmem_wait, which takes them so
// that no use of them moves before it.
__device__ __forceinline__ void tmem_load16(uint32_t addr, float (&x)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]), "=f"(x[8]),
          "=f"(x[9]), "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15])
        : "r"(addr)
        : "memory");
}
// (No instruction: ties the values of other loads that a tmem_wait has waited for to the place behind it.)
__device__ __forceinline__ void tmem_arrived(float (&x)[16], float (&y)[16]) {
    asm volatile(""
                 : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7]),
                   "+f"(x[8]), "+f"(x[9]), "+f"(x[10]), "+f"(x[11]), "+f"(x[12]), "+f"(x[13]), "+f"(x[14]), "+f"(x[15]));
    asm volatile(""
                 : "+f"(y[0]), "+f"(y[1]), "+f"(y[2]), "+f"(y[3]), "+f"(y[4]), "+f"(y[5]), "+f"(y[6]), "+f"(y[7]),
                   "+f"(y[8]), "+f"(y[9]), "+f"(y[10]), "+f"(y[11]), "+f"(y[12]), "+f"(y[13]), "+f"(y[14]), "+f"(y[15]));
}
__device__ __forceinline__ void tmem_wait(float (&x)[16], float (&y)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    tmem_arrived(x, y);
}
// 8 columns of the warp's 32 lanes.
__device__ __forceinline__ void tmem_store8(uint32_t addr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

}  // namespace santa
