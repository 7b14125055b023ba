// More inline-PTX wrappers for sm_100a, for kernels that are chains of small
// MMAs: waits that poll, MMA issue by an elected lane, plain bulk copies,
// stores to tensor memory, operands without swizzle.
#pragma once

#include "sm100.cuh"

namespace retnet {
namespace sm100 {

// As warp_wait, for waits of a few hundred cycles on a chain of hand-overs:
// every lane waits for itself (85 cycles a hand-over against warp_wait's 285,
// whose broadcast and clock reads cost as much as such a wait lasts), and
// only a wait that does not end is handed to warp_wait and its limit.
__device__ __forceinline__ bool warp_spin_wait(uint64_t *bar, uint32_t parity, volatile int *abort,
                                               unsigned *err) {
    bool ok = false;
    for (int i = 0; i < 1024 && !ok; ++i) ok = mbar_try_wait(bar, parity);
    if (__all_sync(0xffffffffu, ok)) return true;
    return warp_wait(bar, parity, abort, err);
}

// A named barrier of whole warps that tells all of them whether any warp
// brought `bad`, so that they leave a loop of barriers together.
__device__ __forceinline__ bool named_barrier_or(int id, int nthreads, bool bad) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)bad), "r"(id), "r"(nthreads)
        : "memory");
    return r != 0;
}

// Contiguous copy global -> shared; both addresses and the size are
// multiples of 16 bytes.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes,
                                          uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
        ::"r"(smem_u32(dst)), "l"((uint64_t)__cvta_generic_to_global(src)), "r"(bytes),
        "r"(smem_u32(bar))
        : "memory");
}
// Contiguous copy shared -> global, same rules.
__device__ __forceinline__ void bulk_store(void *dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                     (uint64_t)__cvta_generic_to_global(dst)),
                 "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}
// Registers -> 32 lanes x 16 consecutive 32-bit columns, as tmem_ld32.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(taddr)
        : "memory");
}
// 32 lanes x 16 consecutive 32-bit columns -> registers, as tmem_ld32.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// One lane of a converged warp, chosen by the hardware.  tcgen05.mma issued
// under this predicate takes its operands from uniform registers (about 10
// cycles an instruction); under `lane == 0` the compiler cannot tell that one
// thread issues and spends 175 (measured), more than a small MMA runs.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(p));
    return p != 0;
}
// A shared-memory matrix descriptor without swizzle, MN-major: 8 MN-elements (16 bytes) by 8 K-rows in
// 128 consecutive bytes, `lbo` between 8-row K groups and `sbo` between
// groups of 8 MN-elements.
__device__ __forceinline__ uint64_t smem_desc_plain(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)((lbo >> 4) & 0x3FFF) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFF) << 32) | ((uint64_t)1 << 46);
}

}  // namespace sm100
}  // namespace retnet
