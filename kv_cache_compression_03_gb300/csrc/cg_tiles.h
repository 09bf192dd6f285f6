// tcgen05: products of tiles in shared and tensor memory, and the waits of kernels whose warps have
// roles.
#pragma once

#include "cg_attention.h"

// ------------------------------------------------------------ instructions

// Descriptor of a shared-memory operand: K-major rows of 128 bytes, 128-byte
// swizzle, 8-row groups 1024 bytes apart. Only the low word, with the address,
// varies; it is passed as 32 bits, so that a product takes few registers over to
// the uniform file (what the issuing thread spends its time on).
constexpr uint32_t kDescHigh = 64u | 1u << 14 | 2u << 29;
// The same of rows of 64 bytes, 64-byte swizzle, groups of 8 rows 512 bytes apart.
constexpr uint32_t kDescHigh64 = 32u | 1u << 14 | 4u << 29;
__device__ __forceinline__ uint32_t smem_desc(uint32_t at) { return (at >> 4 & 0x3FFF) | 1u << 16; }

// bf16 x bf16 -> fp32, both operands K-major, M = 128.
__host__ __device__ constexpr uint32_t mma_desc(int n)
{
    return 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)(n >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
}

// kHigh: the descriptors' high word.
template <uint32_t kHigh = kDescHigh>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t desc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\t"
        "mov.b64 b, {%2, %5};\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(desc), "r"((uint32_t)add), "r"(kHigh)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t desc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(desc), "r"((uint32_t)add), "r"(kDescHigh)
        : "memory");
}

// One lane of the warp, chosen in a way that the compiler knows to be one lane:
// the branch that it takes then needs no care for others at each product.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one;
}

// The barrier is arrived on once all products issued so far are done.
__device__ __forceinline__ void mma_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ void tmem_fence_before()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tmem_fence_after()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of the warp's 32 lanes.
__device__ __forceinline__ void tmem_ld32(float *v, uint32_t at)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(at)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::
            "r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(at)
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t (&v)[16], uint32_t at)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(at)
        : "memory");
}

// Waits that end: false once this wait or another one of the block ran out. The role that
// gets false leaves for good: the other ones then wait for arrivals that do not come, until
// they leave too, and no barrier is ever taken for a phase that it is not in.
__device__ __forceinline__ bool wait_or_leave(uint64_t *bar, uint32_t parity, uint32_t *gave_up,
                                              void *status, bool at_once = false)
{
    const uint32_t at = smem_addr(bar);
    if (!at_once && (bar_poll(at, parity) || bar_wait_long(at, parity, gave_up)))
        return true;
    if (*reinterpret_cast<volatile uint32_t *>(gave_up))
        return false;
    *reinterpret_cast<volatile uint32_t *>(gave_up) = 1;
    int4_set_status(status, CG_ERR_TIMEOUT);
    return false;
}
