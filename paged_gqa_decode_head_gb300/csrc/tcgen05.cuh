// tcgen05.cuh -- wrappers of the fifth-generation tensor core (tcgen05) and
// tensor memory (TMEM) instructions used by libpgqa, as inline PTX.
//
// TMEM addresses: lane in bits 31..16, 32-bit column in bits 15..0. Warp w of
// a warpgroup reaches lanes 32 (w % 4) .. + 31 only.
#pragma once

#include "common.cuh"

namespace pgqa {

constexpr uint32_t kTmemColumns = 512; // all of an SM's tensor memory

// One whole warp allocates / frees all columns; the address lands in *slot.
__device__ __forceinline__ void tmem_alloc_all(uint32_t *slot)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)),
                 "r"(kTmemColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}

__device__ __forceinline__ void tmem_free_all(uint32_t base)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(kTmemColumns));
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Arrive once on `bar` when every tcgen05.mma this thread issued so far has completed.
__device__ __forceinline__ void tc_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// One lane of a converged warp (the same one every time).
__device__ __forceinline__ bool elect_one()
{
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}

// A value that is the same in every lane, marked as such for the compiler: the
// products' operands are uniform registers.
__device__ __forceinline__ uint32_t warp_uniform(uint32_t x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }

// Shared-memory operand descriptor, 128-byte swizzle. Low word: start address
// and leading byte offset, high word: stride byte offset (all in units of 16
// bytes), version 1 (bit 46), swizzle code 2 (bits 61-63).
__device__ __forceinline__ uint32_t tc_desc_low(uint32_t addr, uint32_t lead_bytes)
{
    return (addr >> 4) | lead_bytes >> 4 << 16;
}
__host__ __device__ constexpr uint32_t tc_desc_high(uint32_t stride_bytes) { return stride_bytes >> 4 | 1u << 14 | 2u << 29; }

// d (TMEM) (+)= A B, bf16 operands, fp32 accumulators. A and B by shared-memory
// descriptor (ss) or A in TMEM (ts). accumulate = 0 overwrites d.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint32_t a_low, uint32_t a_high, uint32_t b_low, uint32_t b_high,
                                          uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %6, 0;\n\t"
                 "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
                 "r"(a_low), "r"(a_high), "r"(b_low), "r"(b_high), "r"(idesc), "r"(accumulate)
                 : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint32_t b_low, uint32_t b_high, uint32_t idesc,
                                          uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\t"
                 "mov.b64 b, {%2, %3};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
                 "r"(a), "r"(b_low), "r"(b_high), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// Instruction descriptor of kind::f16 with bf16 A and B, fp32 D, M = 128:
// D format in bits 4-5, A and B formats in 7-9 and 10-12, negate A in 13,
// B "MN-major" (its N dimension contiguous) in 16, N / 8 in 17-22, M / 16 in 24-28.
__host__ __device__ constexpr uint32_t tc_idesc_bf16(uint32_t n, bool negate_a, bool b_mn_major)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((negate_a ? 1u : 0u) << 13) | ((b_mn_major ? 1u : 0u) << 16) |
           ((n >> 3) << 17) | ((128u >> 4) << 24);
}

// Tiled TMA load of a box of a 4-D or 3-D tensor map, default L2 policy for 3-D.
__device__ __forceinline__ void tma_load_4d(void *dst, const void *tmap, int x, int y, int z, int w, uint64_t *bar,
                                            uint64_t policy)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(smem_addr(dst)),
                 "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar)),
                 "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void tma_load_3d_default(void *dst, const void *tmap, int x, int y, int z, uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
                 "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
                 : "memory");
}

// 16 consecutive columns of this warp's 32 lanes <-> 16 registers per thread
// (register i: column i, the thread's own lane). A load's registers pass
// through its wait, so that no use of them moves ahead of it.
__device__ __forceinline__ void tmem_ld16(float *r, uint32_t addr)
{
    uint32_t *u = reinterpret_cast<uint32_t *>(r);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
                 : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_ld16(float *r)
{
    uint32_t *u = reinterpret_cast<uint32_t *>(r);
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(u[0]), "+r"(u[1]), "+r"(u[2]), "+r"(u[3]), "+r"(u[4]), "+r"(u[5]), "+r"(u[6]), "+r"(u[7]), "+r"(u[8]), "+r"(u[9]), "+r"(u[10]), "+r"(u[11]), "+r"(u[12]), "+r"(u[13]), "+r"(u[14]), "+r"(u[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const float *r)
{
    const uint32_t *u = reinterpret_cast<const uint32_t *>(r);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
                 "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
                 : "memory");
}

__device__ __forceinline__ float lds_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.volatile.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Two fp32 operations in one instruction (packed pairs).
struct f32x2 {
    uint64_t bits;
    __device__ __forceinline__ f32x2(float lo, float hi)
    {
        asm("mov.b64 %0, {%1, %2};" : "=l"(bits) : "f"(lo), "f"(hi));
    }
    __device__ __forceinline__ void get(float &lo, float &hi) const
    {
        asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(bits));
    }
};
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c)
{
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c.bits) : "l"(a.bits), "l"(b.bits));
    return c;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b)
{
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a.bits) : "l"(b.bits));
    return a;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(a.bits) : "l"(b.bits));
    return a;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

} // namespace pgqa
