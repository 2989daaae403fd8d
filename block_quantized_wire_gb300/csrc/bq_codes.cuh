// What the kernels that multiply 4-bit codes share: bits picked from words of codes, the matrix
// instruction, words moved through shared memory.
#pragma once

#include "bq_rows.cuh"

namespace bqk {

// (w & mask) ^ x in one instruction
__device__ __forceinline__ uint32_t and_xor(uint32_t w, uint32_t mask, uint32_t x)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(w), "r"(mask), "r"(x));
    return r;
}

// c = a * b, or c += a * b: FP16 operands, binary32 sums.
template <bool kFirst>
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    if constexpr (kFirst)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%10, %10, %10, %10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------- shared memory
__device__ __forceinline__ uint32_t lds_u32(uint32_t a)
{
    uint32_t r;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
    return r;
}

__device__ __forceinline__ uint4 lds_v4(uint32_t a)
{
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "r"(a)
                 : "memory");
    return r;
}

__device__ __forceinline__ void lds_v2(uint32_t a, uint32_t &x, uint32_t &y)
{
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(a) : "memory");
}

// Copies `bytes` of kSize bytes and fills the rest with zeros.
template <int kSize>
__device__ __forceinline__ void lane_copy_part(uint32_t dst, const void *src, int bytes)
{
    if (bytes > 0 && !dbg_ok(src, bytes, false)) bytes = 0;
    if constexpr (kSize == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kSize), "r"(bytes)
                     : "memory");
}

}  // namespace bqk
