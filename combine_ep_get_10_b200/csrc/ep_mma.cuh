// ep_mma.cuh -- device helpers of the kernels that multiply: asynchronous
// 16-byte copies, the warp's matrix product, the three-term bf16 form of an fp32
// operand, and the places of 16-byte chunks in operand tiles.
#pragma once

#include "ep_device.cuh"

namespace ep {

// 16 bytes global -> shared; `bytes` 0 writes zeros and reads nothing.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Arrives on `bar` when this thread's copies so far are done, without waiting
// for them.  Whoever waits on `bar` fences before the tensor core reads: a
// proxy fence of this thread's would wait for every copy it has in flight, the
// later stages' too.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void cp_async_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void cp_async_wait_all()
{
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// d += a (16 x 16, rows) * b (16 x 8, columns), bf16 operands, fp32 sums, by one
// warp from registers.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An fp32 pair as bf16 pairs t[0] + t[1] + t[2], exactly: each term is what the
// upper half of the word holds, 8 of the 24 significant bits, and the next one is
// taken from what is left (cut, not rounded: a rest of the value's own sign, never
// an infinity where the value is finite; below 2^-133 nothing is kept).  An
// infinite value leaves no rest (inf - inf).
__device__ __forceinline__ void split_bf16x2(float a, float b, uint32_t (&t)[3])
{
    t[0] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    a = fabsf(a) == INFINITY ? 0.0f : a - bf16_lo(t[0]);
    b = fabsf(b) == INFINITY ? 0.0f : b - bf16_hi(t[0]);
    t[1] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    a -= bf16_lo(t[1]);
    b -= bf16_hi(t[1]);
    t[2] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}

// Place of 16-byte chunk c of a row in a shared-memory tile of PC (a power of
// two) chunks a row, so that 8 consecutive rows of one chunk lie in different
// banks: what the 32-, 64- and 128-byte swizzles of tensor maps and of operand
// descriptors give.
template <int PC>
__device__ __forceinline__ uint32_t swizzled(int row, int c)
{
    const int f = PC >= 8 ? row & 7 : (row / (8 / PC)) & (PC - 1);
    return static_cast<uint32_t>(row * PC + (c ^ f)) * 16u;
}

} // namespace ep
