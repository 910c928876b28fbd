// ep_tcgen05.cuh -- the 5th-generation tensor core from one CTA: tensor memory,
// shared-memory operand descriptors, the matrix product of bf16 operands with
// fp32 sums, and its completion on an mbarrier.
#pragma once

#include "ep_device.cuh"

namespace ep {

// ------------------------------------------------------------ tensor memory
// One warp; `cols` a power of two of at least 32.  The address lands in *where
// (shared memory).
__device__ __forceinline__ void tmem_alloc(uint32_t* where, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}

// 16 consecutive columns of this warp's 32 lanes (a thread gets its lane's).
__device__ __forceinline__ void tmem_load16(float (&v)[16], uint32_t tmem)
{
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(tmem));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_store16(uint32_t tmem, const float (&v)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
                 "%13, %14, %15};" ::"r"(__float_as_uint(v[0])),
                 "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
                 "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])),
                 "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])),
                 "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])), "r"(__float_as_uint(v[12])),
                 "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15])), "r"(tmem)
                 : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_before_sync()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_after_sync()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// -------------------------------------------------------------- descriptors
// Operand tiles lie in shared memory in rows of 32, 64 or 128 bytes whose
// 16-byte chunks are exchanged by address bits 7.. (swizzled() of ep_mma.cuh).
//   K-major:  a row is one row (column) of the operand, 8 rows to a group,
//             `group` bytes from group to group; a step of 16 along the sum is 32
//             bytes along the row
//   MN-major: a row is one step of the sum, 8 steps to a group, `group` bytes
//             apart; `next` bytes to the rows that hold the following 16, 32 or 64
//             elements
// Tiles start on a multiple of 8 rows' bytes.
enum class Swizzle : uint32_t { k128 = 2, k64 = 4, k32 = 6 };

__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, Swizzle swizzle, uint32_t next, uint32_t group)
{
    return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | static_cast<uint64_t>((next >> 4) & 0x3fffu) << 16 |
           static_cast<uint64_t>((group >> 4) & 0x3fffu) << 32 | uint64_t{1} << 46 |
           static_cast<uint64_t>(swizzle) << 61;
}

// bf16 x bf16 -> fp32, M x N.
__host__ __device__ constexpr uint32_t product_desc(int M, int N, bool a_mn_major, bool b_mn_major)
{
    return 1u << 4 | 1u << 7 | 1u << 10 | (a_mn_major ? 1u << 15 : 0u) | (b_mn_major ? 1u << 16 : 0u) |
           static_cast<uint32_t>(N >> 3) << 17 | static_cast<uint32_t>(M >> 4) << 24;
}

// ------------------------------------------------------------------ product
// d (+)= a * b over 16 steps of the sum; one thread issues it.
__device__ __forceinline__ void tc_product(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(desc), "r"(accumulate ? 1u : 0u)
                 : "memory");
}

// Arrives on `bar` when the products issued by this thread so far are done.
__device__ __forceinline__ void tc_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

} // namespace ep
