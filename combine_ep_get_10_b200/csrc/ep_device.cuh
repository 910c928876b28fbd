// ep_device.cuh -- device-side helpers shared by the sm_100a kernels:
// inline PTX for mbarriers, bulk (TMA engine) copies, non-coherent vector
// loads, streaming stores and the packed bf16 / e4m3 conversions.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "ep.h"

namespace ep {

constexpr uint32_t kFullMask = 0xffffffffu;

// Wall-clock bound on any device-side wait (ns).  A wait that runs out sets
// EP_DEVERR_TIMEOUT and returns; the data it guarded is skipped.
constexpr uint64_t kWaitLimitNs = 2000000000ull;

__device__ __forceinline__ uint32_t smem_addr(const void* p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ uint64_t global_timer_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ void flag_error(uint32_t* err, uint32_t bits)
{
    if (err != nullptr && bits != 0u)
        atomicOr(err, bits);
}

// ------------------------------------------- programmatic dependent launch
// A layout kernel lets the next kernel of the stream start early (when that
// one is launched with programmatic stream serialisation); the dispatch
// kernels issue their input-row loads first and wait for the layout's
// results here before reading them.  Without such a launch both are no-ops.
__device__ __forceinline__ void pdl_launch_dependents()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void pdl_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---------------------------------------------------------------- mbarrier
__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void fence_mbar_init()
{
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return done != 0u;
}

// Wait for phase `parity` of `bar` to complete, for at most kWaitLimitNs from
// the 256th look on (most waits end before, and never read the timer).
__device__ __forceinline__ bool mbar_wait_bounded(uint64_t* bar, uint32_t parity, uint32_t* err)
{
    uint64_t t0 = 0;
    for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
        if ((i & 255u) != 0u)
            continue;
        const uint64_t now = global_timer_ns();
        if (t0 == 0)
            t0 = now;
        if (now - t0 > kWaitLimitNs) {
            flag_error(err, EP_DEVERR_TIMEOUT);
            return false;
        }
    }
    return true;
}

// ------------------------------------------------------ bulk (TMA) copies
// global -> this CTA's shared memory; completes `bytes` of tx on `bar`.
// Addresses 16-byte aligned, bytes a multiple of 16.
__device__ __forceinline__ void bulk_load_g2s(void* dst_smem, const void* src, uint32_t bytes, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_addr(dst_smem)),
        "l"(src), "r"(bytes), "r"(smem_addr(bar))
        : "memory");
}

// shared -> global, tracked by the issuing thread's bulk async-groups.
__device__ __forceinline__ void bulk_store_s2g(void* dst, const void* src_smem, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_addr(src_smem)),
                 "r"(bytes)
                 : "memory");
}

// Order this thread's generic-proxy shared-memory writes before later
// async-proxy (bulk copy) reads of them.
__device__ __forceinline__ void fence_proxy_async_shared()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void bulk_commit()
{
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// All of this thread's bulk groups have finished reading shared memory.
__device__ __forceinline__ void bulk_wait_read_all()
{
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// ------------------------------------------------------------ plain memory
// Loads of the layout's results (slots, offsets, rank rows, counts) in the
// dispatch kernels.  A dispatch runs as a programmatic dependent of the
// kernel before it, and inside the library's one-call entry points that
// kernel is the layout, which lets the dispatch start at once: the
// dispatch's CTAs are then resident while the layout still writes these
// arrays.  After griddepcontrol.wait they are read through L2 (.cg), never
// through the read-only (.nc) path, which was measured returning stale
// values in exactly that situation.  (The combine kernels keep the
// read-only path: no kernel that lets its dependents start early is ever
// launched directly before a combine.)
template <typename T>
__device__ __forceinline__ T ld_meta(const T* p)
{
    return __ldcg(p);
}

__device__ __forceinline__ uint4 ld_nc_v4(const void* p)
{
    uint4 r;
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
        : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
        : "l"(p));
    return r;
}

// Loads that are not waited for before their value is used: predicated, zeros
// where `on` is false.  (A load in a branch is copied at the branch's end, and
// the copy, like any use, waits for it.)
__device__ __forceinline__ uint4 ld_nc_v4_if(const void* p, bool on)
{
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
                 "@p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                 : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w)
                 : "l"(p), "r"(on ? 1u : 0u));
    return r;
}

// The same of memory that the kernel writes too.
__device__ __forceinline__ uint4 ld_v4_if(const void* p, bool on)
{
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
                 "@p ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                 : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w)
                 : "l"(p), "r"(on ? 1u : 0u)
                 : "memory");
    return r;
}

__device__ __forceinline__ uint2 ld_nc_v2_if(const void* p, bool on)
{
    uint2 r = make_uint2(0u, 0u);
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\t"
                 "@p ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];\n\t}"
                 : "+r"(r.x), "+r"(r.y)
                 : "l"(p), "r"(on ? 1u : 0u));
    return r;
}

__device__ __forceinline__ uint32_t ld_nc_u32_if(const void* p, bool on)
{
    uint32_t r = 0u;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p ld.global.nc.u32 %0, [%1];\n\t}"
                 : "+r"(r)
                 : "l"(p), "r"(on ? 1u : 0u));
    return r;
}

// 32 bytes (256-bit load, sm_100) into two 16-byte halves; p 32-byte aligned.
__device__ __forceinline__ void ld_nc_v8(const void* p, uint4& lo, uint4& hi)
{
    asm("ld.global.nc.L1::no_allocate.v8.u32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(lo.x), "=r"(lo.y), "=r"(lo.z), "=r"(lo.w), "=r"(hi.x), "=r"(hi.y), "=r"(hi.z), "=r"(hi.w)
        : "l"(p));
}

__device__ __forceinline__ uint2 ld_nc_v2(const void* p)
{
    uint2 r;
    asm("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}

__device__ __forceinline__ void st_cs_v2(void* p, uint2 v)
{
    asm volatile("st.global.cs.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(v.x), "r"(v.y) : "memory");
}

__device__ __forceinline__ void st_cs_v4(void* p, uint4 v)
{
    asm volatile("st.global.cs.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

__device__ __forceinline__ void st_v4(void* p, uint4 v)
{
    asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

__device__ __forceinline__ void st_v2(void* p, uint2 v)
{
    asm volatile("st.global.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(v.x), "r"(v.y) : "memory");
}

// ------------------------------------------------------------ conversions
// bf16 pair packed in a 32-bit word: element 0 in the low half.
__device__ __forceinline__ float bf16_lo(uint32_t w)
{
    return __uint_as_float(w << 16);
}

__device__ __forceinline__ float bf16_hi(uint32_t w)
{
    return __uint_as_float(w & 0xffff0000u);
}

// Round two floats to bf16 (nearest, ties to even); `lo` lands in the low half.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two floats to e4m3 codes (nearest, ties to even, saturating to +-448);
// `lo` lands in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return static_cast<uint32_t>(r);
}

// Two floats to e5m2 codes (nearest, ties to even, saturating to +-57344);
// `lo` lands in the low byte.
__device__ __forceinline__ uint32_t pack_e5m2x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return static_cast<uint32_t>(r);
}

// Two floats to e2m1 codes (nearest, ties to even, saturating to +-6) in one
// byte; `lo` lands in the low nibble.
__device__ __forceinline__ uint32_t pack_e2m1x2(float lo, float hi)
{
    uint32_t r;
    asm("{\n\t.reg .b8 q;\n\tcvt.rn.satfinite.e2m1x2.f32 q, %1, %2;\n\tcvt.u32.u8 %0, q;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void sts_v2(void* p, uint2 v)
{
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(smem_addr(p)), "r"(v.x), "r"(v.y) : "memory");
}

__device__ __forceinline__ void sts_v4(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint4 lds_v4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ void st_u32(void* p, uint32_t v)
{
    asm volatile("st.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

} // namespace ep
