// Tensor-core plumbing of the tile kernels: mbarriers, TMA loads, tcgen05 instructions and descriptors.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "dr_device.cuh"

namespace dr {
namespace tc {

constexpr long long kWaitLimit = 4LL << 30;   // clock cycles (about 2 s)

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Bounded wait for the phase with the given parity; false on timeout, or soon after *gave_up is set by another wait.
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity, volatile int *gave_up) {
    const uint32_t a = smem_u32(bar);
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done) : "r"(a), "r"(parity) : "memory");
    if (done) return true;
    const long long t0 = clock64();
    while (true) {
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
            : "=r"(done) : "r"(a), "r"(parity) : "memory");
        if (done) return true;
        if (*gave_up) return false;
        if (clock64() - t0 > kWaitLimit) {
            *gave_up = 1;
            return false;
        }
    }
}

// A wait of its own limit, after another has run out: for copies and products that are in flight and end by themselves.
__device__ __forceinline__ void mbar_drain(uint64_t *bar, uint32_t parity) {
    const long long t0 = clock64();
    uint32_t done = 0;
    while (!done && clock64() - t0 <= kWaitLimit)
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
            : "=r"(done) : "r"(smem_u32(bar)), "r"(parity) : "memory");
}

// Whether the phase is over, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return done != 0;
}
// mbar_wait for two barriers: where both phases are over (the usual case) the two tests overlap.
__device__ __forceinline__ bool mbar_wait2(uint64_t *a, uint32_t pa, uint64_t *b, uint32_t pb, volatile int *gave_up) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p, q;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n and.pred p, p, q;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done) : "r"(smem_u32(a)), "r"(pa), "r"(smem_u32(b)), "r"(pb) : "memory");
    if (done) return true;
    return mbar_wait(a, pa, gave_up) && mbar_wait(b, pb, gave_up);
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// Shared-memory matrix descriptor of 128-byte rows with the 128-byte swizzle, 8-row groups 1024 bytes apart.  Rows are
// the M or N index of a K-major operand, or the K index of an MN-major one (one 64-element row wide, so the leading
// offset is not used).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
    return ((uint64_t)(addr & 0x3FFFFu) >> 4) | (1ull << 16) | ((1024ull >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// The same matrix `bytes` further on (a multiple of 16, within shared memory).
__device__ __forceinline__ uint64_t desc_at(uint64_t desc, uint32_t bytes) { return desc + (bytes >> 4); }
// kind::f16 instruction descriptor: fp32 sums, bf16 or f16 operands, A K-major, B K-major or (b_mn) MN-major.
__host__ __device__ constexpr uint32_t instr_desc(int M, int N, bool f16, bool b_mn) {
    return (1u << 4) | ((f16 ? 0u : 1u) << 7) | ((f16 ? 0u : 1u) << 10) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
// A operand in tensor memory
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(
            d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
// One lane of a converged warp, the same each time.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(e));
    return e != 0;
}
__device__ __forceinline__ void commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
// Pairs of CTAs of a cluster (cta_group::2).  The address of a place in the shared memory of the cluster's CTA `rank`:
__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// A copy into this CTA's shared memory that counts on a barrier of either CTA of the pair (a cluster address).
__device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
// Arrives on the barrier at this place in both CTAs (or those in the mask) once the products issued so far are over.
__device__ __forceinline__ void pair_commit(uint64_t *bar, uint16_t mask = 3) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(mask)
        : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

#define DR_TC_R8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), \
                       "=r"(r[o + 6]), "=r"(r[o + 7])
#define DR_TC_W8(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), \
                       "r"(r[o + 6]), "r"(r[o + 7])
// 32 consecutive 32-bit columns of the warp's 32 lanes (one lane per thread)
template <typename T>
__device__ __forceinline__ void ld32(uint32_t taddr, T *r) {
    uint32_t *q = reinterpret_cast<uint32_t *>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : DR_TC_R8(q, 0), DR_TC_R8(q, 8), DR_TC_R8(q, 16), DR_TC_R8(q, 24)
        : "r"(taddr));
}
// Loads that are waited for in the same statement.  To the compiler the outputs of a statement are there when it ends, so it may
// copy or spill them at once, most of all where they cross a loop's edge: registers of a load that is waited for later hold
// nothing yet.
#define DR_TC_E8(r, o) "=&r"(r[o]), "=&r"(r[o + 1]), "=&r"(r[o + 2]), "=&r"(r[o + 3]), "=&r"(r[o + 4]), "=&r"(r[o + 5]), \
                       "=&r"(r[o + 6]), "=&r"(r[o + 7])   // written before the statement's inputs were all read
template <typename T>
__device__ __forceinline__ void ld16_wait(uint32_t taddr, T *r) {
    uint32_t *q = reinterpret_cast<uint32_t *>(r);
    asm volatile(
        "{\n"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];\n"
        " tcgen05.wait::ld.sync.aligned;\n}"
        : DR_TC_E8(q, 0), DR_TC_E8(q, 8)
        : "r"(taddr)
        : "memory");
}
// The same of two places, one latency for both.
template <typename T>
__device__ __forceinline__ void ld16x2_wait(uint32_t at, T *r, uint32_t at2, T *r2) {
    uint32_t *q = reinterpret_cast<uint32_t *>(r), *q2 = reinterpret_cast<uint32_t *>(r2);
    asm volatile(
        "{\n"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%32];\n"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
        "%29, %30, %31}, [%33];\n"
        " tcgen05.wait::ld.sync.aligned;\n}"
        : DR_TC_E8(q, 0), DR_TC_E8(q, 8), DR_TC_E8(q2, 0), DR_TC_E8(q2, 8)
        : "r"(at), "r"(at2)
        : "memory");
}
template <typename T>
__device__ __forceinline__ void ld32_wait(uint32_t taddr, T *r) {
    uint32_t *q = reinterpret_cast<uint32_t *>(r);
    asm volatile(
        "{\n"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
        " tcgen05.wait::ld.sync.aligned;\n}"
        : DR_TC_E8(q, 0), DR_TC_E8(q, 8), DR_TC_E8(q, 16), DR_TC_E8(q, 24)
        : "r"(taddr)
        : "memory");
}
// The same of two places, one latency for both.
template <typename T>
__device__ __forceinline__ void ld32x2_wait(uint32_t at, T *r, uint32_t at2, T *r2) {
    uint32_t *q = reinterpret_cast<uint32_t *>(r), *q2 = reinterpret_cast<uint32_t *>(r2);
    asm volatile(
        "{\n"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, "
        "%45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%65];\n"
        " tcgen05.wait::ld.sync.aligned;\n}"
        : DR_TC_E8(q, 0), DR_TC_E8(q, 8), DR_TC_E8(q, 16), DR_TC_E8(q, 24), DR_TC_E8(q2, 0), DR_TC_E8(q2, 8),
          DR_TC_E8(q2, 16), DR_TC_E8(q2, 24)
        : "r"(at), "r"(at2)
        : "memory");
}
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Ties 32 registers to this point of the program: what reads them afterwards cannot move above a wait_ld before it.
#define DR_TC_P8(r, o) "+r"(r[o]), "+r"(r[o + 1]), "+r"(r[o + 2]), "+r"(r[o + 3]), "+r"(r[o + 4]), "+r"(r[o + 5]), \
                       "+r"(r[o + 6]), "+r"(r[o + 7])
template <typename T>
__device__ __forceinline__ void pin32(T *r) {
    uint32_t *q = reinterpret_cast<uint32_t *>(r);
    asm volatile("" : DR_TC_P8(q, 0), DR_TC_P8(q, 8));
    asm volatile("" : DR_TC_P8(q, 16), DR_TC_P8(q, 24));
}
template <typename T>
__device__ __forceinline__ void st32(uint32_t taddr, const T *r) {
    const uint32_t *q = reinterpret_cast<const uint32_t *>(r);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::DR_TC_W8(q, 0),
        DR_TC_W8(q, 8), DR_TC_W8(q, 16), DR_TC_W8(q, 24), "r"(taddr)
        : "memory");
}
// 16 columns
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t *q) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15};" ::DR_TC_W8(q, 0),
        DR_TC_W8(q, 8), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

}  // namespace tc
}  // namespace dr
