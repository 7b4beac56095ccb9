// The tensor cores' instructions (tcgen05), TMA and cluster barriers, as the product kernels use
// them, and the host's tensor-map encoder.  Internal linkage: each kernel file compiles its own copy.
#pragma once

#include <cuda.h>

#include "device.cuh"

namespace fa {

namespace {

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// One lane of a converged warp.  In this form the compiler knows that a single thread goes
// on: the tensor-core and TMA instructions then take their operands from uniform registers
// directly (with `lane == 0` each MMA took some 290 cycles to issue).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

// Arrive on a barrier of any CTA of the cluster.  What it hands over is TMEM, which the tcgen05
// fences around it order; a release at cluster scope would wait for the thread's memory
// operations besides (the drain forms' main stall).
__device__ __forceinline__ void bar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

constexpr uint32_t kSuspendNs = 1000000;   // a try may sleep this long before it answers no
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(kSuspendNs)
        : "memory");
    return done;
}

// Wait for a phase.  What the barriers guard is read by the tensor cores or from TMEM, which the
// tcgen05 fences order, or came by TMA; no wider acquire is needed.  False where the cluster has
// given up (`gone` is set) or the wait has lasted kMaxWaitClocks (some 20 s): it then sets the
// flag of every CTA of the cluster, so that every role leaves.
constexpr long long kMaxWaitClocks = 40ll * 1000 * 1000 * 1000;
__device__ __forceinline__ void give_up(uint32_t gone, uint32_t ctas) {
    for (uint32_t r = 0; r < ctas; ++r)
        asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], 1;" ::"r"(ctas > 1 ? in_cta(gone, r) : gone) : "memory");
}

__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, uint32_t gone, uint32_t ctas) {
    long long t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (bar_try(bar, parity)) return true;
        uint32_t g;
        asm volatile("ld.relaxed.cluster.shared::cta.u32 %0, [%1];" : "=r"(g) : "r"(gone) : "memory");
        if (g) return false;
        if (t0 == 0) {
            t0 = clock64();
        } else if (clock64() - t0 > kMaxWaitClocks) {
            give_up(gone, ctas);
            return false;
        }
    }
}

template <int kCtas>
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                         uint32_t bar) {
    if constexpr (kCtas == 2)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
            " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
}

// Boxes of the output side, 2-D, 128-byte swizzle: x and y in elements and rows.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y),
                 "r"(src)
                 : "memory");
}

__device__ __forceinline__ uint4 ld_shared4u(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void st_shared4u(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// lo_a, lo_b: the descriptors' low words; `hi` is the high word of both.
template <int kCtas>
__device__ __forceinline__ void mma(uint32_t d, uint32_t lo_a, uint32_t lo_b, uint32_t hi, uint32_t idesc, bool add) {
    if constexpr (kCtas == 2)
        asm volatile(
            "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.u32 p, %5, 0;\n mov.b64 da, {%1, %3};\n"
            " mov.b64 db, {%2, %3};\n tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %4, p;\n}" ::"r"(d), "r"(lo_a),
            "r"(lo_b), "r"(hi), "r"(idesc), "r"(static_cast<uint32_t>(add))
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.u32 p, %5, 0;\n mov.b64 da, {%1, %3};\n"
            " mov.b64 db, {%2, %3};\n tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n}" ::"r"(d), "r"(lo_a),
            "r"(lo_b), "r"(hi), "r"(idesc), "r"(static_cast<uint32_t>(add))
            : "memory");
}

// Arrive on `bar` (the same offset in both CTAs of a pair) when the MMAs issued so far are done.
template <int kCtas>
__device__ __forceinline__ void commit(uint32_t bar) {
    if constexpr (kCtas == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                bar),
            "h"(static_cast<uint16_t>(3))
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

template <int kCtas>
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t cols) {
    if constexpr (kCtas == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}

template <int kCtas>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    if constexpr (kCtas == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}

// 16 columns of this warp's 32 lanes; the values are there after tmem_wait16.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(addr)
        : "memory");
}

// All loads of this warp have completed.  The values pass through, so that no use of them can
// be moved ahead of the wait.
__device__ __forceinline__ void tmem_wait16(float (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const float* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
        "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
        : "memory");
}

// Four floats at `addr` of CTA q's shared memory; parts == 1: this CTA's.
__device__ __forceinline__ float4 ld_part(uint32_t addr, uint32_t q, uint32_t parts) {
    float4 v;
    if (parts == 1)
        asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                     : "r"(addr)
                     : "memory");
    else
        asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                     : "r"(in_cta(addr, q))
                     : "memory");
    return v;
}

__device__ __forceinline__ float ld_part1(uint32_t addr, uint32_t q, uint32_t parts) {
    float v;
    if (parts == 1)
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    else
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(in_cta(addr, q)) : "memory");
    return v;
}

__device__ __forceinline__ void st_shared1(uint32_t addr, float a) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(a) : "memory");
}

__device__ __forceinline__ void st_shared4(uint32_t addr, float a, float b, float c, float d) {
    asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}

// Shared-memory operand descriptor, 128-byte swizzle (version 1 of the format, layout type 2).
// Summed index along the rows (K-major): groups of 8 rows are 1024 bytes apart.  Else
// (MN-major): slabs of 64 x-elements are 8192 bytes apart, groups of 8 summed rows 1024.  The
// address and the slab distance are in the low word.
constexpr uint32_t kDescHi = 1024 >> 4 | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t operand_desc_lo(uint32_t addr, bool kmajor) {
    return (addr & 0x3FFFF) >> 4 | (kmajor ? 1u : 8192u >> 4) << 16;
}

// Swizzled place of float4 `j` (0..7) of row `r` in a 32 x 32 unit: writes by row and reads
// of two adjacent float4 by four lanes of a row are both free of bank conflicts.
__device__ __forceinline__ uint32_t unit_at(uint32_t r, uint32_t j) { return r * 128 + ((j ^ (r & 7)) << 4); }

// ----------------------------------------------------------------- host
typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline cudaError_t tensor_map_encoder(EncodeTiled* out) {
    if (*out) return cudaSuccess;
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
    if (e == cudaSuccess && (q != cudaDriverEntryPointSuccess || !f)) e = cudaErrorNotSupported;
    if (e == cudaSuccess) *out = reinterpret_cast<EncodeTiled>(f);
    return e;
}

}  // namespace

}  // namespace fa
