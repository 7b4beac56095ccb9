// Products on the tensor cores (tcgen05): bf16 operands, fp32 accumulators in TMEM, operands
// staged in shared memory by TMA, the epilogue fused.
//
//   acc[x,y] = sum over pairs (i, j) of planes, sum over kk of P_i(x,kk) Q_j(y,kk)
//
// An operand is 1 plane (bf16 as it is) or 3 (an fp32 operand as the sum of three bf16 terms,
// 24 bits).  Of 3 x 3 planes the six products with i + j <= 2 are taken: the others are below
// 2^-25 of the largest.  Smaller products come first, so that they meet a small accumulator.
//
// A CTA's tile is 128 rows of P (TMEM lanes) by kBN rows of Q (TMEM columns); with kCtas == 2
// a pair of SMs holds 256 rows of P and each half of the Q rows (cta_group::2), which halves
// the operand traffic from L2.  The first warps (4, 8, or 16 in the 256-column forms) drain and
// finish tiles, the next issues TMA loads, the one after it the MMAs.  TMEM holds two
// accumulators, so the next tile's (or chunk's) products run while one is drained.
//
// kDrain: for fp32 results.  The tensor core's fp32 accumulation truncates: 4.4e-6 off over 4096
// terms (relative, 2-norm).  So the accumulator is emptied every 4 blocks of 64 terms into
// registers, which sum with rounding to nearest: 2.4e-7 (every 2 blocks 1.6e-7, every 8 4.8e-7,
// for 2 % of the time).  The products of planes other than the first two have an accumulator of
// their own, which is 2^-8 of the first and is read once a tile.
//
// kSwap: Q (columns) holds the tokens and P the weights -- for few tokens, where the 128 lanes
// are better filled with weights.  The output is then written column by column.
//
// splits > 1 (kCtas == 1): a cluster of `splits` CTAs divides the summed index; each puts its
// part into its own shared memory, and each finishes a share of the tile, summing the parts
// in rank order over distributed shared memory.
//
// What bounds it: the MMAs (measured peak 1954 TFLOP/s) and, before those, the operands' way
// from L2 -- a 256 x 256 tile reads 64 KB per 64 terms, 12 TB/s over all SMs -- and the epilogue
// of tiles with short sums.  Measured, calls queued one after the other:
//   4096 x 4864 x 16384 bf16                    380 us  1718 TFLOP/s  (88 %; 360 and 93 % in a CUDA graph)
//   4096 x 11008 x 4096 bf16, silu and pre      250 us  1480 TFLOP/s  (76 %; tensor pipe 73 % active)
//   1024 x 4096 x 32000 bf16 to fp32            188 us  1425 TFLOP/s  (73 %; 128 CTAs have a tile)
//   32000 x 4096 x 1024 bf16 to fp32            218 us  1231 TFLOP/s  (63 %; a 256 x 256 fp32 tile
//                                               written every 16 blocks, HBM writes 0.52 GB)
//   2056 x 1024 x 4096 bf16, bias, residual     18.9 us  912 TFLOP/s  (47 %: one wave, 4 us of launch)
//   1 x 32000 x 4096 bf16                       41 us   6.4 TB/s of weights (94 % of measured)
//   777 x 4096 x 1024 fp32, bias, gelu          47 us with the pass, 834 TFLOP/s of bf16 products
#include "product_tc.cuh"
#include "product_device.cuh"

namespace fa {

namespace {

constexpr int kBK = 64;                    // summed elements per block: 128 bytes, one swizzle row
// Drain warps: each has the 32 lanes of its quadrant (warp % 4) and a part of the columns.
// The epilogue is bound by instruction latency, so the pair kernel has 16 of them (with 8, the
// adapter merge of 4096 x 4096 took 29 us instead of 16 when this was chosen; with inputs from
// HBM it takes 18).
template <int kBN>
constexpr int kDrainWarps = kBN == 256 ? 16 : kBN >= 64 ? 8 : 4;
// Drain warps sharing a quadrant: a block of outputs by TMA is 64 columns wide, so that the
// 128 x 64 form has one, and half of its drain warps idle.
__host__ __device__ constexpr int drain_parts(int bn, bool swap) { return bn == 256 ? 4 : bn == 128 || (swap && bn == 64) ? 2 : 1; }
// The pair kernel's drain form holds 64 sums per thread: the last warpgroup (loads, MMAs, two
// idle warps) gives registers to the others.  128 x 56 + 512 x 104 <= 640 x 96, what the block
// is launched with.
template <int kBN, bool kDrain>
constexpr bool kRegSplit = kDrain && kBN == 256;
template <int kBN, bool kDrain>
constexpr int kThreads = (kDrainWarps<kBN> + (kRegSplit<kBN, kDrain> ? 4 : 2)) * 32;
constexpr uint32_t kPBytes = 128 * kBK * 2;
constexpr uint32_t kBiasRow = 64 * 4;     // a block's columns of the bias
constexpr uint32_t kUnit = 4096;           // a 32 x 32 block of fp32, or 32 rows x 128 bytes of outputs

// ----------------------------------------------------------------- PTX
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

// ----------------------------------------------------------------- epilogue
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Outputs by TMA: a drain warp's tile part is cut into blocks of 32 rows x 128 bytes, each in
// one of the warp's `slots` buffers.  Without `pre`, a block's residual is loaded into its
// buffer up to slots - 1 blocks ahead (so that HBM-bound products keep some 100 KB of loads in
// flight per SM), replaced by the output in place and stored from there.  With `pre`, the
// block is read from TMEM twice: for `pre`, then for the output, whose residual is read
// directly.
struct OutWarp {
    uint32_t buf, bar, slots;      // this warp's buffers and their load barriers
    uint32_t issued, block;        // loads issued; blocks finished
    uint32_t row_off, col_off;     // of the warp's part within the CTA's tile
    uint32_t blocks;               // per tile
    bool ahead;                    // residuals come by TMA
    TcWalk walk;                   // of the loads
    uint32_t at_tile, at_block, load_slot;    // the next load's
};

template <int kCtas, int kBN>
__device__ __forceinline__ void load_ahead(const TcArgs& a, OutWarp& o, uint32_t upto, uint32_t step, uint32_t width,
                                           uint32_t rank) {
    for (; o.issued < upto && o.at_tile < a.tiles; ++o.issued) {
        const TcTile tile = o.walk.at(a, o.at_tile);
        const uint32_t row = tile.p * 128 * kCtas + (kCtas == 2 ? rank * 128 : 0) + o.row_off;
        const uint32_t col = tile.q * kBN + o.col_off + o.at_block * width;
        const uint32_t s = o.load_slot;
        if (++o.load_slot == o.slots) o.load_slot = 0;
        if (++o.at_block == o.blocks) {
            o.at_block = 0;
            o.at_tile += step;
        }
        // a block outside the output is all zeros: in range for a load
        mbar_expect(o.bar + 8 * s, kUnit);
        tma_load_2d(o.buf + s * kUnit, &a.map_res, col, row, o.bar + 8 * s);
    }
}

// 16 columns of one row (this lane's), sums in v, to the row's 16-byte pieces piece0, ... of
// the output's buffer, which holds the residual there if res_here.  bias: the columns' floats
// in shared memory.  In stages over the 16 values, each stage's choice made once: the code has
// to be small, since a launch starts with a cold instruction cache.
template <bool kBf16>
__device__ __forceinline__ void store_row(uint32_t at, uint32_t piece0, const float (&v)[16]) {
    const uint32_t lane = threadIdx.x % 32;
    if constexpr (kBf16) {
#pragma unroll
        for (int p = 0; p < 2; ++p)
            st_shared4u(at + unit_at(lane, piece0 + p), pack2(v[8 * p], v[8 * p + 1]), pack2(v[8 * p + 2], v[8 * p + 3]),
                        pack2(v[8 * p + 4], v[8 * p + 5]), pack2(v[8 * p + 6], v[8 * p + 7]));
    } else {
#pragma unroll
        for (int p = 0; p < 4; ++p)
            st_shared4(at + unit_at(lane, piece0 + p), v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]);
    }
}

template <int kN>
__device__ __forceinline__ void activate(int act, float (&v)[kN]) {
    if (act == kActRelu) {
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = act_fwd(kActRelu, v[i]);
    } else if (act == kActGelu) {
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = act_fwd(kActGelu, v[i]);
    } else if (act == kActSilu) {
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = act_fwd(kActSilu, v[i]);
    }
}

__device__ __forceinline__ void finish_row(const TcArgs& a, float (&v)[16], uint32_t bias, uint32_t out, uint32_t piece0,
                                           uint32_t row, uint32_t col, bool res_here, bool pre) {
    const uint32_t lane = threadIdx.x % 32;
    const ProdEpilogue& e = a.e;
    const bool bf16 = e.out_dtype != 0;
    if (e.bias) {
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const uint4 b = ld_shared4u(bias + i * 4);
            v[i] = fmaf(e.alpha, v[i], __uint_as_float(b.x));
            v[i + 1] = fmaf(e.alpha, v[i + 1], __uint_as_float(b.y));
            v[i + 2] = fmaf(e.alpha, v[i + 2], __uint_as_float(b.z));
            v[i + 3] = fmaf(e.alpha, v[i + 3], __uint_as_float(b.w));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] *= e.alpha;
    }
    if (!pre) {
    activate(e.act, v);
    if (e.res) {
        if (!res_here) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (row < a.rows && col + i < a.cols)
                    v[i] = fmaf(e.beta, elem(e.res, row * e.ldr + col + i, e.out_dtype), v[i]);
        } else if (bf16) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint4 q = ld_shared4u(out + unit_at(lane, piece0 + p));
                v[8 * p] = fmaf(e.beta, bf16_lo(q.x), v[8 * p]);
                v[8 * p + 1] = fmaf(e.beta, bf16_hi(q.x), v[8 * p + 1]);
                v[8 * p + 2] = fmaf(e.beta, bf16_lo(q.y), v[8 * p + 2]);
                v[8 * p + 3] = fmaf(e.beta, bf16_hi(q.y), v[8 * p + 3]);
                v[8 * p + 4] = fmaf(e.beta, bf16_lo(q.z), v[8 * p + 4]);
                v[8 * p + 5] = fmaf(e.beta, bf16_hi(q.z), v[8 * p + 5]);
                v[8 * p + 6] = fmaf(e.beta, bf16_lo(q.w), v[8 * p + 6]);
                v[8 * p + 7] = fmaf(e.beta, bf16_hi(q.w), v[8 * p + 7]);
            }
        } else {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint4 q = ld_shared4u(out + unit_at(lane, piece0 + p));
                v[4 * p] = fmaf(e.beta, __uint_as_float(q.x), v[4 * p]);
                v[4 * p + 1] = fmaf(e.beta, __uint_as_float(q.y), v[4 * p + 1]);
                v[4 * p + 2] = fmaf(e.beta, __uint_as_float(q.z), v[4 * p + 2]);
                v[4 * p + 3] = fmaf(e.beta, __uint_as_float(q.w), v[4 * p + 3]);
            }
        }
    }
    }
    if (bf16)
        store_row<true>(out, piece0, v);
    else
        store_row<false>(out, piece0, v);
}

// Eight output elements of one row from a unit: lane = columns 8 (lane % 4) of row
// lane / 4 + 8 `part`.  `parts` CTAs hold a share of the sums (1: this CTA's shared memory).
__device__ __forceinline__ void finish_item(const TcArgs& a, uint32_t unit, uint32_t part, uint32_t parts, uint32_t row0,
                                            uint32_t col0) {
    const uint32_t lane = threadIdx.x % 32, r = lane / 4 + 8 * part, j = (lane % 4) * 2;
    const uint32_t row = row0 + r, c = col0 + j * 4;
    if (row >= a.rows || c >= a.cols) return;
    const ProdEpilogue& e = a.e;
    const bool vec = c + 8 <= a.cols, bf16 = e.out_dtype != 0;
    float res[8] = {}, v[8] = {};
    if (e.res) {
        const uint64_t at = row * e.ldr + c;
        if (vec && bf16)
            plain_vec8(static_cast<const uint16_t*>(e.res) + at, res);
        else if (vec)
            plain_vec8(static_cast<const float*>(e.res) + at, res);
        else
            for (int i = 0; i < 8; ++i)
                if (c + i < a.cols) res[i] = elem(e.res, at + i, e.out_dtype);
    }
    float bias[8] = {};
    if (e.bias)
        for (int i = 0; i < 8; ++i)
            if (c + i < a.cols) bias[i] = elem(e.bias, c + i, e.bias_dtype);
    for (uint32_t q = 0; q < parts; ++q) {
        const float4 x = ld_part(unit + unit_at(r, j), q, parts), y = ld_part(unit + unit_at(r, j + 1), q, parts);
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
    }
    const uint64_t at = row * e.ldo + c;
    auto write = [&](void* p) {
        if (vec && bf16)
            store8_global<uint16_t>(p, at, v);
        else if (vec)
            store8_global<float>(p, at, v);
        else
            for (int i = 0; i < 8; ++i)
                if (c + i < a.cols) put(p, at + i, e.out_dtype, v[i]);
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf(e.alpha, v[i], bias[i]);
    if (e.pre) write(e.pre);
    activate(e.act, v);
    if (e.res)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fmaf(e.beta, res[i], v[i]);
    write(e.out);
}

// The same eight rows where outputs are not 16-byte aligned: a lane has kG adjacent columns (as
// many as its stores can be aligned for, a.grain), and a store of the warp covers kG rows.
template <int kG>
__device__ __forceinline__ void finish_rows(const TcArgs& a, uint32_t unit, uint32_t part, uint32_t parts, uint32_t row0,
                                            uint32_t col0) {
    constexpr uint32_t kLanes = 32 / kG, kSteps = 8 / kG;
    const uint32_t lane = threadIdx.x % 32, j0 = lane % kLanes * kG, c = col0 + j0, r0 = 8 * part + lane / kLanes;
    if (c >= a.cols) return;
    const ProdEpilogue& e = a.e;
    const bool whole = c + kG <= a.cols;
    float bias[kG] = {}, res[8] = {}, v[8] = {};
#pragma unroll
    for (int g = 0; g < kG; ++g)
        if (e.bias && c + g < a.cols) bias[g] = elem(e.bias, c + g, e.bias_dtype);
    if (e.res)
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const uint64_t at = (row0 + r0 + i * kG) * e.ldr + c;
            if (row0 + r0 + i * kG >= a.rows) break;
            if (kG == 4 && whole && e.out_dtype) {
                const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(e.res) + at);
                res[i * kG] = bf16_lo(q.x);
                res[i * kG + 1 % kG] = bf16_hi(q.x);
                res[i * kG + 2 % kG] = bf16_lo(q.y);
                res[i * kG + 3 % kG] = bf16_hi(q.y);
            } else {
#pragma unroll
                for (int g = 0; g < kG; ++g)
                    if (c + g < a.cols) res[i * kG + g] = elem(e.res, at + g, e.out_dtype);
            }
        }
    for (uint32_t q = 0; q < parts; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t r = r0 + i / kG * kG, j = j0 + i % kG;
            v[i] += ld_part1(unit + unit_at(r, j / 4) + j % 4 * 4, q, parts);
        }
    const auto write = [&](void* p) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            if (row0 + r0 + i * kG >= a.rows) break;
            const uint64_t at = (row0 + r0 + i * kG) * e.ldo + c;
            const float* x = &v[i * kG];
            if (kG == 4 && whole) {                      // bf16 (16-byte aligned fp32 is not for here)
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + at) = make_uint2(pack2(x[0], x[1 % kG]), pack2(x[2 % kG], x[3 % kG]));
            } else if (kG == 2 && whole && e.out_dtype) {
                *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p) + at) = pack2(x[0], x[1 % kG]);
            } else if (kG == 2 && whole) {
                *reinterpret_cast<float2*>(static_cast<float*>(p) + at) = make_float2(x[0], x[1 % kG]);
            } else {
#pragma unroll
                for (int g = 0; g < kG; ++g)
                    if (c + g < a.cols) put(p, at + g, e.out_dtype, x[g]);
            }
        }
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf(e.alpha, v[i], bias[i % kG]);
    if (e.pre) write(e.pre);
    activate(e.act, v);
    if (e.res)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fmaf(e.beta, res[i], v[i]);
    write(e.out);
}

__device__ __forceinline__ void finish_any(const TcArgs& a, uint32_t unit, uint32_t part, uint32_t parts, uint32_t row0,
                                           uint32_t col0) {
    if (a.vec)
        finish_item(a, unit, part, parts, row0, col0);
    else if (a.grain == 4)
        finish_rows<4>(a, unit, part, parts, row0, col0);
    else if (a.grain == 2)
        finish_rows<2>(a, unit, part, parts, row0, col0);
    else
        finish_rows<1>(a, unit, part, parts, row0, col0);
}

// kSwap: lane = one output column (P row); four output rows, columns 4 `part` of the unit.
__device__ __forceinline__ void finish_item_swapped(const TcArgs& a, uint32_t unit, uint32_t part, uint32_t parts,
                                                    uint32_t prow0, uint32_t qrow0) {
    const uint32_t lane = threadIdx.x % 32, col = prow0 + lane, row0 = qrow0 + part * 4;
    if (col >= a.cols || row0 >= a.rows) return;
    const ProdEpilogue& e = a.e;
    const float bias = e.bias ? elem(e.bias, col, e.bias_dtype) : 0.0f;
    float res[4] = {}, v[4] = {};
    if (e.res)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (row0 + i < a.rows) res[i] = elem(e.res, (row0 + i) * e.ldr + col, e.out_dtype);
    for (uint32_t q = 0; q < parts; ++q) {
        const float4 x = ld_part(unit + unit_at(lane, part), q, parts);
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
    }
    auto write = [&](void* p) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (row0 + i < a.rows) put(p, (row0 + i) * e.ldo + col, e.out_dtype, v[i]);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fmaf(e.alpha, v[i], bias);
    if (e.pre) write(e.pre);
    activate(e.act, v);
    if (e.res)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fmaf(e.beta, res[i], v[i]);
    write(e.out);
}

// ----------------------------------------------------------------- kernel
template <int kCtas, int kBN, bool kDrain, bool kSwap>
__global__ void __launch_bounds__((kThreads<kBN, kDrain>), 1) product_tc_kernel(const __grid_constant__ TcArgs a) {
    constexpr int kQRows = kBN / kCtas;                     // rows of Q that this CTA loads
    constexpr uint32_t kQBytes = kQRows * kBK * 2;
    constexpr int kWarps = kDrainWarps<kBN>, kLoadWarp = kWarps, kMmaWarp = kWarps + 1;
    constexpr int kHalves = drain_parts(kBN, kSwap);
    constexpr int kHalf = kBN / kHalves;                            // columns of each
    constexpr int kUnitCols = kHalf < 32 ? kHalf : 32;      // of a unit of the split exchange
    constexpr int kPieces = kHalf / 16;                     // 16 columns at a time
    // two accumulators; the drain forms of up to 128 columns a third, for the small products
    constexpr uint32_t kTmemWant = kDrain && kBN <= 128 ? 3 * kBN : 2 * kBN;
    constexpr uint32_t kTmemCols = kTmemWant <= 32 ? 32 : kTmemWant <= 64 ? 64 : kTmemWant <= 128 ? 128 : kTmemWant <= 256 ? 256 : 512;
    extern __shared__ __align__(1024) uint8_t dyn[];     // stages, output buffers, bias rows
    __shared__ uint64_t bars[2 * kTcMaxStages + 5 + kWarps * kTcMaxSlots];
    __shared__ uint32_t tmem_slot, gone_flag;
    const uint32_t base = smem_addr(dyn);
    const uint32_t full = smem_addr(&bars[0]), empty = smem_addr(&bars[kTcMaxStages]);
    const uint32_t acc_full = smem_addr(&bars[2 * kTcMaxStages]), acc_empty = acc_full + 16;
    const uint32_t small_empty = acc_full + 32, res_bars = acc_full + 40;
    const bool split_planes = a.planes_p + a.planes_q > 2;
    const uint32_t plane_p = a.sub * kPBytes, plane_q = a.sub * kQBytes;      // of a stage
    const uint32_t stage_bytes = a.planes_p * plane_p + a.planes_q * plane_q;
    const uint32_t warp = __shfl_sync(~0u, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const uint32_t rank = kCtas == 2 || a.splits > 1 ? cluster_rank() : 0;
    const uint32_t split = kCtas == 2 ? 0 : rank;
    const bool leader = kCtas == 1 || rank == 0;
    const uint32_t gone = smem_addr(&gone_flag), ctas = kCtas == 2 ? 2 : a.splits;

    // The next kernel on the stream may set itself up while this one runs; it, as this one,
    // waits for its predecessor's end before it touches global memory.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 0 && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&a.map_p) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&a.map_q) : "memory");
    }
    if (warp == kLoadWarp && lane == 0) {
        for (uint32_t s = 0; s < a.stages; ++s) {
            bar_init(full + 8 * s, 1);
            bar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(acc_full + 8 * b, 1);
            bar_init(acc_empty + 8 * b, kCtas * kHalves * 4);
        }
        bar_init(small_empty, kCtas * kHalves * 4);
        for (uint32_t i = 0; i < kWarps * kTcMaxSlots; ++i) bar_init(res_bars + 8 * i, 1);
        gone_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc<kCtas>(smem_addr(&tmem_slot), kTmemCols);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (kCtas == 2 || a.splits > 1) cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_slot;
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // this cluster's tiles, and this CTA's blocks of the summed index
    const uint32_t group = kCtas == 2 ? 2 : a.splits;
    const uint32_t first = blockIdx.x / group, step = gridDim.x / group;
    const uint32_t kb0 = static_cast<uint64_t>(a.kblocks) * split / a.splits;
    const uint32_t kb1 = static_cast<uint64_t>(a.kblocks) * (split + 1) / a.splits;
    bool ok = true;                      // of this thread: no wait gave up

    if (warp >= kWarps) {
        if constexpr (kRegSplit<kBN, kDrain>) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == kLoadWarp && elect_one()) {
            const uint32_t lead_full = kCtas == 2 ? in_cta(full, 0) : full;
            // the parameters in registers: the asm statements' memory clobbers would have them
            // loaded again for every block, and this thread's latency sets the pace of short tiles
            const bool pk = a.p_kmajor, qk = a.q_kmajor, plain = a.planes_p + a.planes_q == 2;
            const uint32_t sub = a.sub, stages = a.stages, terms = a.k, np = a.planes_p, nq = a.planes_q;
            const uint32_t block_bytes = stage_bytes / sub * kCtas, at_q = base + np * plane_p;
            const CUtensorMap *mp = &a.map_p, *mq = &a.map_q;
            const auto load_p = [&](uint32_t dst, uint32_t k, uint32_t p0, uint32_t z, uint32_t bar) {
                if (pk) {
                    tma_load<kCtas>(dst, mp, k, p0, z, bar);
                } else {
                    tma_load<kCtas>(dst, mp, p0, k, z, bar);
                    tma_load<kCtas>(dst + 8192, mp, p0 + 64, k, z, bar);
                }
            };
            const auto load_q = [&](uint32_t dst, uint32_t k, uint32_t q0, uint32_t z, uint32_t bar) {
                if (qk)
                    tma_load<kCtas>(dst, mq, k, q0, z, bar);
                else
#pragma unroll
                    for (int h = 0; h < kQRows / 64; ++h) tma_load<kCtas>(dst + h * 8192, mq, q0 + 64 * h, k, z, bar);
            };
            uint32_t s = 0, phase = 1;          // the first round of stages is free
            TcWalk walk;
            for (uint32_t t = first; ok && t < a.tiles; t += step) {
                const TcTile tile = walk.at(a, t);
                const uint32_t p0 = tile.p * 128 * kCtas + (kCtas == 2 ? rank * 128 : 0);
                const uint32_t q0 = tile.q * kBN + (kCtas == 2 ? rank * kQRows : 0);
                for (uint32_t kb = kb0; kb < kb1; ++kb) {
                    const uint32_t k0 = kb * sub * kBK, bar = lead_full + 8 * s, off = s * stage_bytes;
                    const bool second = sub == 2 && terms - k0 > kBK;
                    if (!bar_wait(empty + 8 * s, phase, gone, ctas)) {
                        ok = false;
                        break;
                    }
                    if (leader) mbar_expect(full + 8 * s, second ? 2 * block_bytes : block_bytes);
                    if (plain) {
                        load_p(base + off, k0, p0, 0, bar);
                        load_q(at_q + off, k0, q0, 0, bar);
                        if (second) {
                            load_p(base + off + kPBytes, k0 + kBK, p0, 0, bar);
                            load_q(at_q + off + kQBytes, k0 + kBK, q0, 0, bar);
                        }
                    } else {
                        for (uint32_t z = 0; z < np; ++z) load_p(base + off + z * plane_p, k0, p0, z, bar);
                        for (uint32_t z = 0; z < nq; ++z) load_q(at_q + off + z * plane_q, k0, q0, z, bar);
                    }
                    if (++s == stages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
        } else if (warp == kMmaWarp && leader && elect_one()) {
            const uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | (a.p_kmajor ? 0u : 1u << 15) |
                                   (a.q_kmajor ? 0u : 1u << 16) | (kBN / 8) << 17 | (128 * kCtas / 16) << 24;
            const uint32_t step_p = a.p_kmajor ? 32 >> 4 : 2048 >> 4, step_q = a.q_kmajor ? 32 >> 4 : 2048 >> 4;
            const uint32_t desc_p = operand_desc_lo(base, a.p_kmajor);
            const uint32_t desc_q = operand_desc_lo(base + a.planes_p * plane_p, a.q_kmajor);
            const uint32_t small = tmem + 2 * kBN;
            const bool plain = a.planes_p + a.planes_q == 2;
            const uint32_t sub = a.sub, stages = a.stages, terms = a.k, np = a.planes_p, nq = a.planes_q, chunk = a.chunk_kb;
            bool add_small = false;
            uint32_t it = 0, ch = 0, s = 0, phase = 0;      // it: blocks so far; s, phase: its stage
            uint32_t n_tile = 0;
            for (uint32_t t = first; ok && t < a.tiles; t += step, ++n_tile) {
                for (uint32_t kb = kb0; ok && kb < kb1; ++ch) {
                    const uint32_t b = ch & 1;
                    if (ch >= 2 && !bar_wait(acc_empty + 8 * b, (ch / 2 - 1) & 1, gone, ctas)) {
                        ok = false;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    if (kDrain && split_planes && kb == kb0 && t != first &&
                        !bar_wait(small_empty, (n_tile - 1) & 1, gone, ctas)) {
                        ok = false;
                        break;
                    }
                    const uint32_t d = tmem + b * kBN;
                    const uint32_t end = kDrain && kb1 - kb > chunk ? kb + chunk : kb1;
                    bool add = false;
                    if (kb == kb0) add_small = false;
                    for (; kb < end; ++kb, ++it) {
                        const bool second = sub == 2 && terms - kb * 2 * kBK > kBK;
                        // descriptors before the wait: the issuing thread's own latency counts
                        const uint32_t dp = desc_p + (s * stage_bytes >> 4), dq = desc_q + (s * stage_bytes >> 4);
                        uint32_t lp[kBK / 16], lq[kBK / 16];
#pragma unroll
                        for (uint32_t x = 0; x < kBK / 16; ++x) {
                            lp[x] = dp + x * step_p;
                            lq[x] = dq + x * step_q;
                        }
                        if (a.test_expire || !bar_wait(full + 8 * s, phase, gone, ctas)) {
                            ok = false;
                            break;
                        }
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        // all four steps of 16 terms: what lies past the sum's end is zeros
                        if (plain) {
#pragma unroll
                            for (uint32_t x = 0; x < kBK / 16; ++x)
                                mma<kCtas>(d, lp[x], lq[x], kDescHi, idesc, add || x > 0);
                            if (second)
#pragma unroll
                                for (uint32_t x = 0; x < kBK / 16; ++x)
                                    mma<kCtas>(d, lp[x] + (kPBytes >> 4), lq[x] + (kQBytes >> 4), kDescHi, idesc, true);
                        } else {
                            for (uint32_t pair = 0; pair < 6; ++pair) {       // planes: one block per stage
                                // (i, j): 2 0, 1 1, 0 2, 1 0, 0 1, 0 0
                                const uint32_t i = 0x001012 >> (pair * 4) & 3, j = 0x010210 >> (pair * 4) & 3;
                                if (i >= np || j >= nq) continue;
                                const bool main = !kDrain || pair == 5;      // see kDrain above
                                const uint32_t op = i * plane_p >> 4, oq = j * plane_q >> 4;
#pragma unroll
                                for (uint32_t x = 0; x < kBK / 16; ++x)
                                    mma<kCtas>(main ? d : small, lp[x] + op, lq[x] + oq, kDescHi, idesc,
                                               (main ? add : add_small) || x > 0);
                                if (main)
                                    add = true;
                                else
                                    add_small = true;
                            }
                        }
                        add = true;
                        commit<kCtas>(empty + 8 * s);
                        if (++s == stages) {
                            s = 0;
                            phase ^= 1;
                        }
                    }
                    if (ok) commit<kCtas>(acc_full + 8 * b);
                }
            }
            if (!ok) {
                // the loads in flight land before the CTA leaves
                atomicOr(a.err, kErrWaitTimeout);
                give_up(gone, ctas);
                const uint32_t blocks = (kb1 - kb0) * ((a.tiles - first + step - 1) / step);
                for (uint32_t n = 0; n < a.stages && it < blocks; ++n, ++it) {
                    for (uint32_t i = 0; i < 1000 && !bar_try(full + 8 * (it % a.stages), (it / a.stages) & 1); ++i) {}
                }
            }
        }
        __syncwarp();
    } else if (warp / 4 < kHalves) {
        if constexpr (kRegSplit<kBN, kDrain>) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        const uint32_t quad = warp % 4, half = warp / 4;
        const uint32_t mine = tmem + (quad << 21) + half * kHalf;    // lane 32 quad, column half * kHalf
        const uint32_t bias_at = base + a.stages * stage_bytes + 4 * kHalves * a.slots * kUnit + warp * kBiasRow;
        const bool bf16 = a.e.out_dtype != 0;
        const uint32_t width = bf16 ? 64 : 32;           // columns of a block of outputs
        const bool by_tma = !kSwap && a.vec && a.splits == 1;
        OutWarp o;
        o.slots = a.slots;
        o.buf = base + a.stages * stage_bytes + warp * a.slots * kUnit;
        o.bar = res_bars + warp * kTcMaxSlots * 8;
        o.issued = o.block = 0;
        o.at_tile = first;
        o.at_block = o.load_slot = 0;
        o.row_off = quad * 32;
        o.col_off = half * kHalf;
        o.blocks = kHalf / width;
        o.ahead = by_tma && a.e.res && !a.e.pre;
        const uint32_t stage_unit = o.buf;
        if (o.ahead && lane == 0) load_ahead<kCtas, kBN>(a, o, o.slots, step, width, rank);
        const uint32_t lead_empty = kCtas == 2 ? in_cta(acc_empty, 0) : acc_empty, lead_small = lead_empty + 16;
        uint32_t ch = 0, slot = 0, slot_phase = 0;     // slot: of block o.block
        TcWalk walk;
        for (uint32_t t = first; ok && t < a.tiles; t += step) {
            const TcTile tile = walk.at(a, t);
            const uint32_t prow = tile.p * 128 * kCtas + (kCtas == 2 ? rank * 128 : 0) + quad * 32;
            const uint32_t qrow = tile.q * kBN + half * kHalf;
            if constexpr (kDrain) {
                // all chunks but the last are summed in registers; the sums join the last one
                // in TMEM, from where the tile is finished
                const uint32_t chunks = (kb1 - kb0 + a.chunk_kb - 1) / a.chunk_kb;
                float acc[kHalf];
#pragma unroll
                for (int i = 0; i < kHalf; ++i) acc[i] = 0.0f;
                for (uint32_t n = 1; n <= chunks; ++n) {
                    const uint32_t b = ch & 1;
                    if (!bar_wait(acc_full + 8 * b, (ch / 2) & 1, gone, ctas)) {
                        ok = false;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    if (chunks == 1 && !split_planes) break;
#pragma unroll
                    for (int c = 0; c < kPieces; ++c) {
                        float v[16];
                        tmem_ld16(mine + b * kBN + c * 16, v);
                        tmem_wait16(v);
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[c * 16 + i] += v[i];
                    }
                    if (n == chunks) {
                        if (kBN <= 128 && split_planes) {
#pragma unroll
                            for (int c = 0; c < kPieces; ++c) {
                                float v[16];
                                tmem_ld16(mine + 2 * kBN + c * 16, v);
                                tmem_wait16(v);
#pragma unroll
                                for (int i = 0; i < 16; ++i) acc[c * 16 + i] += v[i];
                            }
                            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                            __syncwarp();
                            if (lane == 0) bar_arrive_cluster(lead_small);
                        }
                        break;
                    }
                    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) bar_arrive_cluster(lead_empty + 8 * b);
                    ++ch;
                }
                if (chunks > 1 || split_planes) {
#pragma unroll
                    for (int c = 0; c < kPieces; ++c) tmem_st16(mine + (ch & 1) * kBN + c * 16, acc + c * 16);
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                }
            } else {
                if (!bar_wait(acc_full + 8 * (ch & 1), (ch / 2) & 1, gone, ctas)) ok = false;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            }
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            const uint32_t b = ch & 1;
            const auto release = [&] {       // this warp has read the accumulator
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) bar_arrive_cluster(lead_empty + 8 * b);
            };
            if (!kSwap && by_tma) {
#pragma unroll 1
                for (uint32_t blk = 0; blk < o.blocks; ++blk, ++o.block) {
                    const uint32_t out = o.buf + slot * kUnit, col = qrow + blk * width;
                    // the next residuals are asked for before this block is worked on: buffers
                    // whose last store has been read are free
                    if (o.ahead && o.slots > 1 && lane == 0) {
                        if (o.slots == 2)
                            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                        else
                            asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                        load_ahead<kCtas, kBN>(a, o, o.block + (o.slots == 2 ? 2 : o.slots - 1), step, width, rank);
                    }
                    if (a.e.bias)
                        for (uint32_t i = lane; i < width; i += 32)
                            st_shared1(bias_at + i * 4, col + i < a.cols ? elem(a.e.bias, col + i, a.e.bias_dtype) : 0.0f);
#pragma unroll 1
                    for (int pre = a.e.pre != nullptr; pre >= 0; --pre) {
                        // 32 columns at a time; the first on their way while the block's buffer
                        // is waited for: its residual has come, or its last store has left
                        const uint32_t from = mine + b * kBN + blk * width;
                        float v[16], u[16];
                        tmem_ld16(from, v);
                        tmem_ld16(from + 16, u);
                        if (o.ahead)
                            ok = bar_wait(o.bar + 8 * slot, slot_phase, gone, ctas);
                        else if (lane == 0)              // one buffer
                            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                        __syncwarp();
#pragma unroll 1
                        for (uint32_t in = 0;;) {
                            tmem_wait16(v);
                            tmem_wait16(u);
                            const bool last = in + 32 == width;
                            if (last && blk + 1 == o.blocks && !pre) release();
                            const uint32_t piece = in * (bf16 ? 2 : 4) / 16, row = prow + lane;
                            finish_row(a, v, bias_at + in * 4, out, piece, row, col + in, o.ahead, pre);
                            finish_row(a, u, bias_at + in * 4 + 64, out, piece + (bf16 ? 2 : 4), row, col + in + 16, o.ahead, pre);
                            if (last) break;
                            in += 32;
                            tmem_ld16(from + in, v);
                            tmem_ld16(from + in + 16, u);
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) {
                            if (prow < a.rows && col < a.cols) tma_store_2d(pre ? &a.map_pre : &a.map_out, out, col, prow);
                            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                            if (o.ahead && o.slots == 1) {
                                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                                load_ahead<kCtas, kBN>(a, o, o.block + 2, step, width, rank);
                            }
                        }
                    }
                    if (++slot == o.slots) {
                        slot = 0;
                        slot_phase ^= 1;
                    }
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < kPieces; ++c) {
                    float v[16];
                    tmem_ld16(mine + b * kBN + c * 16, v);
                    tmem_wait16(v);
                    if (c == kPieces - 1) release();
                    // by units of 32 rows x kUnitCols columns, in the exchange's order [quad][half][unit]
                    const uint32_t u = c * 16 / kUnitCols;
                    const uint32_t unit =
                        a.splits > 1 ? base + ((quad * kHalves + half) * (kHalf / kUnitCols) + u) * kUnit : stage_unit;
                    const uint32_t j0 = c * 16 % kUnitCols / 4;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        st_shared4(unit + unit_at(lane, j0 + j), v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    if (a.splits == 1 && (c + 1) * 16 % kUnitCols == 0) {
                        __syncwarp();
#pragma unroll 1
                        for (uint32_t i = 0; i < (kSwap ? kUnitCols / 4 : 4); ++i)
                            if constexpr (kSwap)
                                finish_item_swapped(a, unit, i, 1, prow, qrow + u * 32);
                            else
                                finish_any(a, unit, i, 1, prow, qrow + u * 32);
                        __syncwarp();
                    }
                }
            }
            ++ch;
            ok = __all_sync(~0u, ok);
        }
        if (lane == 0) {
            if (!ok) {
                atomicOr(a.err, kErrWaitTimeout);
                for (; o.block < o.issued; ++o.block)       // the loads in flight land first
                    for (uint32_t i = 0; i < 1000 && !bar_try(o.bar + 8 * (o.block % o.slots), (o.block / o.slots) & 1); ++i) {}
            }
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (kCtas == 2 || a.splits > 1) cluster_sync();
    if (kCtas == 1 && a.splits > 1) {
        // every CTA's part of the one tile is in place: this CTA finishes its share of the rows
        if (warp < kWarps) {
            const TcTile tile = TcWalk().at(a, first);
            constexpr uint32_t kPerQuad = kBN / kUnitCols, kItems = kSwap ? kUnitCols / 4 : 4;
#pragma unroll 1
            for (uint32_t x = rank + a.splits * warp; x < 4 * kPerQuad * kItems; x += a.splits * kWarps) {
                const uint32_t u = x / kItems, i = x % kItems;
                const uint32_t prow = tile.p * 128 + u / kPerQuad * 32, qrow = tile.q * kBN + u % kPerQuad * kUnitCols;
                if constexpr (kSwap)
                    finish_item_swapped(a, base + u * kUnit, i, a.splits, prow, qrow);
                else
                    finish_any(a, base + u * kUnit, i, a.splits, prow, qrow);
            }
        }
        cluster_sync();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        tmem_free<kCtas>(tmem, kTmemCols);
    }
}

// The instantiation for a.cfg: kernel, block-independent facts.
struct Config {
    int ctas, bn;
    bool swap;
};
constexpr Config kConfigs[kTcConfigs] = {{2, 256, false}, {1, 128, false}, {1, 64, false},
                                         {1, 64, true},   {1, 32, true},   {1, 16, true}, {2, 128, false}};
using Kernel = void (*)(TcArgs);
const Kernel kKernels[kTcConfigs][2] = {
    {product_tc_kernel<2, 256, false, false>, product_tc_kernel<2, 256, true, false>},
    {product_tc_kernel<1, 128, false, false>, product_tc_kernel<1, 128, true, false>},
    {product_tc_kernel<1, 64, false, false>, product_tc_kernel<1, 64, true, false>},
    {product_tc_kernel<1, 64, false, true>, product_tc_kernel<1, 64, true, true>},
    {product_tc_kernel<1, 32, false, true>, product_tc_kernel<1, 32, true, true>},
    {product_tc_kernel<1, 16, false, true>, product_tc_kernel<1, 16, true, true>},
    {product_tc_kernel<2, 128, false, false>, product_tc_kernel<2, 128, true, false>}};

constexpr int kTcThreads[kTcConfigs][2] = {{kThreads<256, false>, kThreads<256, true>}, {kThreads<128, false>, kThreads<128, true>},
                                       {kThreads<64, false>, kThreads<64, true>},   {kThreads<64, false>, kThreads<64, true>},
                                       {kThreads<32, false>, kThreads<32, true>},   {kThreads<16, false>, kThreads<16, true>},
                                            {kThreads<128, false>, kThreads<128, true>}};

constexpr uint32_t kSmemMost = 231424;    // dynamic: 227 KB less 1 KB, which the static part begins

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled g_encode = nullptr;

// [planes][outer][inner] bf16, boxes of `rows` x 64 elements, 128-byte swizzle, zeros outside.
bool encode(CUtensorMap* map, const TcOperand& o, uint64_t inner, uint64_t outer, uint32_t rows) {
    const cuuint64_t dims[3] = {inner, outer, o.planes};
    const cuuint64_t strides[2] = {o.ld * 2, o.planes > 1 ? o.plane * 2 : o.ld * 2};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(kBK), rows, 1}, one[3] = {1, 1, 1};
    return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(o.p), dims, strides, box, one,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool out_ready(const void* p, uint64_t ld, int dtype) {
    const uint64_t size = dtype ? 2 : 4;
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0 && ld * size < (1ull << 40);
}

// The output's matrix in boxes of 32 rows x 128 bytes.
bool encode_out(CUtensorMap* map, const void* p, uint64_t ld, const TcArgs& a) {
    const bool bf16 = a.e.out_dtype != 0;
    const cuuint64_t dims[2] = {a.cols, a.rows}, strides[1] = {ld * (bf16 ? 2 : 4)};
    const cuuint32_t box[2] = {bf16 ? 64u : 32u, 32}, one[2] = {1, 1};
    return g_encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
                    const_cast<void*>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t prepare_product_tc(TcShape* shape) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&shape->sms, cudaDevAttrMultiProcessorCount, dev);
    for (int c = 0; c < kTcConfigs; ++c)
        for (int d = 0; d < 2 && e == cudaSuccess; ++d)
            e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kKernels[c][d]),
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost);
    // how many clusters the GPCs hold (of 8 CTAs, fewer than SMs / 8)
    for (int i = 1; i <= 8 && e == cudaSuccess; ++i) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(840 * i);
        cfg.blockDim = dim3(kTcThreads[kTc128][0]);
        cfg.dynamicSmemBytes = kSmemMost;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = i;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, reinterpret_cast<const void*>(kKernels[kTc128][0]), &cfg);
        shape->split_ctas[i] = n * i;
    }
    if (e == cudaSuccess && !g_encode) {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
        if (e == cudaSuccess && (q != cudaDriverEntryPointSuccess || !f)) e = cudaErrorNotSupported;
        if (e == cudaSuccess) g_encode = reinterpret_cast<EncodeTiled>(f);
    }
    return e;
}

cudaError_t launch_product_tc(const TcProduct& p, const TcShape& shape, unsigned int* err, bool test_expire,
                              cudaStream_t stream) {
    TcArgs a{};
    const Config& c = kConfigs[p.cfg];
    const bool drain = p.drain;
    a.e = p.e;
    a.rows = p.m;
    a.cols = p.n;
    a.k = p.k;
    // Two blocks of 64 terms per stage where a tile's MMAs are short: a stage's waits, issue and
    // commit take some 500 cycles, a block of 256 x 256 products 512, of 128 x 128 only 256.
    a.sub = c.bn < 256 && p.a.planes + p.b.planes == 2 && p.k > kBK ? 2 : 1;
    a.kblocks = (p.k + a.sub * kBK - 1) / (a.sub * kBK);
    const TcOperand& P = c.swap ? p.b : p.a;
    const TcOperand& Q = c.swap ? p.a : p.b;
    const uint32_t px = c.swap ? p.n : p.m, qx = c.swap ? p.m : p.n;
    a.p_kmajor = P.kmajor;
    a.q_kmajor = Q.kmajor;
    a.planes_p = P.planes;
    a.planes_q = Q.planes;
    const uint32_t qrows = c.bn / c.ctas;
    const bool okp = P.kmajor ? encode(&a.map_p, P, p.k, px, 128) : encode(&a.map_p, P, px, p.k, kBK);
    const bool okq = Q.kmajor ? encode(&a.map_q, Q, p.k, qx, qrows) : encode(&a.map_q, Q, qx, p.k, kBK);
    if (!okp || !okq) return cudaErrorInvalidValue;
    a.tiles_p = (px + 128 * c.ctas - 1) / (128 * c.ctas);
    a.tiles_q = (qx + c.bn - 1) / c.bn;
    a.tiles = a.tiles_p * a.tiles_q;
    a.splits = c.ctas == 2 ? 1 : p.splits;
    if (a.splits > a.kblocks) a.splits = a.kblocks;
    a.chunk_kb = 4 / a.sub;
    auto vec = [&](const void* q, uint64_t ld) { return !q || out_ready(q, ld, a.e.out_dtype); };
    a.vec = vec(a.e.out, a.e.ldo) && vec(a.e.pre, a.e.ldo) && vec(a.e.res, a.e.ldr);
    // elements that every output row's stores can be aligned for, where not 16 bytes
    a.grain = a.e.out_dtype ? 4 : 2;
    const auto aligned = [&](const void* q, uint64_t ld, uint32_t n) {
        const uint64_t size = a.e.out_dtype ? 2 : 4;
        return !q || (reinterpret_cast<uintptr_t>(q) % (n * size) == 0 && ld % n == 0);
    };
    while (a.grain > 1 && !(aligned(a.e.out, a.e.ldo, a.grain) && aligned(a.e.pre, a.e.ldo, a.grain) &&
                            aligned(a.e.res, a.e.ldr, a.grain)))
        a.grain /= 2;
    const bool by_tma = a.vec && a.splits == 1 && !c.swap;
    if (by_tma && !(encode_out(&a.map_out, a.e.out, a.e.ldo, a) && (!a.e.pre || encode_out(&a.map_pre, a.e.pre, a.e.ldo, a)) &&
                    (!a.e.res || encode_out(&a.map_res, a.e.res, a.e.ldr, a))))
        return cudaErrorInvalidValue;
    const uint32_t stage = a.sub * (P.planes * kPBytes + Q.planes * qrows * kBK * 2);
    const uint32_t warps = 4 * drain_parts(c.bn, c.swap);
    // Short sums with a residual are bound by the output side: more blocks ahead.  Else as many
    // stages as fit.
    a.slots = c.swap ? 1 : by_tma && a.e.res && !a.e.pre && p.k <= 4 * kBK ? (c.bn == 256 ? 2 : kTcMaxSlots) : 1;
    if (warps * (a.slots * kUnit + kBiasRow) + 2 * stage > kSmemMost) a.slots = 1;
    const uint32_t extra = a.splits == 1 ? warps * (a.slots * kUnit + kBiasRow) : 0;
    // two CTAs per SM for the forms that take few registers, if each has three stages
    const auto fit = [&](uint32_t ctas) { return (kSmemMost / ctas - 2048 * (ctas - 1) - extra) / stage; };
    const uint32_t occupancy = c.swap && !drain && fit(2) >= 3 ? 2 : 1;
    uint32_t stages = fit(occupancy);
    if (stages > static_cast<uint32_t>(kTcMaxStages)) stages = kTcMaxStages;
    if (stages < 1) return cudaErrorInvalidValue;
    a.stages = stages;
    uint32_t smem = extra + stages * stage;
    if (a.splits > 1 && smem < 128u * c.bn * 4) smem = 128 * c.bn * 4;
    a.err = err;
    a.test_expire = test_expire;
    const uint32_t per = c.ctas == 2 ? 2 : a.splits;
    uint32_t clusters = a.tiles;
    if (a.splits == 1) {
        const uint32_t room = shape.sms / c.ctas * occupancy;
        if (clusters > room) clusters = room;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(clusters * per);
    cfg.blockDim = dim3(kTcThreads[p.cfg][drain]);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = per;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = per > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kKernels[p.cfg][drain], a);
}

}  // namespace fa
