// The products of an orthogonalised weight step, on the tensor cores (tcgen05): operands as two
// fp16 terms, fp32 sums, results as two fp16 terms again.
//
//   v = c1 * sum_k P(x,k) Q(y,k) + c2 * e1 + c3 * e2
//
// x = hi + lo has 22 bits, so hi lo' + lo hi' + hi hi' is the product to 2^-22 of its size: three
// products of fp16 where three bf16 terms would need six.  The matrices' scales keep |x| below 2^15, and
// their typical elements far above the 2^-24 where fp16 ends.
//
// A CTA's tile is 128 rows of P (TMEM lanes) by kBN rows of Q (TMEM columns); with kCtas == 2 a
// pair of SMs has 256 by 256 (cta_group::2).  The tensor cores' fp32 sum truncates, so it is
// emptied every few blocks of 64 terms into registers, which round to nearest; TMEM has two such
// accumulators.  The last emptying leaves the tile in registers, from where it is finished: the
// accumulators are free for the next tile meanwhile.
//
// Polynomials of a symmetric matrix commute and are symmetric: of these the tiles on and above
// the diagonal are computed, and written twice.
//
// A launch runs a list of products one after the other, for all items: the tiles of a product of
// all items, then those of the next, dealt out to the clusters in turn.  A product of an item needs
// the one before it whole.  A tile's drain warps count it when its stores are done; who works on a
// later product of the item waits for the count (acquire, then a proxy fence before TMA).  All
// clusters are resident (a cooperative launch), and a tile waits for earlier ones alone, so that the
// first that is not done can always go on.  Where the items have a few turns of tiles that fills each
// product's last turn with the next one's tiles: 24 of 1024 x 1024 bf16, 240 and 384 tiles over 76
// pairs, take 1.30 ms so and 1.49 with a launch for each product.  One matrix gains nothing (4096 x
// 4096 fp32 2.89 ms both ways, 512 x 512 bf16 174 us so and 141 by launches, each with the tiles that suit
// it), and is done by launches.
#include <algorithm>

#include <cuda_fp16.h>

#include "ortho.cuh"
#include "tc_ptx.cuh"

namespace fa {

namespace {

constexpr int kBK = 64;                          // summed elements per block: 128 bytes, one swizzle row
constexpr uint32_t kPlane = 128 * kBK * 2;       // of an operand's 128 rows
constexpr uint32_t kStageBytes = 4 * kPlane;
constexpr uint32_t kRing = 3;                    // stages
constexpr uint32_t kUnit = 2048;                 // a drain warp's block of 32 x 32 results on its way out
// Such blocks that a drain warp has under way after the CTA's last tile.  With one alone each store waited
// for the one before to be read.
constexpr uint32_t kUnits = 6;
constexpr uint32_t kSplitUnits = 4;              // of a split tile's block: its four stores
constexpr uint32_t kBand = 8;                    // rows of tiles walked together
constexpr int kCols = 64;                        // of a drain warp

constexpr uint32_t kOrthoSplits = 8;

template <int kBN>
constexpr int kDrain = 4 * kBN / kCols;          // drain warps
// The pair's last warpgroup (loads, MMAs, two idle warps) gives registers to the drain warps, as in
// the product kernels: 128 x 56 + 512 x 104 <= 640 x 96.  At those 96 registers ptxas spills 216 bytes (stores)
// and 428 (loads) of one product's kernel, 40 and 80 of the list's, in the tiles' ends.
template <int kBN>
constexpr int kOrthoThreads = (kDrain<kBN> + (kBN == 256 ? 4 : 2)) * 32;
static_assert(kDrain<128> * kSplitUnits * kUnit <= kStageBytes && kSplitUnits < kUnits);
static_assert(kDrain<256> * kUnits * kUnit <= kRing * kStageBytes && kRing * kStageBytes / kDrain<256> % kUnit == 0);
template <int kBN>
constexpr uint32_t kSmem = kRing * kStageBytes + kDrain<kBN> * kUnit;

struct Op {
    const uint16_t *e1, *e2;
    uint64_t ld, plane;                          // of e1 and e2
    float c1, c2, c3;
    uint32_t rows, cols, kblocks, chunk;         // chunk: blocks between two emptyings
    uint32_t tiles_p, tiles_q, per;              // per: tiles of an item
    uint32_t first, need;                        // the first tile; an item's count when its earlier products are done
    uint8_t p, q, out;                           // maps
    bool p_kmajor, q_kmajor, symmetric;
};

// kMany: a list of products; else one, with what a launch of that needs alone.
template <bool kMany>
struct Args {
    CUtensorMap map[3 * (kMany ? kOrthoBufs : 3)];    // of each buffer: k, mn, out
    Op op[kMany ? kOrthoOps : 1];
    uint32_t* done;                              // [items]
    unsigned int* err;
    uint32_t ops, items, tiles, splits;
    bool test_expire;
};

// A cluster's tiles in turn.
struct Walk {
    uint32_t n = 0;                              // the product
    uint32_t item, p, q;
    template <bool kMany>
    __device__ __forceinline__ const Op& at(const Args<kMany>& a, uint32_t t) {
        if constexpr (kMany)
            while (n + 1 < a.ops && t >= a.op[n + 1].first) ++n;
        const Op& o = a.op[kMany ? n : 0];
        const uint32_t u = t - o.first;
        item = u / o.per;
        uint32_t r = u - item * o.per;
        if (o.symmetric) {                       // column by column, p <= q
            q = static_cast<uint32_t>((sqrtf(8.0f * static_cast<float>(r) + 1.0f) - 1.0f) * 0.5f);
            while (q * (q + 1) / 2 > r) --q;
            while ((q + 1) * (q + 2) / 2 <= r) ++q;
            p = r - q * (q + 1) / 2;
        } else {
            const uint32_t full = kBand * o.tiles_q, band = r / full;
            r -= band * full;
            const uint32_t height = min(kBand, o.tiles_p - band * kBand);
            q = r / height;
            p = band * kBand + r - q * height;
        }
        return o;
    }
};

// Until an item's earlier products are done; false where the cluster has given up, or after some 20 s.
__device__ __forceinline__ bool wait_done(const Args<true>& a, const Op& o, uint32_t item, uint32_t gone, uint32_t ctas) {
    long long t0 = 0;
    for (;;) {
        uint32_t v, g;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(a.done + item) : "memory");
        if (v >= o.need) return true;
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

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y, int32_t z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x), "r"(y),
                 "r"(z), "r"(src)
                 : "memory");
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float half_of(float x) { return __half2float(__float2half_rn(x)); }

// A warp's results as they leave: units of 32 x 32, each free again when its store has read it.
struct Units {
    uint32_t at, n, next;                        // n: kUnits, or 1
    __device__ __forceinline__ uint32_t take() {
        if (threadIdx.x % 32 == 0) {
            if (n == 1)
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            else
                asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kUnits - 1) : "memory");
        }
        __syncwarp();
        const uint32_t u = at + next * kUnit;
        next = next + 1 == n ? 0 : next + 1;
        return u;
    }
    __device__ __forceinline__ void store(const CUtensorMap* out, uint32_t u, uint32_t x, uint32_t y, uint32_t z) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (threadIdx.x % 32 == 0) {
            tma_store_3d(out, u, x, y, z);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
    }
};

// v += c * e: the warp's 32 rows from row0 of kWidth columns from col on, of which v is this lane's row.  Four
// lanes read 64 bytes of a row, and a unit hands the rows over (a row for each lane touched a line for
// each: 3.3 us of the 9 that a product of 230 x 230 took).  kPlanes of a block's two are fetched at a
// time, as registers allow.
template <uint32_t kPlanes, uint32_t kWidth>
__device__ __forceinline__ void add_to(const Op& a, const uint16_t* e, float c, float* v, Units& units, uint32_t item, uint32_t row0,
                                       uint32_t col) {
    const uint32_t lane = threadIdx.x % 32, r0 = lane / 4, j0 = lane % 4;
    const uint16_t* from = e + 2ull * item * a.plane + (row0 + r0) * a.ld + col + 8 * j0;
#pragma unroll
    for (uint32_t n = 0; n < kWidth / 32 * 2; n += kPlanes) {
        const uint32_t h = n / 2;
        uint4 q[kPlanes][4];
        const bool in = col + 32 * h + 8 * j0 < a.cols;
#pragma unroll
        for (uint32_t z = 0; z < kPlanes; ++z)
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) {
                q[z][i] = make_uint4(0, 0, 0, 0);
                // from L2: other SMs may have written them during this launch
                if (in && row0 + r0 + 8 * i < a.rows)
                    q[z][i] = __ldcg(reinterpret_cast<const uint4*>(from + (n + z) % 2 * a.plane + 8 * i * a.ld + 32 * h));
            }
#pragma unroll
        for (uint32_t z = 0; z < kPlanes; ++z) {
            const uint32_t u = units.take();
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) {
                const uint32_t r = r0 + 8 * i;
                st_shared4u(u + r * 64 + ((j0 ^ (r / 2 % 4)) << 4), q[z][i].x, q[z][i].y, q[z][i].z, q[z][i].w);
            }
            __syncwarp();
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) {
                const uint4 w = ld_shared4u(u + lane * 64 + ((j ^ (lane / 2 % 4)) << 4));
                const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x[k]));
                    float* to = v + 32 * h + 8 * j + 2 * k;
                    to[0] = fmaf(c, f.x, to[0]);
                    to[1] = fmaf(c, f.y, to[1]);
                }
            }
        }
    }
}

// The block of 32 x 32 results at (row, col) from v, this lane's row of it: either plane by way of a
// unit, and its mirror image.  64-byte rows in the 64-byte swizzle: 16-byte piece j of row r is at
// j ^ (r / 2 % 4).
__device__ __forceinline__ void finish(const CUtensorMap* out, float* v, Units& units, uint32_t item, uint32_t row0, uint32_t col,
                                       bool mirror) {
    const uint32_t lane = threadIdx.x % 32;
#pragma unroll
    for (uint32_t z = 0; z < 2; ++z) {
        if (z == 1)
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] -= half_of(v[i]);
        uint32_t u = units.take();
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j)
            st_shared4u(u + lane * 64 + ((j ^ (lane / 2 % 4)) << 4), pack_half(v[8 * j], v[8 * j + 1]),
                        pack_half(v[8 * j + 2], v[8 * j + 3]), pack_half(v[8 * j + 4], v[8 * j + 5]),
                        pack_half(v[8 * j + 6], v[8 * j + 7]));
        units.store(out, u, col, row0, 2 * item + z);
        if (!mirror) continue;
        u = units.take();
#pragma unroll
        for (uint32_t c = 0; c < 32; ++c)
            asm volatile("st.shared.b16 [%0], %1;" ::"r"(u + c * 64 + ((lane / 8 ^ (c / 2 % 4)) << 4) + lane % 8 * 2),
                         "h"(__half_as_ushort(__float2half_rn(v[c])))
                         : "memory");
        units.store(out, u, row0, col, 2 * item + z);
    }
}

// A split tile's sums: this warp's to the CTA's shared memory, as 32 x 32 blocks of fp32 (128-byte rows, see
// unit_at); block b is of rows b / 4 * 32 and columns b % 4 * 32 of the tile.
__device__ __forceinline__ void put_sums(uint32_t base, const float (&acc)[kCols], uint32_t quad, uint32_t part) {
    const uint32_t lane = threadIdx.x % 32;
#pragma unroll
    for (uint32_t i = 0; i < kCols; i += 4)
        st_shared4(base + (quad * 4 + part * 2 + i / 32) * 4096 + unit_at(lane, i % 32 / 4), acc[i], acc[i + 1], acc[i + 2],
                   acc[i + 3]);
}

// The blocks that this CTA finishes, 16 / splits of them, summed over the cluster in rank order, to `to`.
__device__ __forceinline__ void sum_blocks(uint32_t base, uint32_t to, uint32_t rank, uint32_t splits) {
    const uint32_t first = rank * (16 / splits) * 4096, bytes = 16 / splits * 4096;
    for (uint32_t at = threadIdx.x * 16; at < bytes; at += kDrain<128> * 32 * 16) {
        float4 v = ld_part(base + first + at, 0, splits);
#pragma unroll 8
        for (uint32_t q = 1; q < splits; ++q) {
            const float4 t = ld_part(base + first + at, q, splits);
            v.x += t.x;
            v.y += t.y;
            v.z += t.z;
            v.w += t.w;
        }
        st_shared4(to + at, v.x, v.y, v.z, v.w);
    }
    asm volatile("barrier.cta.sync 1, %0;" ::"n"(kDrain<128> * 32) : "memory");
}

// kSplit: a cluster of a.splits CTAs has one tile, and each a part of its blocks of terms.  The sums
// meet over distributed shared memory, and each CTA finishes a part of the tile.
template <int kCtas, int kBN, bool kMany, bool kSplit>
__global__ void __launch_bounds__((kOrthoThreads<kBN>), 1) ortho_product_kernel(const __grid_constant__ Args<kMany> a) {
    static_assert(kBN / kCtas == 128, "128 rows of either operand per CTA");
    static_assert(!kSplit || (kCtas == 1 && !kMany), "single SMs, one product");
    constexpr int kWarps = kDrain<kBN>, kLoadWarp = kWarps, kMmaWarp = kWarps + 1;
    extern __shared__ __align__(1024) uint8_t dyn[];
    __shared__ uint64_t bars[2 * kRing + 4];
    __shared__ uint32_t tmem_slot, gone_flag;
    const uint32_t base = smem_addr(dyn), full = smem_addr(&bars[0]), empty = full + 8 * kRing;
    const uint32_t acc_full = full + 16 * kRing, acc_empty = acc_full + 16;
    const uint32_t warp = __shfl_sync(~0u, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const uint32_t rank = kCtas == 2 ? cluster_rank() : 0, gone = smem_addr(&gone_flag);
    const bool leader = rank == 0;
    const uint32_t splits = kSplit ? a.splits : 1, part_rank = kSplit ? cluster_rank() : 0, ctas = kSplit ? splits : kCtas;
    // of a product's blocks, this CTA's
    const auto from_block = [&](uint32_t kblocks) { return kSplit ? part_rank * kblocks / splits : 0; };
    const auto to_block = [&](uint32_t kblocks) { return kSplit ? (part_rank + 1) * kblocks / splits : kblocks; };

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 0 && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&a.map[a.op[0].p]) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&a.map[a.op[0].q]) : "memory");
    }
    if (warp == kLoadWarp && lane == 0) {
        for (uint32_t s = 0; s < kRing; ++s) {
            bar_init(full + 8 * s, 1);
            bar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(acc_full + 8 * b, 1);
            bar_init(acc_empty + 8 * b, kCtas * kWarps);
        }
        gone_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc<kCtas>(smem_addr(&tmem_slot), 2 * kBN);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (kCtas == 2 || kSplit) cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_slot;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t first = blockIdx.x / ctas, step = gridDim.x / ctas;
    bool ok = true;                      // of this thread: no wait gave up

    if (warp >= kWarps) {
        if constexpr (kBN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == kLoadWarp && elect_one()) {
            const uint32_t lead_full = kCtas == 2 ? in_cta(full, 0) : full;
            const auto load = [&](uint32_t dst, const CUtensorMap* m, bool kmajor, uint32_t k, uint32_t x, uint32_t z, uint32_t bar) {
                if (kmajor) {
                    tma_load<kCtas>(dst, m, k, x, z, bar);
                } else {
                    tma_load<kCtas>(dst, m, x, k, z, bar);
                    tma_load<kCtas>(dst + 8192, m, x + 64, k, z, bar);
                }
            };
            uint32_t s = 0, phase = 1;
            Walk tile;
            for (uint32_t t = first; ok && t < a.tiles; t += step) {
                const Op& o = tile.at(a, t);
                const CUtensorMap *mp = &a.map[o.p], *mq = &a.map[o.q];
                const bool pk = o.p_kmajor, qk = o.q_kmajor;
                const uint32_t end = to_block(o.kblocks);
                const uint32_t p0 = tile.p * 128 * kCtas + rank * 128, q0 = tile.q * kBN + rank * 128, z = 2 * tile.item;
                if constexpr (kMany) {
                    if (!wait_done(a, o, tile.item, gone, ctas)) {
                        ok = false;
                        break;
                    }
                    asm volatile("fence.proxy.async;" ::: "memory");
                }
                for (uint32_t kb = from_block(o.kblocks); kb < end; ++kb) {
                    const uint32_t bar = lead_full + 8 * s, at = base + s * kStageBytes;
                    if (!bar_wait(empty + 8 * s, phase, gone, ctas)) {
                        ok = false;
                        break;
                    }
                    if (leader) mbar_expect(full + 8 * s, kStageBytes * kCtas);
                    const uint32_t k = kb * kBK;
                    load(at, mp, pk, k, p0, z, bar);
                    load(at + kPlane, mp, pk, k, p0, z + 1, bar);
                    load(at + 2 * kPlane, mq, qk, k, q0, z, bar);
                    load(at + 3 * kPlane, mq, qk, k, q0, z + 1, bar);
                    if (++s == kRing) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
        } else if (warp == kMmaWarp && leader && elect_one()) {
            uint32_t ch = 0, it = 0, s = 0, phase = 0;
            Walk tile;
            for (uint32_t t = first; ok && t < a.tiles; t += step) {
                const Op& o = tile.at(a, t);
                // fp32 sums of fp16 by fp16
                const uint32_t idesc = 1u << 4 | (o.p_kmajor ? 0u : 1u << 15) | (o.q_kmajor ? 0u : 1u << 16) | (kBN / 8) << 17 |
                                       (128 * kCtas / 16) << 24;
                const uint32_t step_p = o.p_kmajor ? 32 >> 4 : 2048 >> 4, step_q = o.q_kmajor ? 32 >> 4 : 2048 >> 4;
                const uint32_t desc_p = operand_desc_lo(base, o.p_kmajor), desc_q = operand_desc_lo(base + 2 * kPlane, o.q_kmajor);
                const uint32_t kblocks = to_block(o.kblocks), chunk = o.chunk;
                for (uint32_t kb = from_block(o.kblocks); ok && kb < kblocks; ++ch) {
                    const uint32_t b = ch & 1;
                    if (ch >= 2 && !bar_wait(acc_empty + 8 * b, (ch / 2 - 1) & 1, gone, ctas)) {
                        ok = false;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t d = tmem + b * kBN, end = min(kblocks, kb + chunk);
                    bool add = false;
                    for (; kb < end; ++kb, ++it) {
                        const uint32_t dp = desc_p + (s * kStageBytes >> 4), dq = desc_q + (s * kStageBytes >> 4);
                        if (a.test_expire || !bar_wait(full + 8 * s, phase, gone, ctas)) {
                            ok = false;
                            break;
                        }
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        // lo hi, hi lo, hi hi: the small products meet a small accumulator
#pragma unroll
                        for (uint32_t pair = 0; pair < 3; ++pair) {
                            const uint32_t op = pair == 0 ? kPlane >> 4 : 0, oq = pair == 1 ? kPlane >> 4 : 0;
#pragma unroll
                            for (uint32_t x = 0; x < kBK / 16; ++x) {
                                mma<kCtas>(d, dp + op + x * step_p, dq + oq + x * step_q, kDescHi, idesc, add);
                                add = true;
                            }
                        }
                        commit<kCtas>(empty + 8 * s);
                        if (++s == kRing) {
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
                for (uint32_t n = 0; n < kRing; ++n, ++it)
                    for (uint32_t i = 0; i < 1000 && !bar_try(full + 8 * (it % kRing), (it / kRing) & 1); ++i) {}
            }
        }
        __syncwarp();
    } else {
        if constexpr (kBN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        const uint32_t quad = warp % 4, part = warp / 4;
        const uint32_t mine = tmem + (quad << 21) + part * kCols;       // lane 32 quad, column part * kCols
        const uint32_t buf = base + kRing * kStageBytes + warp * kUnit;
        const uint32_t lead_empty = kCtas == 2 ? in_cta(acc_empty, 0) : acc_empty;
        uint32_t ch = 0;
        Walk tile;
        for (uint32_t t = first; ok && t < a.tiles; t += step) {
            const Op& o = kMany ? tile.at(a, t) : a.op[0];      // (the order that spills least)
            const uint32_t chunks = (to_block(o.kblocks) - from_block(o.kblocks) + o.chunk - 1) / o.chunk;
            float acc[kCols];
#pragma unroll
            for (int i = 0; i < kCols; ++i) acc[i] = 0.0f;
            for (uint32_t n = 0; n < chunks; ++n, ++ch) {
                const uint32_t b = ch & 1;
                if (!bar_wait(acc_full + 8 * b, (ch / 2) & 1, gone, ctas)) {
                    ok = false;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
                for (int c = 0; c < kCols; c += 16) {
                    float v[16];
                    tmem_ld16(mine + b * kBN + c, v);
                    tmem_wait16(v);
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[c + i] += v[i];
                }
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) bar_arrive_cluster(lead_empty + 8 * b);
            }
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            if constexpr (kSplit) {
                put_sums(base, acc, quad, part);
                break;
            }
            if constexpr (!kMany) tile.at(a, t);
            const uint32_t row0 = tile.p * 128 * kCtas + rank * 128 + quad * 32, col0 = tile.q * kBN + part * kCols;
            const bool mirror = o.symmetric && tile.p != tile.q;
            if (row0 < o.rows && col0 < o.cols) {
                if constexpr (kMany) {
                    // e1 and e2 are there, as the operands were: seen by every lane
                    ok = __all_sync(~0u, wait_done(a, o, tile.item, gone, ctas));
                    if (!ok) break;
                }
                // the last tile's results leave by way of the stages, which nothing needs any more
                Units units{buf, 1, 0};
                if (t + step >= a.tiles) units = {base + warp * (kRing * kStageBytes / kWarps), kUnits, 0};
#pragma unroll
                for (int i = 0; i < kCols; ++i) acc[i] *= o.c1;
                if (o.e1) add_to<kBN == 128 ? 2 : 1, kCols>(o, o.e1, o.c2, acc, units, tile.item, row0, col0);
                if (o.e2) add_to<kBN == 128 ? 2 : 1, kCols>(o, o.e2, o.c3, acc, units, tile.item, row0, col0);
                finish(&a.map[o.out], acc, units, tile.item, row0, col0, mirror);
                if (col0 + 32 < o.cols) finish(&a.map[o.out], acc + 32, units, tile.item, row0, col0 + 32, mirror);
            }
            if (kMany && lane == 0) {
                // this warp's part of the tile is in memory: for other SMs' TMA and loads
                asm volatile("cp.async.bulk.wait_group 0;\nfence.proxy.async;" ::: "memory");
                asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(a.done + tile.item) : "memory");
            }
        }
        if (lane == 0) {
            if (!ok) atomicOr(a.err, kErrWaitTimeout);
            if (!kSplit) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        }
    }
    if constexpr (kSplit) {
        __syncwarp();
        cluster_sync();
        if (warp < kWarps) {
            const uint32_t sums = base + kStageBytes, own = 16 / splits;
            sum_blocks(base, sums, part_rank, splits);
            Walk tile;
            const Op& o = tile.at(a, first);
            const uint32_t block = part_rank * own + warp;
            const uint32_t row0 = tile.p * 128 + block / 4 * 32, col0 = tile.q * 128 + block % 4 * 32;
            if (warp < own && row0 < o.rows && col0 < o.cols) {
                float v[32];
#pragma unroll
                for (uint32_t i = 0; i < 32; i += 4) {
                    const float4 t = ld_part(sums + warp * 4096 + unit_at(lane, i / 4), 0, 1);
                    v[i] = t.x * o.c1;
                    v[i + 1] = t.y * o.c1;
                    v[i + 2] = t.z * o.c1;
                    v[i + 3] = t.w * o.c1;
                }
                Units units{base + 2 * kStageBytes + warp * kSplitUnits * kUnit, kSplitUnits, 0};
                if (o.e1) add_to<2, 32>(o, o.e1, o.c2, v, units, tile.item, row0, col0);
                if (o.e2) add_to<2, 32>(o, o.e2, o.c3, v, units, tile.item, row0, col0);
                finish(&a.map[o.out], v, units, tile.item, row0, col0, o.symmetric && tile.p != tile.q);
                if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
            }
            __syncwarp();
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (kCtas == 2 || kSplit) cluster_sync();        // no CTA leaves while another may read its sums
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        tmem_free<kCtas>(tmem, 2 * kBN);
    }
}

EncodeTiled g_encode = nullptr;

bool encode(CUtensorMap* map, const OrthoBuf& b, uint32_t items, uint32_t box_x, uint32_t box_y, CUtensorMapSwizzle swizzle) {
    const cuuint64_t dims[3] = {b.cols, b.rows, 2ull * items};
    const cuuint64_t strides[2] = {b.ld * 2, b.plane() * 2};
    const cuuint32_t box[3] = {box_x, box_y, 1}, one[3] = {1, 1, 1};
    return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, b.p, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A list waits within itself and is launched cooperatively; a single product overlaps its start with
// its predecessor's end.
template <int kCtas, int kBN, bool kMany, bool kSplit>
cudaError_t launch(const Args<kMany>& a, uint32_t room, cudaStream_t stream) {
    const uint32_t ctas = kSplit ? a.splits : kCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((kSplit || a.tiles < room ? a.tiles : room) * ctas);
    cfg.blockDim = dim3(kOrthoThreads<kBN>);
    cfg.dynamicSmemBytes = kSmem<kBN>;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    if (kMany) {
        at[0].id = cudaLaunchAttributeCooperative;
        at[0].val.cooperative = 1;
    } else {
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
    }
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = ctas;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, ortho_product_kernel<kCtas, kBN, kMany, kSplit>, a);
}

uint32_t blocks_of(const OrthoProduct& p) { return (p.k + kBK - 1) / kBK; }

uint32_t tiles_of(const OrthoProduct& p, uint32_t side) {
    const uint32_t r = (p.out->rows + side - 1) / side, c = (p.out->cols + side - 1) / side;
    return p.symmetric ? c * (c + 1) / 2 : r * c;
}

// The tile of a launch's products, the CTAs of a tile, and the time that this is thought to take.
struct Plan {
    bool pair;
    uint32_t splits;
    double cost;
    uint32_t side() const { return pair ? 256 : 128; }
};

// Turns over the SMs, in microseconds.  A block of a pair takes 0.8, of a single SM 0.42 or, with all SMs
// loading 64 KB for each, 0.58; a tile's end 1.5, and a product 3 more before its first tile's data is there.
//
// One product whose tiles occupy a part of the SMs has a tile's blocks shared out over a cluster.
// Launching the cluster and exchanging the sums takes 1.9, of eight CTAs 4 (which have to be free in
// one part of the GPU): 512 x 512 bf16, 10 tiles of 8 blocks, 157 us unsplit, 139 by four, 175 by eight;
// 128 x 11008 bf16, first products of one tile and 172 blocks, 299, 178 and 157; 100 x 10000 fp32
// 705, 276 and 201.
Plan plan_of(const OrthoProduct* p, uint32_t n, uint32_t items, bool many, uint32_t sms) {
    const auto cost = [&](bool pair, uint32_t splits) {
        double c = 0.0;
        for (uint32_t i = 0; i < n; ++i) {
            const uint64_t t = static_cast<uint64_t>(tiles_of(p[i], pair ? 256 : 128)) * items, room = pair ? sms / 2 : sms;
            const double busy = std::min(1.0, static_cast<double>(t * splits) / sms);
            const double block = pair ? 0.8 : std::max(0.42, 0.58 * busy);
            // items go on without one another: whole turns for one, parts of turns for many
            const double turns = many ? std::max(1.0, static_cast<double>(t) / room) : static_cast<double>((t + room - 1) / room);
            c += turns * (block * ((blocks_of(p[i]) + splits - 1) / splits) + 1.5) + 3.0 + (splits == 1 ? 0.0 : splits < 8 ? 1.9 : 4.0);
        }
        return c;
    };
    Plan best{true, 1, cost(true, 1)};
    for (uint32_t splits = 1; splits <= (many ? 1 : kOrthoSplits); splits *= 2) {
        if (splits > 1 && (blocks_of(*p) < splits || static_cast<uint64_t>(tiles_of(*p, 128)) * items * splits > sms)) break;
        const double c = cost(false, splits);
        if (c < best.cost) best = {false, splits, c};
    }
    return best;
}

template <bool kMany>
cudaError_t run(const OrthoProduct* p, uint32_t n, uint32_t items, uint32_t* done, uint32_t* count, const OrthoShape& shape,
                unsigned int* err, bool test_expire, cudaStream_t stream) {
    Args<kMany> a{};
    const OrthoBuf* bufs[kOrthoBufs] = {};
    uint32_t held = 0;
    const auto index = [&](const OrthoBuf* b) {
        for (uint32_t i = 0; i < held; ++i)
            if (bufs[i] == b) return 3 * i;
        bufs[held] = b;
        a.map[3 * held] = b->k;
        a.map[3 * held + 1] = b->mn;
        a.map[3 * held + 2] = b->out;
        return 3 * held++;
    };
    a.ops = n;
    a.items = items;
    a.done = done;
    a.err = err;
    a.test_expire = test_expire;
    for (uint32_t i = 0; i < n; ++i) {
        if (held + 3 > kOrthoBufs) return cudaErrorInvalidValue;
        Op& o = a.op[i];
        o.p = static_cast<uint8_t>(index(p[i].P) + (p[i].p_kmajor ? 0 : 1));
        o.q = static_cast<uint8_t>(index(p[i].Q) + (p[i].q_kmajor ? 0 : 1));
        o.out = static_cast<uint8_t>(index(p[i].out) + 2);
        o.e1 = p[i].e1 ? p[i].e1->p : nullptr;
        o.e2 = p[i].e2 ? p[i].e2->p : nullptr;
        o.ld = p[i].out->ld;
        o.plane = p[i].out->plane();
        o.c1 = p[i].c1;
        o.c2 = p[i].c2;
        o.c3 = p[i].c3;
        o.rows = p[i].out->rows;
        o.cols = p[i].out->cols;
        o.kblocks = blocks_of(p[i]);
        o.chunk = p[i].chunk;
        o.p_kmajor = p[i].p_kmajor;
        o.q_kmajor = p[i].q_kmajor;
        o.symmetric = p[i].symmetric;
    }
    const uint32_t sms = static_cast<uint32_t>(shape.sms), pairs = sms / 2;
    const Plan plan = plan_of(p, n, items, kMany, sms);
    const bool pair = plan.pair;
    a.splits = plan.splits;
    a.tiles = 0;
    for (uint32_t i = 0; i < n; ++i) {
        Op& o = a.op[i];
        o.tiles_p = (o.rows + plan.side() - 1) / plan.side();
        o.tiles_q = (o.cols + plan.side() - 1) / plan.side();
        o.per = tiles_of(p[i], plan.side());
        o.first = a.tiles;
        a.tiles += o.per * items;
    }
    const uint32_t warps = pair ? 2 * kDrain<256> : kDrain<128>;
    for (uint32_t i = 0; kMany && i < n; ++i) {
        a.op[i].need = *count;
        *count += warps * a.op[i].per;
    }
    if constexpr (!kMany)
        if (a.splits > 1) return launch<1, 128, false, true>(a, sms, stream);
    return pair ? launch<2, 256, kMany, false>(a, pairs, stream) : launch<1, 128, kMany, false>(a, sms, stream);
}

}  // namespace

cudaError_t prepare_ortho(OrthoShape* shape) {
    if (shape->ready) return cudaSuccess;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&shape->sms, cudaDevAttrMultiProcessorCount, dev);
    const auto room = [&](const void* kernel, uint32_t smem) {
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    };
    room(reinterpret_cast<const void*>(ortho_product_kernel<2, 256, false, false>), kSmem<256>);
    room(reinterpret_cast<const void*>(ortho_product_kernel<2, 256, true, false>), kSmem<256>);
    room(reinterpret_cast<const void*>(ortho_product_kernel<1, 128, false, false>), kSmem<128>);
    room(reinterpret_cast<const void*>(ortho_product_kernel<1, 128, true, false>), kSmem<128>);
    room(reinterpret_cast<const void*>(ortho_product_kernel<1, 128, false, true>), kSmem<128>);
    if (e == cudaSuccess) e = tensor_map_encoder(&g_encode);
    shape->ready = e == cudaSuccess;
    return e;
}

cudaError_t map_ortho(OrthoBuf* b, uint32_t items) {
    return encode(&b->k, *b, items, kBK, 128, CU_TENSOR_MAP_SWIZZLE_128B) &&
                   encode(&b->mn, *b, items, 64, kBK, CU_TENSOR_MAP_SWIZZLE_128B) &&
                   encode(&b->out, *b, items, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B)
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

// Whether a list is launched one at a time: one matrix; turns enough that a part of one does not count; or
// tiles so few that splitting them is worth more (5 of 10192 x 40 bf16 160 us so and 366 by the list).
// *cost: the time.
static bool one_by_one(const OrthoProduct* p, uint32_t n, uint32_t items, uint32_t sms, double* cost) {
    uint64_t most = 0;
    double each = 0.0;
    for (uint32_t i = 0; i < n; ++i) {
        most = std::max<uint64_t>(most, (p[i].out->rows + 255ull) / 256 * ((p[i].out->cols + 255ull) / 256) * items);
        each += plan_of(p + i, 1, items, false, sms).cost;
    }
    const double list = n > 1 ? plan_of(p, n, items, true, sms).cost : each;
    const bool so = n == 1 || items == 1 || most > 8ull * sms / 2 || each < list;
    *cost = so ? each : list;
    return so;
}

double ortho_cost(const OrthoProduct* p, uint32_t n, uint32_t items, uint32_t sms) {
    double c = 0.0, part;
    for (uint32_t at = 0; at < n; at += kOrthoOps) {
        one_by_one(p + at, std::min(kOrthoOps, n - at), items, sms, &part);
        c += part;
    }
    return c;
}

cudaError_t launch_ortho_products(const OrthoProduct* p, uint32_t n, uint32_t items, uint32_t* done, uint32_t* count,
                                  const OrthoShape& shape, unsigned int* err, bool test_expire, cudaStream_t stream, uint64_t* launches) {
    if (n > kOrthoOps) return cudaErrorInvalidValue;
    double cost;
    if (n > 1 && one_by_one(p, n, items, static_cast<uint32_t>(shape.sms), &cost)) {
        cudaError_t e = cudaSuccess;
        for (uint32_t i = 0; i < n && e == cudaSuccess; ++i)
            e = launch_ortho_products(p + i, 1, items, done, count, shape, err, test_expire, stream, launches);
        return e;
    }
    *launches += 1;
    return n == 1 ? run<false>(p, n, items, done, count, shape, err, test_expire, stream)
                  : run<true>(p, n, items, done, count, shape, err, test_expire, stream);
}

}  // namespace fa
