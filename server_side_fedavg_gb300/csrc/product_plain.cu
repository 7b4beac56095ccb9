// Products on the FP32 units: those too small for the tensor cores, and few fp32 rows against
// a weight matrix, where reading the weights is the work.
#include "product_device.cuh"

namespace fa {

namespace {

constexpr int kBlockThreads = 256;

// ----------------------------------------------------------------- tiny products
// One output per kLanes lanes (1 or 32), any storage order.  Bound by launch and load latency: in a
// CUDA graph 4 x 10 x 256 bf16 takes 2.4 us (on the tensor cores 3.1).
template <int kLanes>
__global__ void __launch_bounds__(kBlockThreads) product_tiny_kernel(const __grid_constant__ ProdArgs p) {
    wait_predecessor();
    const uint64_t at = (blockIdx.x * static_cast<uint64_t>(kBlockThreads) + threadIdx.x) / kLanes;
    if (at >= static_cast<uint64_t>(p.m) * p.n) return;
    const uint32_t r = static_cast<uint32_t>(at / p.n), c = static_cast<uint32_t>(at - static_cast<uint64_t>(r) * p.n);
    const uint64_t sa = p.a.kmajor ? 1 : p.a.ld, sb = p.b.kmajor ? 1 : p.b.ld;
    const uint64_t a0 = p.a.kmajor ? r * p.a.ld : r, b0 = p.b.kmajor ? c * p.b.ld : c;
    float sum = 0.0f;
    for (uint32_t kk = threadIdx.x % kLanes; kk < p.k; kk += kLanes)
        sum = fmaf(elem(p.a.p, a0 + kk * sa, p.a.dtype), elem(p.b.p, b0 + kk * sb, p.b.dtype), sum);
#pragma unroll
    for (int d = kLanes / 2; d; d /= 2) sum += __shfl_xor_sync(~0u, sum, d);
    if (threadIdx.x % kLanes == 0) finish_one(p.e, sum, r, c);
}

// ----------------------------------------------------------------- few rows
// A CTA has kCols columns of the output (rows of b, which is K-major as a is) and walks over
// the rows of a in groups of kRows.  Its eight warps divide the summed index; a lane loads 16
// bytes of each of its rows at a time (kVec; else one element), so that a warp keeps
// kCols x 512 bytes of weights in flight.  Bound by HBM for the weights up to some 16 rows, by
// the FMA rate beyond.  Sums: per lane, then over the lanes by halving (a lane ends up with
// one output of the group), then over the warps in order.
// Measured in fp32: one row by 32000 x 4096 80 us, 6.6 TB/s (97 % of the measured copy rate);
// 16 rows by 4096 x 4096 23.5 us.
template <int kRows>
constexpr int kCols = kRows == 8 ? 8 : 4;      // 8 x 8: as many loads from L1 as FMAs can feed on

// Value i of a group of kN, summed over the lanes, ends in the lanes with lane % kN == i.
template <int kN, int kAll = kN>
__device__ __forceinline__ float reduce_lanes(const float (&v)[kN]) {
    constexpr int kHalf = kN / 2;
    const bool up = threadIdx.x & kHalf;
    float h[kHalf];
#pragma unroll
    for (int i = 0; i < kHalf; ++i)
        h[i] = (up ? v[i + kHalf] : v[i]) + __shfl_xor_sync(~0u, up ? v[i] : v[i + kHalf], kHalf);
    if constexpr (kHalf > 1) {
        return reduce_lanes<kHalf, kAll>(h);
    } else {
#pragma unroll
        for (int d = kAll; d < 32; d *= 2) h[0] += __shfl_xor_sync(~0u, h[0], d);
        return h[0];
    }
}

template <typename T, bool kVec>
struct Piece {                          // what a lane loads of a row at a time
    static constexpr int kElems = kVec ? 16 / sizeof(T) : 1;
    float x[kElems];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (!kVec) {
            x[0] = elem(p, 0, sizeof(T) == 2);
        } else if constexpr (sizeof(T) == 2) {
            plain_vec8(p, x);
        } else {
            const float4 v = *reinterpret_cast<const float4*>(p);
            x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
        }
    }
};

template <typename T, int kRows, bool kVec>
__global__ void __launch_bounds__(kBlockThreads) product_thin_kernel(const __grid_constant__ ProdArgs p) {
    constexpr int kC = kCols<kRows>, kWarps = kBlockThreads / 32, kOut = kRows * kC, kE = Piece<T, kVec>::kElems;
    constexpr int kGroup = kOut < 32 ? kOut : 32;
    __shared__ float part[kWarps][kOut];
    wait_predecessor();
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint32_t c0 = blockIdx.x * kC;
    const T *a = static_cast<const T*>(p.a.p), *b = static_cast<const T*>(p.b.p);
    const T* rows[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) rows[c] = b + min(c0 + c, p.n - 1) * p.b.ld;     // past the end: the last row again
    for (uint32_t r0 = 0; r0 < p.m; r0 += kRows) {
        float acc[kOut] = {};
        for (uint32_t k0 = (warp * 32 + lane) * kE; k0 < p.k; k0 += kBlockThreads * kE) {
            Piece<T, kVec> w[kC];
#pragma unroll
            for (int c = 0; c < kC; ++c) w[c].load(rows[c] + k0);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                Piece<T, kVec> x;
                x.load(a + min(r0 + r, p.m - 1) * p.a.ld + k0);
#pragma unroll
                for (int c = 0; c < kC; ++c)
#pragma unroll
                    for (int i = 0; i < kE; ++i) acc[r * kC + c] = fmaf(x.x[i], w[c].x[i], acc[r * kC + c]);
            }
        }
#pragma unroll
        for (int g = 0; g < kOut; g += kGroup) {
            float v[kGroup];
#pragma unroll
            for (int i = 0; i < kGroup; ++i) v[i] = acc[g + i];
            const float mine = reduce_lanes<kGroup>(v);
            if (lane < kGroup) part[warp][g + lane] = mine;
        }
        __syncthreads();
        if (threadIdx.x < kOut) {
            float sum = 0.0f;
            for (int w = 0; w < kWarps; ++w) sum += part[w][threadIdx.x];
            const uint32_t r = r0 + threadIdx.x / kC, c = c0 + threadIdx.x % kC;
            if (r < p.m && c < p.n) finish_one(p.e, sum, r, c);
        }
        __syncthreads();
    }
}

// The same with b stored [k, n]: a lane per column (kVec: two), the eight warps and up to eight
// CTAs of a cluster divide the summed index; a's rows are staged in shared memory, transposed,
// and read as broadcasts.  Sums: per lane, over the warps in order, over the cluster in order.
// Bound by the latency of a warp's walk down its share of the rows.  Measured: 8 rows by
// 4096 x 4096 fp32 15.5 us, 4.3 TB/s.
constexpr int kStage = 256;            // summed elements of a staged at a time

template <typename T, int kRows, bool kVec>
__global__ void __launch_bounds__(kBlockThreads) product_thin_n_kernel(const __grid_constant__ ProdArgs p, uint32_t splits) {
    constexpr int kWarps = kBlockThreads / 32, kC = kVec ? 2 : 1, kOut = kRows * 32 * kC;
    __shared__ __align__(16) float staged[kStage][kRows];
    __shared__ float part[kWarps][kOut];
    wait_predecessor();
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const uint32_t c0 = blockIdx.x / splits * 32 * kC, col = c0 + lane * kC;
    const uint32_t k_lo = static_cast<uint64_t>(p.k) * rank / splits, k_hi = static_cast<uint64_t>(p.k) * (rank + 1) / splits;
    const T *a = static_cast<const T*>(p.a.p), *b = static_cast<const T*>(p.b.p) + min(col, p.n - kC);
    for (uint32_t r0 = 0; r0 < p.m; r0 += kRows) {
        float acc[kRows][kC] = {};
        for (uint32_t k0 = k_lo; k0 < k_hi; k0 += kStage) {
            const uint32_t many = min(static_cast<uint32_t>(kStage), k_hi - k0);
            __syncthreads();
            for (uint32_t i = threadIdx.x; i < kStage * kRows; i += kBlockThreads) {
                const uint32_t r = i / kStage, kk = i % kStage;
                staged[kk][r] = kk < many && r0 + r < p.m ? elem(a, (r0 + r) * p.a.ld + k0 + kk, sizeof(T) == 2) : 0.0f;
            }
            __syncthreads();
#pragma unroll 8
            for (uint32_t kk = warp; kk < many; kk += kWarps) {
                float w[kC];
                const T* at = b + (k0 + kk) * p.b.ld;
                if constexpr (kVec && sizeof(T) == 4) {
                    const float2 v = *reinterpret_cast<const float2*>(at);
                    w[0] = v.x;
                    w[1] = v.y;
                } else if constexpr (kVec) {
                    const uint32_t v = *reinterpret_cast<const uint32_t*>(at);
                    w[0] = bf16_lo(v);
                    w[1] = bf16_hi(v);
                } else {
                    w[0] = elem(at, 0, sizeof(T) == 2);
                }
#pragma unroll
                for (int r = 0; r < kRows; ++r)
#pragma unroll
                    for (int c = 0; c < kC; ++c) acc[r][c] = fmaf(staged[kk][r], w[c], acc[r][c]);
            }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int c = 0; c < kC; ++c) part[warp][(r * 32 + lane) * kC + c] = acc[r][c];
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < kOut; i += kBlockThreads) {
            float sum = part[0][i];
            for (int w = 1; w < kWarps; ++w) sum += part[w][i];
            part[0][i] = sum;
        }
        if (splits > 1) {
            asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
            if (rank != 0) {
                // rank 0 reads this CTA's sums before it goes on
                asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
                continue;
            }
        } else {
            __syncthreads();
        }
        for (uint32_t i = threadIdx.x; i < kOut; i += kBlockThreads) {
            float sum = part[0][i];
            for (uint32_t q = 1; q < splits; ++q) {
                float v;
                asm volatile("{\n .reg .u32 r;\n mapa.shared::cluster.u32 r, %1, %2;\n ld.shared::cluster.f32 %0, [r];\n}"
                             : "=f"(v)
                             : "r"(smem_addr(&part[0][i])), "r"(q)
                             : "memory");
                sum += v;
            }
            const uint32_t r = r0 + i / (32 * kC), c = c0 + i % (32 * kC);
            if (r < p.m && c < p.n) finish_one(p.e, sum, r, c);
        }
        if (splits > 1) asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        __syncthreads();
    }
}

template <typename T, int kRows, bool kVec>
cudaError_t thin_n(const ProdArgs& p, cudaStream_t stream) {
    const uint32_t cols = kVec ? 64 : 32, blocks = (p.n + cols - 1) / cols;
    // enough CTAs for four per SM, each with a stage's worth of the sum
    uint32_t splits = 1;
    while (splits < 8 && blocks * splits < 608 && p.k >= splits * 2 * 64) splits *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks * splits);
    cfg.blockDim = dim3(kBlockThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = splits;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, product_thin_n_kernel<T, kRows, kVec>, p, splits);
}

template <typename T, bool kVec>
cudaError_t thin_n_rows(const ProdArgs& p, cudaStream_t stream) {
    if (p.m == 1) return thin_n<T, 1, kVec>(p, stream);
    if (p.m <= 4) return thin_n<T, 4, kVec>(p, stream);
    return thin_n<T, 8, kVec>(p, stream);
}

template <typename T, bool kVec>
cudaError_t thin(const ProdArgs& p, cudaStream_t stream) {
    if (p.m == 1)
        return launch_next(product_thin_kernel<T, 1, kVec>, dim3((p.n + kCols<1> - 1) / kCols<1>), kBlockThreads, stream, p);
    if (p.m <= 4)
        return launch_next(product_thin_kernel<T, 4, kVec>, dim3((p.n + kCols<4> - 1) / kCols<4>), kBlockThreads, stream, p);
    return launch_next(product_thin_kernel<T, 8, kVec>, dim3((p.n + kCols<8> - 1) / kCols<8>), kBlockThreads, stream, p);
}

}  // namespace

cudaError_t launch_product_tiny(const ProdArgs& p, cudaStream_t stream) {
    // short sums: a thread per output
    const uint64_t lanes = p.k <= 32 ? 1 : 32;
    const uint64_t grid = (static_cast<uint64_t>(p.m) * p.n * lanes + kBlockThreads - 1) / kBlockThreads;
    if (grid >= (1ull << 31)) return cudaErrorInvalidConfiguration;
    return launch_next(lanes == 1 ? product_tiny_kernel<1> : product_tiny_kernel<32>, dim3(static_cast<uint32_t>(grid)),
                       kBlockThreads, stream, p);
}

cudaError_t launch_product_thin(const ProdArgs& p, cudaStream_t stream) {
    const uint64_t size = p.a.dtype ? 2 : 4;
    if (!p.b.kmajor) {
        const bool two = reinterpret_cast<uintptr_t>(p.b.p) % (2 * size) == 0 && p.b.ld % 2 == 0 && p.n % 2 == 0;
        if (p.a.dtype) return two ? thin_n_rows<uint16_t, true>(p, stream) : thin_n_rows<uint16_t, false>(p, stream);
        return two ? thin_n_rows<float, true>(p, stream) : thin_n_rows<float, false>(p, stream);
    }
    const auto aligned = [&](const ProdOperand& o) {
        return reinterpret_cast<uintptr_t>(o.p) % 16 == 0 && o.ld * size % 16 == 0;
    };
    const bool vec = aligned(p.a) && aligned(p.b) && p.k * size % 16 == 0;
    if (p.a.dtype) return vec ? thin<uint16_t, true>(p, stream) : thin<uint16_t, false>(p, stream);
    return vec ? thin<float, true>(p, stream) : thin<float, false>(p, stream);
}

}  // namespace fa
