// The first pass and the last of an orthogonalised weight step: momentum and the update's norm, the
// scaled update as two fp16 terms, and the result joined to the weight.  Streaming passes, bound by
// HBM: the three of 24 of 1024 x 1024 bf16 with momentum and weight take 116 us, 6.1 TB/s of what they
// read and write.  (The norm has to be known before the first term, so the update is read twice.)
#include <algorithm>

#include <cuda_fp16.h>

#include "ortho_device.cuh"

namespace fa {

namespace {

constexpr uint32_t kEndThreads = 256;

__global__ void __launch_bounds__(kEndThreads) ortho_norm_kernel(const __grid_constant__ OrthoEnds a, Vecs v) {
    __shared__ Squares sums[kEndThreads / 32];
    wait_predecessor();
    const uint32_t item = blockIdx.y, per = (a.cols + 7) / 8, all = per * a.rows;
    Squares s;
    for (uint32_t i = blockIdx.x * kEndThreads + threadIdx.x; i < all; i += gridDim.x * kEndThreads) {
        const uint32_t r = i / per, c = (i - r * per) * 8;
        float x[8], g[8];
        step_of(a, v, item, r, c, false, x, g);
        if (a.momentum_out.p) store8(a.momentum_out, row_of(a.momentum_out, item, r), c, a.cols, v.momentum_out, g);
        s.add(x);
    }
    s.over_warp();
    if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x > 0) return;
    if (blockIdx.x == 0) a.done[item] = 0;
    for (uint32_t w = 1; w < kEndThreads / 32; ++w) s.add(sums[w]);
    a.part[static_cast<uint64_t>(item) * a.blocks + blockIdx.x] = make_float3(s.mid, s.high, s.low);
}

// x / (|x| + eps) * 2^shift as two fp16 terms.
__global__ void __launch_bounds__(kEndThreads) ortho_scale_kernel(const __grid_constant__ OrthoEnds a, Vecs v) {
    __shared__ float2 factor;
    wait_predecessor();
    const uint32_t item = blockIdx.y, per = static_cast<uint32_t>(a.ld / 8), all = per * a.rows;
    if (threadIdx.x < 32) {
        Squares s;
        for (uint32_t i = threadIdx.x; i < a.blocks; i += 32) {
            const float3 p = a.part[static_cast<uint64_t>(item) * a.blocks + i];
            s.mid += p.x;
            s.high += p.y;
            s.low += p.z;
        }
        s.over_warp();
        if (threadIdx.x == 0) {
            factor = s.factor(a.eps);
            factor.x = ldexpf(factor.x, a.shift);
        }
    }
    __syncthreads();
    const float f0 = factor.x, f1 = factor.y;
    const uint64_t plane = a.rows * a.ld;
    uint16_t* to = a.x + 2 * item * plane;
    for (uint32_t i = blockIdx.x * kEndThreads + threadIdx.x; i < all; i += gridDim.x * kEndThreads) {
        const uint32_t r = i / per, c = (i - r * per) * 8;
        float x[8], g[8];
        step_of(a, v, item, r, c, true, x, g);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float p = x[2 * j] * f1 * f0, q = x[2 * j + 1] * f1 * f0;
            const __half2 h = __floats2half2_rn(p, q);
            const float2 f = __half22float2(h);
            const __half2 l = __floats2half2_rn(p - f.x, q - f.y);
            hi[j] = *reinterpret_cast<const uint32_t*>(&h);
            lo[j] = *reinterpret_cast<const uint32_t*>(&l);
        }
        const uint64_t at = static_cast<uint64_t>(i) * 8;
        st_v4u(to + at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
        st_v4u(to + plane + at, make_uint4(lo[0], lo[1], lo[2], lo[3]));
    }
}

// out = alpha * (hi + lo) + beta * residual, rounded once.
__global__ void __launch_bounds__(kEndThreads) ortho_finish_kernel(const __grid_constant__ OrthoEnds a, Vecs v) {
    wait_predecessor();
    const uint32_t item = blockIdx.y, per = static_cast<uint32_t>(a.ld / 8), all = per * a.rows;
    const uint64_t plane = a.rows * a.ld;
    const uint16_t* from = a.x + 2 * item * plane;
    for (uint32_t i = blockIdx.x * kEndThreads + threadIdx.x; i < all; i += gridDim.x * kEndThreads) {
        const uint32_t r = i / per, c = (i - r * per) * 8;
        const uint64_t at = static_cast<uint64_t>(i) * 8;
        const uint4 h = ld_plain_v4(from + at), l = ld_plain_v4(from + plane + at);
        const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
        float x[8], res[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&hw[j]));
            const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&lw[j]));
            x[2 * j] = a.alpha * (p.x + q.x);
            x[2 * j + 1] = a.alpha * (p.y + q.y);
        }
        if (a.residual.p) {
            load8(a.residual, row_of(a.residual, item, r), c, a.cols, v.residual, res);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = fmaf(a.beta, res[j], x[j]);
        }
        store8(a.out, row_of(a.out, item, r), c, a.cols, v.out, x);
    }
}

}  // namespace

// Blocks per item: eight per SM over all items, with two steps for a thread at least where there are fewer.
uint32_t ortho_blocks(uint32_t items, uint32_t rows, uint32_t cols, uint32_t sms) {
    const uint64_t steps = (static_cast<uint64_t>(rows) * ((cols + 7) / 8) + kEndThreads - 1) / kEndThreads;
    const uint64_t most = std::max<uint64_t>(1, 8ull * sms / items);
    return static_cast<uint32_t>(std::max<uint64_t>(1, std::min<uint64_t>((steps + 1) / 2, most)));
}

cudaError_t launch_ortho_norm(const OrthoEnds& a, cudaStream_t stream) {
    return launch_next(ortho_norm_kernel, dim3(a.blocks, a.items), kEndThreads, stream, a, vecs(a));
}

cudaError_t launch_ortho_scale(const OrthoEnds& a, cudaStream_t stream) {
    return launch_next(ortho_scale_kernel, dim3(a.blocks, a.items), kEndThreads, stream, a, vecs(a));
}

cudaError_t launch_ortho_finish(const OrthoEnds& a, cudaStream_t stream) {
    return launch_next(ortho_finish_kernel, dim3(a.blocks, a.items), kEndThreads, stream, a, vecs(a));
}

}  // namespace fa
