// The first pass and the last of an orthogonalised weight step: momentum and the update's norm, the
// scaled update as two fp16 terms, and the result joined to the weight.  Streaming passes, bound by
// HBM.
#include <algorithm>

#include <cuda_fp16.h>

#include "ortho.cuh"
#include "product_device.cuh"

namespace fa {

namespace {

constexpr uint32_t kEndThreads = 256;

// Eight elements of a row from column c on; those past its end as 0.
__device__ __forceinline__ void load8(const OrthoMat& m, uint64_t row_at, uint32_t c, uint32_t cols, bool vec, float (&x)[8]) {
    if (vec && c + 8 <= cols) {
        if (m.dtype)
            plain_vec8(static_cast<const uint16_t*>(m.p) + row_at + c, x);
        else
            plain_vec8(static_cast<const float*>(m.p) + row_at + c, x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = c + i < cols ? elem(m.p, row_at + c + i, m.dtype) : 0.0f;
    }
}

__device__ __forceinline__ void store8(const OrthoMat& m, uint64_t row_at, uint32_t c, uint32_t cols, bool vec, const float (&x)[8]) {
    void* p = const_cast<void*>(m.p);
    if (vec && c + 8 <= cols) {
        if (m.dtype)
            store8_global<uint16_t>(p, row_at + c, x);
        else
            store8_global<float>(p, row_at + c, x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < cols) put(p, row_at + c + i, m.dtype, x[i]);
    }
}

struct Vecs {
    bool update, momentum, momentum_out, residual, out;
};

__device__ __forceinline__ uint64_t row_of(const OrthoMat& m, uint32_t item, uint32_t r) { return item * m.step + r * m.ld; }

// g' = mu m + u, to `g`; x = u + mu g' or g'.  kept: g' is read from momentum_out, where the first
// pass has put it (over m, it may be).
__device__ __forceinline__ void step_of(const OrthoEnds& a, const Vecs& v, uint32_t item, uint32_t r, uint32_t c, bool kept,
                                        float (&x)[8], float (&g)[8]) {
    load8(a.update, row_of(a.update, item, r), c, a.cols, v.update, x);
    if (kept && a.momentum_out.p) {
        load8(a.momentum_out, row_of(a.momentum_out, item, r), c, a.cols, v.momentum_out, g);
    } else if (a.momentum.p) {
        load8(a.momentum, row_of(a.momentum, item, r), c, a.cols, v.momentum, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = fmaf(a.mu, g[i], x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = x[i];
        if (!a.momentum_out.p) return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = a.nesterov ? fmaf(a.mu, g[i], x[i]) : g[i];
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

__global__ void __launch_bounds__(kEndThreads) ortho_norm_kernel(const __grid_constant__ OrthoEnds a, Vecs v) {
    __shared__ double sums[kEndThreads / 32];
    wait_predecessor();
    const uint32_t item = blockIdx.y, per = (a.cols + 7) / 8, all = per * a.rows;
    double s = 0.0;
    for (uint32_t i = blockIdx.x * kEndThreads + threadIdx.x; i < all; i += gridDim.x * kEndThreads) {
        const uint32_t r = i / per, c = (i - r * per) * 8;
        float x[8], g[8];
        step_of(a, v, item, r, c, false, x, g);
        if (a.momentum_out.p) store8(a.momentum_out, row_of(a.momentum_out, item, r), c, a.cols, v.momentum_out, g);
        // eight squares in fp32 where none can leave its range, else in fp64
        float most = 0.0f, q = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            most = fmaxf(most, fabsf(x[j]));
            q = fmaf(x[j], x[j], q);
        }
        if (most < 0x1p60f && (most > 0x1p-40f || most == 0.0f) && q == q) {
            s += static_cast<double>(q);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) s += static_cast<double>(x[j]) * static_cast<double>(x[j]);
        }
    }
    s = warp_sum(s);
    if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x > 0) return;
    for (uint32_t w = 1; w < kEndThreads / 32; ++w) s += sums[w];
    a.part[static_cast<uint64_t>(item) * a.blocks + blockIdx.x] = s;
}

// x / (|x| + eps) * 2^shift as two fp16 terms.
__global__ void __launch_bounds__(kEndThreads) ortho_scale_kernel(const __grid_constant__ OrthoEnds a, Vecs v) {
    __shared__ float factor[2];
    wait_predecessor();
    const uint32_t item = blockIdx.y, per = static_cast<uint32_t>(a.ld / 8), all = per * a.rows;
    if (threadIdx.x < 32) {
        double s = 0.0;
        for (uint32_t i = threadIdx.x; i < a.blocks; i += 32) s += a.part[static_cast<uint64_t>(item) * a.blocks + i];
        s = warp_sum(s);
        if (threadIdx.x == 0) {
            // the factor as a fraction of 1 and a power of two, which fp32 has down to 2^-149
            int e;
            factor[0] = static_cast<float>(frexp(1.0 / (sqrt(s) + a.eps), &e));
            factor[1] = ldexpf(1.0f, e + a.shift);
        }
    }
    __syncthreads();
    const float f0 = factor[0], f1 = factor[1];
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

bool vec_ok(const OrthoMat& m, uint32_t items) {
    const uint64_t size = m.dtype ? 2 : 4;
    return reinterpret_cast<uintptr_t>(m.p) % 16 == 0 && m.ld * size % 16 == 0 && (items == 1 || m.step * size % 16 == 0);
}

Vecs vecs(const OrthoEnds& a) {
    return {vec_ok(a.update, a.items), vec_ok(a.momentum, a.items), vec_ok(a.momentum_out, a.items), vec_ok(a.residual, a.items),
            vec_ok(a.out, a.items)};
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
