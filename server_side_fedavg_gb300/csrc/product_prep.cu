// What goes before the products: operands laid out as bf16 planes, and the elementwise part
// of the gradients with the bias gradient's column sums.  Streaming passes, bound by HBM (or L2,
// which holds what a pass has just written for the product after it).  Measured: 6262 x 7231
// fp32 into three planes 71 us, 6.4 TB/s of bytes read and written; gelu's gradient of
// 2056 x 4096 bf16 with the column sums 17 us, issue slots 59 % busy with the activations.
// Two operands of one product share a launch (777 x 1024 and 4096 x 1024 fp32: 48.0 us for the
// product and its passes in two launches, 44.6 in one).
#include <algorithm>

#include "product_device.cuh"

namespace fa {

namespace {

// x as three bf16 terms: each the remainder so far rounded to nearest even, so that 24 bits
// of x are kept.  A finite x that would round to infinity takes the largest finite bf16
// first.  An infinity or NaN is the first term alone.
__device__ __forceinline__ void split3(float x, uint16_t (&t)[3]) {
    uint16_t h = __bfloat16_as_ushort(__float2bfloat16_rn(x));
    if ((h & 0x7FFF) == 0x7F80 && isfinite(x)) h = (h & 0x8000) | 0x7F7F;
    t[0] = h;
    t[1] = t[2] = 0;
    if (!isfinite(x)) return;
    float r = x - __uint_as_float(static_cast<uint32_t>(h) << 16);     // exact
    t[1] = __bfloat16_as_ushort(__float2bfloat16_rn(r));
    r -= __uint_as_float(static_cast<uint32_t>(t[1]) << 16);           // exact
    t[2] = __bfloat16_as_ushort(__float2bfloat16_rn(r));
}

// Eight values to each of the planes at element `at` (a multiple of 8 from a 16-byte
// aligned base).
__device__ __forceinline__ void store_planes(uint16_t* dst, uint64_t at, uint64_t plane, int planes,
                                             const float (&x)[8]) {
    if (planes == 1) {
        store8_global<uint16_t>(dst, at, x);
        return;
    }
    uint32_t w[3][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint16_t lo[3], hi[3];
        split3(x[2 * i], lo);
        split3(x[2 * i + 1], hi);
#pragma unroll
        for (int p = 0; p < 3; ++p) w[p][i] = lo[p] | static_cast<uint32_t>(hi[p]) << 16;
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) st_v4u(dst + p * plane + at, make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]));
}

// Columns c .. c + 7 of a row of `cols` (those past its end as 0).
__device__ __forceinline__ void load8(const void* p, uint64_t row_at, uint32_t c, uint32_t cols, int dt, bool vec,
                                      float (&x)[8]) {
    if (vec && c + 8 <= cols) {
        if (dt)
            plain_vec8(static_cast<const uint16_t*>(p) + row_at + c, x);
        else
            plain_vec8(static_cast<const float*>(p) + row_at + c, x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = c + i < cols ? elem(p, row_at + c + i, dt) : 0.0f;
    }
}

// Eight elements per thread and step, rows in turn; the blocks from `second` on have the second
// operand.
struct SplitArgs {
    SplitJob job[2];
    bool vec[2];
    uint32_t second;
};

__global__ void __launch_bounds__(256) split_kernel(const __grid_constant__ SplitArgs a) {
    wait_predecessor();
    const bool last = blockIdx.x >= a.second;
    const SplitJob& j = a.job[last];
    const uint32_t block = last ? blockIdx.x - a.second : blockIdx.x, blocks = last ? gridDim.x - a.second : a.second;
    const void* src = j.src;
    const bool vec = a.vec[last];
    const int dtype = j.dtype;
    const uint32_t cols = j.cols, planes = j.planes;
    const uint64_t ld = j.ld, ldd = j.ldd, per = ldd / 8, all = per * j.rows, plane = j.rows * ldd;
    uint16_t* dst = static_cast<uint16_t*>(j.dst);
    for (uint64_t i = block * 256ull + threadIdx.x; i < all; i += blocks * 256ull) {
        const uint64_t r = i / per;
        const uint32_t c = static_cast<uint32_t>(i - r * per) * 8;
        float x[8];
        load8(src, r * ld, c, cols, dtype, vec, x);
        store_planes(dst, r * ldd + c, plane, planes, x);
    }
}

template <int kAct>
__device__ __forceinline__ void times_grad(float (&d)[8], const float (&z)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j] *= act_grad(kAct, z[j]);
}

// Columns c .. c + 7 at p (those past the row's end as 0).
template <typename T>
__device__ __forceinline__ void load8t(const T* p, uint32_t c, uint32_t cols, bool vec, float (&x)[8]) {
    if (vec && c + 8 <= cols)
        plain_vec8(p, x);
    else
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = c + i < cols ? elem(p, i, sizeof(T) == 2) : 0.0f;
}

// A block of a.rows rows by 256 columns per CTA: a lane holds 8 columns, a warp every
// eighth row; the column sums join over the warps in warp order.
template <typename T>
__global__ void __launch_bounds__(256, 4) act_grad_kernel(const __grid_constant__ ActGradArgs a, bool vec, bool vz) {
    __shared__ float sums[8][256];
    wait_predecessor();
    const uint32_t c = blockIdx.x * 256 + threadIdx.x % 32 * 8, warp = threadIdx.x / 32;
    const uint32_t blocks = (a.m + a.rows - 1) / a.rows;
    const uint64_t plane = a.m * a.ldz;
    const T *dout = static_cast<const T*>(a.dout), *pre = static_cast<const T*>(a.pre);
    for (uint32_t blk = blockIdx.y; blk < blocks; blk += gridDim.y) {
        float s[8] = {};
        if (c < a.n)
            // a row at a time, in small code: four CTAs per SM keep 32 KB of loads in flight
#pragma unroll 1
            for (uint32_t r = blk * a.rows + warp; r < min(a.m, (blk + 1) * a.rows); r += 8) {
                float d[8], z[8];
                load8t(dout + r * a.ldd + c, c, a.n, vec, d);
                if (pre) load8t(pre + r * a.ldp + c, c, a.n, vec, z);
                if (a.act == kActGelu)
                    times_grad<kActGelu>(d, z);
                else if (a.act == kActSilu)
                    times_grad<kActSilu>(d, z);
                else if (a.act == kActRelu)
                    times_grad<kActRelu>(d, z);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] += d[j];
                if (!a.dz) continue;
                if (a.dz_planes) {
                    store_planes(static_cast<uint16_t*>(a.dz), r * a.ldz + c, plane, a.dz_planes, d);
                } else if (vz && c + 8 <= a.n) {
                    store8_global<float>(a.dz, r * a.ldz + c, d);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (c + j < a.n) static_cast<float*>(a.dz)[r * a.ldz + c + j] = d[j];
                }
            }
        if (!a.part) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) sums[warp][threadIdx.x % 32 * 8 + j] = s[j];
        __syncthreads();
        const uint32_t col = blockIdx.x * 256 + threadIdx.x;
        if (col < a.n) {
            float t = 0.0f;
            for (int w = 0; w < 8; ++w) t += sums[w][threadIdx.x];
            a.part[static_cast<uint64_t>(blk) * a.n + col] = t;
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(256) col_sum_kernel(const float* part, uint32_t blocks, uint32_t n, void* out,
                                                      int out_dtype) {
    wait_predecessor();
    const uint32_t c = blockIdx.x * 256 + threadIdx.x;
    if (c >= n) return;
    float s = 0.0f;
#pragma unroll 16
    for (uint32_t b = 0; b < blocks; ++b) s += part[static_cast<uint64_t>(b) * n + c];
    put(out, c, out_dtype, s);
}

bool vec_ok(const void* p, uint64_t ld, int dtype) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (dtype ? 2 : 4) % 16 == 0;
}

}  // namespace

cudaError_t launch_split(const SplitJob* jobs, int n, cudaStream_t stream) {
    constexpr uint64_t kMost = 152 * 8;
    SplitArgs a = {};
    uint64_t blocks[2] = {};
    for (int i = 0; i < n; ++i) {
        a.job[i] = jobs[i];
        a.vec[i] = vec_ok(jobs[i].src, jobs[i].ld, jobs[i].dtype);
        blocks[i] = (jobs[i].ldd / 8 * jobs[i].rows + 255) / 256;
    }
    // shares of the most that run at one time, at least one each
    const uint64_t all = blocks[0] + blocks[1];
    if (all > kMost)
        for (int i = 0; i < n; ++i) blocks[i] = std::max<uint64_t>(1, blocks[i] * kMost / all);
    a.second = static_cast<uint32_t>(blocks[0]);
    return launch_next(split_kernel, dim3(static_cast<uint32_t>(blocks[0] + blocks[1])), 256, stream, a);
}

cudaError_t launch_act_grad(const ActGradArgs& a, cudaStream_t stream) {
    const uint32_t blocks = (a.m + a.rows - 1) / a.rows;
    return launch_next(a.dtype ? act_grad_kernel<uint16_t> : act_grad_kernel<float>,
                       dim3((a.n + 255) / 256, blocks < 65535 ? blocks : 65535), 256, stream, a,
                       vec_ok(a.dout, a.ldd, a.dtype) && vec_ok(a.pre, a.ldp, a.dtype), vec_ok(a.dz, a.ldz, 0));
}

cudaError_t launch_col_sum(const float* part, uint32_t blocks, uint32_t n, void* out, int out_dtype,
                           cudaStream_t stream) {
    return launch_next(col_sum_kernel, dim3((n + 255) / 256), 256, stream, part, blocks, n, out, out_dtype);
}

}  // namespace fa
