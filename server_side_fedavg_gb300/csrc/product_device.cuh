// Device helpers of the product kernels: typed element access, activations and their
// derivatives, the epilogue's arithmetic.  Internal linkage: each kernel file compiles its
// own copy.
#pragma once

#include "device.cuh"
#include "product.cuh"

namespace fa {

namespace {

constexpr int kActRelu = 1, kActGelu = 2, kActSilu = 3;

// Element e of an array of dtype code dt (0 fp32, 1 bf16), plain (coherent) loads.
__device__ __forceinline__ float elem(const void* p, uint64_t e, int dt) {
    return dt ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[e]) << 16)
              : static_cast<const float*>(p)[e];
}

__device__ __forceinline__ void put(void* p, uint64_t e, int dt, float v) {
    if (dt)
        static_cast<uint16_t*>(p)[e] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    else
        static_cast<float*>(p)[e] = v;
}

// exp(x), off by up to 2^-22 and |x| 2^-23 of its value.
__device__ __forceinline__ float exp_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}

// Phi(z), the normal distribution: its tail beyond |z| is exp(-z^2 / 2) times a polynomial in
// t = 1 / (1 + 0.48 |z|), fitted to it here by weighted least squares, relative error up to 8.6e-8
// for |z| up to 14.  With so large a factor of |z| the rounding of t costs little at 0: over
// normally distributed z gelu in fp32 is off by 2.5e-8 (root mean square), as z times half of
// 1 + erf is, its derivative by 3.8e-8 (2.8e-8); below -1 both are relatively exact.  `bell`
// receives exp(-z^2 / 2), which the derivative needs too.  A third of the instructions of erff and
// expf, with which the activation gradient took 27 us at 2056 x 4096 (now 17).  Five terms, good to
// 1.5e-7 absolute (2.2 times the error over normal z), saved 1 % of bf16 products and gradients with gelu.
__device__ __forceinline__ float normal_cdf(float z, float& bell) {
    const float t = __fdividef(1.0f, fmaf(0.48f, fabsf(z), 1.0f));
    float s = fmaf(t, 0.053876061f, -0.282321781f);
    s = fmaf(t, s, 0.584696114f);
    s = fmaf(t, s, -0.54503572f);
    s = fmaf(t, s, 0.137284324f);
    s = fmaf(t, s, 0.0152480444f);
    s = fmaf(t, s, 0.153758347f);
    s = fmaf(t, s, 0.19098562f);
    s = fmaf(t, s, 0.191509038f);
    bell = exp_fast(-0.5f * z * z);
    const float tail = t * s * bell;
    return z >= 0.0f ? 1.0f - tail : tail;
}

// act(z).  A NaN stays a NaN in each.
__device__ __forceinline__ float act_fwd(int act, float z) {
    if (act == kActRelu) return z < 0.0f ? 0.0f : z;
    if (act == kActGelu) {
        float bell;
        return z * normal_cdf(z, bell);
    }
    if (act == kActSilu) return __fdividef(z, 1.0f + exp_fast(-z));
    return z;
}

// act'(z):  relu [z > 0];  gelu Phi(z) + z phi(z);  silu s (1 + z (1 - s)), s = 1 / (1 + exp(-z)).
__device__ __forceinline__ float act_grad(int act, float z) {
    if (act == kActRelu) return z > 0.0f ? 1.0f : 0.0f;
    if (act == kActGelu) {
        float bell;
        const float cdf = normal_cdf(z, bell);
        return fmaf(z * bell, 0.39894228040143268f, cdf);
    }
    if (act == kActSilu) {
        const float s = __fdividef(1.0f, 1.0f + exp_fast(-z));
        return s * fmaf(z, 1.0f - s, 1.0f);
    }
    return 1.0f;
}

// One output element from its fp32 sum: bias, activation and residual in fp32, one
// rounding at the store.
__device__ __forceinline__ void finish_one(const ProdEpilogue& e, float sum, uint64_t row, uint32_t col) {
    float z = e.alpha * sum;
    if (e.bias) z += elem(e.bias, col, e.bias_dtype);
    if (e.pre) put(e.pre, row * e.ldo + col, e.out_dtype, z);
    float y = act_fwd(e.act, z);
    if (e.res) y = fmaf(e.beta, elem(e.res, row * e.ldr + col, e.out_dtype), y);
    put(e.out, row * e.ldo + col, e.out_dtype, y);
}

// Every kernel of the products is launched as a programmatic dependent of its predecessor on the
// stream: its launch and set-up overlap that kernel's end.  Each thread begins with
// wait_predecessor before it touches global memory.
__device__ __forceinline__ void wait_predecessor() {
    asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;" ::: "memory");
}

template <typename... Params, typename... Args>
cudaError_t launch_next(void (*kern)(Params...), dim3 grid, uint32_t block, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
}

}  // namespace

}  // namespace fa
