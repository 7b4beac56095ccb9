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

// Phi(z), the normal distribution, by the rational approximation 7.1.26 of Abramowitz and Stegun,
// "Handbook of Mathematical Functions": erfc(x) = exp(-x^2) (a1 t + ... + a5 t^5), t = 1 / (1 + p x),
// for x >= 0, absolute error up to 1.5e-7 -- of the size of fp32's rounding of Phi near 1.  `bell`
// receives exp(-z^2 / 2), which the derivative needs too.  A third of the instructions of erff
// and expf, which bounded the activation gradient (27 us at 2056 x 4096).
__device__ __forceinline__ float normal_cdf(float z, float& bell) {
    const float t = __fdividef(1.0f, fmaf(0.3275911f * 0.70710678118654752f, fabsf(z), 1.0f));
    float s = fmaf(t, 1.061405429f, -1.453152027f);
    s = fmaf(t, s, 1.421413741f);
    s = fmaf(t, s, -0.284496736f);
    s = fmaf(t, s, 0.254829592f);
    bell = exp_fast(-0.5f * z * z);
    const float tail = 0.5f * t * s * bell;
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
