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

// act(z).  A NaN stays a NaN in each.
__device__ __forceinline__ float act_fwd(int act, float z) {
    if (act == kActRelu) return z < 0.0f ? 0.0f : z;
    if (act == kActGelu) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    if (act == kActSilu) return __fdividef(z, 1.0f + expf(-z));
    return z;
}

// act'(z):  relu [z > 0];  gelu Phi(z) + z phi(z);  silu s (1 + z (1 - s)), s = 1 / (1 + exp(-z)).
__device__ __forceinline__ float act_grad(int act, float z) {
    if (act == kActRelu) return z > 0.0f ? 1.0f : 0.0f;
    if (act == kActGelu)
        return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) + z * expf(-0.5f * z * z) * 0.39894228040143268f;
    if (act == kActSilu) {
        const float s = __fdividef(1.0f, 1.0f + expf(-z));
        return s * (1.0f + z * (1.0f - s));
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
