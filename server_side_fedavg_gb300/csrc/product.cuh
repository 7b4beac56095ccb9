// Matrix products with bias, activation and residual in their epilogue, and what their
// gradients need: the launch interface (internal to the library).
//
//   out[m,n] = act(alpha * sum_k A(m,k) B(k,n) + bias[n]) + beta * residual[m,n]
//
// dtype codes as in kernels.cuh: 0 = fp32, 1 = bf16.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fa {

// One operand: element (x, kk) -- x is m of A or n of B -- at p[x * ld + kk] if kmajor
// (the summed index runs along a row), else at p[kk * ld + x].
struct ProdOperand {
    const void* p;
    uint64_t ld;
    int dtype;
    bool kmajor;
};

struct ProdEpilogue {
    float alpha, beta;
    const void* bias;       // [n] of bias_dtype, or nullptr
    const void* res;        // [m,n] of out_dtype, or nullptr; may be out
    void* out;              // [m,n] of out_dtype
    void* pre;              // [m,n] of out_dtype with stride ldo, or nullptr
    uint64_t ldr, ldo;
    int bias_dtype, out_dtype, act;
};

struct ProdArgs {
    uint32_t m, n, k;
    ProdOperand a, b;
    ProdEpilogue e;
};

// Any types, strides and storage orders; for small m * n * k (and k == 0).
cudaError_t launch_product_tiny(const ProdArgs& p, cudaStream_t stream);

// Few rows of a; a K-major, both operands of one type.
cudaError_t launch_product_thin(const ProdArgs& p, cudaStream_t stream);

// The products' operands where they are not as the tensor-core kernel reads them (bf16,
// 16-byte aligned base and row stride): the matrix [rows][cols] as `planes` bf16 planes
// [plane][rows][ldd], ldd a multiple of 8 -- one plane for bf16 sources, three for fp32:
// x = x0 + x1 + x2, each term the remainder rounded to nearest, 24 bits in all.
struct SplitJob {
    const void* src;
    uint64_t ld;
    int dtype;
    uint32_t rows, cols, planes;
    void* dst;
    uint64_t ldd;
};
// One or two operands in one launch.
cudaError_t launch_split(const SplitJob* jobs, int n, cudaStream_t stream);

// dZ[m,n] = dout * act'(pre), computed in fp32 and written (dz != nullptr) with row stride
// ldz as fp32 (dz_planes 0), rounded to bf16 (1) or as three bf16 planes (3), m * ldz
// elements apart; and its column sums over blocks of `rows` rows (a multiple of 8),
// to part[ceil(m / rows)][n] (part != nullptr).
struct ActGradArgs {
    uint32_t m, n, rows;
    const void* dout;
    const void* pre;        // nullptr: act is none
    uint64_t ldd, ldp;
    int dtype, act;
    void* dz;
    uint64_t ldz;
    int dz_planes;
    float* part;
};
cudaError_t launch_act_grad(const ActGradArgs& a, cudaStream_t stream);

// out[n] = sum over blocks of part[blocks][n], in block order, rounded to out_dtype.
cudaError_t launch_col_sum(const float* part, uint32_t blocks, uint32_t n, void* out, int out_dtype,
                           cudaStream_t stream);

}  // namespace fa
