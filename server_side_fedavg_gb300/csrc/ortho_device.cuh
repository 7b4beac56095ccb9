// What the orthogonalised weight step's own passes share: rows eight elements at a time, momentum,
// the norm's factor.  Internal linkage: each kernel file compiles its own copy.
#pragma once

#include "ortho.cuh"
#include "product_device.cuh"

namespace fa {

namespace {

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

// x: u, then u + mu g' or g'; g: m, then g' = mu m + u (u itself without a momentum).
__device__ __forceinline__ void momentum_step(const OrthoEnds& a, float (&x)[8], float (&g)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = a.momentum.p ? fmaf(a.mu, g[i], x[i]) : x[i];
    if (!a.momentum.p && !a.momentum_out.p) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = a.nesterov ? fmaf(a.mu, g[i], x[i]) : g[i];
}

// The same from memory.  kept: g' is read from momentum_out, where the first pass has put it (over
// m, it may be).
__device__ __forceinline__ void step_of(const OrthoEnds& a, const Vecs& v, uint32_t item, uint32_t r, uint32_t c, bool kept,
                                        float (&x)[8], float (&g)[8]) {
    load8(a.update, row_of(a.update, item, r), c, a.cols, v.update, x);
    if (kept && a.momentum_out.p) {
        load8(a.momentum_out, row_of(a.momentum_out, item, r), c, a.cols, v.momentum_out, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = a.nesterov ? fmaf(a.mu, g[i], x[i]) : g[i];
        return;
    }
    if (a.momentum.p) load8(a.momentum, row_of(a.momentum, item, r), c, a.cols, v.momentum, g);
    momentum_step(a, x, g);
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// Sum of eight squares: in fp32 where none can leave its range, else in fp64.
__device__ __forceinline__ double squares(const float (&x)[8]) {
    float most = 0.0f, q = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        most = fmaxf(most, fabsf(x[j]));
        q = fmaf(x[j], x[j], q);
    }
    if (most < 0x1p60f && (most > 0x1p-40f || most == 0.0f) && q == q) return static_cast<double>(q);
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) s += static_cast<double>(x[j]) * static_cast<double>(x[j]);
    return s;
}

// 2^shift / (root of s + eps) as a fraction of 1 and a power of two, which fp32 has down to 2^-149.
__device__ __forceinline__ float2 factor_of(double s, double eps, int shift) {
    int e;
    const float f = static_cast<float>(frexp(1.0 / (sqrt(s) + eps), &e));
    return make_float2(f, ldexpf(1.0f, e + shift));
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

}  // namespace fa
