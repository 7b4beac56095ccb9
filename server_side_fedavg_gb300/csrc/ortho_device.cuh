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

// x: u, then u + mu g' or g'; g: m, then g' = mu m + u.  Without a momentum both are u: mu is not read.
__device__ __forceinline__ void momentum_step(const OrthoEnds& a, float (&x)[8], float (&g)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = a.momentum.p ? fmaf(a.mu, g[i], x[i]) : x[i];
    if (!a.momentum.p) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = a.nesterov ? fmaf(a.mu, g[i], x[i]) : g[i];
}

// The same from memory.  kept: g' is read from momentum_out, where the first pass has put it (over
// m, it may be).
__device__ __forceinline__ void step_of(const OrthoEnds& a, const Vecs& v, uint32_t item, uint32_t r, uint32_t c, bool kept,
                                        float (&x)[8], float (&g)[8]) {
    load8(a.update, row_of(a.update, item, r), c, a.cols, v.update, x);
    if (kept && a.momentum.p && a.momentum_out.p) {
        load8(a.momentum_out, row_of(a.momentum_out, item, r), c, a.cols, v.momentum_out, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = a.nesterov ? fmaf(a.mu, g[i], x[i]) : g[i];
        return;
    }
    if (a.momentum.p) load8(a.momentum, row_of(a.momentum, item, r), c, a.cols, v.momentum, g);
    momentum_step(a, x, g);
}

// A sum of squares of fp32 numbers of any size, in fp32: those from 2^-50 to 2^45 as they are,
// smaller and larger ones scaled by 2^84 and 2^-84, so that no square of up to 2^32 of them leaves
// fp32's range.  (In fp64, whose units are few on this GPU, the sum and the root took 5 us of a small
// matrix's 20.)
struct Squares {
    float mid = 0.0f, high = 0.0f, low = 0.0f;
    __device__ __forceinline__ void add(const float (&x)[8]) {
        float most = 0.0f, least = 0x1p45f, q = 0.0f;
        bool nan = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = fabsf(x[j]);
            most = fmaxf(most, v);
            if (v > 0.0f) least = fminf(least, v);
            nan |= v != v;
            q = fmaf(v, v, q);
        }
        if (most < 0x1p45f && least >= 0x1p-50f && !nan) {
            mid += q;
            return;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = fabsf(x[j]), h = v * 0x1p-84f, l = v * 0x1p84f;
            if (!(v < 0x1p45f))
                high = fmaf(h, h, high);
            else if (v < 0x1p-50f)
                low = fmaf(l, l, low);
            else
                mid = fmaf(v, v, mid);
        }
    }
    __device__ __forceinline__ void add(const Squares& o) {
        mid += o.mid;
        high += o.high;
        low += o.low;
    }
    __device__ __forceinline__ void over_warp() {
#pragma unroll
        for (int o = 16; o > 0; o /= 2) {
            mid += __shfl_xor_sync(~0u, mid, o);
            high += __shfl_xor_sync(~0u, high, o);
            low += __shfl_xor_sync(~0u, low, o);
        }
    }
    // 1 / (root + eps) as x * y, y a power of two that brings the largest element into fp32's middle
    __device__ __forceinline__ float2 factor(double eps) const {
        if (high > 0.0f || high != high)
            return make_float2(1.0f / (sqrtf(high + mid * 0x1p-84f * 0x1p-84f) + static_cast<float>(eps * 0x1p-84)), 0x1p-84f);
        const float s = mid + low * 0x1p-84f * 0x1p-84f;
        if (mid > 0.0f) return make_float2(1.0f / (sqrtf(s) + static_cast<float>(eps)), 1.0f);
        const double e = eps * 0x1p84;
        return make_float2(1.0f / (sqrtf(low) + static_cast<float>(e < 1e38 ? e : 1e38)), 0x1p84f);
    }
};

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
