// What the group norm kernels share: vectors of channels, arithmetic on them two at a time, the
// activations.  Internal linkage: each kernel file compiles its own copy.
#pragma once

#include "group_norm.cuh"
#include "product_device.cuh"

namespace fa {

namespace {

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};

// By a load that stays where it is written: the loops below ask for several, then use them.
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_raw(const T* p) {
    Vec<T, V> q;
    constexpr size_t kSize = sizeof(T) * V;
    if constexpr (kSize == 16) {
        const uint4 w = ld_plain_v4(p);
        memcpy(&q, &w, kSize);
    } else if constexpr (kSize == 8) {
        uint2 w;
        asm volatile("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(w.x), "=r"(w.y) : "l"(p));
        memcpy(&q, &w, kSize);
    } else if constexpr (kSize == 4) {
        uint32_t w;
        asm volatile("ld.global.u32 %0, [%1];" : "=r"(w) : "l"(p));
        memcpy(&q, &w, kSize);
    } else {
        uint16_t w;
        asm volatile("ld.global.u16 %0, [%1];" : "=h"(w) : "l"(p));
        memcpy(&q, &w, kSize);
    }
    return q;
}

template <typename T, int V>
__device__ __forceinline__ void widen(const Vec<T, V>& q, float (&x)[V]) {
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {
        uint32_t w[V / 2];
        memcpy(w, &q, sizeof w);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        }
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = __uint_as_float(static_cast<uint32_t>(q.e[i]) << 16);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = q.e[i];
    }
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[V]) {
    Vec<T, V> q;
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {
        uint32_t w[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        memcpy(&q, w, sizeof w);
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < V; ++i) q.e[i] = __bfloat16_as_ushort(__float2bfloat16_rn(x[i]));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) q.e[i] = x[i];
    }
    *reinterpret_cast<Vec<T, V>*>(p) = q;
}

// Element by element, two at a time: d = a + b, a * b, a * b + c.
template <int V>
__device__ __forceinline__ void add(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
#pragma unroll
    for (int i = 0; i + 1 < V; i += 2)
        asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n"
            " mov.b64 {%0, %1}, d;\n}"
            : "=f"(d[i]), "=f"(d[i + 1])
            : "f"(a[i]), "f"(a[i + 1]), "f"(b[i]), "f"(b[i + 1]));
    if (V % 2) d[V - 1] = a[V - 1] + b[V - 1];
}

template <int V>
__device__ __forceinline__ void mul(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
#pragma unroll
    for (int i = 0; i + 1 < V; i += 2)
        asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 d, a, b;\n"
            " mov.b64 {%0, %1}, d;\n}"
            : "=f"(d[i]), "=f"(d[i + 1])
            : "f"(a[i]), "f"(a[i + 1]), "f"(b[i]), "f"(b[i + 1]));
    if (V % 2) d[V - 1] = a[V - 1] * b[V - 1];
}

template <int V>
__device__ __forceinline__ void fma(float (&d)[V], const float (&a)[V], const float (&b)[V], const float (&c)[V]) {
#pragma unroll
    for (int i = 0; i + 1 < V; i += 2)
        asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
            " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
            : "=f"(d[i]), "=f"(d[i + 1])
            : "f"(a[i]), "f"(a[i + 1]), "f"(b[i]), "f"(b[i + 1]), "f"(c[i]), "f"(c[i + 1]));
    if (V % 2) d[V - 1] = fmaf(a[V - 1], b[V - 1], c[V - 1]);
}

// 1 / (1 + exp(-z)).
template <int V>
__device__ __forceinline__ void sigmoid(float (&s)[V], const float (&z)[V]) {
    float one[V], scale[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        one[i] = 1.0f;
        scale[i] = -1.4426950408889634f;
    }
    mul(s, z, scale);
#pragma unroll
    for (int i = 0; i < V; ++i) asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(s[i]));
    add(s, s, one);
#pragma unroll
    for (int i = 0; i < V; ++i) asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(s[i]));
}

template <int V>
__device__ __forceinline__ void act_of(int act, float (&z)[V]) {
    if (act == kActSilu) {
        float s[V];
        sigmoid(s, z);
        mul(z, z, s);
    } else {
        activate(act, z);
    }
}

// d *= act'(z)
template <int V>
__device__ __forceinline__ void times_act_grad(int act, float (&d)[V], const float (&z)[V]) {
    if (act == kActRelu) {
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] *= act_grad(kActRelu, z[i]);
    } else if (act == kActGelu) {
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] *= act_grad(kActGelu, z[i]);
    } else if (act == kActSilu) {
        // s (1 + z (1 - s)) = s + (z s) (1 - s)
        float s[V], t[V], one[V], r[V];
        sigmoid(s, z);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            one[i] = 1.0f;
            r[i] = -s[i];
        }
        mul(t, z, s);
        add(r, one, r);
        fma(t, t, r, s);
        mul(d, d, t);
    }
}

// Over `lanes` neighbouring lanes, a power of two.
__device__ __forceinline__ float lane_sum(float v, uint32_t lanes) {
    for (uint32_t o = lanes / 2; o > 0; o /= 2) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// A thread's sums over the positions of its run: s[0] of d = x - reference, s[1] of d^2, for each channel,
// and how the variance comes from them without cancelling.  A run's squares about a point r are its squares
// about its mean m and n (m - r)^2.  Where r is the mean of the first k positions, these have at least
// k (m - r)^2 of the squares about m, so that the second part is at most n / k times the first, whatever
// the values are.  The reference begins as the thread's first value and is moved to the mean so far after
// the first few positions and whenever the run has grown kGrow times: no sum is more than some ten times
// what is kept of it.  (With one reference for a run, its first value, one voxel 1000 spreads off left 3
// digits of the variance.)
constexpr uint32_t kGrow = 8;
template <int V>
struct Moments {
    float less[V] = {}, s[2][V] = {};                // less: the reference, negated
    __device__ __forceinline__ void begin(const float (&x)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) less[i] = -x[i];
    }
    __device__ __forceinline__ void step(float (&x)[V]) {
        add(x, x, less);
        add(s[0], s[0], x);
        fma(s[1], x, x, s[1]);
    }
    // to the mean of the n positions so far
    __device__ __forceinline__ void move(float n) {
        const float inv = 1.0f / n;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float to = less[i] - s[0][i] * inv, by = less[i] - to, rest = fmaf(-n, by, s[0][i]);
            s[1][i] = fmaf(-by, s[0][i] + rest, s[1][i]);
            s[0][i] = rest;
            less[i] = to;
        }
    }
    // this thread's part of the mean of `count` positions, n of them its own (if n is 0, all here is 0)
    __device__ __forceinline__ void mean_part(float n, float count, float (&to)[V]) const {
        const float inv = 1.0f / count, share = n * inv;
#pragma unroll
        for (int i = 0; i < V; ++i) to[i] = fmaf(-less[i], share, s[0][i] * inv);
    }
    // the same sums about `base`
    __device__ __forceinline__ void about(float n, const float* base) {
        const float inv = n > 0.0f ? 1.0f / n : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float m = s[0][i] * inv, d = (-less[i] - base[i]) + m;
            s[1][i] = fmaf(n * d, d, fmaxf(fmaf(-s[0][i], m, s[1][i]), 0.0f));
            s[0][i] = n * d;
        }
    }
};

// What a thread keeps of its channels: with h = x - mean, z = h scale + beta, scale = rstd gamma.
template <int V>
struct Channels {
    float less[V], scale[V], beta[V];
    Channels() = default;
    __device__ __forceinline__ Channels(const NormArgs& a, uint32_t sample, uint32_t c) {
        const uint32_t per = a.channels / a.groups;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint64_t g = static_cast<uint64_t>(sample) * a.groups + (c + i) / per;
            less[i] = -a.mean[g];
            scale[i] = a.rstd[g] * (a.gamma ? elem(a.gamma, c + i, a.param_dtype) : 1.0f);
            beta[i] = a.beta ? elem(a.beta, c + i, a.param_dtype) : 0.0f;
        }
    }
    // x to h, d to dz
    __device__ __forceinline__ void step(int act, float (&x)[V], float (&d)[V]) const {
        add(x, x, less);
        if (act == 0) return;
        float z[V];
        fma(z, x, scale, beta);
        times_act_grad(act, d, z);
    }
};

}  // namespace

}  // namespace fa
