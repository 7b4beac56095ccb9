// Distillation kernels: one CTA per row of logits.
//
//   loss  reads the row twice (maximum, then the sum of exponentials)
//   grad  reads it a third time and writes w T (q - share), share being nonzero at the
//         lists' entries alone
//
// The shares of the entries are gathered in a hash table in shared memory (entry -> sum of
// (n_j / total) p_jc): several clients name the same entry, and 64-bit integer adds of
// 2^-62 units give the same sum in any order.  The row is written without the shares
// first, then the table's entries are written over it.
#include "distill.cuh"
#include "device.cuh"

namespace fa {

namespace {

constexpr int kDThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kFix = 4611686018427387904.0f;           // 2^62
constexpr unsigned long long kPoison = 1ull << 63;       // the sum is NaN

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, d));
    return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    return v;
}

// Over the CTA, in a fixed order; every thread gets the result.
template <bool kMax>
__device__ __forceinline__ float block_reduce(float v, float* tmp) {
    v = kMax ? warp_max(v) : warp_sum(v);
    __syncthreads();
    if (threadIdx.x % 32 == 0) tmp[threadIdx.x / 32] = v;
    __syncthreads();
    float r = tmp[0];
    for (int i = 1; i < kDThreads / 32; ++i) r = kMax ? fmaxf(r, tmp[i]) : r + tmp[i];
    return r;
}

__device__ __forceinline__ float value_at(const void* p, uint64_t e, int dt) {
    return dt ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[e]) << 16)
              : static_cast<const float*>(p)[e];
}

template <typename T>
__device__ __forceinline__ float at(const T* p, uint64_t e) {
    if constexpr (sizeof(T) == 2)
        return __uint_as_float(static_cast<uint32_t>(p[e]) << 16);
    else
        return p[e];
}

template <typename T>
__device__ __forceinline__ void set(T* p, uint64_t e, float v) {
    if constexpr (sizeof(T) == 2)
        p[e] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    else
        p[e] = v;
}

__device__ __forceinline__ uint32_t hash_of(int32_t key, uint32_t slots) {
    return (static_cast<uint32_t>(key) * 2654435761u) >> (__clz(slots) + 1);   // top log2(slots) bits
}

template <typename T, bool kGrad>
__global__ void __launch_bounds__(kDThreads) distill_kernel(const __grid_constant__ DistillArgs a) {
    extern __shared__ unsigned long long sums[];                 // [slots]
    int32_t* keys = reinterpret_cast<int32_t*>(sums + a.slots);  // [slots], -1 free
    __shared__ float tmp[kDThreads / 32];
    __shared__ float cl_loss[kMaxDistillClients], cl_mass[kMaxDistillClients], cl_on[kMaxDistillClients];
    const uint32_t row = blockIdx.x;
    const float w = a.row_weight ? a.row_weight[row] : 1.0f;
    const T* z = static_cast<const T*>(a.logits) + row * a.ld;
    T* g = kGrad ? static_cast<T*>(a.grad) + row * a.ldg : nullptr;
    if (!(w > 0.0f)) {
        if (kGrad)
            for (uint32_t i = threadIdx.x; i < a.vocab; i += kDThreads) set(g, i, 0.0f);
        if (threadIdx.x == 0) {
            if (a.loss) a.loss[row] = 0.0f;
            if (a.lse_out) a.lse_out[row] = 0.0f;
        }
        return;
    }
    if (kGrad)
        for (uint32_t i = threadIdx.x; i < a.slots; i += kDThreads) {
            sums[i] = 0;
            keys[i] = -1;
        }
    // the row's statistics
    float m = 0.0f, s = 1.0f, lse;
    const float c = a.inv_t * kLog2e;
    if (a.lse_in) {
        lse = a.lse_in[row];
    } else {
        float v = -INFINITY;
        for (uint32_t i = threadIdx.x; i < a.vocab; i += kDThreads) v = fmaxf(v, at(z, i));
        m = block_reduce<true>(v, tmp);
        v = 0.0f;
        // (z - m) first, then the scale: exact or rounded once where z is near m, and no
        // overflow of z * c for values near the type's lowest
        for (uint32_t i = threadIdx.x; i < a.vocab; i += kDThreads) v += ex2((at(z, i) - m) * c);
        s = block_reduce<false>(v, tmp);
        lse = fmaf(m, a.inv_t, logf(s));
    }
    __syncthreads();
    // the clients' lists, a warp each
    const int lane = threadIdx.x % 32;
    for (uint32_t j = threadIdx.x / 32; j < a.nclients; j += kDThreads / 32) {
        const DistillClient& cl = a.client[j];
        const uint64_t base = static_cast<uint64_t>(row) * cl.topk;
        float top = -INFINITY;
        bool nan = false;
        for (uint32_t i = lane; i < cl.topk; i += 32) {
            const int32_t e = cl.index[base + i];
            if (e >= 0 && static_cast<uint32_t>(e) >= a.vocab) atomicOr(a.err, kErrListIndex);
            if (static_cast<uint32_t>(e) < a.vocab) {
                const float u = value_at(cl.value, base + i, a.value_dtype);
                nan |= u != u;
                top = fmaxf(top, u);
            }
        }
        top = warp_max(top);
        const bool on = __any_sync(~0u, nan) || top > -INFINITY;
        float sum = 0.0f;
        for (uint32_t i = lane; i < cl.topk; i += 32)
            if (static_cast<uint32_t>(cl.index[base + i]) < a.vocab)
                sum += ex2((value_at(cl.value, base + i, a.value_dtype) - top) * c);
        sum = warp_sum(sum);
        const float inv = 1.0f / sum, logsum = logf(sum);
        float loss = 0.0f, mass = 0.0f;
        if (on)
            for (uint32_t i = lane; i < cl.topk; i += 32) {
                const int32_t e = cl.index[base + i];
                if (static_cast<uint32_t>(e) >= a.vocab) continue;
                const float d = (value_at(cl.value, base + i, a.value_dtype) - top) * a.inv_t;
                const float p = ex2(d * kLog2e) * inv;
                if (p == 0.0f) continue;      // nothing, also where the student's logit is -inf
                loss += p * (d - logsum - at(z, e) * a.inv_t);
                mass += p;
                if (kGrad) {
                    uint32_t h = hash_of(e, a.slots);
                    for (;; h = (h + 1) & (a.slots - 1)) {
                        const int32_t was = atomicCAS(&keys[h], -1, e);
                        if (was == -1 || was == e) break;
                    }
                    if (p != p)
                        atomicOr(&sums[h], kPoison);
                    else
                        atomicAdd(&sums[h], __float2ull_rn(p * cl.share * kFix));
                }
            }
        loss = warp_sum(loss);
        mass = warp_sum(mass);
        if (lane == 0) {
            cl_loss[j] = loss;
            cl_mass[j] = mass;
            cl_on[j] = on ? cl.weight : 0.0f;
        }
    }
    __syncthreads();
    float total = 0.0f, loss = 0.0f;
    for (uint32_t j = 0; j < a.nclients; ++j) total += cl_on[j];
    const bool some = total > 0.0f;
    // n_j / N first: the terms of a logit near the type's lowest are near fp32's range
    for (uint32_t j = 0; j < a.nclients; ++j)
        if (cl_on[j] > 0.0f) loss = fmaf(cl_on[j] / total, fmaf(lse, cl_mass[j], cl_loss[j]), loss);
    if (threadIdx.x == 0) {
        if (a.loss) a.loss[row] = some ? w * a.temperature * a.temperature * loss : 0.0f;
        if (a.lse_out) a.lse_out[row] = lse;
    }
    if constexpr (kGrad) {
        const float coef = some ? w * a.temperature : 0.0f;
        const float scale = coef / s, back = some ? a.total / total : 0.0f;
        auto q = [&](float x) { return a.lse_in ? ex2(fmaf(x, a.inv_t, -lse) * kLog2e) : ex2((x - m) * c); };
        // the entries' values are taken before the row is written: grad may be logits
        float mine[2 * kMaxDistillTopk / kDThreads];
        for (uint32_t i = threadIdx.x, t = 0; i < a.slots; i += kDThreads, ++t)
            if (keys[i] >= 0) {
                const float share = sums[i] & kPoison ? NAN : static_cast<float>(sums[i]) * (1.0f / kFix) * back;
                mine[t] = coef * (q(at(z, keys[i])) / s - share);
            }
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < a.vocab; i += kDThreads) set(g, i, some ? q(at(z, i)) * scale : 0.0f);
        __syncthreads();
        if (some)
            for (uint32_t i = threadIdx.x, t = 0; i < a.slots; i += kDThreads, ++t)
                if (keys[i] >= 0) set(g, keys[i], mine[t]);
    }
}

}  // namespace

cudaError_t prepare_distill() {
    const int most = static_cast<int>(2 * kMaxDistillTopk * 12);
    cudaError_t e = cudaFuncSetAttribute(distill_kernel<uint16_t, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(distill_kernel<float, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    return e;
}

cudaError_t launch_distill(DistillArgs& a, cudaStream_t stream) {
    uint32_t entries = 0;
    for (uint32_t j = 0; j < a.nclients; ++j) entries += a.client[j].topk;
    a.slots = 2;
    while (a.slots < 2 * entries) a.slots *= 2;
    const size_t smem = a.grad ? static_cast<size_t>(a.slots) * 12 : 0;
    if (a.grad) {
        if (a.dtype)
            distill_kernel<uint16_t, true><<<a.rows, kDThreads, smem, stream>>>(a);
        else
            distill_kernel<float, true><<<a.rows, kDThreads, smem, stream>>>(a);
    } else if (a.dtype) {
        distill_kernel<uint16_t, false><<<a.rows, kDThreads, smem, stream>>>(a);
    } else {
        distill_kernel<float, false><<<a.rows, kDThreads, smem, stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace fa
