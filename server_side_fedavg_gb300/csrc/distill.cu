// Distillation kernels.
//
//   loss   log sum exp of the row, and over the clients' lists sum p (log p - log q)
//   grad   w T (q - share), share being nonzero at the lists' entries alone
//
// Rows of up to 8 x 64 KB are held in registers: a CTA (or a cluster of 2, 4 or 8, each with a
// slice) loads its row once with every load in flight at the same time, finds maximum and sum
// together -- each thread over its own maximum, pairs (maximum, sum) merged over warp, CTA and,
// through distributed shared memory, cluster -- and writes the gradient from the registers.
// The row is read once and written once: bound by HBM.  Longer rows are streamed from memory
// (and L2) twice or three times.
//
// An exponential is 2^(z c - k) with c = log2(e) / T and k = maximum c rounded: one FMA and one
// ex2.  k's rounding is the same in every term and in the statistic that is formed with the
// same k, so it cancels.  Rows whose maximum is beyond 2^20 T / log2(e) in size (rows masked by
// the type's lowest value throughout, or with infinities) take 2^((z - maximum) c) instead.
//
// The shares of the entries are gathered in a hash table in shared memory (entry -> sum of
// (n_j / total) p_jc): several clients name the same entry, and 64-bit integer adds of
// 2^-62 units give the same sum in any order.  The row is written without the shares
// first, then the table's entries are written over it.
#include "distill.cuh"
#include "device.cuh"

namespace fa {

namespace {

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
template <int kThreads, bool kMax>
__device__ __forceinline__ float block_reduce(float v, float* tmp) {
    v = kMax ? warp_max(v) : warp_sum(v);
    __syncthreads();
    if (threadIdx.x % 32 == 0) tmp[threadIdx.x / 32] = v;
    __syncthreads();
    float r = tmp[0];
    for (int i = 1; i < kThreads / 32; ++i) r = kMax ? fmaxf(r, tmp[i]) : r + tmp[i];
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

// ----------------------------------------------------------------- the clients' lists
struct Lists {
    float loss[kMaxDistillClients];     // sum p (log p - z / T) of client j
    float mass[kMaxDistillClients];     // sum p: 1 (or 0) up to rounding
    float on[kMaxDistillClients];       // n_j, 0 if absent
};

// A warp per client: softmax of its values over its used places, its part of the loss (kLoss)
// and its shares into the table, as far as they fall into [lo, hi) (kGrad).
template <typename T, bool kGrad, int kThreads>
__device__ __forceinline__ void read_lists(const DistillArgs& a, const T* z, uint32_t row, bool want_loss, uint32_t lo,
                                           uint32_t hi, Lists& l, unsigned long long* sums, int32_t* keys) {
    const int lane = threadIdx.x % 32;
    const float c = a.inv_t * kLog2e;
    for (uint32_t j = threadIdx.x / 32; j < a.nclients; j += kThreads / 32) {
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
                mass += p;
                if (want_loss) loss += p * (d - logsum - at(z, e) * a.inv_t);
                if (kGrad && static_cast<uint32_t>(e) >= lo && static_cast<uint32_t>(e) < hi) {
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
            l.loss[j] = loss;
            l.mass[j] = mass;
            l.on[j] = on ? cl.weight : 0.0f;
        }
    }
}

// N_r; 0: no client.  The lists have been read by the whole CTA.
__device__ __forceinline__ float total_weight(const DistillArgs& a, const Lists& l) {
    float total = 0.0f;
    for (uint32_t j = 0; j < a.nclients; ++j) total += l.on[j];
    return total;
}

__device__ __forceinline__ void write_loss(const DistillArgs& a, const Lists& l, uint32_t row, float w, float total, float lse) {
    float loss = 0.0f;
    // n_j / N first: the terms of a logit near the type's lowest are near fp32's range
    for (uint32_t j = 0; j < a.nclients; ++j)
        if (l.on[j] > 0.0f) loss = fmaf(l.on[j] / total, fmaf(lse, l.mass[j], l.loss[j]), loss);
    if (a.loss) a.loss[row] = total > 0.0f ? w * a.temperature * a.temperature * loss : 0.0f;
    if (a.lse_out) a.lse_out[row] = lse;
}

// An exponential's form in one row: fast 2^(z c - k), else 2^((z p - k) r).
struct Exp {
    float c, k, p, r;
    bool fast;
    __device__ __forceinline__ float quick(float z) const { return ex2(fmaf(z, c, -k)); }
    __device__ __forceinline__ float slow(float z) const { return ex2(fmaf(z, p, -k) * r); }
    __device__ __forceinline__ float operator()(float z) const { return fast ? quick(z) : slow(z); }
};

// The fast form's k is at most 2^20 in size: its rounding, up to 2^-5, is in every exponent.
constexpr float kFastMost = 1048576.0f;

// From a kept statistic: q = 2^(z c - lse log2 e), the product's rounding error moved to `scale`
// (log2 e is kLog2e + 1.92596303e-8).
__device__ __forceinline__ Exp from_lse(const DistillArgs& a, float lse, float& scale) {
    const float k = lse * kLog2e;
    if (!(fabsf(k) < kFastMost)) return {0.0f, lse, a.inv_t, kLog2e, false};
    scale = ex2(-fmaf(lse, 1.92596303e-8f, fmaf(lse, kLog2e, -k)));
    return {a.inv_t * kLog2e, k, 0.0f, 0.0f, true};
}

// The entries' values of the gradient, into the table in place of the sums -- before the row is
// written, since grad may be logits; then, after a barrier, over the written row.
template <typename T, int kThreads>
__device__ __forceinline__ void entry_values(const DistillArgs& a, const T* z, const Exp& e, float coef, float scale,
                                             float back, unsigned long long* sums, const int32_t* keys) {
    for (uint32_t h = threadIdx.x; h < a.slots; h += kThreads)
        if (keys[h] >= 0) {
            const float share = sums[h] & kPoison ? NAN : static_cast<float>(sums[h]) * (1.0f / kFix) * back;
            sums[h] = __float_as_uint(coef * (e(at(z, keys[h])) * scale - share));
        }
}

template <typename T, int kThreads>
__device__ __forceinline__ void write_entries(const DistillArgs& a, T* g, const unsigned long long* sums, const int32_t* keys) {
    for (uint32_t h = threadIdx.x; h < a.slots; h += kThreads)
        if (keys[h] >= 0) set(g, keys[h], __uint_as_float(static_cast<uint32_t>(sums[h])));
}

// ----------------------------------------------------------------- rows in registers
constexpr int kMaxSlice = 65536;       // bytes of a row that a CTA of 512 threads holds

__device__ __forceinline__ uint32_t rank_in_cluster() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void sync_cluster() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float2 peer2(const float2* p, uint32_t rank) {
    uint32_t addr;
    float2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

// The elements of 16 loaded bytes.
template <typename T>
__device__ __forceinline__ void unpack(const uint4& q, float (&x)[16 / sizeof(T)]) {
    if constexpr (sizeof(T) == 2) {
        x[0] = bf16_lo(q.x); x[1] = bf16_hi(q.x); x[2] = bf16_lo(q.y); x[3] = bf16_hi(q.y);
        x[4] = bf16_lo(q.z); x[5] = bf16_hi(q.z); x[6] = bf16_lo(q.w); x[7] = bf16_hi(q.w);
    } else {
        x[0] = __uint_as_float(q.x); x[1] = __uint_as_float(q.y);
        x[2] = __uint_as_float(q.z); x[3] = __uint_as_float(q.w);
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack(const float (&x)[16 / sizeof(T)]) {
    if constexpr (sizeof(T) == 2) {
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        return make_uint4(r[0], r[1], r[2], r[3]);
    } else {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
}

// (m, s): the sum of 2^(z c) is s 2^(m c) -- with m c rounded as Exp has it.
__device__ __forceinline__ void merge(float& m, float& s, float m2, float s2, float c) {
    const float top = fmaxf(m, m2), k = top * c;
    s = s * ex2(m * c - k) + s2 * ex2(m2 * c - k);
    m = top;
}

// One row (or slice) in the registers of kThreads threads, kNv x 16 bytes each.  A slice starts
// anywhere: elements before its first 16-byte boundary and after its last are held one per
// thread in `edge`.
template <typename T, bool kGrad, int kThreads, int kNv>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) distill_row_kernel(const __grid_constant__ DistillArgs a) {
    constexpr int kV = 16 / sizeof(T), kWarps = kThreads / 32;
    extern __shared__ unsigned long long sums[];                 // [slots]
    int32_t* keys = reinterpret_cast<int32_t*>(sums + a.slots);  // [slots], -1 free
    __shared__ float tmp[kWarps], tmp2[kWarps];
    __shared__ float2 mine;
    __shared__ Lists lists;
    const uint32_t ctas = a.cluster, rank = ctas > 1 ? rank_in_cluster() : 0;
    const uint32_t row = blockIdx.x / ctas, t = threadIdx.x;
    const float w = a.row_weight ? a.row_weight[row] : 1.0f;
    const T* z = static_cast<const T*>(a.logits) + row * a.ld;
    T* g = kGrad ? static_cast<T*>(a.grad) + row * a.ldg : nullptr;
    const uint32_t lo = rank * a.slice, hi = min(lo + a.slice, a.vocab), n = hi > lo ? hi - lo : 0;
    const T* zs = z + lo;
    T* gs = kGrad ? g + lo : nullptr;
    // 16-byte vectors of the slice: `head` elements before them, `tail` after
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(zs) % 16 / sizeof(T));
    const uint32_t head = min(off ? kV - off : 0, n), nvec = (n - head) / kV, tail = n - head - nvec * kV;
    const bool has_edge = t < head || (t >= kV && t - kV < tail);
    const uint32_t edge_at = t < head ? t : head + nvec * kV + t - kV;
    const bool same_phase = kGrad && reinterpret_cast<uintptr_t>(gs) % 16 == reinterpret_cast<uintptr_t>(zs) % 16;
    const auto put_vec = [&](uint32_t v, const float (&x)[kV]) {
        T* p = gs + head + v * kV;
        if (same_phase) {
            st_v4u(p, pack<T>(x));
        } else {
#pragma unroll
            for (int i = 0; i < kV; ++i) set(p, i, x[i]);
        }
    };
    const auto write_zeros = [&] {
        const float zero[kV] = {};
#pragma unroll
        for (int i = 0; i < kNv; ++i)
            if (t + i * kThreads < nvec) put_vec(t + i * kThreads, zero);
        if (has_edge) set(gs, edge_at, 0.0f);
    };
    if (!(w > 0.0f)) {
        if (kGrad) write_zeros();
        if (t == 0 && rank == 0) {
            if (a.loss) a.loss[row] = 0.0f;
            if (a.lse_out) a.lse_out[row] = 0.0f;
        }
        return;
    }
    // the row, all loads in flight; what is not there counts as -inf
    constexpr uint32_t kNone = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
    uint4 q[kNv];
#pragma unroll
    for (int i = 0; i < kNv; ++i)
        q[i] = t + i * kThreads < nvec ? ld_plain_v4(zs + head + (t + i * kThreads) * kV) : make_uint4(kNone, kNone, kNone, kNone);
    const float edge = has_edge ? at(zs, edge_at) : -INFINITY;
    if (kGrad) {
        for (uint32_t i = t; i < a.slots; i += kThreads) {
            sums[i] = 0;
            keys[i] = -1;
        }
        __syncthreads();
    }
    read_lists<T, kGrad, kThreads>(a, z, row, rank == 0 && a.loss, lo, hi, lists, sums, keys);

    const float c = a.inv_t * kLog2e;
    const float most = kFastMost / c;      // of a maximum, for the fast form
    Exp e{c, 0.0f, 0.0f, 0.0f, true};
    float scale = 1.0f, lse;               // q = e(z) * scale
    if (a.lse_in) {
        lse = a.lse_in[row];
        e = from_lse(a, lse, scale);
        __syncthreads();
    } else {
        // each thread's own maximum, floored where the fast form ends
        float m = fmaxf(edge, -most);
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            float x[kV];
            unpack<T>(q[i], x);
#pragma unroll
            for (int j = 0; j < kV; ++j) m = fmaxf(m, x[j]);
        }
        e.k = m * c;
        float s = e.quick(edge);
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            float x[kV], part = 0.0f;
            unpack<T>(q[i], x);
#pragma unroll
            for (int j = 0; j < kV; ++j) part += e.quick(x[j]);
            s += part;
        }
        // merged over the warp, the CTA and the cluster, in a fixed order
#pragma unroll
        for (int d = 16; d; d >>= 1) merge(m, s, __shfl_xor_sync(~0u, m, d), __shfl_xor_sync(~0u, s, d), c);
        if (t % 32 == 0) {
            tmp[t / 32] = m;
            tmp2[t / 32] = s;
        }
        __syncthreads();
        m = tmp[t % kWarps];
        s = tmp2[t % kWarps];
#pragma unroll
        for (int d = kWarps / 2; d; d >>= 1) merge(m, s, __shfl_xor_sync(~0u, m, d), __shfl_xor_sync(~0u, s, d), c);
        if (ctas > 1) {
            if (t == 0) mine = make_float2(m, s);
            sync_cluster();
            const float2 first = peer2(&mine, 0);
            m = first.x;
            s = first.y;
            for (uint32_t r = 1; r < ctas; ++r) {
                const float2 v = peer2(&mine, r);
                merge(m, s, v.x, v.y, c);
            }
        }
        if (!(fabsf(m) < most)) {
            // the same for every thread of the cluster: the plain form, maximum first
            m = edge;
#pragma unroll 1
            for (uint32_t v = t; v < nvec; v += kThreads) {
                float x[kV];
                unpack<T>(ld_plain_v4(zs + head + v * kV), x);
#pragma unroll
                for (int j = 0; j < kV; ++j) m = fmaxf(m, x[j]);
            }
            m = block_reduce<kThreads, true>(m, tmp);
            if (ctas > 1) {
                sync_cluster();
                if (t == 0) mine.x = m;
                sync_cluster();
                for (uint32_t r = 0; r < ctas; ++r) m = fmaxf(m, peer2(&mine, r).x);
            }
            e = {0.0f, m, 1.0f, c, false};
            s = has_edge ? e.slow(edge) : 0.0f;
#pragma unroll 1
            for (uint32_t v = t; v < nvec; v += kThreads) {
                float x[kV];
                unpack<T>(ld_plain_v4(zs + head + v * kV), x);
#pragma unroll
                for (int j = 0; j < kV; ++j) s += e.slow(x[j]);
            }
            s = block_reduce<kThreads, false>(s, tmp);
            if (ctas > 1) {
                sync_cluster();
                if (t == 0) mine.x = s;
                sync_cluster();
                s = 0.0f;
                for (uint32_t r = 0; r < ctas; ++r) s += peer2(&mine, r).x;
            }
            lse = fmaf(m, a.inv_t, logf(s));
        } else {
            e.k = m * c;
            lse = (e.k + log2f(s)) * 0.69314718055994531f;
        }
        scale = 1.0f / s;
    }
    const float total = total_weight(a, lists);
    if (t == 0 && rank == 0) write_loss(a, lists, row, w, total, lse);
    if constexpr (kGrad) {
        if (total > 0.0f) {
            const float coef = w * a.temperature, back = a.total / total;
            entry_values<T, kThreads>(a, z, e, coef, scale, back, sums, keys);
            __syncthreads();
            const float by = scale * coef;
            if (e.fast) {
#pragma unroll
                for (int i = 0; i < kNv; ++i)
                    if (t + i * kThreads < nvec) {
                        float x[kV];
                        unpack<T>(q[i], x);
#pragma unroll
                        for (int j = 0; j < kV; ++j) x[j] = e.quick(x[j]) * by;
                        put_vec(t + i * kThreads, x);
                    }
            } else {
#pragma unroll 1
                for (uint32_t v = t; v < nvec; v += kThreads) {
                    float x[kV];
                    unpack<T>(ld_plain_v4(zs + head + v * kV), x);
#pragma unroll
                    for (int j = 0; j < kV; ++j) x[j] = e.slow(x[j]) * by;
                    put_vec(v, x);
                }
            }
            if (has_edge) set(gs, edge_at, e(edge) * by);
            __syncthreads();
            write_entries<T, kThreads>(a, g, sums, keys);
        } else {
            write_zeros();
        }
    }
    if (ctas > 1) sync_cluster();          // a peer may still read `mine`
}

// ----------------------------------------------------------------- rows streamed
constexpr int kDThreads = 512;

template <typename T, bool kGrad>
__global__ void __launch_bounds__(kDThreads) distill_stream_kernel(const __grid_constant__ DistillArgs a) {
    extern __shared__ unsigned long long sums[];                 // [slots]
    int32_t* keys = reinterpret_cast<int32_t*>(sums + a.slots);  // [slots], -1 free
    __shared__ float tmp[kDThreads / 32];
    __shared__ Lists lists;
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
    if (kGrad) {
        for (uint32_t i = threadIdx.x; i < a.slots; i += kDThreads) {
            sums[i] = 0;
            keys[i] = -1;
        }
        __syncthreads();
    }
    read_lists<T, kGrad, kDThreads>(a, z, row, a.loss != nullptr, 0, a.vocab, lists, sums, keys);
    const float c = a.inv_t * kLog2e;
    Exp e{0.0f, 0.0f, 1.0f, c, false};
    float scale = 1.0f, lse;
    if (a.lse_in) {
        lse = a.lse_in[row];
        e = from_lse(a, lse, scale);
        __syncthreads();
    } else {
        float v = -INFINITY;
#pragma unroll 8
        for (uint32_t i = threadIdx.x; i < a.vocab; i += kDThreads) v = fmaxf(v, at(z, i));
        e.k = block_reduce<kDThreads, true>(v, tmp);
        v = 0.0f;
#pragma unroll 8
        for (uint32_t i = threadIdx.x; i < a.vocab; i += kDThreads) v += e(at(z, i));
        const float s = block_reduce<kDThreads, false>(v, tmp);
        lse = fmaf(e.k, a.inv_t, logf(s));
        scale = 1.0f / s;
    }
    const float total = total_weight(a, lists);
    if (threadIdx.x == 0) write_loss(a, lists, row, w, total, lse);
    if constexpr (kGrad) {
        const bool some = total > 0.0f;
        const float coef = some ? w * a.temperature : 0.0f, back = some ? a.total / total : 0.0f, by = scale * coef;
        if (some) entry_values<T, kDThreads>(a, z, e, coef, scale, back, sums, keys);
        __syncthreads();
#pragma unroll 8
        for (uint32_t i = threadIdx.x; i < a.vocab; i += kDThreads) set(g, i, some ? e(at(z, i)) * by : 0.0f);
        __syncthreads();
        if (some) write_entries<T, kDThreads>(a, g, sums, keys);
    }
}

// The row kernels by type, direction and vectors per thread: 128 threads (1, 2, 4, 8), 512
// threads (4, 8).
using DistillKernel = void (*)(DistillArgs);
template <typename T, bool kGrad>
constexpr DistillKernel kRowKernels[6] = {
    distill_row_kernel<T, kGrad, 128, 1>, distill_row_kernel<T, kGrad, 128, 2>, distill_row_kernel<T, kGrad, 128, 4>,
    distill_row_kernel<T, kGrad, 128, 8>, distill_row_kernel<T, kGrad, 512, 4>, distill_row_kernel<T, kGrad, 512, 8>};

}  // namespace

cudaError_t prepare_distill() {
    const int most = static_cast<int>(2 * kMaxDistillTopk * 12);
    cudaError_t e = cudaSuccess;
    const auto allow = [&](DistillKernel k) {
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(reinterpret_cast<const void*>(k), cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    };
    for (int i = 0; i < 6; ++i) {
        allow(kRowKernels<uint16_t, true>[i]);
        allow(kRowKernels<float, true>[i]);
    }
    allow(distill_stream_kernel<uint16_t, true>);
    allow(distill_stream_kernel<float, true>);
    return e;
}

cudaError_t launch_distill(DistillArgs& a, cudaStream_t stream) {
    uint32_t entries = 0;
    for (uint32_t j = 0; j < a.nclients; ++j) entries += a.client[j].topk;
    a.slots = 2;
    while (a.slots < 2 * entries) a.slots *= 2;
    const bool grad = a.grad != nullptr;
    const uint64_t size = a.dtype ? 2 : 4, bytes = a.vocab * size;
    cudaLaunchConfig_t cfg = {};
    cfg.dynamicSmemBytes = grad ? static_cast<size_t>(a.slots) * 12 : 0;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    DistillKernel kern;
    uint32_t cluster = 1;
    while (cluster < 8 && bytes > static_cast<uint64_t>(cluster) * kMaxSlice) cluster *= 2;
    if (bytes > static_cast<uint64_t>(cluster) * kMaxSlice || static_cast<uint64_t>(a.rows) * cluster >= (1ull << 31)) {
        kern = a.dtype ? (grad ? distill_stream_kernel<uint16_t, true> : distill_stream_kernel<uint16_t, false>)
                       : (grad ? distill_stream_kernel<float, true> : distill_stream_kernel<float, false>);
        a.cluster = 1;
        cfg.blockDim = dim3(kDThreads);
    } else {
        // slices of whole vectors, so that they have the row's alignment
        a.cluster = cluster;
        a.slice = static_cast<uint32_t>((a.vocab + cluster * 16ull - 1) / (cluster * 16ull) * 16);
        const uint64_t vecs = a.slice * size / 16 + 1;
        int k = 5;
        cfg.blockDim = dim3(512);
        if (vecs <= 128 * 8) {
            k = vecs <= 128 ? 0 : vecs <= 256 ? 1 : vecs <= 512 ? 2 : 3;
            cfg.blockDim = dim3(128);
        } else if (vecs <= 512 * 4) {
            k = 4;
        }
        kern = a.dtype ? (grad ? kRowKernels<uint16_t, true>[k] : kRowKernels<uint16_t, false>[k])
                       : (grad ? kRowKernels<float, true>[k] : kRowKernels<float, false>[k]);
    }
    at[0].val.clusterDim.x = a.cluster;
    cfg.numAttrs = a.cluster > 1 ? 1 : 0;
    cfg.gridDim = dim3(a.rows * a.cluster);
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace fa
