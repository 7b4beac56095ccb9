// Distillation kernels.
//
//   loss   log sum exp of the row, and over the clients' lists sum p (log p - log q)
//   grad   w T (q - share), share being nonzero at the lists' entries alone
//
// Rows of up to 8 x 66 KB are held in shared memory: a CTA (or a cluster of 2, 4 or 8, each with
// a slice) loads its row once with every load in flight at the same time, sums its exponentials
// -- each warp over a reference of its own, pairs (reference, sum) merged over the CTA and, through
// distributed shared memory, the cluster -- and writes the gradient from there.
// The row is read once and written once: bound by HBM, with the exponentials (two per element of
// a gradient) close behind.  Longer rows are streamed from memory (and L2) twice or three times.
// Of rows whose statistic is given the slices are independent, and of any number.
//
// Measured, back to back (the measured copy rate is 6.77 TB/s): gradient and loss of 4096 rows of
// 32000 bf16 logits, 8 lists of 32, a tenth of the rows masked and a fifth of the lists empty,
// 99 us, 5.4 TB/s (issue slots 52 % busy, HBM at 4.7 TB/s, the rest of the traffic in L2), all rows
// and lists full 114; gradient of 700 x 131075 bf16 from a kept statistic 77 us, 4.8 TB/s; loss
// of 1531 x 32003 fp32 38 us, 5.2 TB/s; one row of 32000 5.2 us.
//
// An exponential is 2^(z c - k) with c = log2(e) / T and k = reference c rounded: one FMA and one
// ex2.  k's rounding is the same in every term and in the statistic that is formed with the
// same k, so it cancels.  Rows whose reference is beyond 2^20 T / log2(e) in size or whose sum is
// beyond 2^90 (masked by the type's lowest value or -inf where the reference was looked for, or
// with infinities) take 2^((z - maximum) c) instead, in further passes over memory.
//
// The shares of the entries are gathered in a hash table in shared memory (entry -> sum of
// (n_j / total) p_jc, total being all the clients' weight): several clients name the same entry,
// and integer adds of fixed-point units give the same sum in any order.  Which clients a row has
// is known after its lists have been read; where they have less than 2^-12 of the total, so that
// the units would be beyond 2^-40 of N_r, the shares are taken once more as parts of N_r.  Only
// calls with such a client have kernels that do (kLight): 4096 rows of 32000 bf16 logits with 8
// lists of 32 in each take 133 us with them and 114 without.  The row is written without the
// shares first, then the table's entries are written over it.
#include <algorithm>

#include "distill.cuh"
#include "device.cuh"

namespace fa {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// A table slot: an entry and the sum of its shares in 2^-51 units, as two 32-bit words (2^-30
// units, and the 21 bits below them: the low words of 2048 terms cannot overflow).  32-bit
// adds in shared memory are single instructions, 64-bit ones loops.
struct Slots {
    int32_t* key;          // -1: free
    uint32_t* hi;          // bit 31: the sum is NaN; once the sums are used, the value's bits
    uint32_t* lo;
    uint16_t* taken;       // the slots in use, in no particular order
    uint32_t* count;       // of them
};
constexpr uint32_t kPoison = 1u << 31;

constexpr uint32_t kSlotBytes = 13;       // 12, and 2 for every two slots: half of them can be taken

__device__ __forceinline__ Slots slots_at(void* p, uint32_t n, uint32_t* count) {
    int32_t* key = static_cast<int32_t*>(p);
    return {key, reinterpret_cast<uint32_t*>(key + n), reinterpret_cast<uint32_t*>(key + 2 * n),
            reinterpret_cast<uint16_t*>(key + 3 * n), count};
}

template <int kThreads>
__device__ __forceinline__ void empty_table(const Slots& s, uint32_t n) {
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
        s.key[i] = -1;
        s.hi[i] = s.lo[i] = 0;
    }
    if (threadIdx.x == 0) *s.count = 0;
}

__device__ __forceinline__ void add_share(const Slots& s, uint32_t h, float x) {
    const float units = x * 1073741824.0f;                       // 2^30: exact
    const uint32_t hi = __float2uint_rz(units);
    atomicAdd(&s.hi[h], hi);
    atomicAdd(&s.lo[h], __float2uint_rn((units - __uint2float_rn(hi)) * 2097152.0f));
}

__device__ __forceinline__ float share_of(const Slots& s, uint32_t h) {
    if (s.hi[h] & kPoison) return NAN;
    const unsigned long long v = (static_cast<unsigned long long>(s.hi[h]) << 21) + s.lo[h];
    return static_cast<float>(v) * 4.4408920985006262e-16f;      // 2^-51
}

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

// ----------------------------------------------------------------- the clients' lists
// The warp's lanes each put a share of entry e into the table (if `mine`).  All lanes stay
// together: lanes that leave the search one by one would each do the rest on their own.
__device__ __forceinline__ void put_shares(const DistillArgs& a, const Slots& table, bool mine, int32_t e, float x) {
    // two multiplications with the high bits folded down between: one alone leaves evenly spaced
    // entries in clusters
    uint32_t h = static_cast<uint32_t>(e) * 2654435761u;
    h = (h ^ h >> 15) * 2246822519u >> a.hash_shift;
    bool search = mine, won = false;
    while (__any_sync(~0u, search))
        if (search) {
            const int32_t was = atomicCAS(&table.key[h], -1, e);
            won = was == -1;
            search = !won && was != e;
            if (search) h = (h + 1) & (a.slots - 1);
        }
    __syncwarp();
    const uint32_t winners = __ballot_sync(~0u, won), lane = threadIdx.x % 32;
    if (winners) {
        uint32_t base = 0;
        if (lane == 0) base = atomicAdd(table.count, static_cast<uint32_t>(__popc(winners)));
        base = __shfl_sync(~0u, base, 0);
        if (won) table.taken[base + __popc(winners & ((1u << lane) - 1))] = static_cast<uint16_t>(h);
    }
    if (mine) {
        if (x != x)
            atomicOr(&table.hi[h], kPoison);
        else
            add_share(table, h, x);
    }
    __syncwarp();
}

struct Lists {
    float on[kMaxDistillClients];       // n_j, 0 if absent (zeroed before)
    float loss[kMaxDistillClients];     // sum p (log p - z / T) of client j
    float mass[kMaxDistillClients];     // sum p: 1 (or 0) up to rounding
};

// The largest value over client cl's used places of a row and the sum of the exponentials over
// it, by one warp; false: the client has nothing for the row, or no weight (then its values are
// nothing to the row, whatever they are).
__device__ __forceinline__ bool list_statistics(const DistillArgs& a, const DistillClient& cl, uint64_t base, float& top,
                                                float& sum) {
    const int lane = threadIdx.x % 32;
    const float c = a.inv_t * kLog2e;
    top = -INFINITY;
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
    const bool on = cl.weight > 0.0f && (__any_sync(~0u, nan) || top > -INFINITY);
    sum = 0.0f;
    for (uint32_t i = lane; i < cl.topk; i += 32)
        if (static_cast<uint32_t>(cl.index[base + i]) < a.vocab)
            sum += ex2((value_at(cl.value, base + i, a.value_dtype) - top) * c);
    sum = warp_sum(sum);
    return on;
}

// A warp per client: softmax of its values over its used places, its part of the loss (kLoss)
// and its shares into the table, as far as they fall into [lo, hi) (kGrad).
template <typename T, bool kGrad, int kThreads>
__device__ __forceinline__ void read_lists(const DistillArgs& a, const T* z, uint32_t row, bool want_loss, uint32_t lo,
                                           uint32_t hi, Lists& l, const Slots& table) {
    const int lane = threadIdx.x % 32;
    for (uint32_t j = threadIdx.x / 32; j < a.nclients; j += kThreads / 32) {
        const DistillClient& cl = a.client[j];
        const uint64_t base = static_cast<uint64_t>(row) * cl.topk;
        float top, sum;
        const bool on = list_statistics(a, cl, base, top, sum);
        const float inv = 1.0f / sum, logsum = logf(sum);
        float loss = 0.0f, mass = 0.0f;
        if (on)
            for (uint32_t i0 = 0; i0 < cl.topk; i0 += 32) {
                const uint32_t i = i0 + lane;
                const int32_t e = i < cl.topk ? cl.index[base + i] : -1;
                const bool used = static_cast<uint32_t>(e) < a.vocab;
                const float d = used ? (value_at(cl.value, base + i, a.value_dtype) - top) * a.inv_t : 0.0f;
                const float p = used ? ex2(d * kLog2e) * inv : 0.0f;
                // a p of 0 is nothing, also where the student's logit is -inf
                const bool some = !(p == 0.0f);
                mass += p;
                if (want_loss && some) loss += p * (d - logsum - at(z, e) * a.inv_t);
                if (kGrad)
                    put_shares(a, table, some && static_cast<uint32_t>(e) >= lo && static_cast<uint32_t>(e) < hi, e, p * cl.share);
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

// Lists of up to 64 places, a warp each: the places are loaded before anything else of the row,
// and the student's logits there (for the loss) are asked for as soon as the places are known
// and used after the row's statistics, so that no memory latency of the lists is waited for.  More
// places, or more lists than the CTA has warps (8; 4 for rows of up to 16 KB), are read in place,
// which is slower: the gradient of 4096 x 32000 bf16 logits takes 114 us with 8 lists of 32 and 176
// with 9, 160 with 8 lists of 64 and 194 with 8 of 65; of 16384 x 8000 127 us with 4 lists of 32
// and 171 with 5.
constexpr int kShortTopk = 64;

struct ShortList {
    int32_t e[2];
    float u[2];       // the client's value, then d - log sum
    float p[2], z[2];
};

__device__ __forceinline__ void load_short(const DistillArgs& a, uint32_t row, uint32_t j, ShortList& s) {
    const DistillClient& cl = a.client[j];
    const uint64_t base = static_cast<uint64_t>(row) * cl.topk;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t at = threadIdx.x % 32 + 32 * i;
        s.e[i] = -1;
        s.u[i] = 0.0f;
        if (at < cl.topk) {
            s.e[i] = cl.index[base + at];
            s.u[i] = value_at(cl.value, base + at, a.value_dtype);
        }
    }
}

template <typename T, bool kGrad>
__device__ __forceinline__ void use_short(const DistillArgs& a, const T* z, uint32_t j, bool want_loss, uint32_t lo,
                                          uint32_t hi, ShortList& s, Lists& l, const Slots& table) {
    const DistillClient& cl = a.client[j];
    float top = -INFINITY;
    bool nan = false, used[2] = {false, false};
    const int places = cl.topk > 32 ? 2 : 1;      // of a lane
    s.z[1] = s.p[1] = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (i >= places) break;
        used[i] = static_cast<uint32_t>(s.e[i]) < a.vocab;
        if (s.e[i] >= 0 && !used[i]) atomicOr(a.err, kErrListIndex);
        s.z[i] = used[i] && want_loss ? at(z, s.e[i]) : 0.0f;
        nan |= used[i] && s.u[i] != s.u[i];
        if (used[i]) top = fmaxf(top, s.u[i]);
    }
    top = warp_max(top);
    const bool on = cl.weight > 0.0f && (__any_sync(~0u, nan) || top > -INFINITY);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (i >= places) break;
        s.u[i] = (s.u[i] - top) * a.inv_t;
        s.p[i] = used[i] ? ex2(s.u[i] * kLog2e) : 0.0f;
        sum += s.p[i];
    }
    sum = warp_sum(sum);
    const float inv = on ? 1.0f / sum : 0.0f, logsum = logf(sum);
    float mass = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (i >= places) break;
        s.p[i] = on ? s.p[i] * inv : 0.0f;
        s.u[i] -= logsum;
        mass += s.p[i];
        const uint32_t e = static_cast<uint32_t>(s.e[i]);
        if (kGrad) put_shares(a, table, !(s.p[i] == 0.0f) && e >= lo && e < hi, s.e[i], s.p[i] * cl.share);
    }
    mass = warp_sum(mass);
    if (threadIdx.x % 32 == 0) {
        l.mass[j] = mass;
        l.on[j] = on ? cl.weight : 0.0f;
    }
}

// Its part of the loss, once the row's statistics have been taken.
__device__ __forceinline__ void end_short(const DistillArgs& a, uint32_t j, const ShortList& s, Lists& l) {
    float loss = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (!(s.p[i] == 0.0f)) loss += s.p[i] * (s.u[i] - s.z[i] * a.inv_t);
    loss = warp_sum(loss);
    if (threadIdx.x % 32 == 0) l.loss[j] = loss;
}

// The shares again, as parts of the row's own weight: the sums taken so far are discarded (their
// slots stay).  By the whole CTA, after a barrier behind the lists.
template <int kThreads>
__device__ __noinline__ void share_again(const DistillArgs& a, uint32_t row, uint32_t lo, uint32_t hi, const Lists& l, float total,
                                         Slots table) {
    for (uint32_t i = threadIdx.x; i < *table.count; i += kThreads) {
        const uint32_t h = table.taken[i];
        table.hi[h] = table.lo[h] = 0;
    }
    __syncthreads();
    for (uint32_t j = threadIdx.x / 32; j < a.nclients; j += kThreads / 32) {
        if (!(l.on[j] > 0.0f)) continue;
        const DistillClient& cl = a.client[j];
        const uint64_t base = static_cast<uint64_t>(row) * cl.topk;
        float top, sum;
        list_statistics(a, cl, base, top, sum);
        const float inv = 1.0f / sum, share = l.on[j] / total;
        for (uint32_t i0 = 0; i0 < cl.topk; i0 += 32) {
            const uint32_t i = i0 + threadIdx.x % 32;
            const int32_t e = i < cl.topk ? cl.index[base + i] : -1;
            const bool used = static_cast<uint32_t>(e) < a.vocab;
            const float d = used ? (value_at(cl.value, base + i, a.value_dtype) - top) * a.inv_t : 0.0f;
            const float p = used ? ex2(d * kLog2e) * inv : 0.0f;
            put_shares(a, table, !(p == 0.0f) && static_cast<uint32_t>(e) >= lo && static_cast<uint32_t>(e) < hi, e, p * share);
        }
    }
    __syncthreads();
}

// What the table's sums are to be multiplied by to be parts of N_r.
template <int kThreads, bool kLight>
__device__ __forceinline__ float shares_scale(const DistillArgs& a, uint32_t row, uint32_t lo, uint32_t hi, const Lists& l,
                                              float total, const Slots& table) {
    const float back = a.total / total;
    if constexpr (kLight)
        if (total > 0.0f && back > kLightest) {
            share_again<kThreads>(a, row, lo, hi, l, total, table);
            return 1.0f;
        }
    return back;
}

// N_r; 0: no client.  The lists have been read by the whole CTA.
__device__ __forceinline__ float total_weight(const DistillArgs& a, const Lists& l) {
    float total = 0.0f;
    for (uint32_t j = 0; j < a.nclients; j += 4) {
        const float4 v = *reinterpret_cast<const float4*>(&l.on[j]);
        total += (v.x + v.y) + (v.z + v.w);
    }
    return total;
}

// By one whole warp, a lane per client.
__device__ __forceinline__ void write_loss(const DistillArgs& a, const Lists& l, uint32_t row, float w, float total, float lse) {
    const uint32_t j = threadIdx.x % 32;
    float loss = 0.0f;
    // n_j / N first: the terms of a logit near the type's lowest are near fp32's range
    if (a.loss && j < a.nclients && l.on[j] > 0.0f) loss = l.on[j] / total * fmaf(lse, l.mass[j], l.loss[j]);
    loss = warp_sum(loss);
    if (j != 0) return;
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
// Every partial sum is held to this before it is scaled to a larger reference: the scale is 0
// beyond a gap of 126 (ex2.approx flushes), and a sum that may be dropped then has to be small
// beside the larger reference's own term of 1 -- 2^90 leaves 2^-36 of it.
constexpr float kSumMost = 0x1p90f;
// A partial sum beyond it (or NaN) is passed on as an infinity, which no scale turns into a
// number below kSumMost: the row takes the plain form.
__device__ __forceinline__ float bounded(float s) { return s < kSumMost ? s : INFINITY; }

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
template <int kThreads, typename At>
__device__ __forceinline__ void entry_values(const DistillArgs& a, At z_at, const Exp& e, float coef, float scale, float back,
                                             const Slots& table) {
    for (uint32_t i = threadIdx.x; i < *table.count; i += kThreads) {
        const uint32_t h = table.taken[i];
        table.hi[h] = __float_as_uint(coef * (e(z_at(table.key[h])) * scale - share_of(table, h) * back));
    }
}

// ... leaving the slots free for the next row (the count is the caller's to reset).
template <typename T, int kThreads>
__device__ __forceinline__ void write_entries(const DistillArgs& a, T* g, bool some, const Slots& table) {
    for (uint32_t i = threadIdx.x; i < *table.count; i += kThreads) {
        const uint32_t h = table.taken[i];
        if (some) set(g, table.key[h], __uint_as_float(table.hi[h]));
        table.key[h] = -1;
        table.hi[h] = table.lo[h] = 0;
    }
}

// ----------------------------------------------------------------- rows held on chip
// Bytes of a row that a CTA holds: three CTAs per SM.  With 48 KB, four of them: the gradient of 4096
// x 32000 bf16 149 us (this way 102), of 2048 x 65536 149 (110), of 1531 x 32003 fp32 95 (75).
constexpr uint32_t kMaxSlice = 66 * 1024;
constexpr uint32_t kSmallSlice = 16 * 1024; // held by 128 threads, larger ones by 256
constexpr uint32_t kSharedBytes = 227 * 1024, kSliceCost = 16 * 1024;

__device__ __forceinline__ uint32_t rank_in_cluster() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// A pair from every CTA of a cluster to every CTA, in shared memory: two sets in turn, since a
// peer that has this CTA's pair may go on to the next exchange while this one still waits for
// others'.  The pairs are sent by st.async, which counts their bytes at the receiver's barrier:
// a cluster barrier's release would wait for the row's stores and the next row's loads as well
// (the loss of 1531 rows of 32003 fp32 logits: 42.9 us, against 39.4 this way).
constexpr uint32_t kMaxCluster = 8;
constexpr long long kMaxWaitClocks = 40ll * 1000 * 1000 * 1000;      // some 20 s
struct Exchange {
    unsigned long long bar[2];
    float2 pair[2][kMaxCluster];
    uint32_t gone;                         // a wait has run out: the CTA leaves
};

__device__ __forceinline__ void open_exchange(Exchange& x) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\nmbarrier.init.shared::cta.b64 [%1], 1;\n"
                 "fence.mbarrier_init.release.cluster;" ::"r"(smem_addr(&x.bar[0])), "r"(smem_addr(&x.bar[1])) : "memory");
    x.gone = 0;
}

// By one warp.  False: the peers' pairs have not come.
__device__ __forceinline__ bool swap_pairs(Exchange& x, uint32_t turn, uint32_t ctas, uint32_t rank, float2 v, bool expire) {
    const uint32_t lane = threadIdx.x % 32, bar = smem_addr(&x.bar[turn % 2]), to = smem_addr(&x.pair[turn % 2][rank]);
    if (lane == 0)
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(ctas * 8) : "memory");
    if (lane < ctas)
        asm volatile(
            "{\n .reg .b32 to, bar;\n mapa.shared::cluster.u32 to, %0, %2;\n mapa.shared::cluster.u32 bar, %1, %2;\n"
            " st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [to], {%3, %4}, [bar];\n}" ::"r"(to),
            "r"(bar), "r"(lane), "f"(v.x), "f"(v.y)
            : "memory");
    const long long t0 = clock64();
    for (uint32_t done = 0; !done;) {
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, 1000000;\n"
            " selp.u32 %0, 1, 0, p;\n}"
            : "=r"(done)
            : "r"(bar), "r"(turn / 2 % 2)
            : "memory");
        if (!done && clock64() - t0 > kMaxWaitClocks) return false;
    }
    return !expire;
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

// Pairs (m, s), a reference and a sum: the sum of 2^(z c) is s 2^(m c), m c rounded as in Exp.
// Over the warp's lanes (kLanes: the first so many hold pairs, the others repeat them).
__device__ __forceinline__ float warp_largest(float m) {
    float top;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(top) : "f"(m));
    return top;
}

template <int kLanes>
__device__ __forceinline__ void merge_lanes(float& m, float& s, float c) {
    const float top = warp_largest(m);
    s *= ex2(__fmul_rn(m, c) - __fmul_rn(top, c));      // the rounded products, as in k
#pragma unroll
    for (int d = kLanes / 2; d; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
    m = top;
}

__device__ __forceinline__ void merge(float& m, float& s, float m2, float s2, float c) {
    const float top = fmaxf(m, m2), k = __fmul_rn(top, c);
    s = __fmaf_rn(s2, ex2(__fmul_rn(m2, c) - k), __fmul_rn(s, ex2(__fmul_rn(m, c) - k)));
    m = top;
}

// Two floats at a time (packed fp32 arithmetic).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
        " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n"
        " mov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 d, a, b;\n"
        " mov.b64 {%0, %1}, d;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// The larger of m and the elements of 16 bytes (NaNs left out).
template <typename T>
__device__ __forceinline__ float max_of(float m, const uint4& q) {
    if constexpr (sizeof(T) == 2) {
        const auto two = [](uint32_t x, uint32_t y) {
            uint32_t r;
            asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
            return r;
        };
        const uint32_t r = two(two(q.x, q.y), two(q.z, q.w));
        return fmaxf(m, fmaxf(bf16_lo(r), bf16_hi(r)));
    } else {
        return fmaxf(fmaxf(m, fmaxf(__uint_as_float(q.x), __uint_as_float(q.y))),
                     fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
    }
}

// Where a row's slice lies: 16-byte vectors with `head` elements before them and `tail` after.
template <typename T>
struct Place {
    static constexpr uint32_t kV = 16 / sizeof(T);
    const T* z;             // the slice's first element
    uint32_t head, nvec, tail;
    __device__ __forceinline__ Place(const DistillArgs& a, uint32_t row, uint32_t lo, uint32_t n)
        : z(static_cast<const T*>(a.logits) + row * a.ld + lo) {
        const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(z) % 16 / sizeof(T));
        head = min(off ? kV - off : 0, n);
        nvec = (n - head) / kV;
        tail = n - head - nvec * kV;
    }
    // elements outside the vectors, one per thread: thread t's, if it has one
    __device__ __forceinline__ bool edge(uint32_t t) const { return t < head || (t >= kV && t - kV < tail); }
    __device__ __forceinline__ uint32_t edge_at(uint32_t t) const { return t < head ? t : head + nvec * kV + t - kV; }
};

// Rows (or slices of them: kJoint, a cluster's, kSlices, independent ones) held in shared memory.
// Three or four CTAs of 256 threads per SM, whose slices in flight hide HBM's latency.  Slices of
// a cluster are larger, three per SM, and take the registers for it (1531 x 32003 fp32: 37.3 us,
// with a bound for four 39.0); whole rows fit four (6000 rows of 20000 bf16, with the gradient:
// 98 us, with three 107).  Each thread copies its own 16-byte vectors there (cp.async: no registers held, no barrier needed) and
// goes over them twice; as it leaves a vector for the last time it asks for the next row's in
// its place, and the next row's lists and weight are loaded as early, so that HBM is read while
// a row is being worked on.  Elements beside the vectors are held one per thread in `edge`.
enum RowForm { kWhole, kSlices, kJoint };
template <typename T, bool kGrad, int kThreads, RowForm kForm, bool kLight = false>
__global__ void __launch_bounds__(kThreads, kThreads == 128 ? 8 : kForm == kWhole ? 4 : 3) distill_row_kernel(const __grid_constant__ DistillArgs a) {
    constexpr uint32_t kV = 16 / sizeof(T), kWarps = kThreads / 32;
    extern __shared__ __align__(16) uint8_t dyn[];               // the slice's vectors, the table
    __shared__ float tmp[kWarps], tmp2[kWarps];
    __shared__ Exchange exchange;
    __shared__ __align__(16) Lists lists;
    __shared__ uint32_t taken;
    const uint32_t ctas = kForm == kWhole ? 1 : a.parts;
    const uint32_t rank = kForm == kJoint ? rank_in_cluster() : kForm == kSlices ? blockIdx.x % ctas : 0;
    if constexpr (kForm == kJoint) {
        if (threadIdx.x == 0) open_exchange(exchange);
        __syncwarp();
        cluster_arrive();
    }
    const uint32_t t = threadIdx.x, step = gridDim.x / ctas;
    const uint32_t lo = rank * a.slice, hi = min(lo + a.slice, a.vocab), n = hi > lo ? hi - lo : 0;
    const bool brief = a.short_lists && a.nclients <= kWarps, has_list = brief && t / 32 < a.nclients;
    const bool want_loss = rank == 0 && a.loss;
    const uint4* held = reinterpret_cast<const uint4*>(dyn);
    const uint32_t held_at = smem_addr(dyn);
    const Slots table = slots_at(dyn + a.table_at, a.slots, &taken);
    const auto weight_of = [&](uint32_t row) { return row < a.rows ? (a.row_weight ? a.row_weight[row] : 1.0f) : 0.0f; };
    const auto fetch = [&](const uint4* mem, uint32_t v) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(held_at + v * 16), "l"(mem + v) : "memory");
    };

    uint32_t row = blockIdx.x / ctas;
    ShortList list;
    if (has_list) load_short(a, row, t / 32, list);
    float w = weight_of(row);
    if (kGrad) empty_table<kThreads>(table, a.slots);
    Place<T> at_row(a, row, lo, n);
    float edge = -INFINITY;
    if (w > 0.0f) {
        const uint4* mem = reinterpret_cast<const uint4*>(at_row.z + at_row.head);
        for (uint32_t v = t; v < at_row.nvec; v += kThreads) fetch(mem, v);
        if (at_row.edge(t)) edge = at(at_row.z, at_row.edge_at(t));
    }
    const float c = a.inv_t * kLog2e, most = kFastMost / c;      // of a maximum, for the fast form

    uint32_t turn = 0;                     // exchanges so far
    const float2* pairs = nullptr;         // the last one's
    const auto give = [&](float x, float y) {          // the same in every thread; false: the CTA leaves
        if (t < 32 && !swap_pairs(exchange, turn, ctas, rank, make_float2(x, y), a.test_expire)) {
            exchange.gone = 1;
            atomicOr(a.err, kErrWaitTimeout);
        }
        pairs = exchange.pair[turn++ % 2];
        __syncthreads();
        return exchange.gone == 0;
    };
    if (kForm == kJoint) cluster_wait();           // the peers' barriers are set up
    while (row < a.rows) {
        const uint32_t next = row + step;
        const float w_next = weight_of(next);
        const Place<T> place = at_row;
        at_row = Place<T>(a, next < a.rows ? next : row, lo, n);
        const uint4 *mem = reinterpret_cast<const uint4*>(place.z + place.head),
                    *mem_next = reinterpret_cast<const uint4*>(at_row.z + at_row.head);
        const T* z = place.z - lo;
        T* g = kGrad ? static_cast<T*>(a.grad) + row * a.ldg : nullptr;
        T* gs = kGrad ? g + lo : nullptr;
        const uint32_t nvec = place.nvec, head = place.head;
        const bool has_edge = place.edge(t);
        const bool same_phase = kGrad && reinterpret_cast<uintptr_t>(gs) % 16 == reinterpret_cast<uintptr_t>(place.z) % 16;
        const auto put_vec = [&](uint32_t v, const uint4& x) {
            T* p = gs + head + v * kV;
            if (same_phase) {
                st_v4u(p, x);
            } else {
                const T* e = reinterpret_cast<const T*>(&x);
#pragma unroll
                for (uint32_t i = 0; i < kV; ++i) p[i] = e[i];
            }
        };
        const auto write_zeros = [&] {
            for (uint32_t v = t; v < nvec; v += kThreads) put_vec(v, make_uint4(0, 0, 0, 0));
            if (has_edge) set(gs, place.edge_at(t), 0.0f);
        };
        // a thread's vectors of the next row from v on, once the present ones are not needed
        const auto fetch_next = [&](uint32_t v) {
            if (w_next > 0.0f)
                for (; v < at_row.nvec; v += kThreads) fetch(mem_next, v);
        };
        if (!(w > 0.0f)) {
            if (kGrad) write_zeros();
            if (t == 0 && rank == 0) {
                if (a.loss) a.loss[row] = 0.0f;
                if (a.lse_out) a.lse_out[row] = 0.0f;
            }
            fetch_next(t);
        } else {
            if (t < kMaxDistillClients) lists.on[t] = 0.0f;
            __syncthreads();
            if (has_list)
                use_short<T, kGrad>(a, z, t / 32, want_loss, lo, hi, list, lists, table);
            else if (!brief)
                read_lists<T, kGrad, kThreads>(a, z, row, want_loss, lo, hi, lists, table);
            asm volatile("cp.async.wait_all;" ::: "memory");

            Exp e{c, 0.0f, 0.0f, 0.0f, true};
            float scale = 1.0f, sum = 1.0f;        // q = e(z) * scale
            if (a.lse_in) {
                e = from_lse(a, a.lse_in[row], scale);
                if (has_list && want_loss) end_short(a, t / 32, list, lists);
                __syncthreads();
                // in place, the peers may write their slices only when rank 0 has taken the
                // loss's logits (below, the exchange of statistics sees to that)
                if (kForm == kJoint && !give(0.0f, 0.0f)) break;
            } else {
                // One pass: the sum over a reference, the largest of what the warp has at two
                // places of the row, in place of the maximum.  Terms over it are no harm up to
                // kSumMost (beyond, the plain form below).
                float m = fmaxf(edge, -most);
                if (t < nvec) {
                    m = max_of<T>(m, held[t]);
                    m = max_of<T>(m, held[t + (nvec - 1 - t) / (2 * kThreads) * kThreads]);
                }
                m = warp_largest(m);
                e.k = __fmul_rn(m, c);
                float2 s2 = make_float2(e.quick(edge), 0.0f);
                const float2 cc = make_float2(c, c), kk = make_float2(-e.k, -e.k);
#pragma unroll 4
                for (uint32_t v = t; v < nvec; v += kThreads) {
                    float x[kV];
                    unpack<T>(held[v], x);
                    if (!kGrad && w_next > 0.0f && v < at_row.nvec) fetch(mem_next, v);
                    float2 part = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (uint32_t j = 0; j < kV; j += 2) {
                        const float2 y = fma2(make_float2(x[j], x[j + 1]), cc, kk);
                        part = add2(part, make_float2(ex2(y.x), ex2(y.y)));
                    }
                    s2 = add2(s2, part);
                }
                if (!kGrad) fetch_next(t < nvec ? t + (nvec - t + kThreads - 1) / kThreads * kThreads : t);
                // merged over the warp, the CTA and the cluster, in a fixed order
                float s = bounded(warp_sum(s2.x + s2.y));
                if (t % 32 == 0) {
                    tmp[t / 32] = m;
                    tmp2[t / 32] = s;
                }
                if (has_list && want_loss) end_short(a, t / 32, list, lists);
                __syncthreads();
                m = tmp[t % kWarps];
                s = tmp2[t % kWarps];
                merge_lanes<kWarps>(m, s, c);
                if constexpr (kForm == kJoint) {
                    if (!give(m, bounded(s))) break;
                    m = pairs[0].x;
                    s = pairs[0].y;
                    for (uint32_t r = 1; r < ctas; ++r) merge(m, s, pairs[r].x, pairs[r].y, c);
                }
                if (!(fabsf(m) < most && s < kSumMost)) {
                    // the same for every thread of the cluster: the plain form from memory,
                    // maximum first
                    m = edge;
                    for (uint32_t v = t; v < nvec; v += kThreads) m = max_of<T>(m, ld_plain_v4(mem + v));
                    m = block_reduce<kThreads, true>(m, tmp);
                    if constexpr (kForm == kJoint) {
                        if (!give(m, 0.0f)) break;
                        for (uint32_t r = 0; r < ctas; ++r) m = fmaxf(m, pairs[r].x);
                    }
                    e = {0.0f, m, 1.0f, c, false};
                    s = has_edge ? e.slow(edge) : 0.0f;
                    for (uint32_t v = t; v < nvec; v += kThreads) {
                        float x[kV];
                        unpack<T>(ld_plain_v4(mem + v), x);
#pragma unroll
                        for (uint32_t j = 0; j < kV; ++j) s += e.slow(x[j]);
                    }
                    s = block_reduce<kThreads, false>(s, tmp);
                    if constexpr (kForm == kJoint) {
                        if (!give(s, 0.0f)) break;
                        s = 0.0f;
                        for (uint32_t r = 0; r < ctas; ++r) s += pairs[r].x;
                    }
                } else {
                    e.k = __fmul_rn(m, c);
                }
                scale = __frcp_rn(s);
                sum = s;
            }
            if (has_list && next < a.rows) load_short(a, next, t / 32, list);
            const float total = total_weight(a, lists);
            if constexpr (kGrad) {
                const float back = shares_scale<kThreads, kLight>(a, row, lo, hi, lists, total, table);
                const float coef = w * a.temperature, by = scale * coef;
                const auto z_at = [&](int32_t key) {
                    const uint32_t i = key - lo - head;          // below 0: beyond nvec * kV
                    return i < nvec * kV ? at(reinterpret_cast<const T*>(dyn), i) : at(z, key);
                };
                if (total > 0.0f) entry_values<kThreads>(a, z_at, e, coef, scale, back, table);
                __syncthreads();
                const auto grad_of = [&](uint32_t v) {
                    const float2 cc = make_float2(e.c, e.c), kk = make_float2(-e.k, -e.k), bb = make_float2(by, by);
                    float x[kV];
                    unpack<T>(held[v], x);
#pragma unroll
                    for (uint32_t j = 0; j < kV; j += 2) {
                        float2 y = fma2(make_float2(x[j], x[j + 1]), cc, kk);
                        y = mul2(make_float2(ex2(y.x), ex2(y.y)), bb);
                        x[j] = y.x;
                        x[j + 1] = y.y;
                    }
                    return pack<T>(x);
                };
                if (!(total > 0.0f)) {
                    write_zeros();
                    fetch_next(t);
                } else if (e.fast && same_phase) {
                    uint4* to = reinterpret_cast<uint4*>(gs + head);
                    const uint32_t ahead = w_next > 0.0f ? at_row.nvec : 0;
#pragma unroll 4
                    for (uint32_t v = t; v < nvec; v += kThreads) {
                        st_v4u(to + v, grad_of(v));
                        if (v < ahead) fetch(mem_next, v);
                    }
                    fetch_next(t < nvec ? t + (nvec - t + kThreads - 1) / kThreads * kThreads : t);
                } else {
                    for (uint32_t v = t; v < nvec; v += kThreads) {
                        if (e.fast) {
                            put_vec(v, grad_of(v));
                        } else {
                            float x[kV];
                            unpack<T>(held[v], x);
#pragma unroll
                            for (uint32_t j = 0; j < kV; ++j) x[j] = e.slow(x[j]) * by;
                            put_vec(v, pack<T>(x));
                        }
                    }
                    fetch_next(t);
                }
                if (has_edge && total > 0.0f) set(gs, place.edge_at(t), e(edge) * by);
                __syncthreads();
                write_entries<T, kThreads>(a, g, total > 0.0f, table);
            }
            // by the warp that has the fewest lists
            if (t / 32 == kWarps - 1 && rank == 0 && (a.loss || a.lse_out)) {
                const float lse = a.lse_in  ? a.lse_in[row]
                                  : e.fast ? (e.k + log2f(sum)) * 0.69314718055994531f
                                           : fmaf(e.k, a.inv_t, logf(sum));
                write_loss(a, lists, row, w, total, lse);
            }
            __syncthreads();                   // the lists' and the reductions' places are free
            if (kGrad && t == 0) taken = 0;
        }
        if (!(w > 0.0f) && has_list && next < a.rows) load_short(a, next, t / 32, list);
        edge = w_next > 0.0f && at_row.edge(t) ? at(at_row.z, at_row.edge_at(t)) : -INFINITY;
        w = w_next;
        row = next;
    }
    if constexpr (kForm == kJoint) {
        asm volatile("cp.async.wait_all;" ::: "memory");     // a wait has run out: loads of the next row
        // a peer may still send to this CTA
        cluster_arrive();
        cluster_wait();
    }
}

// ----------------------------------------------------------------- rows streamed
constexpr int kDThreads = 512;

template <typename T, bool kGrad>
__global__ void __launch_bounds__(kDThreads) distill_stream_kernel(const __grid_constant__ DistillArgs a) {
    extern __shared__ __align__(16) uint8_t dyn[];               // the table
    __shared__ float tmp[kDThreads / 32];
    __shared__ __align__(16) Lists lists;
    __shared__ uint32_t taken;
    const Slots table = slots_at(dyn, a.slots, &taken);
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
    if (kGrad) empty_table<kDThreads>(table, a.slots);
    if (threadIdx.x < kMaxDistillClients) lists.on[threadIdx.x] = 0.0f;
    __syncthreads();
    read_lists<T, kGrad, kDThreads>(a, z, row, a.loss != nullptr, 0, a.vocab, lists, table);
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
    if (threadIdx.x < 32) write_loss(a, lists, row, w, total, lse);
    if constexpr (kGrad) {
        const bool some = total > 0.0f;
        const float back = shares_scale<kDThreads, true>(a, row, 0, a.vocab, lists, total, table);
        const float coef = some ? w * a.temperature : 0.0f, by = scale * coef;
        if (some) entry_values<kDThreads>(a, [&](int32_t i) { return at(z, i); }, e, coef, scale, back, table);
        __syncthreads();
#pragma unroll 8
        for (uint32_t i = threadIdx.x; i < a.vocab; i += kDThreads) set(g, i, some ? e(at(z, i)) * by : 0.0f);
        __syncthreads();
        write_entries<T, kDThreads>(a, g, some, table);
    }
}

using DistillKernel = void (*)(DistillArgs);
// A kernel for a row's form and a slice's size (a cluster's slices are of 33 KB and more).  The
// gradients of calls with a light client are few: 256 threads for slices of any size.
template <typename T, bool kGrad>
DistillKernel row_kernel(RowForm form, bool small, bool light) {
    if constexpr (kGrad)
        if (light)
            return form == kJoint    ? distill_row_kernel<T, true, 256, kJoint, true>
                   : form == kSlices ? distill_row_kernel<T, true, 256, kSlices, true>
                                     : distill_row_kernel<T, true, 256, kWhole, true>;
    if (form == kJoint) return distill_row_kernel<T, kGrad, 256, kJoint>;
    if constexpr (kGrad)
        if (form == kSlices) return small ? distill_row_kernel<T, true, 128, kSlices> : distill_row_kernel<T, true, 256, kSlices>;
    return small ? distill_row_kernel<T, kGrad, 128, kWhole> : distill_row_kernel<T, kGrad, 256, kWhole>;
}

}  // namespace

cudaError_t prepare_distill() {
    cudaError_t e = cudaSuccess;
    const auto allow = [&](DistillKernel k) {
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(reinterpret_cast<const void*>(k), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kMaxSlice + kSlotBytes * 2 * kMaxDistillTopk);
    };
    for (RowForm form : {kWhole, kSlices, kJoint})
        for (bool small : {false, true}) {
            allow(row_kernel<uint16_t, false>(form, small, false));
            allow(row_kernel<uint16_t, true>(form, small, small));
            allow(row_kernel<uint16_t, true>(form, small, false));
            allow(row_kernel<float, false>(form, small, false));
            allow(row_kernel<float, true>(form, small, small));
            allow(row_kernel<float, true>(form, small, false));
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
    a.hash_shift = 32;
    for (uint32_t n = a.slots; n > 1; n /= 2) --a.hash_shift;          // the top log2(slots) bits
    a.short_lists = true;
    for (uint32_t j = 0; j < a.nclients; ++j) a.short_lists = a.short_lists && a.client[j].topk <= kShortTopk;
    const bool grad = a.grad != nullptr;
    const uint32_t size = a.dtype ? 2 : 4, table = grad ? a.slots * kSlotBytes : 0;
    const uint64_t bytes = static_cast<uint64_t>(a.vocab) * size;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    DistillKernel kern;
    // slices of 16 elements' multiples, so that they all have the row's alignment
    const auto slice_of = [&](uint64_t n) { return static_cast<uint32_t>((a.vocab + n * 16 - 1) / (n * 16) * 16); };
    bool held = true;                      // rows on chip
    uint64_t parts = 1;
    // With the statistic given, a row's slices need nothing of one another -- but for the loss at
    // the logits that the gradient replaces.  Their number is then free: the one with the least
    // work on the SM that has the most, a slice's lists and barriers costing as much as some
    // kSliceCost bytes.  Against the least power of two: 700 rows of 131075 bf16 logits 77.3 us
    // and 81.2, 1000 of 50000 42.9 and 47.1, 8 of 131075 8.2 and 10.3 (700 of 131072 in fp32
    // 134.0 and 131.8).
    const bool apart = grad && a.lse_in && !(a.loss && a.grad == a.logits);
    if (apart) {
        const uint64_t least = (bytes + kMaxSlice - 1) / kMaxSlice, top = std::max<uint64_t>(16, std::min(4 * least, least + 64));
        uint64_t best = ~0ull;
        for (uint64_t n = least; n <= top && n * 1024 <= bytes + 1024 * least; ++n) {
            const uint64_t held_bytes = static_cast<uint64_t>(slice_of(n)) * size;
            const uint64_t fit = kSharedBytes / (held_bytes + table + 2048), most = held_bytes > kSmallSlice ? 3 : 8;
            const uint64_t per_sm = std::min({fit, most, (a.rows * n + a.sms - 1) / a.sms});
            const uint64_t at_once = std::max<uint64_t>(1, a.sms * per_sm / n);      // rows
            const uint64_t turns = (a.rows + at_once - 1) / at_once;
            if (turns * per_sm * (held_bytes + kSliceCost) < best) {
                best = turns * per_sm * (held_bytes + kSliceCost);
                parts = n;
            }
        }
    } else {
        while (parts < kMaxCluster && bytes > parts * kMaxSlice) parts *= 2;
    }
    a.joint = !apart && parts > 1;
    // Rows that a cluster does not hold, and without a statistic, are streamed: of 1024 fp32 rows with
    // 4 lists of 32, loss and gradient take 100 and 212 us at 135168 entries (held), 174 and 723 at
    // 135200 (streamed); of 512 bf16 rows 57 and 121 at 270336, 142 and 703 at 270400.
    if (bytes > parts * kMaxSlice || a.rows * parts >= (1ull << 31)) {
        kern = a.dtype ? (grad ? distill_stream_kernel<uint16_t, true> : distill_stream_kernel<uint16_t, false>)
                       : (grad ? distill_stream_kernel<float, true> : distill_stream_kernel<float, false>);
        held = false;
        a.parts = 1;
        cfg.blockDim = dim3(kDThreads);
        cfg.dynamicSmemBytes = table;
    } else {
        a.parts = static_cast<uint32_t>(parts);
        a.slice = slice_of(parts);
        a.table_at = (a.slice < a.vocab ? a.slice : a.vocab) * size / 16 * 16;
        const bool light = grad && a.light, small = !a.joint && a.table_at <= kSmallSlice && !light;
        const RowForm form = a.joint ? kJoint : parts > 1 ? kSlices : kWhole;
        cfg.blockDim = dim3(small ? 128 : 256);
        cfg.dynamicSmemBytes = a.table_at + table;
        kern = a.dtype ? (grad ? row_kernel<uint16_t, true>(form, small, light) : row_kernel<uint16_t, false>(form, small, false))
                       : (grad ? row_kernel<float, true>(form, small, light) : row_kernel<float, false>(form, small, false));
    }
    const uint32_t cluster = a.joint ? a.parts : 1;
    at[0].val.clusterDim.x = cluster;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    cfg.gridDim = dim3(a.rows * a.parts);
    if (held) {
        // as many rows as run at one time; the same kernel and sizes as in the last call of this
        // thread are not asked for again
        static thread_local struct {
            DistillKernel kern = nullptr;
            uint32_t cluster = 0;
            size_t smem = 0;
            int device = -1, clusters = 0;
        } last;
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess &&
            !(last.kern == kern && last.cluster == cluster && last.smem == cfg.dynamicSmemBytes && last.device == dev)) {
            int n = 0;
            cudaLaunchConfig_t ask = cfg;
            ask.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&n, reinterpret_cast<const void*>(kern), &ask);
            last = {kern, cluster, cfg.dynamicSmemBytes, dev, n};
        }
        if (e != cudaSuccess) return e;
        const uint32_t rows = static_cast<uint32_t>(last.clusters) * cluster / a.parts;
        if (rows > 0 && a.rows > rows) cfg.gridDim = dim3(rows * a.parts);
    }
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace fa
