// Rotary positions of queries and keys.
//
//   (u, v) -> scale * (u cos t - v sin t, v cos t + u sin t),   t = position * frequency of the pair
//
// The gradient is the same map with -t.  A position is an integer and a frequency is held as a
// whole number of 2^-64 turns, so that their product modulo 2^64 is the angle modulo a turn,
// exactly: no table of cosines is read, and a far position is as exact as a near one.  The
// quadrant is taken off in integers too; the rest, |t| <= pi / 4, goes through sincospif.
//
// Two forms.  rotary_kernel: a thread has V pairs (its vectors are V elements) and turns them in
// several heads of one token, so that the sines are computed once for all of these.
// rotary_ring_kernel, for many 16-bit tokens whose heads lie side by side: CTAs that stay, a ring of stages of
// a few tokens in shared memory, filled and emptied by bulk copies of a warp of its own; the others
// turn a stage where it lies, and compute the next one's sines.
//
// What bounds it: HBM, each element read and written once.  268 MB of bf16, both directions' traffic
// 537 MB: 82.7 us, 6.49 TB/s of the 6.69 of a copy; one token of 32 + 32 heads: 2.7 us, a launch's latency.
#include "product_device.cuh"
#include "rotary.cuh"

namespace fa {

namespace {

constexpr uint32_t kRotThreads = 256;
constexpr uint32_t kAhead = 2;            // heads whose loads are in flight together

// V elements of T, as they lie in memory.
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
    T e[V];
};

// (16 bytes by a load that stays where it is written)
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p) {
    Pack<T, V> q;
    if constexpr (sizeof(T) * V == 16) {
        const uint4 w = ld_plain_v4(p);
        memcpy(&q, &w, 16);
    } else {
        q = *reinterpret_cast<const Pack<T, V>*>(p);
    }
    return q;
}

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }
__device__ __forceinline__ void narrow(float x, float& y) { y = x; }
__device__ __forceinline__ void narrow(float x, uint16_t& y) { y = __bfloat16_as_ushort(__float2bfloat16_rn(x)); }

__device__ __forceinline__ void sin_cos_turn(uint64_t turn, float& s, float& c) {
    // to the nearest quarter, and what is left in 2^-33 of half a turn
    const uint64_t q = turn + (1ull << 61);
    const int32_t rest = static_cast<int32_t>(static_cast<int64_t>(turn - (q >> 62 << 62)) >> 30);
    float sn, cs;
    sincospif(static_cast<float>(rest) * 0x1p-33f, &sn, &cs);
    const uint32_t quad = static_cast<uint32_t>(q >> 62);
    s = quad & 1 ? cs : sn;
    c = quad & 1 ? sn : cs;
    if (quad & 2) s = -s;
    if (quad == 1 || quad == 2) c = -c;
}

// The pairs of two vectors: (i, i) of them, or interleaved elements 2 i and 2 i + 1 of the two in a row.
template <typename T, int V, bool kInterleaved>
__device__ __forceinline__ void turn_pairs(Pack<T, V>& u, Pack<T, V>& v, const float (&cs)[V], const float (&sn)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        T& p = !kInterleaved ? u.e[i] : 2 * i < V ? u.e[2 * i % V] : v.e[2 * i % V];
        T& q = !kInterleaved ? v.e[i] : 2 * i + 1 < V ? u.e[(2 * i + 1) % V] : v.e[(2 * i + 1) % V];
        const float f = widen(p), g = widen(q);
        narrow(fmaf(f, cs[i], -(g * sn[i])), p);
        narrow(fmaf(g, cs[i], f * sn[i]), q);
    }
}

// V floats of shared memory, at a multiple of V.
template <int V>
__device__ __forceinline__ void load_table(const float* p, float (&x)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += V < 4 ? V : 4) {
        const Pack<float, (V < 4 ? V : 4)> q = *reinterpret_cast<const Pack<float, (V < 4 ? V : 4)>*>(p + i);
#pragma unroll
        for (int j = 0; j < (V < 4 ? V : 4); ++j) x[i + j] = q.e[j];
    }
}

template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kRotThreads, sizeof(T) * V == 16 ? 4 : 1) rotary_kernel(const __grid_constant__ RotaryArgs a) {
    typedef Pack<T, V> P;
    __shared__ uint64_t turns[kRotaryMaxPairs];
    const uint32_t half = a.rotary_dim / 2;
    for (uint32_t i = threadIdx.x; i < half; i += kRotThreads) turns[i] = a.turns[i];
    __syncthreads();
    wait_predecessor();
    const uint64_t at = blockIdx.x * static_cast<uint64_t>(kRotThreads) + threadIdx.x;
    const uint32_t per = a.chunks * a.slots;
    const uint64_t which = at >> 32 ? at / per : static_cast<uint32_t>(at) / per;
    if (which >= a.tokens) return;
    const uint32_t token = static_cast<uint32_t>(which), in = static_cast<uint32_t>(at - which * per);
    const uint32_t slot = in / a.chunks, chunk = in - slot * a.chunks;
    const uint32_t b = token / a.seq, s = token - b * a.seq;
    // the two vectors of this thread in a head
    const bool turn = chunk < a.turning;
    const uint32_t e0 = !turn ? a.rotary_dim + (chunk - a.turning) * 2 * V : kInterleaved ? chunk * 2 * V : chunk * V;
    const uint32_t e1 = turn && !kInterleaved ? e0 + half : e0 + V;
    const bool second = e1 < a.head_dim;
    const uint32_t heads0 = a.part[0].heads, heads = heads0 + a.part[1].heads;
    const T* x0 = static_cast<const T*>(a.part[0].x) + b * a.part[0].xb + s * a.part[0].xt;
    const T* x1 = static_cast<const T*>(a.part[1].x) + b * a.part[1].xb + s * a.part[1].xt;
    T* o0 = static_cast<T*>(a.part[0].out) + b * a.part[0].ob + s * a.part[0].ot;
    T* o1 = static_cast<T*>(a.part[1].out) + b * a.part[1].ob + s * a.part[1].ot;
    P u[kAhead], v[kAhead];
    const auto fetch = [&](uint32_t h0) {
#pragma unroll
        for (uint32_t k = 0; k < kAhead; ++k) {
            const uint32_t h = h0 + k * a.slots;
            if (h >= heads) break;
            const T* x = h < heads0 ? x0 + h * a.part[0].xh : x1 + (h - heads0) * a.part[1].xh;
            u[k] = load_pack<T, V>(x + e0);
            if (second) v[k] = load_pack<T, V>(x + e1);
        }
    };
    fetch(slot);                         // on their way while the sines are computed
    uint64_t pos;
    if (a.position) {
        const int32_t p = a.position[token];
        if (p < 0) return;               // padding: left as it is
        pos = static_cast<uint64_t>(p);
    } else {
        pos = static_cast<uint64_t>(a.first) + s;
    }
    float cs[V], sn[V];
    if (turn) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint64_t t = pos * turns[chunk * V + i];
            sin_cos_turn(a.inverse ? 0 - t : t, sn[i], cs[i]);
            sn[i] *= a.scale;
            cs[i] *= a.scale;
        }
    }
    for (uint32_t h0 = slot;;) {
#pragma unroll
        for (uint32_t k = 0; k < kAhead; ++k) {
            const uint32_t h = h0 + k * a.slots;
            if (h >= heads) break;
            T* o = h < heads0 ? o0 + h * a.part[0].oh : o1 + (h - heads0) * a.part[1].oh;
            if (turn) turn_pairs<T, V, kInterleaved>(u[k], v[k], cs, sn);
            *reinterpret_cast<P*>(o + e0) = u[k];
            if (second) *reinterpret_cast<P*>(o + e1) = v[k];
        }
        h0 += kAhead * a.slots;
        if (h0 >= heads) return;
        fetch(h0);
    }
}

// ----------------------------------------------------------------- ring
// The stage, slots and CTAs that were fastest of those that were tried: 268 MB of bf16 (32 + 32 heads of
// 128) in 82.7 us, 6.49 TB/s; six slots of 16 KB 85.0, three CTAs of four such 92.8, one CTA of three
// slots of 64 KB 83.8.
constexpr uint32_t kRingStage = 32768, kRingSlots = 3, kRingTokens = 8, kRingCtas = 2;
constexpr uint32_t kRingMost = kRingSlots * kRingStage + 2 * kRingTokens * 2 * kRotaryMaxPairs * 4;    // shared memory

// The computing warps of a CTA; whether all of their threads say so.
__device__ __forceinline__ bool sync_and(bool ok) {
    uint32_t all;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.and.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
        : "=r"(all)
        : "r"(static_cast<uint32_t>(ok)), "n"(kRotThreads)
        : "memory");
    return all;
}

template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kRotThreads + 32, kRingCtas) rotary_ring_kernel(const __grid_constant__ RotaryArgs a) {
    typedef Pack<T, V> P;
    extern __shared__ __align__(128) uint8_t dyn[];      // stages, then [2][tokens][cos, sin][rotary_dim / 2]
    __shared__ uint64_t bars[2 * kRingSlots];
    __shared__ uint32_t live[kRingSlots];                 // of a stage's tokens, a bit each: the fetching thread's own
    float* table = reinterpret_cast<float*>(dyn + kRingSlots * kRingStage);
    const uint32_t full = smem_addr(bars), done = full + 8 * kRingSlots;
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < kRingSlots; ++s) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(full + 8 * s) : "memory");
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(done + 8 * s), "r"(kRotThreads / 32) : "memory");
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    wait_predecessor();
    const uint32_t per = a.cta_tokens, stages = (a.tokens + per - 1) / per;
    const uint32_t n = blockIdx.x < stages ? (stages - blockIdx.x - 1) / gridDim.x + 1 : 0;
    const uint32_t half = a.rotary_dim / 2, heads = a.part[0].heads + a.part[1].heads;
    const uint32_t bytes0 = a.part[0].heads * a.head_dim * sizeof(T), bytes1 = a.part[1].heads * a.head_dim * sizeof(T);
    const auto token0_of = [&](uint32_t i) { return (blockIdx.x + i * gridDim.x) * per; };
    const auto tokens_of = [&](uint32_t i) { return min(per, a.tokens - token0_of(i)); };

    if (threadIdx.x >= kRotThreads) {
        if (threadIdx.x > kRotThreads) return;
        const auto fetch = [&](uint32_t i) {
            const uint32_t s = i % kRingSlots, tokens = tokens_of(i);
            uint32_t mask = 0;
            mbar_expect(full + 8 * s, tokens * (bytes0 + bytes1));
            for (uint32_t t = 0; t < tokens; ++t) {
                const uint32_t token = token0_of(i) + t, b = token / a.seq, at = token - b * a.seq;
                uint8_t* to = dyn + s * kRingStage + t * (bytes0 + bytes1);
                if (bytes0) bulk_load(to, static_cast<const T*>(a.part[0].x) + b * a.part[0].xb + at * a.part[0].xt, bytes0, full + 8 * s);
                if (bytes1)
                    bulk_load(to + bytes0, static_cast<const T*>(a.part[1].x) + b * a.part[1].xb + at * a.part[1].xt, bytes1, full + 8 * s);
                mask |= (!a.position || a.position[token] >= 0 ? 1u : 0u) << t;
            }
            live[s] = mask;
        };
        for (uint32_t i = 0; i < min(n, kRingSlots); ++i) fetch(i);
        bool ok = true;
        uint32_t i = 0;
        for (; i < n; ++i) {
            const uint32_t s = i % kRingSlots, tokens = tokens_of(i);
            if (!mbar_wait(done + 8 * s, (i / kRingSlots) & 1)) {
                ok = false;
                break;
            }
            for (uint32_t t = 0; t < tokens; ++t) {
                if (!(live[s] >> t & 1)) continue;                // padding: left as it is
                const uint32_t token = token0_of(i) + t, b = token / a.seq, at = token - b * a.seq;
                const uint8_t* from = dyn + s * kRingStage + t * (bytes0 + bytes1);
                if (bytes0) bulk_store(static_cast<T*>(a.part[0].out) + b * a.part[0].ob + at * a.part[0].ot, from, bytes0);
                if (bytes1) bulk_store(static_cast<T*>(a.part[1].out) + b * a.part[1].ob + at * a.part[1].ot, from + bytes0, bytes1);
            }
            bulk_commit();
            if (i >= 1 && i - 1 + kRingSlots < n) {
                asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");     // the stage before has left
                fetch(i - 1 + kRingSlots);
            }
        }
        if (!ok) {
            atomicOr(a.err, kErrWaitTimeout);
            // the loads in flight land before the CTA leaves
            const uint32_t fetched = min(n, i < 1 ? kRingSlots : i - 1 + kRingSlots);
            for (; i < fetched; ++i) mbar_wait(full + 8 * (i % kRingSlots), (i / kRingSlots) & 1);
        }
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        return;
    }

    const uint32_t tall = kRotThreads / a.turning, chunk = threadIdx.x % a.turning, row0 = threadIdx.x / a.turning;
    const uint32_t e0 = kInterleaved ? chunk * 2 * V : chunk * V, e1 = kInterleaved ? e0 + V : e0 + half;
    const auto sines = [&](uint32_t i) {
        float* to = table + (i & 1) * per * a.rotary_dim;
        const uint32_t tokens = tokens_of(i);
        for (uint32_t j = threadIdx.x; j < tokens * half; j += kRotThreads) {
            const uint32_t t = j / half, pair = j - t * half, token = token0_of(i) + t;
            const uint64_t pos = a.position ? static_cast<uint64_t>(static_cast<int64_t>(a.position[token]))
                                            : static_cast<uint64_t>(a.first) + token % a.seq;
            float s, c;
            const uint64_t angle = pos * a.turns[pair];
            sin_cos_turn(a.inverse ? 0 - angle : angle, s, c);
            to[2 * t * half + pair] = c * a.scale;
            to[(2 * t + 1) * half + pair] = s * a.scale;
        }
    };
    if (n) sines(0);
    bool ok = sync_and(true);
    for (uint32_t i = 0; ok && i < n; ++i) {
        const uint32_t s = i % kRingSlots;
        ok = mbar_wait(full + 8 * s, (i / kRingSlots) & 1);
        if (ok && row0 < tall) {
            const float* of = table + (i & 1) * per * a.rotary_dim + chunk * V;
            const uint32_t rows = tokens_of(i) * heads;
            T* at = reinterpret_cast<T*>(dyn + s * kRingStage);
            uint32_t t = row0 / heads, next = (t + 1) * heads;
#pragma unroll 2
            for (uint32_t row = row0; row < rows; row += tall) {
                while (row >= next) {
                    ++t;
                    next += heads;
                }
                T* x = at + row * a.head_dim;
                P u = *reinterpret_cast<const P*>(x + e0), v = *reinterpret_cast<const P*>(x + e1);
                float cs[V], sn[V];
                load_table(of + 2 * t * half, cs);
                load_table(of + (2 * t + 1) * half, sn);
                turn_pairs<T, V, kInterleaved>(u, v, cs, sn);
                *reinterpret_cast<P*>(x + e0) = u;
                *reinterpret_cast<P*>(x + e1) = v;
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (threadIdx.x % 32 == 0) mbar_arrive(done + 8 * s);
        if (i + 1 < n) sines(i + 1);
        ok = sync_and(ok);
    }
    if (!ok && threadIdx.x == 0) atomicOr(a.err, kErrWaitTimeout);
}

// Whether the ring takes the call; sets cta_tokens.  A token's heads lie side by side in runs of 16-byte
// pieces, and:
// - 16-bit elements.  4 MB to 384 MB of fp32 took the same time to 3 % in both forms (128 MB: 42.1 and
//   42.3 us), but those that the L2 holds (64 MB: 22.4 against 20.6).  Half as many bytes an element are
//   twice as many instructions a byte, where bulk copies save most (256 MB: 84 against 108 to 115).
// - 4 KB a token or more, so that its sines are few beside its elements.  Of 16 MB of bf16, heads of 128,
//   2 + 8 heads took 13.6 us here and 15.7 by the other form, 24 MB 20.0 and 17.1; 16 + 4 heads 9.0 and
//   15.3; a single head 78 and 15.
// - a stage for each SM.  16 + 4 to 32 + 32 heads, 4 MB (about 130 stages): 4.8 to 6.3 us against 5.4 to
//   5.6; 6 MB: 5.2 to 6.6 against 7.3 to 7.7.
bool ring_suits(RotaryArgs& a, uint32_t size, uint32_t sms) {
    uint64_t row = 0;
    for (const RotaryPart& p : a.part) {
        if (!p.heads) continue;
        const uint64_t bytes = static_cast<uint64_t>(p.heads) * a.head_dim * size;
        const bool dense = p.heads == 1 || (p.xh == a.head_dim && p.oh == a.head_dim);
        const auto whole = [&](uint64_t elements) { return elements * size % 16 == 0; };
        if (!dense || bytes % 16 || !whole(p.xb) || !whole(p.xt) || !whole(p.ob) || !whole(p.ot) ||
            reinterpret_cast<uintptr_t>(p.x) % 16 || reinterpret_cast<uintptr_t>(p.out) % 16)
            return false;
        row += bytes;
    }
    if (row < kRingStage / kRingTokens || row > kRingStage) return false;
    a.cta_tokens = static_cast<uint32_t>(kRingStage / row);
    return a.tokens / a.cta_tokens >= sms;
}

template <int V>
cudaError_t launch_ring(const RotaryArgs& a, uint32_t sms, cudaStream_t stream) {
    const auto kernel = a.interleaved ? rotary_ring_kernel<uint16_t, V, true> : rotary_ring_kernel<uint16_t, V, false>;
    const uint32_t smem = kRingSlots * kRingStage + 2 * a.cta_tokens * a.rotary_dim * 4;
    const cudaError_t e = allow_shared(reinterpret_cast<const void*>(kernel), kRingMost);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(std::min((a.tokens + a.cta_tokens - 1) / a.cta_tokens, kRingCtas * sms));
    cfg.blockDim = dim3(kRotThreads + 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T, int V>
cudaError_t launch_v(RotaryArgs& a, uint32_t sms, cudaStream_t stream) {
    a.turning = a.rotary_dim / 2 / V;
    if constexpr (sizeof(T) == 2)
        if (ring_suits(a, sizeof(T), sms)) return launch_ring<V>(a, sms, stream);
    a.chunks = a.turning + (a.copy ? (a.head_dim - a.rotary_dim + 2 * V - 1) / (2 * V) : 0);
    // Eight heads a thread where that leaves the SMs full (1536 threads each, twice over), else
    // fewer, down to one.
    const uint32_t heads = a.part[0].heads + a.part[1].heads;
    const uint64_t each = static_cast<uint64_t>(a.tokens) * a.chunks, want = 2ull * 1536 * sms;
    uint64_t slots = std::max<uint64_t>((heads + 7) / 8, (want + each - 1) / each);
    a.slots = static_cast<uint32_t>(std::min<uint64_t>(slots, heads));
    const uint64_t blocks = (each * a.slots + kRotThreads - 1) / kRotThreads;
    if (blocks >= 1ull << 31) return cudaErrorInvalidValue;
    return launch_next(a.interleaved ? rotary_kernel<T, V, true> : rotary_kernel<T, V, false>,
                       dim3(static_cast<uint32_t>(blocks)), kRotThreads, stream, a);
}

}  // namespace

cudaError_t launch_rotary(RotaryArgs& a, uint32_t sms, cudaStream_t stream) {
    // the longest vectors that every address of the call is aligned for
    const uint32_t size = a.dtype ? 2 : 4;
    const auto fits = [&](uint32_t v) {
        bool ok = a.rotary_dim / 2 % v == 0 && a.head_dim % v == 0;
        for (const RotaryPart& p : a.part)
            if (p.heads)
                ok = ok && reinterpret_cast<uintptr_t>(p.x) % (v * size) == 0 && reinterpret_cast<uintptr_t>(p.out) % (v * size) == 0 &&
                     p.xb % v == 0 && p.xt % v == 0 && p.xh % v == 0 && p.ob % v == 0 && p.ot % v == 0 && p.oh % v == 0;
        return ok;
    };
    if (a.dtype) {
        if (fits(8)) return launch_v<uint16_t, 8>(a, sms, stream);
        if (fits(4)) return launch_v<uint16_t, 4>(a, sms, stream);
        if (fits(2)) return launch_v<uint16_t, 2>(a, sms, stream);
        return launch_v<uint16_t, 1>(a, sms, stream);
    }
    if (fits(4)) return launch_v<float, 4>(a, sms, stream);
    if (fits(2)) return launch_v<float, 2>(a, sms, stream);
    return launch_v<float, 1>(a, sms, stream);
}

}  // namespace fa
