// Rotary positions of queries and keys.
//
//   (u, v) -> scale * (u cos t - v sin t, v cos t + u sin t),   t = position * frequency of the pair
//
// The gradient is the same map with -t.  A position is an integer and a frequency is held as a
// whole number of 2^-64 turns, so that their product modulo 2^64 is the angle modulo a turn,
// exactly: no table of cosines is read, and a far position is as exact as a near one.  The
// quadrant is taken off in integers too; the rest, |t| <= pi / 4, goes through sincospif.
//
// A thread has V pairs (its vectors are V elements) and turns them in several heads of one token,
// so that the sines are computed once for all of these.  What bounds it: HBM, each element read
// and written once.
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
            if (turn) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    // interleaved: pair i is elements 2 i and 2 i + 1 of the two vectors in a row
                    T& p = !kInterleaved ? u[k].e[i] : 2 * i < V ? u[k].e[2 * i % V] : v[k].e[2 * i % V];
                    T& q = !kInterleaved ? v[k].e[i] : 2 * i + 1 < V ? u[k].e[(2 * i + 1) % V] : v[k].e[(2 * i + 1) % V];
                    const float f = widen(p), g = widen(q);
                    narrow(fmaf(f, cs[i], -(g * sn[i])), p);
                    narrow(fmaf(g, cs[i], f * sn[i]), q);
                }
            }
            *reinterpret_cast<P*>(o + e0) = u[k];
            if (second) *reinterpret_cast<P*>(o + e1) = v[k];
        }
        h0 += kAhead * a.slots;
        if (h0 >= heads) return;
        fetch(h0);
    }
}

template <typename T, int V>
cudaError_t launch_v(RotaryArgs& a, uint32_t sms, cudaStream_t stream) {
    a.turning = a.rotary_dim / 2 / V;
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
