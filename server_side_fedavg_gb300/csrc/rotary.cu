// Rotary positions of queries and keys.
//
//   (u, v) -> scale * (u cos t - v sin t, v cos t + u sin t),   t = position * frequency of the pair
//
// The gradient is the same map with -t.  A position is an integer and a frequency is held as a
// whole number of 2^-64 turns, so that their product modulo 2^64 is the angle modulo a turn,
// exactly: no table of cosines is read, and a far position is as exact as a near one.  The
// quadrant is taken off in integers too; the rest, |t| <= pi / 4, goes through sincospif.
//
// A CTA has a few tokens, or for a few tokens some of their heads.  Its threads compute the sines of
// the tokens' pairs into shared memory, each once, while their first vectors are on their way;
// then each takes the vectors of one place in the heads, all heads and tokens in turn.
//
// What bounds it: HBM, each element read and written once.
#include "product_device.cuh"
#include "rotary.cuh"

namespace fa {

namespace {

constexpr uint32_t kRotThreads = 256;
constexpr uint32_t kRotTokens = 4;        // of a CTA
constexpr uint32_t kAhead = 4;            // heads whose loads a thread has in flight

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

__device__ __forceinline__ float2 cos_sin_turn(uint64_t turn) {
    // to the nearest quarter, and what is left in 2^-33 of half a turn
    const uint64_t q = turn + (1ull << 61);
    const int32_t rest = static_cast<int32_t>(static_cast<int64_t>(turn - (q >> 62 << 62)) >> 30);
    float sn, cs;
    sincospif(static_cast<float>(rest) * 0x1p-33f, &sn, &cs);
    const uint32_t quad = static_cast<uint32_t>(q >> 62);
    const float c = quad & 1 ? sn : cs, s = quad & 1 ? cs : sn;
    return make_float2(quad == 1 || quad == 2 ? -c : c, quad & 2 ? -s : s);
}

template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kRotThreads, 4) rotary_kernel(const __grid_constant__ RotaryArgs a) {
    typedef Pack<T, V> P;
    extern __shared__ __align__(16) float table[];      // [tokens][cos, sin][rotary_dim / 2]
    __shared__ int live[kRotTokens];
    wait_predecessor();
    const uint32_t half = a.rotary_dim / 2;
    const uint32_t token0 = blockIdx.x * a.cta_tokens, tokens = min(a.cta_tokens, a.tokens - token0);
    const uint32_t heads0 = a.part[0].heads, heads = heads0 + a.part[1].heads;
    const uint32_t head0 = blockIdx.y * a.cta_heads, mine = min(a.cta_heads, heads - head0);

    // This thread's place in a head, its two vectors there, and the row (token, head) it begins with;
    // the CTA has `tall` rows at a time.
    const uint32_t tall = kRotThreads / a.chunks, chunk = threadIdx.x % a.chunks, row0 = threadIdx.x / a.chunks;
    const bool on = row0 < tall, turn = chunk < a.turning;
    const uint32_t e0 = !turn ? a.rotary_dim + (chunk - a.turning) * 2 * V : kInterleaved ? chunk * 2 * V : chunk * V;
    const uint32_t e1 = turn && !kInterleaved ? e0 + half : e0 + V;
    const bool second = e1 < a.head_dim;
    const uint32_t rows = tokens * mine;
    P u[kAhead], v[kAhead];
    const auto place = [&](uint32_t row, uint32_t& t, bool out) {
        t = row / mine;
        const uint32_t h = head0 + row - t * mine, token = token0 + t, b = token / a.seq, s = token - b * a.seq;
        const bool k = h >= heads0;
        const RotaryPart& p = a.part[k];
        return out ? b * p.ob + s * p.ot + (k ? h - heads0 : h) * p.oh : b * p.xb + s * p.xt + (k ? h - heads0 : h) * p.xh;
    };
    const auto is_k = [&](uint32_t row) { return head0 + row % mine >= heads0; };
    const auto fetch = [&](uint32_t row) {
#pragma unroll
        for (uint32_t i = 0; i < kAhead; ++i) {
            if (row + i * tall >= rows) break;
            uint32_t t;
            const uint64_t at = place(row + i * tall, t, false);
            const T* x = static_cast<const T*>(a.part[is_k(row + i * tall)].x) + at;
            u[i] = load_pack<T, V>(x + e0);
            if (second) v[i] = load_pack<T, V>(x + e1);
        }
    };
    if (on) fetch(row0);
    for (uint32_t i = threadIdx.x; i < tokens * half; i += kRotThreads) {
        const uint32_t t = i / half, pair = i - t * half, token = token0 + t;
        uint64_t pos;
        if (a.position) {
            const int32_t p = a.position[token];
            if (pair == 0) live[t] = p >= 0;             // negative: padding, left as it is
            pos = static_cast<uint64_t>(static_cast<int64_t>(p));
        } else {
            if (pair == 0) live[t] = 1;
            pos = static_cast<uint64_t>(a.first) + token % a.seq;
        }
        const uint64_t angle = pos * a.turns[pair];
        const float2 cs = cos_sin_turn(a.inverse ? 0 - angle : angle);
        table[2 * t * half + pair] = cs.x * a.scale;
        table[(2 * t + 1) * half + pair] = cs.y * a.scale;
    }
    __syncthreads();
    if (!on) return;
    for (uint32_t row = row0;;) {
#pragma unroll
        for (uint32_t i = 0; i < kAhead; ++i) {
            if (row + i * tall >= rows) break;
            uint32_t t;
            const uint64_t at = place(row + i * tall, t, true);
            if (!live[t]) continue;
            T* o = static_cast<T*>(a.part[is_k(row + i * tall)].out) + at;
            if (turn) {
                const float *cs = table + 2 * t * half + chunk * V, *sn = cs + half;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    // interleaved: pair j is elements 2 j and 2 j + 1 of the two vectors in a row
                    T& p = !kInterleaved ? u[i].e[j] : 2 * j < V ? u[i].e[2 * j % V] : v[i].e[2 * j % V];
                    T& q = !kInterleaved ? v[i].e[j] : 2 * j + 1 < V ? u[i].e[(2 * j + 1) % V] : v[i].e[(2 * j + 1) % V];
                    const float f = widen(p), g = widen(q);
                    narrow(fmaf(f, cs[j], -(g * sn[j])), p);
                    narrow(fmaf(g, cs[j], f * sn[j]), q);
                }
            }
            *reinterpret_cast<P*>(o + e0) = u[i];
            if (second) *reinterpret_cast<P*>(o + e1) = v[i];
        }
        row += kAhead * tall;
        if (row >= rows) return;
        fetch(row);
    }
}

template <typename T, int V>
cudaError_t launch_v(RotaryArgs& a, uint32_t sms, cudaStream_t stream) {
    a.turning = a.rotary_dim / 2 / V;
    a.chunks = a.turning + (a.copy ? (a.head_dim - a.rotary_dim + 2 * V - 1) / (2 * V) : 0);
    // kRotTokens tokens a CTA where that leaves eight CTAs per SM, else fewer; for fewer tokens than
    // twice the SMs the heads are shared out too.
    const uint32_t heads = a.part[0].heads + a.part[1].heads;
    a.cta_tokens = std::max(1u, std::min(kRotTokens, a.tokens / (8 * sms)));
    const uint32_t blocks = (a.tokens + a.cta_tokens - 1) / a.cta_tokens, share = std::min(heads, std::max(1u, 2 * sms / blocks));
    a.cta_heads = (heads + share - 1) / share;
    if (a.chunks > kRotThreads) return launch_rotary_wide(a, stream);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks, (heads + a.cta_heads - 1) / a.cta_heads);
    cfg.blockDim = dim3(kRotThreads);
    cfg.dynamicSmemBytes = a.cta_tokens * a.rotary_dim * 4;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, a.interleaved ? rotary_kernel<T, V, true> : rotary_kernel<T, V, false>, a);
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
