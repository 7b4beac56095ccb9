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
constexpr uint32_t kAhead = 2;            // heads whose loads a thread has in flight

// V elements of T, as they lie in memory.
template <typename T, int V>
struct alignas(sizeof(T) * V < 16 ? sizeof(T) * V : 16) Pack {
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

// V floats of shared memory, at a multiple of V.
template <int V>
__device__ __forceinline__ void load_table(const float* p, float (&x)[V]) {
    const Pack<float, V> q = *reinterpret_cast<const Pack<float, V>*>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = q.e[i];
}

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
    __shared__ uint64_t at_in[kRotTokens][2], at_out[kRotTokens][2];
    __shared__ int64_t position[kRotTokens];             // -1: padding, left as it is
    wait_predecessor();
    const uint32_t half = a.rotary_dim / 2;
    const uint32_t token0 = blockIdx.x * a.cta_tokens, tokens = min(a.cta_tokens, a.tokens - token0);
    const uint32_t heads0 = a.part[0].heads, heads = heads0 + a.part[1].heads;
    const uint32_t head0 = blockIdx.y * a.cta_heads, mine = min(a.cta_heads, heads - head0);
    if (threadIdx.x < tokens) {
        const uint32_t t = threadIdx.x, b = (token0 + t) / a.seq, s = token0 + t - b * a.seq;
        const int32_t p = a.position ? a.position[token0 + t] : 0;
        position[t] = a.position ? (p < 0 ? -1 : p) : a.first + s;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            at_in[t][k] = b * a.part[k].xb + s * a.part[k].xt;
            at_out[t][k] = b * a.part[k].ob + s * a.part[k].ot;
        }
    }
    __syncthreads();

    // This thread's place in a head, its two vectors there, and the row (token, head) it begins with;
    // the CTA has `tall` rows at a time.
    const uint32_t chunk0 = blockIdx.z * kRotThreads, width = min(a.chunks - chunk0, kRotThreads), tall = kRotThreads / width;
    const uint32_t chunk = chunk0 + threadIdx.x % width, row0 = threadIdx.x / width;
    const bool turn = chunk < a.turning;
    const uint32_t e0 = !turn ? a.rotary_dim + (chunk - a.turning) * 2 * V : kInterleaved ? chunk * 2 * V : chunk * V;
    const uint32_t e1 = turn && !kInterleaved ? e0 + half : e0 + V;
    const bool second = e1 < a.head_dim;
    struct Row {
        uint32_t t, h;                       // of the CTA's tokens and heads
    };
    const auto on = [&](Row r) {             // tall rows on
        r.h += tall;
        while (r.h >= mine) {
            r.h -= mine;
            ++r.t;
        }
        return r;
    };
    Row row = {0, row0};
    while (row.h >= mine) {
        row.h -= mine;
        ++row.t;
    }
    if (row0 >= tall) row.t = tokens;
    P u[kAhead], v[kAhead];
    const auto fetch = [&](Row r) {
#pragma unroll
        for (uint32_t i = 0; i < kAhead; ++i, r = on(r)) {
            if (r.t >= tokens) break;
            const bool k = head0 + r.h >= heads0;
            const T* x = static_cast<const T*>(a.part[k].x) + at_in[r.t][k] + (head0 + r.h - (k ? heads0 : 0)) * a.part[k].xh;
            u[i] = load_pack<T, V>(x + e0);
            if (second) v[i] = load_pack<T, V>(x + e1);
        }
    };
    fetch(row);
    for (uint32_t t = 0; t < tokens; ++t)
        for (uint32_t pair = threadIdx.x; pair < half; pair += kRotThreads) {
            const uint64_t angle = static_cast<uint64_t>(position[t]) * a.turns[pair];
            const float2 cs = cos_sin_turn(a.inverse ? 0 - angle : angle);
            table[2 * t * half + pair] = cs.x * a.scale;
            table[(2 * t + 1) * half + pair] = cs.y * a.scale;
        }
    __syncthreads();
    while (row.t < tokens) {
#pragma unroll
        for (uint32_t i = 0; i < kAhead; ++i, row = on(row)) {
            if (row.t >= tokens) return;
            if (position[row.t] < 0) continue;
            const bool k = head0 + row.h >= heads0;
            T* o = static_cast<T*>(a.part[k].out) + at_out[row.t][k] + (head0 + row.h - (k ? heads0 : 0)) * a.part[k].oh;
            if (turn) {
                float cs[V], sn[V];
                load_table(table + 2 * row.t * half + chunk * V, cs);
                load_table(table + (2 * row.t + 1) * half + chunk * V, sn);
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks, (heads + a.cta_heads - 1) / a.cta_heads, (a.chunks + kRotThreads - 1) / kRotThreads);
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
