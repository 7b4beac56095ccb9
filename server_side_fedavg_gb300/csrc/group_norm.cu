// Group norm with an activation, channels last, and its gradients.
//
//   xhat = (x - mean) * rstd,  z = xhat * gamma + beta,  y = act(z)
//   dz = dout * act'(z),  d_beta = sum dz,  d_gamma = sum dz xhat
//   dx = rstd * (gamma dz - mean_g(gamma dz) - xhat * mean_g(gamma dz xhat))
//
// mean and rstd are over a sample's positions and a group's channels, mean_g likewise.
//
// Two passes over the data: the statistics, then the result.  A thread keeps V channels (one
// vector) and walks down positions, so that nothing of a channel is fetched twice; a CTA has a
// run of a sample's positions.  The second pass walks its run backwards: what the first pass read
// last is still in L2.  A thread's sums are taken of x less a reference that follows the mean (see
// Moments).  Threads, a run's channels, and then the runs, are joined in a fixed order as means and sums of
// squares about them, by their differences from a point near the common mean: for threads that mean
// itself, for channels the mean of up to 32, for runs the first one's.  (The mean of 1 / k of the positions
// is within k^(1/2) spreads of the whole's: such a point costs roundings of that size, nothing squared.)
// So neither an offset far larger than the spread nor positions unlike the others cost digits, and the
// kept mean is off by its own rounding.
//
// What bounds it: small samples, the launches (4 x 9216 x 64 fp32 11.7 us, 1 x 216 x 256 6.8); large ones
// that the one kernel does not take, HBM, x read twice and the result written once: 2 x 128^3 x 32 bf16 in
// rows of 40 elements 278 us, 3.4 TB/s of whole lines, gradients of 2 x 96^3 in such rows 182.
#include <algorithm>

#include "group_norm_device.cuh"

namespace fa {

namespace {

constexpr uint32_t kNormThreads = 256, kNormWarps = kNormThreads / 32;
constexpr uint32_t kNormCtas = 4, kNormGradCtas = 2;                     // per SM
constexpr uint32_t kNormMost = 16 * kNormMaxChannels + 2 * 8 * kNormThreads * 4;   // bytes of shared memory

// A CTA's columns in turn: `width` vectors by `tall` positions at a time.
struct Tile {
    uint32_t width, tall, col, row;
    bool on;
    __device__ __forceinline__ Tile(uint32_t vectors, uint32_t c0)
        : width(min(vectors - c0, kNormThreads)), tall(kNormThreads / width), col(threadIdx.x % width),
          row(threadIdx.x / width), on(row < tall) {}
};

// Lanes for each of a warp's sums of n terms: a power of two.
__device__ __forceinline__ uint32_t lanes_for(uint32_t n) { return n >= 32 ? 32 : n <= 1 ? 1 : 2u << (31 - __clz(n - 1)); }

// Sums over a tile's positions: s[i][j] of every thread of a column end up in its first one.
template <int N, int V>
__device__ __forceinline__ void sum_rows(float (&s)[N][V], float* red, const Tile& t) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) red[(i * V + j) * kNormThreads + threadIdx.x] = s[i][j];
    __syncthreads();
    for (uint32_t left = t.tall; left > 1;) {
        const uint32_t half = (left + 1) / 2;
        if (t.row < left - half)
#pragma unroll
            for (int k = 0; k < N * V; ++k) {
                s[k / V][k % V] += red[k * kNormThreads + threadIdx.x + half * t.width];
                red[k * kNormThreads + threadIdx.x] = s[k / V][k % V];
            }
        left = half;
        __syncthreads();
    }
}

template <typename T>
__device__ __forceinline__ const T* at(const NormTensor& t, uint32_t sample) {
    return static_cast<const T*>(t.p) + sample * t.step;
}

// How many positions of [r0, r1) are this thread's.
__device__ __forceinline__ uint32_t rows_mine(const Tile& t, uint32_t r0, uint32_t r1) {
    return t.on && r0 + t.row < r1 ? (r1 - r0 - t.row + t.tall - 1) / t.tall : 0;
}

// f(vector of p0, vector of p1, position) for this thread's positions `from` to `to` of [r0, r1), channels
// from c.
template <typename T, int V>
constexpr uint32_t kAtOnce = sizeof(T) * V >= 16 ? 4 : 8;    // 64 bytes of a stream in flight, no more than eight positions
template <bool kReverse, int kStreams, int V, typename T, typename F>
__device__ __forceinline__ void over_rows(const Tile& t, const T* p0, uint64_t ld0, const T* p1, uint64_t ld1, uint32_t r0,
                                          uint32_t r1, uint32_t c, F f, uint32_t from = 0, uint32_t to = ~0u) {
    if (!t.on) return;
    constexpr uint32_t kU = kAtOnce<T, V>;
    const uint32_t mine = rows_mine(t, r0, r1), end = min(mine, to);
    const auto row_of = [&](uint32_t i) { return r0 + t.row + (kReverse ? mine - 1 - i : i) * t.tall; };
    uint32_t i = from;
    for (; i + kU <= end; i += kU) {
        Vec<T, V> q[kU], p[kU];
#pragma unroll
        for (uint32_t u = 0; u < kU; ++u) {
            q[u] = load_raw<T, V>(p0 + row_of(i + u) * ld0 + c);
            p[u] = kStreams == 2 ? load_raw<T, V>(p1 + row_of(i + u) * ld1 + c) : q[u];
        }
#pragma unroll
        for (uint32_t u = 0; u < kU; ++u) f(q[u], p[u], row_of(i + u));
    }
    for (; i < end; ++i) {
        const Vec<T, V> q = load_raw<T, V>(p0 + row_of(i) * ld0 + c);
        f(q, kStreams == 2 ? load_raw<T, V>(p1 + row_of(i) * ld1 + c) : q, row_of(i));
    }
}

// ----------------------------------------------------------------- forward
// stat[sample][group][chunk] = (mean, as a sum of two; sum of squares about it) over the chunk's positions.
template <typename T, int V>
__global__ void __launch_bounds__(kNormThreads, kNormCtas) norm_stat_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ float sm[];
    float *mean = sm, *sq = mean + a.channels, *base = sq + a.channels, *red = base + a.channels;
    wait_predecessor();
    const uint32_t vectors = a.channels / V, per = a.channels / a.groups, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t r0 = blockIdx.x * a.rows, r1 = min(a.positions, r0 + a.rows);
    const float count = static_cast<float>(r1 - r0), inv = 1.0f / count, inv_per = 1.0f / static_cast<float>(per);
    for (uint32_t sample = a.first + blockIdx.y; sample < a.last; sample += gridDim.y) {
        const T* x = at<T>(a.x, sample);
        for (uint32_t c0 = 0; c0 < vectors; c0 += kNormThreads) {
            const Tile t(vectors, c0);
            const uint32_t c = (c0 + t.col) * V;
            Moments<V> o;
            const uint32_t mine = rows_mine(t, r0, r1);
            {
                // (where a thread has no position, the last one's: it then weighs nothing)
                float from[V];
                widen(load_raw<T, V>(x + min(r0 + t.row, r1 - 1) * a.x.ld + c), from);
                o.begin(from);
            }
            for (uint32_t i = 0, end = kAtOnce<T, V>;; i = end, end *= kGrow) {
                over_rows<false, 1, V>(
                    t, x, a.x.ld, x, a.x.ld, r0, r1, c,
                    [&](const Vec<T, V>& q, const Vec<T, V>&, uint32_t) {
                        float d[V];
                        widen(q, d);
                        o.step(d);
                    },
                    i, end);
                if (end >= mine) break;
                o.move(static_cast<float>(end));
            }
            // the threads' common mean, then their sums about it
            const float n = static_cast<float>(mine);
            float m[1][V];
            o.mean_part(n, count, m[0]);
            sum_rows<1, V>(m, red, t);
            if (t.row == 0)
#pragma unroll
                for (int i = 0; i < V; ++i) base[c + i] = m[0][i];
            __syncthreads();
            if (t.on) o.about(n, base + c);
            sum_rows<2, V>(o.s, red, t);
            if (t.row == 0)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = o.s[0][i] * inv;
                    mean[c + i] = d;
                    sq[c + i] = fmaxf(fmaf(-o.s[0][i], d, o.s[1][i]), 0.0f);
                }
            __syncthreads();
        }
        // a group per `lanes` lanes
        const uint32_t lanes = lanes_for(per), sub = lane % lanes;
        for (uint32_t g0 = warp * (32 / lanes); g0 < a.groups; g0 += kNormWarps * (32 / lanes)) {
            const uint32_t g = g0 + lane / lanes, end = g < a.groups ? (g + 1) * per : 0;
            // a point near the group's mean: that of its first channels, one a lane
            float hi = g * per + sub < end ? base[g * per + sub] + mean[g * per + sub] : 0.0f, m = 0.0f, q = 0.0f;
            hi = lane_sum(hi * (1.0f / static_cast<float>(min(lanes, per))), lanes);
            for (uint32_t c = g * per + sub; c < end; c += lanes) {
                mean[c] += base[c] - hi;
                m += mean[c];
            }
            m = lane_sum(m, lanes) * inv_per;
            for (uint32_t c = g * per + sub; c < end; c += lanes) {
                const float d = mean[c] - m;
                q += fmaf(count * d, d, sq[c]);
            }
            q = lane_sum(q, lanes);
            if (sub == 0 && g < a.groups)
                a.stat[(static_cast<uint64_t>(sample) * a.groups + g) * a.chunks + blockIdx.x] = make_float4(hi, m, q, 0.0f);
        }
        __syncthreads();
    }
}

// A sample's mean, what its rounding to fp32 left, and 1 / sqrt(variance + eps) per group, from its chunks'
// parts, into shared memory.
__device__ __forceinline__ void join_chunks(const NormArgs& a, uint32_t sample, float* mean, float* left, float* rstd) {
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, per = a.channels / a.groups;
    const uint32_t lanes = lanes_for(a.chunks), sub = lane % lanes;
    const float all = static_cast<float>(a.positions);
    const auto rows_of = [&](uint32_t i) { return static_cast<float>(min(a.rows, a.positions - i * a.rows)); };
    for (uint32_t g0 = warp * (32 / lanes); g0 < a.groups; g0 += kNormWarps * (32 / lanes)) {
        const uint32_t g = g0 + lane / lanes, end = g < a.groups ? a.chunks : 0;
        const float4* part = a.stat + (static_cast<uint64_t>(sample) * a.groups + g) * a.chunks;
        float m = 0.0f, q = 0.0f, hi = 0.0f;       // hi: a point near the mean, the first chunk's
        float4 own = make_float4(0.0f, 0.0f, 0.0f, 0.0f);        // this lane's first: with few chunks its only one
        if (sub < end) own = part[sub];
        hi = __shfl_sync(~0u, own.x + own.y, lane - sub);
        const auto rest = [&](float4 p, uint32_t i, float to) { return fmaf((p.x - hi) + p.y, rows_of(i), to); };
        if (sub < end) m = rest(own, sub, 0.0f);
#pragma unroll 4
        for (uint32_t i = sub + lanes; i < end; i += lanes) m = rest(part[i], i, m);
        m = lane_sum(m, lanes) / all;
        const auto square = [&](float4 p, uint32_t i) {
            const float d = ((p.x - hi) + p.y) - m;
            return fmaf(rows_of(i) * static_cast<float>(per) * d, d, p.z);
        };
        if (sub < end) q = square(own, sub);
#pragma unroll 4
        for (uint32_t i = sub + lanes; i < end; i += lanes) q += square(part[i], i);
        q = lane_sum(q, lanes) / (all * static_cast<float>(per));
        if (sub == 0 && g < a.groups) {
            mean[g] = hi + m;
            left[g] = (hi - mean[g]) + m;
            rstd[g] = 1.0f / sqrtf(q + a.eps);
        }
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kNormThreads, kNormCtas) norm_apply_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ float sm[];
    float *mean = sm, *rstd = mean + a.groups, *left = rstd + a.groups;
    wait_predecessor();
    const uint32_t vectors = a.channels / V, per = a.channels / a.groups;
    const uint32_t r0 = blockIdx.x * a.rows, r1 = min(a.positions, r0 + a.rows);
    const int act = a.act;
    for (uint32_t sample = a.first + blockIdx.y; sample < a.last; sample += gridDim.y) {
        const uint64_t first = static_cast<uint64_t>(sample) * a.groups;
        join_chunks(a, sample, mean, left, rstd);
        __syncthreads();
        if (blockIdx.x == 0 && a.mean_out)
            for (uint32_t g = threadIdx.x; g < a.groups; g += kNormThreads) a.mean_out[first + g] = mean[g];
        if (blockIdx.x == 0 && a.rstd_out)
            for (uint32_t g = threadIdx.x; g < a.groups; g += kNormThreads) a.rstd_out[first + g] = rstd[g];
        const T* x = at<T>(a.x, sample);
        T* y = const_cast<T*>(at<T>(a.out, sample));
        for (uint32_t c0 = 0; c0 < vectors; c0 += kNormThreads) {
            const Tile t(vectors, c0);
            const uint32_t c = (c0 + t.col) * V;
            // y = act((x - mean) scale + shift): what the mean's rounding left is in the shift
            float less[V] = {}, scale[V] = {}, shift[V] = {};
            if (t.on)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const uint32_t g = (c + i) / per;
                    less[i] = -mean[g];
                    scale[i] = rstd[g] * (a.gamma ? elem(a.gamma, c + i, a.param_dtype) : 1.0f);
                    shift[i] = fmaf(-left[g], scale[i], a.beta ? elem(a.beta, c + i, a.param_dtype) : 0.0f);
                }
            over_rows<true, 1, V>(t, x, a.x.ld, x, a.x.ld, r0, r1, c, [&](const Vec<T, V>& q, const Vec<T, V>&, uint32_t r) {
                float v[V];
                widen(q, v);
                add(v, v, less);
                fma(v, v, scale, shift);
                act_of(act, v);
                store_vec<T, V>(y + r * a.out.ld + c, v);
            });
        }
        __syncthreads();
    }
}

// ----------------------------------------------------------------- backward
// part[sample][chunk][group] = sums of gamma dz and gamma dz xhat over the chunk;
// cpart[its CTA][channel] = sums of dz and dz xhat over the CTA's chunks.
template <typename T, int V>
__global__ void __launch_bounds__(kNormThreads, kNormGradCtas) norm_grad_stat_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ float sm[];
    float *s0 = sm, *s1 = s0 + a.channels, *t0 = s1 + a.channels, *t1 = t0 + a.channels,
          *red = t1 + a.channels;
    wait_predecessor();
    const uint32_t vectors = a.channels / V, per = a.channels / a.groups, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t r0 = blockIdx.x * a.rows, r1 = min(a.positions, r0 + a.rows);
    const int act = a.act;
    for (uint32_t c = threadIdx.x; c < a.channels; c += kNormThreads) t0[c] = t1[c] = 0.0f;
    __syncthreads();
    for (uint32_t sample = a.first + blockIdx.y; sample < a.last; sample += gridDim.y) {
        const T *x = at<T>(a.x, sample), *dout = at<T>(a.dout, sample);
        for (uint32_t c0 = 0; c0 < vectors; c0 += kNormThreads) {
            const Tile t(vectors, c0);
            const uint32_t c = (c0 + t.col) * V;
            float s[2][V] = {};
            const Channels<V> ch(a, sample, t.on ? c : 0);
            over_rows<false, 2, V>(t, x, a.x.ld, dout, a.dout.ld, r0, r1, c,
                                          [&](const Vec<T, V>& q, const Vec<T, V>& p, uint32_t) {
                                              float v[V], d[V];
                                              widen(q, v);
                                              widen(p, d);
                                              ch.step(act, v, d);
                                              add(s[0], s[0], d);
                                              fma(s[1], d, v, s[1]);
                                          });
            // sums of dz h so far: of dz xhat
            if (t.on)
#pragma unroll
                for (int i = 0; i < V; ++i) s[1][i] *= a.rstd[static_cast<uint64_t>(sample) * a.groups + (c + i) / per];
            sum_rows<2, V>(s, red, t);
            if (t.row == 0)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float g = a.gamma ? elem(a.gamma, c + i, a.param_dtype) : 1.0f;
                    s0[c + i] = g * s[0][i];
                    s1[c + i] = g * s[1][i];
                    t0[c + i] += s[0][i];
                    t1[c + i] += s[1][i];
                }
            __syncthreads();
        }
        const uint32_t lanes = lanes_for(per), sub = lane % lanes;
        for (uint32_t g0 = warp * (32 / lanes); g0 < a.groups; g0 += kNormWarps * (32 / lanes)) {
            const uint32_t g = g0 + lane / lanes, end = g < a.groups ? (g + 1) * per : 0;
            float p = 0.0f, q = 0.0f;
            for (uint32_t c = g * per + sub; c < end; c += lanes) {
                p += s0[c];
                q += s1[c];
            }
            p = lane_sum(p, lanes);
            q = lane_sum(q, lanes);
            if (sub == 0 && g < a.groups)
                a.part[(static_cast<uint64_t>(sample) * a.chunks + blockIdx.x) * a.groups + g] = make_float2(p, q);
        }
        __syncthreads();
    }
    if (a.cpart) {
        float2* to = a.cpart + (static_cast<uint64_t>(a.row0 + blockIdx.y) * a.chunks + blockIdx.x) * a.channels;
        for (uint32_t c = threadIdx.x; c < a.channels; c += kNormThreads) to[c] = make_float2(t0[c], t1[c]);
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kNormThreads, kNormGradCtas) norm_grad_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ float sm[];
    float *c1 = sm, *c2 = c1 + a.groups;
    wait_predecessor();
    const uint32_t vectors = a.channels / V, per = a.channels / a.groups, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t r0 = blockIdx.x * a.rows, r1 = min(a.positions, r0 + a.rows);
    const int act = a.act;
    const float inv = 1.0f / (static_cast<float>(a.positions) * static_cast<float>(per));
    for (uint32_t sample = a.first + blockIdx.y; sample < a.last; sample += gridDim.y) {
        const uint32_t lanes = lanes_for(a.chunks), sub = lane % lanes;
        for (uint32_t g0 = warp * (32 / lanes); g0 < a.groups; g0 += kNormWarps * (32 / lanes)) {
            const uint32_t g = g0 + lane / lanes, end = g < a.groups ? a.chunks : 0;
            const float2* part = a.part + static_cast<uint64_t>(sample) * a.chunks * a.groups + g;
            float p = 0.0f, q = 0.0f;
#pragma unroll 4
            for (uint32_t i = sub; i < end; i += lanes) {
                const float2 v = part[static_cast<uint64_t>(i) * a.groups];
                p += v.x;
                q += v.y;
            }
            p = lane_sum(p, lanes);
            q = lane_sum(q, lanes);
            if (sub == 0 && g < a.groups) {
                c1[g] = p * inv;
                c2[g] = q * inv;
            }
        }
        __syncthreads();
        const T *x = at<T>(a.x, sample), *dout = at<T>(a.dout, sample);
        T* dx = const_cast<T*>(at<T>(a.out, sample));
        for (uint32_t c0 = 0; c0 < vectors; c0 += kNormThreads) {
            const Tile t(vectors, c0);
            const uint32_t c = (c0 + t.col) * V;
            const Channels<V> ch(a, sample, t.on ? c : 0);
            // dx = scale dz - rstd m1 - h rstd^2 m2
            float k1[V] = {}, k2[V] = {};
            if (t.on)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const uint32_t g = (c + i) / per;
                    const float r = a.rstd[static_cast<uint64_t>(sample) * a.groups + g];
                    k1[i] = -r * c1[g];
                    k2[i] = -r * r * c2[g];
                }
            over_rows<true, 2, V>(t, x, a.x.ld, dout, a.dout.ld, r0, r1, c,
                                         [&](const Vec<T, V>& q, const Vec<T, V>& p, uint32_t r) {
                                             float v[V], d[V];
                                             widen(q, v);
                                             widen(p, d);
                                             ch.step(act, v, d);
                                             fma(v, v, k2, k1);
                                             fma(d, d, ch.scale, v);
                                             store_vec<T, V>(dx + r * a.out.ld + c, d);
                                         });
        }
        __syncthreads();
    }
}

// The parameters' gradients: columns of cpart, eight a block, summed in 128 strands of rows and these
// in order.
__global__ void __launch_bounds__(1024) norm_param_kernel(const float2* part, uint32_t rows, uint32_t channels, void* d_gamma,
                                                          void* d_beta, int dtype) {
    __shared__ float2 sums[1024];
    wait_predecessor();
    const uint32_t c = blockIdx.x * 8 + threadIdx.x % 8;
    float2 s = make_float2(0.0f, 0.0f);
    if (c < channels)
#pragma unroll 8
        for (uint32_t r = threadIdx.x / 8; r < rows; r += 128) {
            const float2 v = part[static_cast<uint64_t>(r) * channels + c];
            s.x += v.x;
            s.y += v.y;
        }
    sums[threadIdx.x] = s;
    for (uint32_t left = 512; left >= 8; left /= 2) {
        __syncthreads();
        if (threadIdx.x < left) {
            s.x += sums[threadIdx.x + left].x;
            s.y += sums[threadIdx.x + left].y;
            sums[threadIdx.x] = s;
        }
    }
    if (threadIdx.x >= 8 || c >= channels) return;
    if (d_beta) put(d_beta, c, dtype, s.x);
    if (d_gamma) put(d_gamma, c, dtype, s.y);
}

using Kernel = void (*)(NormArgs);
struct Set {
    Kernel stat, apply, grad_stat, grad;
};
template <typename T, int V>
constexpr Set set_of() {
    return {norm_stat_kernel<T, V>, norm_apply_kernel<T, V>, norm_grad_stat_kernel<T, V>, norm_grad_kernel<T, V>};
}

// The longest vectors that the channels and every address allow.
uint32_t vector_of(const NormArgs& a, bool backward) {
    const uint32_t size = a.dtype ? 2 : 4;
    const auto ok = [&](const NormTensor& t, uint32_t v) {
        return reinterpret_cast<uintptr_t>(t.p) % (v * size) == 0 && t.ld % v == 0 && (a.n == 1 || t.step % v == 0);
    };
    for (uint32_t v = 16 / size; v > 1; v = v == 8 ? 2 : v / 2)
        if (a.channels % v == 0 && ok(a.x, v) && ok(a.out, v) && (!backward || ok(a.dout, v))) return v;
    return 1;
}

const Set& kernels(const NormArgs& a, uint32_t v) {
    static const Set sets[2][3] = {{set_of<float, 1>(), set_of<float, 2>(), set_of<float, 4>()},
                                   {set_of<uint16_t, 1>(), set_of<uint16_t, 2>(), set_of<uint16_t, 8>()}};
    return sets[a.dtype][v == 1 ? 0 : v == 2 ? 1 : 2];
}

cudaError_t launch_one(Kernel k, const NormArgs& a, uint32_t smem, cudaStream_t stream) {
    if (smem > 48 * 1024) {
        const cudaError_t e = allow_shared(reinterpret_cast<const void*>(k), kNormMost);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.chunks, std::min(a.across, a.last - a.first));
    cfg.blockDim = dim3(kNormThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a);
}

cudaError_t passes(NormArgs a, bool backward, cudaStream_t stream, unsigned* launches) {
    const uint32_t v = vector_of(a, backward), red = 2 * v * kNormThreads * 4;
    const Set& k = kernels(a, v);
    cudaError_t e = cudaSuccess;
    const uint32_t n = a.n;
    a.row0 = 0;
    for (a.first = 0; a.first < n && e == cudaSuccess; a.first = a.last) {
        a.last = a.first + std::min(n - a.first, a.batch);
        e = launch_one(backward ? k.grad_stat : k.stat, a, (backward ? 16 : 12) * a.channels + red, stream);
        if (e == cudaSuccess) e = launch_one(backward ? k.grad : k.apply, a, (backward ? 8 : 12) * a.groups, stream);
        *launches += 2;
        a.row0 += a.across;
    }
    return e;
}

}  // namespace

void plan_norm(NormArgs& a, bool backward, uint32_t sms) {
    // Samples per pair of launches: as many as L2 holds for the second pass (64 MB of its 129), one at
    // least; and as many CTAs as run at one time over all of these.
    const uint64_t sample = static_cast<uint64_t>(a.positions) * a.channels * (a.dtype ? 2 : 4) * (backward ? 2 : 1);
    a.batch = static_cast<uint32_t>(std::min<uint64_t>(a.n, std::max<uint64_t>(1, (64ull << 20) / sample)));
    const uint32_t ctas = (backward ? kNormGradCtas : kNormCtas) * sms;
    a.across = std::min(a.batch, ctas);
    const uint32_t v = vector_of(a, backward), vectors = std::min(a.channels / v, kNormThreads), tall = kNormThreads / vectors;
    const uint64_t want = std::max(1u, ctas / std::max(1u, a.across)), least = 4ull * tall;
    uint64_t rows = (a.positions + want - 1) / want;
    rows = std::max((rows + tall - 1) / tall * tall, least);
    a.rows = static_cast<uint32_t>(std::min<uint64_t>(rows, a.positions));
    a.chunks = (a.positions + a.rows - 1) / a.rows;
}

cudaError_t launch_norm(const NormArgs& a, cudaStream_t stream, unsigned* launches) { return passes(a, false, stream, launches); }

cudaError_t launch_norm_param(const NormArgs& a, uint32_t rows, cudaStream_t stream) {
    return launch_next(norm_param_kernel, dim3((a.channels + 7) / 8), 1024, stream, a.cpart, rows, a.channels, a.d_gamma, a.d_beta,
                       a.param_dtype);
}

cudaError_t launch_norm_backward(const NormArgs& a, cudaStream_t stream, unsigned* launches) { return passes(a, true, stream, launches); }

}  // namespace fa
