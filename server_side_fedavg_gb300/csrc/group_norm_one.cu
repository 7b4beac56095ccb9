// Group norm and its gradients in one kernel, where a sample's positions are one run of bytes.
//
// k CTAs share a sample, each every k-th stage of its positions; one CTA per SM, launched
// cooperatively or as clusters.  A warp of its own fetches them by bulk copies into a ring of 40 KB
// stages; 20 warps compute, which leaves each thread 80 registers.
// After the statistics' pass the CTAs meet at a counter in global memory, join their parts, and
// walk their stages backwards for the result: the stages fetched last are still in shared memory,
// some 28 MB of a sample over all SMs, and are not fetched again; the next sample's first stages
// are fetched meanwhile.  A sample that fits is read once.
//
// What bounds it: HBM, x (and dout) read once and beyond 28 MB a second time, the result written once.  2 x
// 128^3 x 32 bf16 135 us, 698 MB moved at 5.2 TB/s; gradients of 2 x 96^3 x 32 bf16 with silu 97 us, instruction
// issue (62 % of the slots), those of 3 x 107865 x 64 fp32 68 us.
#include <algorithm>

#include "group_norm_device.cuh"

namespace fa {

namespace {

constexpr uint32_t kOneThreads = 640, kOneWarps = kOneThreads / 32;           // that compute
constexpr uint32_t kOneStage = 40960, kOneSlots = 5;
constexpr uint32_t kOneRed = 128 * (kOneWarps + 2);   // floats: the sums over the positions
static_assert(kOneRed >= 4 * kOneThreads, "four of every thread's sums");
constexpr uint32_t kOneChunks = 160;                  // CTAs of a sample: five per lane of a warp
// Bytes of a sample's inputs from which on one kernel is faster: 32 of 4096 x 128 bf16 (1 MB) take 28
// us so and 22 in two passes, one of 32768 x 64 bf16 (4 MB) 14 and 15, 2 of 32768 x 256 fp32 31 and 36.
constexpr double kOneLeast = 4e6;
constexpr uint32_t kOneMost = 225 * 1024;             // dynamic shared memory
constexpr uint32_t kOneGroups = 80;                   // counters for samples at one time, and one for the end

// The computing warps of a CTA; whether all of their threads say so.
__device__ __forceinline__ void sync_compute() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(kOneThreads) : "memory"); }

__device__ __forceinline__ bool sync_and(bool ok) {
    uint32_t all;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.and.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
        : "=r"(all)
        : "r"(static_cast<uint32_t>(ok)), "n"(kOneThreads)
        : "memory");
    return all;
}

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// Until `counter` has reached `target`; false after some 20 s.
constexpr long long kMeetClocks = 40ll * 1000 * 1000 * 1000;
__device__ __forceinline__ bool meet(uint32_t* counter, uint32_t target) {
    __threadfence();
    atomicAdd(counter, 1u);
    const long long t0 = clock64();
    while (ld_acquire(counter) < target)
        if (clock64() - t0 > kMeetClocks) return false;
    return true;
}

// The ring's slots in the order of their use.  A sample's n stages go to slots b, b + d, ... (d is 1
// or -1); the result's pass takes them from the last to the first, so that slots come free in the
// order b + d (n - 1), ..., b, and the next sample starts at b - d the other way round.
struct Slots {
    uint32_t count;
    int b = 0, d = 1;
    uint32_t full = 0, empty = 0, used = 0;           // a bit per slot: phases, and whether it has been filled
    __device__ __forceinline__ uint32_t at(uint32_t i) const {
        const int n = static_cast<int>(count), s = (b + d * static_cast<int>(i % count)) % n;
        return s < 0 ? s + n : s;
    }
    __device__ __forceinline__ uint32_t after(uint32_t s) const { return d > 0 ? (s + 1 == count ? 0 : s + 1) : (s == 0 ? count : s) - 1; }
    __device__ __forceinline__ uint32_t before(uint32_t s) const { return d < 0 ? (s + 1 == count ? 0 : s + 1) : (s == 0 ? count : s) - 1; }
    __device__ __forceinline__ void next() {
        b = (b - d + static_cast<int>(count)) % static_cast<int>(count);
        d = -d;
    }
};

// Stages of a sample's CTA, and the positions in them.
__device__ __forceinline__ uint32_t stages_of(const NormArgs& a, uint32_t rank) {
    return ((a.positions + a.stage_rows - 1) / a.stage_rows + a.chunks - 1 - rank) / a.chunks;
}
__device__ __forceinline__ float rows_of(const NormArgs& a, uint32_t rank) {
    const uint32_t n = stages_of(a, rank), last = ((n - 1) * a.chunks + rank) * a.stage_rows;
    return static_cast<float>((n - 1) * a.stage_rows + min(a.stage_rows, a.positions - last));
}

template <typename T>
__device__ __forceinline__ const T* at(const NormTensor& t, uint32_t sample) {
    return static_cast<const T*>(t.p) + sample * t.step;
}

// The threads' sums over the positions, for each channel, in its first thread.  Where lanes of a warp
// share columns by a power of two, over these first, then over the warps in order.  Else four sums at a time over a tree.
template <int N, int V>
__device__ __forceinline__ void over_positions(float (&s)[N][V], float* red, uint32_t vectors, uint32_t tall) {
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, my_row = threadIdx.x / vectors;
    if (vectors <= 32 && 32 % vectors == 0 && N * V * vectors <= 4 * 32) {
        float v[N * V];
#pragma unroll
        for (int k = 0; k < N * V; ++k) v[k] = s[k / V][k % V];
        for (uint32_t o = 16; o >= vectors; o /= 2)
#pragma unroll
            for (int k = 0; k < N * V; ++k) v[k] += __shfl_xor_sync(~0u, v[k], o);
        // [sum][warp][column]
        if (lane < vectors)
#pragma unroll
            for (int k = 0; k < N * V; ++k) red[(k * kOneWarps + warp) * vectors + lane] = v[k];
        sync_compute();
        for (uint32_t i = threadIdx.x; i < N * V * vectors; i += kOneThreads) {
            float t = 0.0f;
#pragma unroll
            for (uint32_t w = 0; w < kOneWarps; ++w) t += red[(i / vectors * kOneWarps + w) * vectors + i % vectors];
            red[N * V * kOneWarps * vectors + i] = t;
        }
        sync_compute();
        if (threadIdx.x < vectors)
#pragma unroll
            for (int k = 0; k < N * V; ++k) s[k / V][k % V] = red[N * V * (kOneWarps * vectors) + k * vectors + threadIdx.x];
        return;
    }
#pragma unroll
    for (int k0 = 0; k0 < N * V; k0 += 4) {
#pragma unroll
        for (int k = 0; k < 4; ++k) red[k * kOneThreads + threadIdx.x] = s[(k0 + k) / V][(k0 + k) % V];
        sync_compute();
        for (uint32_t left = tall; left > 1;) {
            const uint32_t half = (left + 1) / 2;
            if (my_row < left - half)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float& v = s[(k0 + k) / V][(k0 + k) % V];
                    v += red[k * kOneThreads + threadIdx.x + half * vectors];
                    red[k * kOneThreads + threadIdx.x] = v;
                }
            left = half;
            sync_compute();
        }
    }
}

template <typename T, int V, bool kBackward>
__global__ void __launch_bounds__(kOneThreads + 32) norm_one_kernel(const __grid_constant__ NormArgs a) {
    constexpr uint32_t kStreams = kBackward ? 2 : 1, kPlane = kOneStage / kStreams;
    extern __shared__ __align__(128) uint8_t dyn[];
    __shared__ uint64_t bars[2 * kOneSlots];
    float* red = reinterpret_cast<float*>(dyn + a.slots * kOneStage);
    float *s0 = red + kOneRed, *s1 = s0 + a.channels;                      // of a channel
    float *t0 = s1 + a.channels, *t1 = t0 + (kBackward ? a.channels : 0);          // gradients so far; forward: means
    float *g0 = t1 + a.channels, *g1 = g0 + a.groups, *left = g1 + a.groups;
    const uint32_t full = smem_addr(bars), empty = full + 8 * kOneSlots;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < a.slots; ++s) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(full + 8 * s) : "memory");
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(empty + 8 * s), "r"(kOneWarps) : "memory");
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    wait_predecessor();

    const uint32_t group = blockIdx.x / a.chunks, rank = blockIdx.x % a.chunks, row = a.channels * sizeof(T);
    // this CTA's stages: rank, rank + k, ...: what all fetch at one time lies together
    const uint32_t n = stages_of(a, rank);
    const auto first_of = [&](uint32_t stage) { return (stage * a.chunks + rank) * a.stage_rows; };
    Slots ring;
    ring.count = a.slots;
    bool ok = true;

    if (warp == kOneWarps) {
        if (lane == 0) {
            const auto fetch = [&](const T* x, const T* dout, uint32_t stage, uint32_t s) {
                if (ring.used >> s & 1) {
                    ok = mbar_wait(empty + 8 * s, ring.empty >> s & 1);
                    ring.empty ^= 1u << s;
                    if (!ok) return;
                }
                ring.used |= 1u << s;
                const uint32_t first = first_of(stage), bytes = min(a.stage_rows, a.positions - first) * row;
                mbar_expect(full + 8 * s, bytes * kStreams);
                bulk_load(dyn + s * kOneStage, x + static_cast<uint64_t>(first) * a.channels, bytes, full + 8 * s);
                if (kBackward) bulk_load(dyn + s * kOneStage + kPlane, dout + static_cast<uint64_t>(first) * a.channels, bytes, full + 8 * s);
                ring.full ^= 1u << s;
            };
            for (uint32_t sample = group; ok && sample < a.n; sample += a.across) {
                const T *x = at<T>(a.x, sample), *dout = kBackward ? at<T>(a.dout, sample) : nullptr;
                for (uint32_t i = 0; ok && i < n; ++i) fetch(x, dout, i, ring.at(i));
                for (uint32_t i = a.slots; ok && i < n; ++i) fetch(x, dout, n - 1 - i, ring.at(n - 1 - i));
                ring.next();
            }
            if (!ok) {
                atomicOr(a.err, kErrWaitTimeout);
                // the loads in flight land before the CTA leaves: the last phase of every slot's
                for (uint32_t s = 0; s < a.slots; ++s)
                    if (ring.used >> s & 1) mbar_wait(full + 8 * s, (ring.full >> s & 1) ^ 1);
            }
        }
        return;
    }

    const uint32_t vectors = a.channels / V, per = a.channels / a.groups;
    const uint32_t tall = kOneThreads / vectors, my_row = threadIdx.x / vectors, c = threadIdx.x % vectors * V;
    const uint32_t stage_each = a.stage_rows / tall;           // of a whole stage's positions, a thread's
    const bool on = my_row < tall;
    const float count = rows_of(a, rank), inv_count = 1.0f / count, all = static_cast<float>(a.positions);
    const int act = a.act;
    const auto wait_full = [&](uint32_t s) {
        const bool got = mbar_wait(full + 8 * s, ring.full >> s & 1);
        ring.full ^= 1u << s;
        return got;
    };
    const auto release = [&](uint32_t s) {
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + 8 * s);
    };
    // f(vector of x, vector of dout, where its result goes) of a stage, four at a time
    const uint32_t step = tall * row, mine = my_row * row + c * sizeof(T);
    const uint64_t step_out = tall * a.out.ld;
    const auto over = [&](uint32_t stage, uint32_t s, T* out, auto f) {
        if (!on) return;
        const uint32_t first = first_of(stage), rows = min(a.stage_rows, a.positions - first);
        const uint8_t* from = dyn + s * kOneStage + mine;
        T* to = out + (first + my_row) * a.out.ld + c;
        uint32_t r = my_row;
        for (; r + 3 * tall < rows; r += 4 * tall) {
            Vec<T, V> q[4], p[4];
#pragma unroll
            for (uint32_t u = 0; u < 4; ++u) {
                q[u] = *reinterpret_cast<const Vec<T, V>*>(from + u * step);
                if (kBackward) p[u] = *reinterpret_cast<const Vec<T, V>*>(from + kPlane + u * step);
            }
#pragma unroll
            for (uint32_t u = 0; u < 4; ++u) f(q[u], kBackward ? p[u] : q[u], to + u * step_out);
            from += 4 * step;
            to += 4 * step_out;
        }
        for (; r < rows; r += tall, from += step, to += step_out) {
            const Vec<T, V> q = *reinterpret_cast<const Vec<T, V>*>(from);
            f(q, kBackward ? *reinterpret_cast<const Vec<T, V>*>(from + kPlane) : q, to);
        }
    };
    if (kBackward) {
        for (uint32_t i = threadIdx.x; i < a.channels; i += kOneThreads) t0[i] = t1[i] = 0.0f;
        sync_compute();
    }
    uint32_t round = 0;
    for (uint32_t sample = group; ok && sample < a.n; sample += a.across, ++round) {
        const T* x = at<T>(a.x, sample);
        T* out = const_cast<T*>(at<T>(a.out, sample));
        // the statistics' pass
        Moments<V> o;                                          // (backward: its sums alone)
        float (&s)[2][V] = o.s;
        Channels<V> ch;
        if (kBackward && on) ch = Channels<V>(a, sample, c);
        uint32_t my_rows = 0, next = 1;                        // forward: positions so far; stages when the reference moves
        for (uint32_t i = 0, slot = ring.at(0); ok && i < n; ++i, slot = ring.after(slot)) {
            ok = __all_sync(~0u, wait_full(slot));
            if (!ok) break;
            if (!kBackward && on) {
                const uint32_t rows = min(a.stage_rows, a.positions - first_of(i));
                if (i == 0 && my_row < rows) {
                    float from[V];
                    widen(*reinterpret_cast<const Vec<T, V>*>(dyn + slot * kOneStage + mine), from);
                    o.begin(from);
                }
                my_rows += rows == a.stage_rows ? stage_each : my_row < rows ? (rows - my_row + tall - 1) / tall : 0;
            }
            over(i, slot, out, [&](const Vec<T, V>& q, const Vec<T, V>& p, T*) {
                float v[V], d[V];
                widen(q, v);
                if constexpr (kBackward) {
                    widen(p, d);
                    ch.step(act, v, d);
                    add(s[0], s[0], d);
                    fma(s[1], d, v, s[1]);
                } else {
                    o.step(v);
                }
            });
            if (i + a.slots < n) release(slot);               // the last ones are kept
            if (!kBackward && i + 1 == next && my_rows > 0) {
                o.move(static_cast<float>(my_rows));
                next *= kGrow;
            }
        }
        if constexpr (!kBackward) {
            // the threads' common mean, then their sums about it
            float m[1][V];
            o.mean_part(static_cast<float>(my_rows), count, m[0]);
            over_positions(m, red, vectors, tall);
            if (my_row == 0)
#pragma unroll
                for (int i = 0; i < V; ++i) t0[c + i] = m[0][i];
            sync_compute();
            if (on) o.about(static_cast<float>(my_rows), t0 + c);
        }
        over_positions(s, red, vectors, tall);
        if (my_row == 0)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if constexpr (kBackward) {
                    const float rstd = a.rstd[static_cast<uint64_t>(sample) * a.groups + (c + i) / per];
                    const float g = a.gamma ? elem(a.gamma, c + i, a.param_dtype) : 1.0f;
                    s[1][i] *= rstd;                          // from dz h to dz xhat
                    s0[c + i] = g * s[0][i];
                    s1[c + i] = g * s[1][i];
                    t0[c + i] += s[0][i];
                    t1[c + i] += s[1][i];
                } else {
                    const float m = s[0][i] * inv_count;
                    s0[c + i] = m;
                    s1[c + i] = fmaxf(fmaf(-s[0][i], m, s[1][i]), 0.0f);
                }
            }
        sync_compute();
        // of each group, for the sample's other CTAs
        const uint64_t parts = static_cast<uint64_t>(sample) * a.chunks * a.groups;
        for (uint32_t g = warp; g < a.groups; g += kOneWarps) {
            float p = 0.0f, q = 0.0f;
            if constexpr (kBackward) {
                for (uint32_t k = g * per + lane; k < (g + 1) * per; k += 32) {
                    p += s0[k];
                    q += s1[k];
                }
                p = warp_sum(p);
                q = warp_sum(q);
                if (lane == 0) __stcg(a.part + parts + rank * a.groups + g, make_float2(p, q));
            } else {
                // a point near the group's mean: that of its first channels, one a lane
                float hi = lane < per ? t0[g * per + lane] + s0[g * per + lane] : 0.0f;
                hi = warp_sum(hi) / static_cast<float>(min(per, 32u));
                for (uint32_t k = g * per + lane; k < (g + 1) * per; k += 32) {
                    s0[k] += t0[k] - hi;
                    p += s0[k];
                }
                p = warp_sum(p) / static_cast<float>(per);
                for (uint32_t k = g * per + lane; k < (g + 1) * per; k += 32) {
                    const float d = s0[k] - p;
                    q += fmaf(count * d, d, s1[k]);
                }
                q = warp_sum(q);
                if (lane == 0) __stcg(a.stat + parts + g * a.chunks + rank, make_float4(hi, p, q, 0.0f));
            }
        }
        ok = sync_and(ok);
        if (a.chunks > 1) {
            if (threadIdx.x == 0) ok = meet(a.counters + group, (round + 1) * a.chunks) && ok;
            ok = sync_and(ok);
        }
        for (uint32_t g = warp; g < a.groups; g += kOneWarps) {
            float p = 0.0f, q = 0.0f;
            if constexpr (kBackward) {
                float2 v[kOneChunks / 32];
#pragma unroll
                for (uint32_t u = 0; u < kOneChunks / 32; ++u) {
                    const uint32_t i = lane + 32 * u;
                    v[u] = i < a.chunks ? __ldcg(a.part + parts + i * a.groups + g) : make_float2(0.0f, 0.0f);
                }
#pragma unroll
                for (uint32_t u = 0; u < kOneChunks / 32; ++u) {
                    p += v[u].x;
                    q += v[u].y;
                }
                const float inv = 1.0f / (all * static_cast<float>(per));
                p = warp_sum(p) * inv;
                q = warp_sum(q) * inv;
            } else {
                float4 v[kOneChunks / 32];                     // w: its positions
#pragma unroll
                for (uint32_t u = 0; u < kOneChunks / 32; ++u) {
                    const uint32_t i = lane + 32 * u;
                    v[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (i >= a.chunks) continue;
                    v[u] = __ldcg(a.stat + parts + g * a.chunks + i);
                    v[u].w = rows_of(a, i);
                }
                const float hi = __shfl_sync(~0u, v[0].x + v[0].y, 0);       // a point near the mean, the first CTA's
                float m = 0.0f;
#pragma unroll
                for (uint32_t u = 0; u < kOneChunks / 32; ++u) m = v[u].w > 0.0f ? fmaf((v[u].x - hi) + v[u].y, v[u].w, m) : m;
                m = warp_sum(m) / all;
#pragma unroll
                for (uint32_t u = 0; u < kOneChunks / 32; ++u) {
                    const float d = ((v[u].x - hi) + v[u].y) - m;
                    q += v[u].w > 0.0f ? fmaf(v[u].w * static_cast<float>(per) * d, d, v[u].z) : 0.0f;
                }
                p = hi + m;
                q = 1.0f / sqrtf(warp_sum(q) / (all * static_cast<float>(per)) + a.eps);
                if (lane == 0) {
                    left[g] = (hi - p) + m;
                    const uint64_t to = static_cast<uint64_t>(sample) * a.groups + g;
                    if (rank == 0 && a.mean_out) a.mean_out[to] = p;
                    if (rank == 0 && a.rstd_out) a.rstd_out[to] = q;
                }
            }
            if (lane == 0) {
                g0[g] = p;
                g1[g] = q;
            }
        }
        sync_compute();
        // the result's pass, from the last stage to the first
        float less[V] = {}, k1[V] = {}, k2[V] = {};
        if (on)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint32_t g = (c + i) / per;
                if constexpr (kBackward) {
                    // dx = scale dz - rstd m1 - h rstd^2 m2
                    const float r = a.rstd[static_cast<uint64_t>(sample) * a.groups + g];
                    k1[i] = -r * g0[g];
                    k2[i] = -r * r * g1[g];
                } else {
                    // y = act((x - mean) scale + shift): what the mean's rounding left is in the shift
                    less[i] = -g0[g];
                    k1[i] = g1[g] * (a.gamma ? elem(a.gamma, c + i, a.param_dtype) : 1.0f);
                    k2[i] = fmaf(-left[g], k1[i], a.beta ? elem(a.beta, c + i, a.param_dtype) : 0.0f);
                }
            }
        for (uint32_t i = 0, slot = ring.at(n - 1); ok && i < n; ++i, slot = ring.before(slot)) {
            if (i >= a.slots) {
                ok = __all_sync(~0u, wait_full(slot));
                if (!ok) break;
            }
            over(n - 1 - i, slot, out, [&](const Vec<T, V>& q, const Vec<T, V>& p, T* to) {
                float v[V], d[V];
                widen(q, v);
                if constexpr (kBackward) {
                    widen(p, d);
                    ch.step(act, v, d);
                    fma(v, v, k2, k1);
                    fma(v, d, ch.scale, v);
                } else {
                    add(v, v, less);
                    fma(v, v, k1, k2);
                    act_of(act, v);
                }
                store_vec<T, V>(to, v);
            });
            release(slot);
        }
        ring.next();
        ok = sync_and(ok);
    }
    if (kBackward && a.cpart)
        for (uint32_t i = threadIdx.x; i < a.channels; i += kOneThreads)
            a.cpart[static_cast<uint64_t>(blockIdx.x) * a.channels + i] = make_float2(t0[i], t1[i]);
    if (threadIdx.x == 0) {
        if (!ok) atomicOr(a.err, kErrWaitTimeout);
        // the last CTA to leave sets the counters back
        if (a.chunks > 1 && atomicAdd(a.counters + kOneGroups, 1u) == gridDim.x - 1) {
            for (uint32_t i = 0; i <= kOneGroups; ++i) a.counters[i] = 0;
            __threadfence();
        }
    }
}

// Shared memory beside the ring.
uint32_t fixed_bytes(const NormArgs& a, bool backward) {
    return (kOneRed + (backward ? 4 : 3) * a.channels + 3 * a.groups) * 4;
}
// Channels of a thread: 16 bytes, but for the gradients of bf16 four, whose state would not fit its
// registers otherwise.
uint32_t channels_of(int dtype, bool backward) { return dtype && !backward ? 8 : 4; }

}  // namespace

bool plan_norm_one(NormArgs& a, bool backward, uint32_t sms) {
    const uint32_t size = a.dtype ? 2 : 4, v = 16 / size, streams = backward ? 2 : 1;
    if (a.channels % v || a.channels > 1024) return false;
    const auto dense = [&](const NormTensor& t) {
        return reinterpret_cast<uintptr_t>(t.p) % 16 == 0 && (a.positions == 1 || t.ld == a.channels) && (a.n == 1 || t.step % v == 0);
    };
    const auto aligned = [&](const NormTensor& t) {
        return reinterpret_cast<uintptr_t>(t.p) % 16 == 0 && t.ld % v == 0 && (a.n == 1 || t.step % v == 0);
    };
    if (!dense(a.x) || (backward && !dense(a.dout)) || !aligned(a.out)) return false;
    const uint32_t row = a.channels * size, tall = kOneThreads / (a.channels / channels_of(a.dtype, backward));
    a.stage_rows = kOneStage / streams / row / tall * tall;
    a.slots = std::min(kOneSlots, (kOneMost - fixed_bytes(a, backward)) / kOneStage);
    // Samples at one time, each with its share of the SMs: the least by a model of the rounds that takes.
    // A round moves its samples' bytes, with what is not kept in shared memory read again, at the SMs'
    // share of 6.5 TB/s, and has some 9 us of sums and waiting.  Two of 128^3 x 32 bf16 take 135 us side
    // by side and 141 one after the other, the gradients of three of 45 x 47 x 51 x 64 fp32 68 and 80.
    const uint64_t stages = (a.positions + a.stage_rows - 1) / a.stage_rows;
    const double out = static_cast<double>(a.positions) * row, in = out * streams;
    if (in < kOneLeast) return false;
    double best = 1e300;
    for (uint32_t rounds = 1; rounds <= std::min(a.n, 64u); ++rounds) {
        const uint32_t g = (a.n + rounds - 1) / rounds;
        if (g > sms) continue;
        const uint32_t k = static_cast<uint32_t>(std::min<uint64_t>({sms / g, stages, kOneChunks}));
        if (k > 1 && g > kOneGroups) continue;
        const double again = std::max(0.0, in - static_cast<double>(k) * a.slots * kOneStage);
        const double cost = rounds * ((in + again + out) / (6.5e6 * k / sms) + 9.0);
        if (cost < best) {
            best = cost;
            a.chunks = k;
            a.across = g;
        }
    }
    if (best > 1e299) return false;
    return true;
}

cudaError_t launch_norm_one(const NormArgs& a, bool backward, cudaStream_t stream) {
    using Kernel = void (*)(NormArgs);
    static const Kernel kernels[2][2] = {{norm_one_kernel<float, 4, false>, norm_one_kernel<float, 4, true>},
                                         {norm_one_kernel<uint16_t, 8, false>, norm_one_kernel<uint16_t, 4, true>}};
    const Kernel k = kernels[a.dtype][backward];
    const uint32_t smem = a.slots * kOneStage + fixed_bytes(a, backward);
    const cudaError_t e = allow_shared(reinterpret_cast<const void*>(k), kOneMost);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.across * a.chunks);
    cfg.blockDim = dim3(kOneThreads + 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    // CTAs that meet run at the same time: those of a cluster do, others in a cooperative launch
    cudaLaunchAttribute at[1];
    if (a.chunks <= 8) {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = a.chunks;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    } else {
        at[0].id = cudaLaunchAttributeCooperative;
        at[0].val.cooperative = 1;
    }
    cfg.attrs = at;
    cfg.numAttrs = a.chunks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k, a);
}

}  // namespace fa
