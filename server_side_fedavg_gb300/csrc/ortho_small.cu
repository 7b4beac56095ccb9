// A whole orthogonalised weight step for matrices with a short side of up to 64 (adapters, small
// classifiers), in fp32: one kernel, a matrix per cluster.
//
// Each CTA of the cluster holds a run of the long side in shared memory, as fp32 rows x_j of kM
// elements, from the first pass to the last.  A = sum_j x_j x_j^T: every CTA sums its run, and all
// read each other's sums over distributed shared memory, in rank order.  The steps' polynomials in A
// are then kM x kM products in shared memory, which every CTA does for itself, and x_j <- (q + Q) x_j
// closes a segment of up to three steps (see the host's `segments`).
//
// What bounds it: the chain of phases.  10 x 256 16 us, 128 of 16 x 4096 bf16 with momentum 80 us (100 MB, 15
// us of HBM): two turns of CTAs, each 11 us loading, 24 in two segments, 4 storing.
//
// Rows are kM + 4 floats apart: lanes that read 16 bytes of rows next to each other then meet no
// bank conflict.
#include <algorithm>

#include "ortho_device.cuh"
#include "tc_ptx.cuh"

namespace fa {

namespace {

constexpr uint32_t kSmallThreads = 256, kSmallWarps = kSmallThreads / 32, kSmallCtas = 8;
// Rows per CTA, unless eight CTAs have to hold more: for a few matrices, and for more than would
// fill the SMs twice.  What every CTA does for itself counts: one of 16 x 4096 bf16 takes 17 us with
// runs of 512 and 25 with 1024; 128 take 98 and 79 us.
constexpr uint32_t kSmallRun = 512, kManyRun = 1024, kMany = 304;
// Sides above 32, an SM's registers to a CTA: 128 rows, or 256, while the SMs (of which whole clusters of
// eight find 14 to 16 places) hold all clusters at once.  1 x 64 x 1024 fp32 71 us in runs of 128 and 92 of
// 256, 16 x 48 x 1000 bf16 141 and 93.  Others are left to the tensor cores: 1 x 64 x 1024 117 us there, 1 x
// 33 x 3000 bf16 119 and 133 here, 16 x 48 x 1000 124, 4 x 64 x 4096 125 and 164, 300 x 48 x 700 328 and 520.
constexpr uint32_t kRun64 = 128, kMany64 = 112;
constexpr uint32_t kSmallMost = 226 * 1024;    // bytes of shared memory
constexpr uint32_t kSmallAhead = 4;            // pieces of eight elements whose loads a thread has in flight

template <int kM>
constexpr uint32_t kPitch = kM + 4;
template <int kM>
constexpr uint32_t kMat = kM * kPitch<kM>;     // floats of a kM x kM matrix
// six matrices (two where segments are of one step), two buffers of this CTA's sums for the others,
// the warps' sums
template <int kM>
constexpr uint32_t kMats = kM == 64 ? 2 : 6;
template <int kM>
constexpr uint32_t kFixed = (kMats<kM> * kMat<kM> + 2 * kM * kM + (kM == 64 ? 0 : kSmallWarps * kM * kM)) * 4;

__device__ __forceinline__ void fma2(float2& d, float2 a, float2 b) {
    asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 d, {%0, %1};\n"
        " fma.rn.f32x2 d, a, b, d;\n mov.b64 {%0, %1}, d;\n}"
        : "+f"(d.x), "+f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
}

// C = c1 A B + c2 E + c3 F, all symmetric; C is none of the others.  A thread has kB x kB elements.
template <int kM>
__device__ __forceinline__ void mul(float* C, const float* A, const float* B, float c1, const float* E, float c2, const float* F,
                                    float c3) {
    constexpr uint32_t kB = kM <= 16 ? 1 : kM / 16, kSide = kM / kB;
    if (threadIdx.x < kSide * kSide) {
        const uint32_t r = threadIdx.x / kSide, c = threadIdx.x % kSide;
        float2 s[kB][kB];
#pragma unroll
        for (uint32_t i = 0; i < kB * kB; ++i) s[i / kB][i % kB] = make_float2(0.0f, 0.0f);
#pragma unroll 8
        for (uint32_t k = 0; k < kM; k += 4) {
            float4 x[kB], y[kB];
#pragma unroll
            for (uint32_t i = 0; i < kB; ++i) {
                x[i] = *reinterpret_cast<const float4*>(A + (r + kSide * i) * kPitch<kM> + k);
                y[i] = *reinterpret_cast<const float4*>(B + (c + kSide * i) * kPitch<kM> + k);
            }
#pragma unroll
            for (uint32_t i = 0; i < kB * kB; ++i) {
                const float4 p = x[i / kB], q = y[i % kB];
                fma2(s[i / kB][i % kB], make_float2(p.x, p.y), make_float2(q.x, q.y));
                fma2(s[i / kB][i % kB], make_float2(p.z, p.w), make_float2(q.z, q.w));
            }
        }
#pragma unroll
        for (uint32_t i = 0; i < kB * kB; ++i) {
            const uint32_t at = (r + kSide * (i / kB)) * kPitch<kM> + c + kSide * (i % kB);
            float v = fmaf(c2, E[at], c1 * (s[i / kB][i % kB].x + s[i / kB][i % kB].y));
            if (F) v = fmaf(c3, F[at], v);
            C[at] = v;
        }
    }
    __syncthreads();
}

// Element i of 8 of a piece `at`: four rows (or columns) of either half of the matrix, so that lanes with
// neighbouring pieces read neighbouring 16 bytes.
template <int kM>
__device__ __forceinline__ uint32_t piece_row(uint32_t at, uint32_t i) {
    return 4 * at + i % 4 + i / 4 * (kM / 2);
}

// This CTA's sum of x_j x_j^T over its run, to out[kM][kM].  A lane has an 8 x 8 tile of the result
// and every so-manieth row; lanes with one tile, then warps, are summed in a fixed order.  kM == 64: the
// tiles on and above the diagonal alone.
template <int kM>
__device__ __forceinline__ void gram(const float* xs, uint32_t run, float* red, float* out) {
    constexpr bool kHalf = kM == 64;
    constexpr uint32_t kSide = kM / 8, kTiles = kHalf ? kSide * (kSide + 1) / 2 : kSide * kSide, kStrands = kSmallThreads / kTiles;
    const uint32_t tile = threadIdx.x % kTiles, strand = threadIdx.x / kTiles;
    uint32_t ti = tile / kSide, tk = tile % kSide;
    if constexpr (kHalf) {
        uint32_t r = tile;
        for (ti = 0; r >= kSide - ti; ++ti) r -= kSide - ti;
        tk = ti + r;
    }
    float2 s[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[i][k] = make_float2(0.0f, 0.0f);
    for (uint32_t j = strand < kStrands ? strand : run; j < run; j += kStrands) {
        const float* x = xs + j * kPitch<kM>;
        const float4 a0 = *reinterpret_cast<const float4*>(x + 4 * ti), a1 = *reinterpret_cast<const float4*>(x + 4 * ti + kM / 2);
        const float4 b0 = *reinterpret_cast<const float4*>(x + 4 * tk), b1 = *reinterpret_cast<const float4*>(x + 4 * tk + kM / 2);
        const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
        const float2 bv[4] = {make_float2(b0.x, b0.y), make_float2(b0.z, b0.w), make_float2(b1.x, b1.y), make_float2(b1.z, b1.w)};
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) fma2(s[i][k], make_float2(av[i], av[i]), bv[k]);
    }
    if constexpr (!kHalf) {
        float* v = &s[0][0].x;
        // lanes with one tile: each exchange halves what a lane keeps
        const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        uint32_t first = 0;
#pragma unroll
        for (uint32_t o = 16, half = 32; o >= kTiles; o /= 2, half /= 2) {
            const bool upper = lane & o;
#pragma unroll
            for (uint32_t e = 0; e < half; ++e) {
                const float got = __shfl_xor_sync(~0u, upper ? v[e] : v[e + half], o);
                v[e] = (upper ? v[e + half] : v[e]) + got;
            }
            if (upper) first += half;
        }
        constexpr uint32_t kKeep = 64 * kTiles / 32;
#pragma unroll
        for (uint32_t e = 0; e < kKeep; ++e)
            red[(warp * kM + piece_row<kM>(ti, (first + e) / 8)) * kM + piece_row<kM>(tk, (first + e) % 8)] = v[e];
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < kM * kM; i += kSmallThreads) {
            float t = 0.0f;
#pragma unroll
            for (uint32_t w = 0; w < kSmallWarps; ++w) t += red[w * kM * kM + i];
            out[i] = t;
        }
    } else {
        for (uint32_t turn = 0; turn < kStrands; ++turn) {
            if (strand == turn)
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i)
#pragma unroll
                    for (uint32_t h = 0; h < 2; ++h) {
                        float4* to = reinterpret_cast<float4*>(out + piece_row<kM>(ti, i) * kM + piece_row<kM>(tk, 4 * h));
                        float4 t = turn ? *to : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        t.x += s[i][2 * h].x;
                        t.y += s[i][2 * h].y;
                        t.z += s[i][2 * h + 1].x;
                        t.w += s[i][2 * h + 1].y;
                        *to = t;
                    }
            __syncthreads();
        }
    }
}

// A = f * the CTAs' sums, in rank order.
template <int kM>
__device__ __forceinline__ void join(float* A, const float* own, uint32_t ctas, float f) {
    if constexpr (kM < 64) {
        for (uint32_t i = threadIdx.x; i < kM * kM; i += kSmallThreads) {
            float v = 0.0f;
            for (uint32_t q = 0; q < ctas; ++q) v += ld_part1(smem_addr(own + i), q, ctas);
            A[i / kM * kPitch<kM> + i % kM] = v * f;
        }
    } else {
        for (uint32_t i = threadIdx.x; i < kM * kM / 4; i += kSmallThreads) {
            const uint32_t r = i / (kM / 4), c = i % (kM / 4) * 4, pr = r % (kM / 2) / 4, pc = c % (kM / 2) / 4;
            if (pr > pc) continue;                   // below the diagonal
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (uint32_t q = 0; q < ctas; ++q) {
                const float4 t = ld_part(smem_addr(own + 4 * i), q, ctas);
                v.x += t.x;
                v.y += t.y;
                v.z += t.z;
                v.w += t.w;
            }
            v = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
            *reinterpret_cast<float4*>(A + r * kPitch<kM> + c) = v;
            if (pr < pc) {
                float* to = A + c * kPitch<kM> + r;
                to[0] = v.x;
                to[kPitch<kM>] = v.y;
                to[2 * kPitch<kM>] = v.z;
                to[3 * kPitch<kM>] = v.w;
            }
        }
    }
    __syncthreads();
}

// x_j <- q x_j + Q x_j.  A thread has kRows rows, 256 kRows 8 / kM apart, by 8 elements, kM / 8 apart:
// neighbouring lanes read neighbouring rows.
template <int kM>
__device__ __forceinline__ void apply(float* xs, uint32_t run, const float* Q, float q) {
    constexpr uint32_t kSide = kM / 8, kGroups = kSmallThreads / kSide, kRows = kM == 32 ? 8 : kM == 64 ? 4 : kM / 4;
    const uint32_t i0 = threadIdx.x % kSide, g = threadIdx.x / kSide;
    for (uint32_t j0 = 0; j0 < run; j0 += kGroups * kRows) {
        float y[kRows][8];
        uint32_t at[kRows];
#pragma unroll
        for (uint32_t n = 0; n < kRows; ++n) {
            at[n] = min(j0 + g + kGroups * n, run - 1) * kPitch<kM>;
#pragma unroll
            for (uint32_t e = 0; e < 8; ++e) y[n][e] = 0.0f;
        }
#pragma unroll 2
        for (uint32_t k = 0; k < kM; k += 4) {
            float4 x[kRows];
#pragma unroll
            for (uint32_t n = 0; n < kRows; ++n) x[n] = *reinterpret_cast<const float4*>(xs + at[n] + k);
#pragma unroll
            for (uint32_t e = 0; e < 8; ++e) {
                const float4 v = *reinterpret_cast<const float4*>(Q + (i0 + kSide * e) * kPitch<kM> + k);
#pragma unroll
                for (uint32_t n = 0; n < kRows; ++n)
                    y[n][e] = fmaf(v.w, x[n].w, fmaf(v.z, x[n].z, fmaf(v.y, x[n].y, fmaf(v.x, x[n].x, y[n][e]))));
            }
        }
        __syncthreads();                 // every lane of these rows has read them
#pragma unroll
        for (uint32_t n = 0; n < kRows; ++n)
            if (j0 + g + kGroups * n < run)
#pragma unroll
                for (uint32_t e = 0; e < 8; ++e) {
                    float* to = xs + at[n] + i0 + kSide * e;
                    *to = fmaf(q, *to, y[n][e]);
                }
    }
}

// x[k] <- x[(k + by) % 8].  Lanes that write (or read) a column of xs each, eight rows apart, start at
// different rows of their eight, so that they meet no bank conflict: kPitch is four times an odd number.
__device__ __forceinline__ void rotate(float (&x)[8], uint32_t by) {
#pragma unroll
    for (uint32_t b = 1; b < 8; b *= 2) {
        float y[8];
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) y[k] = by & b ? x[(k + b) % 8] : x[k];
#pragma unroll
        for (uint32_t k = 0; k < 8; ++k) x[k] = y[k];
    }
}

struct SmallArgs {
    OrthoEnds e;
    OrthoSmall s;
    Vecs v;
    uint32_t run, ctas;                        // run: a multiple of 8
};

template <int kM>
__global__ void __launch_bounds__(kSmallThreads, kM <= 16 ? 2 : 1) ortho_small_kernel(const __grid_constant__ SmallArgs a) {
    extern __shared__ __align__(16) float sm[];
    __shared__ Squares sums[kSmallWarps], mine;
    __shared__ float2 factor;
    const OrthoEnds& e = a.e;
    float *A = sm, *P0 = A + kMat<kM>, *P1 = P0 + kMat<kM>, *R = P1 + kMat<kM>, *Q0 = R + kMat<kM>, *Q1 = Q0 + kMat<kM>;
    float *part = sm + kMats<kM> * kMat<kM>, *red = part + 2 * kM * kM, *xs = sm + kFixed<kM> / 4;
    const uint32_t rank = a.ctas > 1 ? cluster_rank() : 0, item = blockIdx.x / a.ctas;
    const bool wide = e.rows <= e.cols;
    const uint32_t n = wide ? e.cols : e.rows, m = wide ? e.rows : e.cols;
    const uint32_t j0 = min(n, rank * a.run), run = min(a.run, n - j0), run8 = (run + 7) / 8 * 8;
    wait_predecessor();

    // The rows eight elements at a time: along the long side of the matrix (wide), or of a row x_j.  Wide,
    // eight neighbouring lanes have neighbouring pieces of one row of the matrix, a line of memory, and a
    // warp four rows (lanes with a row each took three times as long: 128 of 16 x 4096 98 us, so 79).
    const uint32_t pieces = run8 / 8, all = wide ? (pieces + 7) / 8 * 8 * kM : run * (kM / 8), turn = threadIdx.x % 8;
    // a piece's row of the matrix less m's part, or of x_j; and its place along the other side
    const auto row_in = [&](uint32_t t) { return wide ? t / 32 % (kM / 4) * 4 + t % 32 / 8 : t / (kM / 8); };
    const auto piece_in = [&](uint32_t t) { return wide ? t / (8 * kM) * 8 + t % 8 : t % (kM / 8); };
    const auto row_at = [&](uint32_t t) { return wide ? row_in(t) : j0 + row_in(t); };
    const auto col_at = [&](uint32_t t) { return wide ? j0 + piece_in(t) * 8 : piece_in(t) * 8; };
    const auto held = [&](uint32_t t) { return t < all && (!wide || piece_in(t) < pieces); };
    const auto in_use = [&](uint32_t t) { return held(t) && (wide ? row_in(t) : piece_in(t) * 8) < m; };
    Squares sum;
    for (uint32_t t0 = threadIdx.x; t0 < all; t0 += kSmallAhead * kSmallThreads) {
        float x[kSmallAhead][8], g[kSmallAhead][8];
#pragma unroll
        for (uint32_t u = 0; u < kSmallAhead; ++u) {
            const uint32_t t = t0 + u * kSmallThreads;
            if (!in_use(t)) continue;
            load8(e.update, row_of(e.update, item, row_at(t)), col_at(t), e.cols, a.v.update, x[u]);
            if (e.momentum.p) load8(e.momentum, row_of(e.momentum, item, row_at(t)), col_at(t), e.cols, a.v.momentum, g[u]);
        }
#pragma unroll
        for (uint32_t u = 0; u < kSmallAhead; ++u) {
            const uint32_t t = t0 + u * kSmallThreads;
            if (!held(t)) break;
            if (in_use(t)) {
                momentum_step(e, x[u], g[u]);
                if (e.momentum_out.p)
                    store8(e.momentum_out, row_of(e.momentum_out, item, row_at(t)), col_at(t), e.cols, a.v.momentum_out, g[u]);
                sum.add(x[u]);
            } else {
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k) x[u][k] = 0.0f;
            }
            if (wide) {
                float* to = xs + piece_in(t) * 8 * kPitch<kM> + row_in(t);
                rotate(x[u], turn);
#pragma unroll
                for (uint32_t k = 0; k < 8; ++k) to[((k + turn) % 8) * kPitch<kM>] = x[u][k];
            } else {
                float* to = xs + row_in(t) * kPitch<kM> + piece_in(t) * 8;
                *reinterpret_cast<float4*>(to) = make_float4(x[u][0], x[u][1], x[u][2], x[u][3]);
                *reinterpret_cast<float4*>(to + 4) = make_float4(x[u][4], x[u][5], x[u][6], x[u][7]);
            }
        }
    }
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    sum.over_warp();
    if (lane == 0) sums[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (uint32_t w = 1; w < kSmallWarps; ++w) sum.add(sums[w]);
        mine = sum;
    }
    if (a.ctas > 1)
        cluster_sync();
    else
        __syncthreads();
    if (threadIdx.x == 0) {
        sum = Squares();
        for (uint32_t q = 0; q < a.ctas; ++q) {
            sum.mid += ld_part1(smem_addr(&mine.mid), q, a.ctas);
            sum.high += ld_part1(smem_addr(&mine.high), q, a.ctas);
            sum.low += ld_part1(smem_addr(&mine.low), q, a.ctas);
        }
        factor = sum.factor(e.eps);
    }
    __syncthreads();
    // The rows stay as they are, but for a power of two where their squares could leave fp32's
    // range; A and the result take the factor.
    const float f0 = factor.x, f1 = factor.y;
    if (f1 != 1.0f) {
        for (uint32_t t = threadIdx.x; t < run * kM; t += kSmallThreads) xs[t / kM * kPitch<kM> + t % kM] *= f1;
        __syncthreads();
    }

    uint32_t left = a.s.steps, parity = 0;
    for (uint32_t n_part = a.s.parts; n_part > 0; --n_part, parity ^= 1) {
        const uint32_t steps = (left + n_part - 1) / n_part;
        left -= steps;
        float* own = part + parity * kM * kM;
        gram<kM>(xs, run, red, own);
        // the others' sums; they have read this buffer's last ones before the last exchange
        if (a.ctas > 1)
            cluster_sync();
        else
            __syncthreads();
        join<kM>(A, own, a.ctas, f0 * f0);
        float *P = P0, *Q = P0, *next = Q0;
        float q = 1.0f;
        for (uint32_t j = 0; j < steps; ++j) {
            P = j % 2 ? P1 : P0;                 // (kM == 64: one step, P0 alone)
            mul<kM>(P, A, A, a.s.c, A, a.s.b, nullptr, 0.0f);
            if (j == 0) {
                Q = P;
                q = a.s.a;
            } else {
                mul<kM>(next, P, Q, 1.0f, Q, a.s.a, P, q);
                Q = next;
                next = next == Q0 ? Q1 : Q0;
                q *= a.s.a;
            }
            if (j + 1 < steps) {
                mul<kM>(R, A, P, 1.0f, A, a.s.a, nullptr, 0.0f);
                mul<kM>(A, R, P, 1.0f, R, a.s.a, nullptr, 0.0f);
            }
        }
        apply<kM>(xs, run, Q, q);
        __syncthreads();
    }

    for (uint32_t t0 = threadIdx.x; t0 < all; t0 += kSmallAhead * kSmallThreads) {
        float res[kSmallAhead][8];
        if (e.residual.p)
#pragma unroll
            for (uint32_t u = 0; u < kSmallAhead; ++u) {
                const uint32_t t = t0 + u * kSmallThreads;
                if (in_use(t)) load8(e.residual, row_of(e.residual, item, row_at(t)), col_at(t), e.cols, a.v.residual, res[u]);
            }
#pragma unroll
        for (uint32_t u = 0; u < kSmallAhead; ++u) {
            const uint32_t t = t0 + u * kSmallThreads;
            if (!in_use(t)) continue;
            float x[8];
            const float* from = wide ? xs + piece_in(t) * 8 * kPitch<kM> + row_in(t) : xs + row_in(t) * kPitch<kM> + piece_in(t) * 8;
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) x[k] = from[wide ? (k + turn) % 8 * kPitch<kM> : k];
            if (wide) rotate(x, 8 - turn);
#pragma unroll
            for (uint32_t k = 0; k < 8; ++k) {
                x[k] = e.alpha * (f0 * x[k]);
                if (e.residual.p) x[k] = fmaf(e.beta, res[u][k], x[k]);
            }
            store8(e.out, row_of(e.out, item, row_at(t)), col_at(t), e.cols, a.v.out, x);
        }
    }
    if (a.ctas > 1) cluster_sync();          // no CTA leaves while another may read its sums
}

uint32_t side(uint32_t m) { return m <= 8 ? 8 : m <= 16 ? 16 : m <= 32 ? 32 : 64; }

uint32_t fixed(uint32_t m) { return m <= 8 ? kFixed<8> : m <= 16 ? kFixed<16> : m <= 32 ? kFixed<32> : kFixed<64>; }

// CTAs of a cluster (a power of two), and rows of each; false where the matrices are not for this kernel.
bool split(uint32_t m, uint32_t n, uint64_t items, uint32_t* ctas, uint32_t* run) {
    if (m > 64) return false;
    const auto fill = [&](uint32_t rows) {
        *ctas = 1;
        while (*ctas < kSmallCtas && *ctas * rows < n) *ctas *= 2;
        *run = ((n + *ctas - 1) / *ctas + 7) / 8 * 8;
        return static_cast<uint64_t>(*run) * (side(m) + 4) * 4 + fixed(m) <= kSmallMost;
    };
    if (side(m) == 64) {
        for (const uint32_t rows : {kRun64, 2 * kRun64})
            if (fill(rows) && *run <= rows && items * *ctas <= kMany64) return true;
        return false;
    }
    const bool few = fill(kSmallRun);
    if (items * *ctas <= kMany || !few) return few;
    return fill(kManyRun) || fill(kSmallRun);
}

template <int kM>
cudaError_t launch(SmallArgs a, cudaStream_t stream) {
    const uint32_t smem = kFixed<kM> + a.run * kPitch<kM> * 4;
    const cudaError_t r = allow_shared(reinterpret_cast<const void*>(ortho_small_kernel<kM>), kSmallMost);
    if (r != cudaSuccess) return r;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.e.items * a.ctas);
    cfg.blockDim = dim3(kSmallThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = a.ctas;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = a.ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, ortho_small_kernel<kM>, a);
}

}  // namespace

bool ortho_small_fits(uint64_t items, uint32_t rows, uint32_t cols) {
    uint32_t ctas, run;
    return split(std::min(rows, cols), std::max(rows, cols), items, &ctas, &run);
}

cudaError_t launch_ortho_small(const OrthoEnds& e, const OrthoSmall& s, cudaStream_t stream) {
    SmallArgs a{};
    a.e = e;
    a.s = s;
    a.v = vecs(e);
    const uint32_t m = std::min(e.rows, e.cols);
    split(m, std::max(e.rows, e.cols), e.items, &a.ctas, &a.run);
    if (side(m) == 64) a.s.parts = a.s.steps;    // no room for the squares of longer segments
    switch (side(m)) {
    case 8: return launch<8>(a, stream);
    case 16: return launch<16>(a, stream);
    case 32: return launch<32>(a, stream);
    default: return launch<64>(a, stream);
    }
}

}  // namespace fa
