// Products in plain fp32 arithmetic for any type, stride and size.
#include "product_device.cuh"

namespace fa {

namespace {

constexpr int kPt = 64;    // outputs per tile side
constexpr int kPk = 16;    // summed elements per step
constexpr int kPlainBlock = 128;

// out tile 64 x 64 per CTA of 256 threads, 4 x 4 outputs each; both operands staged as
// fp32 in shared memory, [kk][x], with the summed index or x along the global row.
__global__ void __launch_bounds__(256) product_plain_kernel(const __grid_constant__ ProdArgs p) {
    __shared__ float sa[kPk][kPt + 4], sb[kPk][kPt + 4];
    const uint32_t m0 = blockIdx.y * kPt, n0 = blockIdx.x * kPt;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    // sums over blocks of kPlainBlock terms, then over the blocks: a single chain of 11008
    // additions was 2e-6 off, twice what blocks leave
    float acc[4][4] = {}, tot[4][4] = {};
    for (uint32_t k0 = 0; k0 < p.k; k0 += kPk) {
        for (int i = threadIdx.x; i < kPk * kPt; i += 256) {
            int kk = p.a.kmajor ? i % kPk : i / kPt, x = p.a.kmajor ? i / kPk : i % kPt;
            bool in = m0 + x < p.m && k0 + kk < p.k;
            uint64_t at = p.a.kmajor ? (uint64_t)(m0 + x) * p.a.ld + k0 + kk : (uint64_t)(k0 + kk) * p.a.ld + m0 + x;
            sa[kk][x] = in ? elem(p.a.p, at, p.a.dtype) : 0.0f;
            kk = p.b.kmajor ? i % kPk : i / kPt, x = p.b.kmajor ? i / kPk : i % kPt;
            in = n0 + x < p.n && k0 + kk < p.k;
            at = p.b.kmajor ? (uint64_t)(n0 + x) * p.b.ld + k0 + kk : (uint64_t)(k0 + kk) * p.b.ld + n0 + x;
            sb[kk][x] = in ? elem(p.b.p, at, p.b.dtype) : 0.0f;
        }
        __syncthreads();
        const int kn = p.k - k0 < kPk ? p.k - k0 : kPk;
        for (int kk = 0; kk < kn; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[kk][ty * 4 + i], sb[kk][tx + 16 * j], acc[i][j]);
        __syncthreads();
        if ((k0 / kPk + 1) % (kPlainBlock / kPk) == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    tot[i][j] += acc[i][j];
                    acc[i][j] = 0.0f;
                }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t r = m0 + ty * 4 + i, c = n0 + tx + 16 * j;
            if (r < p.m && c < p.n) finish_one(p.e, tot[i][j] + acc[i][j], r, c);
        }
}

}  // namespace

cudaError_t launch_product_plain(const ProdArgs& p, cudaStream_t stream) {
    // rows beyond 65535 tiles (4 M rows) go in several launches
    const uint32_t per = 65535u * kPt;
    for (uint32_t r = 0; r < p.m; r += per) {
        ProdArgs q = p;
        const uint64_t so = p.e.out_dtype ? 2 : 4, sa = p.a.dtype ? 2 : 4;
        q.m = p.m - r < per ? p.m - r : per;
        q.a.p = static_cast<const char*>(p.a.p) + (p.a.kmajor ? r * p.a.ld : r) * sa;
        q.e.out = static_cast<char*>(p.e.out) + r * p.e.ldo * so;
        if (p.e.pre) q.e.pre = static_cast<char*>(p.e.pre) + r * p.e.ldo * so;
        if (p.e.res) q.e.res = static_cast<const char*>(p.e.res) + r * p.e.ldr * so;
        product_plain_kernel<<<dim3((p.n + kPt - 1) / kPt, (q.m + kPt - 1) / kPt), 256, 0, stream>>>(q);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace fa
