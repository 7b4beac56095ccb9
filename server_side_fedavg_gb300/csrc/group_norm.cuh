// Group norm with an activation, channels last: launch interface (internal to the library).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fa {

constexpr uint32_t kNormMaxChannels = 8192;

// A tensor [n][positions][channels]: positions `ld` elements apart, samples `step`.
struct NormTensor {
    const void* p;
    uint64_t ld, step;
};

struct NormArgs {
    NormTensor x, dout, out;       // out: y, or the gradient of x
    const void *gamma, *beta;      // of param_dtype, or nullptr (1 and 0)
    const float *mean, *rstd;      // backward: [n][groups]
    float *mean_out, *rstd_out;    // forward, or nullptr
    void *d_gamma, *d_beta;        // backward, of param_dtype, or nullptr
    float4* stat;                  // forward: [n][groups][chunks] of the statistics' parts, the mean as a sum of two
    float2* part;                  // backward: [n][chunks][groups] of the sums' parts
    float2* cpart;                 // [norm_rows * chunks][channels] of the parameters' gradients, or nullptr
    uint32_t n, positions, channels, groups;
    uint32_t rows, chunks;         // positions per CTA, and CTAs of a sample
    uint32_t stage_rows, slots;    // one kernel: positions per stage, stages in shared memory
    uint32_t* counters;            // one kernel: 81, zero between launches
    unsigned int* err;
    uint32_t batch, across;        // samples per pair of launches, and of these at work at one time
    uint32_t first, last, row0;    // samples of this launch, and its first row of across in cpart
    int dtype, param_dtype, act;
    float eps;
};

// In one kernel, where the positions are one run of 16-byte pieces: false where they are not.  Else
// fills in rows, chunks (CTAs per sample), across (samples at one time), stage_rows and slots; cpart is
// [across * chunks][channels].
bool plan_norm_one(NormArgs& a, bool backward, uint32_t sms);
cudaError_t launch_norm_one(const NormArgs& a, bool backward, cudaStream_t stream);

// In two passes: rows, chunks, batch and across for these sizes; the workspace of `stat`, `part` and `cpart` follows from them.
void plan_norm(NormArgs& a, bool backward, uint32_t sms);
// Rows of `across` over all launches.
inline uint64_t norm_rows(const NormArgs& a) {
    const uint64_t whole = (a.n - 1) / a.batch, rest = a.n - whole * a.batch;
    return whole * a.across + (rest < a.across ? rest : a.across);
}
cudaError_t launch_norm(const NormArgs& a, cudaStream_t stream, unsigned* launches);
cudaError_t launch_norm_backward(const NormArgs& a, cudaStream_t stream, unsigned* launches);
// d_gamma and d_beta from `rows` rows of cpart.
cudaError_t launch_norm_param(const NormArgs& a, uint32_t rows, cudaStream_t stream);

}  // namespace fa
