// Test-only: fakes of the launches that layers.cpp and orthogonalise.cpp make, beside those of
// work_shim.cpp (compiled with g++ on the CPU, no CUDA device code).
#include <cuda_runtime.h>

#include <cstdint>

#include "group_norm.cuh"
#include "ortho.cuh"
#include "rotary.cuh"

namespace {

struct Seen {
    uint32_t launches = 0, products = 0, small = 0, fail_at = 0;
    fa::RotaryArgs rotary;
    fa::OrthoEnds ends;
} seen;

cudaError_t call() { return ++seen.launches == seen.fail_at ? cudaErrorUnknown : cudaSuccess; }

}  // namespace

namespace fa {

cudaError_t launch_rotary(RotaryArgs& a, uint32_t, cudaStream_t) {
    seen.rotary = a;
    return call();
}

bool plan_norm_one(NormArgs&, bool, uint32_t) { return false; }
cudaError_t launch_norm_one(const NormArgs&, bool, cudaStream_t) { return call(); }
void plan_norm(NormArgs& a, bool, uint32_t) {
    a.rows = a.positions;
    a.chunks = 1;
    a.batch = a.across = a.n;
}
cudaError_t launch_norm(const NormArgs&, cudaStream_t, unsigned* launches) {
    *launches += 2;
    return call();
}
cudaError_t launch_norm_backward(const NormArgs&, cudaStream_t, unsigned* launches) {
    *launches += 2;
    return call();
}
cudaError_t launch_norm_param(const NormArgs&, uint32_t, cudaStream_t) { return call(); }

cudaError_t prepare_ortho(OrthoShape* shape) {
    shape->sms = 152;
    shape->ready = true;
    return cudaSuccess;
}
cudaError_t map_ortho(OrthoBuf*, uint32_t) { return cudaSuccess; }
// by their operations
double ortho_cost(const OrthoProduct* p, uint32_t n, uint32_t, uint32_t) {
    double c = 0.0;
    for (uint32_t i = 0; i < n; ++i) c += (p[i].symmetric ? 0.5 : 1.0) * p[i].out->rows * p[i].out->cols * p[i].k;
    return c;
}
cudaError_t launch_ortho_products(const OrthoProduct*, uint32_t n, uint32_t, uint32_t*, uint32_t*, const OrthoShape&, unsigned int*, bool,
                                  cudaStream_t, uint64_t* launches) {
    seen.products += n;
    *launches += n;
    return call();
}
uint32_t ortho_blocks(uint32_t, uint32_t, uint32_t, uint32_t) { return 4; }
cudaError_t launch_ortho_norm(const OrthoEnds& e, cudaStream_t) {
    seen.ends = e;
    return call();
}
cudaError_t launch_ortho_scale(const OrthoEnds&, cudaStream_t) { return call(); }
cudaError_t launch_ortho_finish(const OrthoEnds&, cudaStream_t) { return call(); }
bool ortho_small_fits(uint64_t, uint32_t rows, uint32_t cols) { return rows <= 32 || cols <= 32; }
cudaError_t launch_ortho_small(const OrthoEnds& e, const OrthoSmall&, cudaStream_t) {
    seen.ends = e;
    ++seen.small;
    return call();
}

}  // namespace fa

extern "C" {

void ss_reset(uint32_t fail_at) {
    seen = Seen();
    seen.fail_at = fail_at;
}
uint32_t ss_launches() { return seen.launches; }
uint32_t ss_products() { return seen.products; }
uint32_t ss_small() { return seen.small; }
uint64_t ss_turn(uint32_t i) { return seen.rotary.turns[i]; }
int ss_copies() { return seen.rotary.copy; }

}  // extern "C"
