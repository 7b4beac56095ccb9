// Test-only: work.cpp over a fake of the CUDA runtime and of the kernels' launches (compiled
// with g++ on the CPU, no CUDA device code).  The CPU suite makes a call of either fail, and
// reads in which order streams, events and launches were used.
#include <fedavg.h>

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdlib>
#include <map>
#include <new>
#include <string>
#include <vector>

#include "distill.cuh"
#include "product_tc.cuh"

namespace {

struct Fake {
    std::string log;                     // a word per call: name[:stream]
    std::string fail_at;                 // the call of this name fails,
    int fail_in = 0;                     // after so many others of its name,
    bool fail_by_throwing = false;       // by an exception in place of an error code
    bool pending = false;                // events stay incomplete
    int cfg = -1;                        // of the last tensor-core product
    uint32_t splits = 0;
    bool drain = false;
    uintptr_t next = 0x1000;
} fake;

cudaError_t call(const std::string& name, cudaError_t error = cudaErrorUnknown) {
    fake.log += name + " ";
    const std::string bare = name.substr(0, name.find(':'));
    if (bare != fake.fail_at || fake.fail_in-- != 0) return cudaSuccess;
    if (fake.fail_by_throwing) throw std::bad_alloc();
    return error;
}

std::string on(const char* name, cudaStream_t s) { return std::string(name) + ":" + std::to_string(reinterpret_cast<uintptr_t>(s)); }

template <typename T>
cudaError_t make(const char* name, T* out) {
    const cudaError_t e = call(name, cudaErrorMemoryAllocation);
    if (e == cudaSuccess) *out = reinterpret_cast<T>(fake.next += 1ull << 40);
    return e;
}

}  // namespace

extern "C" {

cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorName(cudaError_t) { return "name"; }
const char* cudaGetErrorString(cudaError_t) { return "text"; }
cudaError_t cudaMalloc(void** p, size_t) { return make("malloc", p); }
cudaError_t cudaFree(void*) { return call("free"); }
cudaError_t cudaHostAlloc(void** p, size_t, unsigned) {
    *p = std::calloc(1, 64);
    return call("host_alloc", cudaErrorMemoryAllocation);
}
cudaError_t cudaFreeHost(void* p) { std::free(p); return cudaSuccess; }
cudaError_t cudaMemset(void*, int, size_t) { return call("memset:0"); }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t s) { return call(on("memset", s)); }
cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t s) { return call(on("copy", s)); }
cudaError_t cudaStreamCreateWithFlags(cudaStream_t* s, unsigned) { return make("stream", s); }
cudaError_t cudaStreamDestroy(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t s) { return call(on("synchronize", s)); }
cudaError_t cudaDeviceSynchronize() { return call("synchronize:0"); }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* c) { *c = cudaStreamCaptureStatusNone; return cudaSuccess; }
cudaError_t cudaStreamGetId(cudaStream_t s, unsigned long long* id) { *id = reinterpret_cast<uintptr_t>(s); return cudaSuccess; }
cudaError_t cudaStreamWaitEvent(cudaStream_t s, cudaEvent_t, unsigned) { return call(on("wait", s)); }
cudaError_t cudaEventCreateWithFlags(cudaEvent_t* e, unsigned) { return make("event", e); }
cudaError_t cudaEventDestroy(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t s) { return call(on("record", s)); }
cudaError_t cudaEventQuery(cudaEvent_t) {
    const cudaError_t e = call("query");
    return e == cudaSuccess && fake.pending ? cudaErrorNotReady : e;
}
cudaError_t cudaPointerGetAttributes(cudaPointerAttributes* a, const void*) {
    *a = {};
    a->type = cudaMemoryTypeDevice;
    return cudaSuccess;
}

const char* fa_strerror(fa_status) { return ""; }

}  // extern "C"

namespace fa {

cudaError_t launch_product_tiny(const ProdArgs&, cudaStream_t s) { return call(on("tiny", s)); }
cudaError_t launch_product_thin(const ProdArgs&, cudaStream_t s) { return call(on("thin", s)); }
cudaError_t launch_split(const SplitJob*, int, cudaStream_t s) { return call(on("split", s)); }
cudaError_t launch_act_grad(const ActGradArgs&, cudaStream_t s) { return call(on("act_grad", s)); }
cudaError_t launch_col_sum(const float*, uint32_t, uint32_t, void*, int, cudaStream_t s) { return call(on("col_sum", s)); }
cudaError_t launch_distill(DistillArgs&, cudaStream_t s) { return call(on("distill", s)); }
cudaError_t prepare_distill() { return cudaSuccess; }
cudaError_t prepare_product_tc(TcShape* shape) {
    shape->sms = 152;
    for (int i = 1; i <= 8; ++i) shape->split_ctas[i] = 152 / i * i;
    return cudaSuccess;
}
cudaError_t launch_product_tc(const TcProduct& p, const TcShape&, unsigned int*, bool, cudaStream_t s) {
    fake.cfg = p.cfg;
    fake.splits = p.splits;
    fake.drain = p.drain;
    return call(on("product", s));
}

}  // namespace fa

extern "C" {

void ws_reset() { fake = Fake(); }
const char* ws_log() { return fake.log.c_str(); }
void ws_clear_log() { fake.log.clear(); }
void ws_fail(const char* name, int in, int throwing) {
    fake.fail_at = name;
    fake.fail_in = in;
    fake.fail_by_throwing = throwing != 0;
}
void ws_pending(int yes) { fake.pending = yes != 0; }
// The last tensor-core product's configuration, splits and whether its result is fp32.
void ws_choice(int* cfg, uint32_t* splits, int* drain) {
    *cfg = fake.cfg;
    *splits = fake.splits;
    *drain = fake.drain;
}
// fa_work_sync and fa_work_close; -99 where an exception leaves them.
int32_t ws_sync(fa_work* w) {
    try {
        return fa_work_sync(w);
    } catch (...) {
        return -99;
    }
}
int32_t ws_close(fa_work* w) {
    try {
        return fa_work_close(w);
    } catch (...) {
        return -99;
    }
}

}  // extern "C"
