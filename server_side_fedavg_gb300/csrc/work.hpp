// Work handles as the operators' entry points share them (internal to the library): the handle,
// argument checks, workspace, order of a handle's calls.  The helpers have internal linkage: each
// file of entry points compiles its own copy.
#pragma once

#include <fedavg.h>

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <chrono>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <limits>
#include <mutex>
#include <new>
#include <string>
#include <thread>
#include <vector>

#include "kernels.cuh"
#include "ortho.cuh"
#include "product_tc.cuh"

struct fa_work {
    std::mutex mu;
    int device = 0;
    uint32_t timeout_ms = 60000;
    uint32_t flags = 0;
    uint8_t* ws = nullptr;               // the workspace shared by the handle's calls
    uint64_t ws_bytes = 0;
    bool ws_captured = false;            // a captured call uses it: a graph may still
    std::vector<void*> retired;          // workspaces that were, kept for such graphs
    cudaEvent_t chain = nullptr;         // recorded after the last queued call
    bool chain_valid = false;
    unsigned long long chain_stream_id = 0;
    unsigned int* err_dev = nullptr;     // kErrBytes, zero at first: error word (kernels OR bits in), counters
    unsigned int* err_host = nullptr;    // pinned copy
    cudaStream_t err_stream = nullptr;
    cudaEvent_t err_ev = nullptr;
    fa::TcShape tc;
    fa::OrthoShape ortho;                // filled in by the first fa_orthogonalise
    fa_work_stats stats{};
    std::string err;
};

namespace {

struct Range {
    explicit Range(const char* name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
};

class DeviceGuard {
public:
    explicit DeviceGuard(int dev) {
        if (cudaGetDevice(&prev_) == cudaSuccess && prev_ != dev) restore_ = cudaSetDevice(dev) == cudaSuccess;
    }
    ~DeviceGuard() {
        if (restore_) cudaSetDevice(prev_);
    }

private:
    int prev_ = 0;
    bool restore_ = false;
};

fa_status fail(fa_work* w, fa_status s, const std::string& what) {
    w->err = what;
    const char* v = std::getenv("FA_LOG");
    if (v != nullptr && v[0] != '\0' && std::strcmp(v, "0") != 0)
        std::fprintf(stderr, "[fedavg] %s: %s\n", fa_strerror(s), what.c_str());
    return s;
}

fa_status cuda_fail(fa_work* w, cudaError_t e, const char* where) {
    cudaGetLastError();
    return fail(w, e == cudaErrorMemoryAllocation ? FA_ERR_NOMEM : FA_ERR_CUDA,
                std::string(where) + ": " + cudaGetErrorName(e) + " (" + cudaGetErrorString(e) + ")");
}

#define FW_CUDA(w, call)                                       \
    do {                                                       \
        const cudaError_t e_ = (call);                         \
        if (e_ != cudaSuccess) return cuda_fail(w, e_, #call); \
    } while (0)

fa_status wait_event(fa_work* w, cudaEvent_t ev, const char* what) {
    const auto t0 = std::chrono::steady_clock::now();
    for (uint32_t spins = 0;; ++spins) {
        const cudaError_t e = cudaEventQuery(ev);
        if (e == cudaSuccess) return FA_OK;
        if (e != cudaErrorNotReady) return cuda_fail(w, e, what);
        const auto ms =
            std::chrono::duration_cast<std::chrono::milliseconds>(std::chrono::steady_clock::now() - t0).count();
        if (ms > static_cast<long long>(w->timeout_ms))
            return fail(w, FA_ERR_TIMEOUT, std::string(what) + ": no completion within timeout_ms");
        if (spins < 64)
            std::this_thread::yield();
        else
            std::this_thread::sleep_for(std::chrono::microseconds(50));
    }
}

bool capturing(cudaStream_t s) {
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    return cudaStreamIsCapturing(s, &st) == cudaSuccess && st != cudaStreamCaptureStatusNone;
}

// Make `s` wait for the handle's earlier calls.  Captured work is ordered by the stream
// its graph is replayed on.
fa_status chain_in(fa_work* w, cudaStream_t s, bool capture) {
    if (!w->chain_valid || capture) return FA_OK;
    unsigned long long id = 0;
    FW_CUDA(w, cudaStreamGetId(s, &id));
    if (id != w->chain_stream_id) FW_CUDA(w, cudaStreamWaitEvent(s, w->chain, 0));
    return FA_OK;
}

// From a call's first launch to its end, however it ends: the handle's next call, and a wait for
// the handle, come after everything that this call has queued.  A call that fails half-way has
// kernels on its stream that still use the workspace.
class ChainOut {
public:
    ChainOut(fa_work* w, cudaStream_t s, bool capture) : w_(w), s_(s), open_(!capture) {}
    ChainOut(const ChainOut&) = delete;
    ChainOut& operator=(const ChainOut&) = delete;
    ~ChainOut() {
        if (open_ && record() != cudaSuccess) cudaGetLastError();
    }
    // r, or the event's own error where r is none.
    fa_status end(fa_status r) {
        if (r != FA_OK || !open_) return r;
        open_ = false;
        const cudaError_t e = record();
        return e == cudaSuccess ? FA_OK : cuda_fail(w_, e, "cudaEventRecord");
    }

private:
    cudaError_t record() {
        unsigned long long id = 0;
        cudaError_t e = cudaEventRecord(w_->chain, s_);
        if (e == cudaSuccess) e = cudaStreamGetId(s_, &id);
        if (e != cudaSuccess) return e;
        w_->chain_stream_id = id;
        w_->chain_valid = true;
        return e;
    }
    fa_work* w_;
    cudaStream_t s_;
    bool open_;
};

// At least `bytes` of workspace.  Growing waits for the handle's queued calls, which may
// still use the old one.
fa_status ensure_ws(fa_work* w, uint64_t bytes, bool capture) {
    if (bytes <= w->ws_bytes) {
        w->ws_captured |= capture && bytes > 0;
        return FA_OK;
    }
    if (capture)
        return fail(w, FA_ERR_STATE, "the workspace would have to grow during capture: run the call once before, "
                                     "or open the handle with workspace_bytes");
    if (w->chain_valid) {
        const fa_status r = wait_event(w, w->chain, "workspace growth");
        if (r != FA_OK) return r;
    }
    bytes = (bytes + (1ull << 21) - 1) >> 21 << 21;
    if (w->ws && w->ws_captured) {
        w->retired.push_back(w->ws);
    } else if (w->ws) {
        FW_CUDA(w, cudaFree(w->ws));
    }
    w->ws = nullptr;
    w->ws_bytes = w->stats.workspace_bytes = 0;
    w->ws_captured = false;
    FW_CUDA(w, cudaMalloc(reinterpret_cast<void**>(&w->ws), bytes));
    w->ws_bytes = bytes;
    w->stats.workspace_bytes = bytes;
    return FA_OK;
}

// A tensor the kernels read or write: in this device's memory.
fa_status check_ptr(fa_work* w, const void* p, const char* name) {
    if (p == nullptr) return fail(w, FA_ERR_ARG, std::string(name) + " is NULL");
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
        cudaGetLastError();
        return fail(w, FA_ERR_ARG, std::string(name) + " is not device memory");
    }
    if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged)
        return fail(w, FA_ERR_ARG, std::string(name) + " is not device memory");
    if (at.type == cudaMemoryTypeDevice && at.device != w->device)
        return fail(w, FA_ERR_ARG, std::string(name) + " is on another device");
    return FA_OK;
}

bool dtype_ok(int32_t d) { return d == FA_F32 || d == FA_BF16; }
uint64_t size_of(int32_t d) { return d == FA_F32 ? 4 : 2; }
int code_of(int32_t d) { return d == FA_F32 ? 0 : 1; }

// A matrix argument: rows of `width` elements `ld` apart, `rows` of them.
fa_status check_mat(fa_work* w, const void* p, uint64_t rows, uint64_t width, uint64_t ld, int32_t dt,
                    const char* name) {
    if (rows == 0 || width == 0) return FA_OK;      // not read
    if (ld < width) return fail(w, FA_ERR_RANGE, std::string(name) + ": stride shorter than a row");
    if (ld >> 40) return fail(w, FA_ERR_RANGE, std::string(name) + ": stride of 2^40 or more");
    if (reinterpret_cast<uintptr_t>(p) % size_of(dt))
        return fail(w, FA_ERR_ARG, std::string(name) + " is not aligned to its element type");
    return check_ptr(w, p, name);
}

// Whether two matrices share an element: rows of `width` elements of `size` bytes, `ld` apart.
// Exact where one of them is one run of bytes or both have rows the same distance apart (column
// slices of one buffer); else where their spans meet.
struct Extent {
    const void* p;
    uint64_t rows, width, ld, size;
};

bool overlap(const Extent& x, const Extent& y) {
    if (!x.p || !y.p || !x.rows || !x.width || !y.rows || !y.width) return false;
    typedef __int128 Wide;               // 2^31 rows of 2^40 elements
    const auto rows = [](const Extent& e) -> Wide { return e.width == e.ld ? 1 : e.rows; };
    const auto row = [](const Extent& e) -> Wide { return Wide(e.width == e.ld ? e.rows * e.width : e.width) * e.size; };
    const Wide x_row = row(x), y_row = row(y), x_rows = rows(x), y_rows = rows(y);
    const Wide x_step = Wide(x.ld) * x.size, y_step = Wide(y.ld) * y.size;
    // from x's first byte to y's
    const Wide apart = Wide(reinterpret_cast<uintptr_t>(y.p)) - Wide(reinterpret_cast<uintptr_t>(x.p));
    if (apart >= (x_rows - 1) * x_step + x_row || -apart >= (y_rows - 1) * y_step + y_row) return false;
    if (x_rows > 1 && y_rows > 1 && x_step != y_step) return true;
    const Wide step = x_rows > 1 ? x_step : y_step;
    // Row j of y begins apart + (j - i) step bytes after row i of x: they meet where that lies in
    // (-y_row, x_row).  The least difference of rows that is above the lower end:
    const Wide from = -y_row - apart;
    Wide least = from / step;                                     // rounded towards 0
    if (from % step != 0 && from < 0) --least;                    // down
    least = std::max<Wide>(least + 1, 1 - x_rows);
    return least <= y_rows - 1 && apart + least * step < x_row;
}

constexpr uint64_t kMaxSize = 1ull << 31;

// err_dev: the error word, and from word kNormCounters on those in which the CTAs of a group norm meet.
constexpr uint32_t kErrBytes = 1024, kNormCounters = 16;

fa_status launched(fa_work* w, cudaError_t e, const char* what) {
    if (e != cudaSuccess) return cuda_fail(w, e, what);
    w->stats.kernel_launches++;
    return FA_OK;
}

uint64_t pad256(uint64_t b) { return (b + 255) / 256 * 256; }

// Workspace handed out piece by piece.  A first run with base 0 adds the sizes up.
struct Carve {
    uint8_t* base;
    uint64_t used = 0;
    void* take(uint64_t bytes) {
        uint8_t* p = base ? base + used : nullptr;
        used += pad256(bytes);
        return p;
    }
};

// No exception past the C boundary.
template <typename F>
fa_status guarded(F f) {
    try {
        return f();
    } catch (const std::bad_alloc&) {
        return FA_ERR_NOMEM;
    } catch (...) {
        return FA_ERR_INTERNAL;
    }
}

// Every operator entry point: the argument struct checked for its size, the handle locked, its
// device current.
template <typename Args, typename F>
fa_status enter(const char* name, fa_work* w, const Args* args, F f) {
    if (!w) return FA_ERR_ARG;
    return guarded([&] {
        Range range(name);
        std::lock_guard<std::mutex> lk(w->mu);
        DeviceGuard dg(w->device);
        w->err.clear();
        if (!args || args->size < sizeof(Args)) return fail(w, FA_ERR_ARG, "args is NULL or args.size too small");
        return f(*args);
    });
}

}  // namespace
