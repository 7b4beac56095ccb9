// Distillation from the clients' top logits: the launch interface (internal to the
// library).  Formulas in include/fedavg.h.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fa {

constexpr int kMaxDistillClients = 16;
constexpr uint32_t kMaxDistillTopk = 2048;   // summed over the clients

constexpr float kLightest = 4096.0f;         // all weight / a client's: above, it is a light one

constexpr unsigned int kErrListIndex = 2u;   // device error bit: a list entry >= vocab

struct DistillClient {
    const int32_t* index;   // [rows][topk]
    const void* value;      // [rows][topk]
    uint32_t topk;
    float weight;           // n_j, times a power of two that the call's weights share
    float share;            // n_j / (sum of all n_j), 0 if that sum is 0
};

struct DistillArgs {
    const void* logits;
    void* grad;                // nullptr: loss only
    const float* row_weight;   // nullptr: 1
    float* loss;               // or nullptr
    const float* lse_in;       // nullptr: computed
    float* lse_out;            // or nullptr
    unsigned int* err;
    uint64_t ld, ldg;
    uint32_t rows, vocab;
    uint32_t nclients;
    uint32_t slots;            // hash slots: a power of two >= 2 * (sum of topk)
    uint32_t hash_shift;
    uint32_t parts, slice;     // CTAs per row and the elements of each
    uint32_t sms;              // of the device
    uint32_t table_at;         // bytes of a slice's vectors in shared memory: the table follows
    float temperature, inv_t;
    float total;               // sum of all weights
    int dtype, value_dtype;
    bool short_lists;          // every list has at most 64 places
    bool light;                // a client has a weight, but less than 1 / kLightest of all
    bool joint;                // a row's CTAs are a cluster and exchange their statistics
    bool test_expire;          // the first exchange's wait counts as run out
    DistillClient client[kMaxDistillClients];
};

// Fills slots, hash_shift, parts, slice, table_at, short_lists and joint; the caller fills the
// rest.
cudaError_t launch_distill(DistillArgs& a, cudaStream_t stream);
cudaError_t prepare_distill();   // shared-memory limits, for the current device

}  // namespace fa
