// Rotary positions: launch interface (internal to the library).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fa {

constexpr uint32_t kRotaryMaxPairs = 256;

// One of the tensors turned in a call: element e of head h of token s of batch entry b at
// x[b xb + s xt + h xh + e].
struct RotaryPart {
    const void* x;
    void* out;
    uint64_t xb, xt, xh, ob, ot, oh;
    uint32_t heads;
};

struct RotaryArgs {
    RotaryPart part[2];
    const int32_t* position;    // [tokens], or nullptr: first + the token's place in its sequence
    int64_t first;
    uint32_t tokens, seq;       // batch * seq of them
    uint32_t head_dim, rotary_dim;
    uint32_t chunks, turning;   // per head: pieces of 2 V elements, and those of them that turn
    uint32_t slots;             // heads of a token are shared out over so many threads per piece
    uint32_t cta_tokens;        // the ring's, of a stage
    unsigned int* err;
    int dtype;
    float scale;
    bool interleaved, inverse, copy;   // copy: what does not turn goes to out too
    uint64_t turns[kRotaryMaxPairs];   // of a pair per position, in 2^-64 of a whole turn
};

// Fills in chunks, turning and slots.
cudaError_t launch_rotary(RotaryArgs& a, uint32_t sms, cudaStream_t stream);

}  // namespace fa
