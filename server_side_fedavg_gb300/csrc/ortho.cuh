// Orthogonalised weight steps: launch interface (internal to the library).
//
// Matrices between the first pass and the last are held as two fp16 terms, x * 2^s = hi + lo, hi
// rounded to nearest and lo the remainder rounded: 22 bits, in planes [item][hi, lo][rows][ld].
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace fa {

struct OrthoBuf {
    uint16_t* p = nullptr;
    uint32_t rows = 0, cols = 0;
    uint64_t ld = 0;                   // a multiple of 8
    uint64_t plane() const { return rows * ld; }
    CUtensorMap k, mn, out;            // summed index along rows, across them; as a result
};

constexpr uint32_t kOrthoOps = 24, kOrthoBufs = 12;    // products of a launch; buffers of these, and three

// out = c1 * sum_k P(x,k) Q(y,k) + c2 * e1 + c3 * e2 of every item, on the tensor cores.  An
// operand's element (x, k) is at its row x if it is K-major, else at its row k.
struct OrthoProduct {
    const OrthoBuf *P, *Q, *out, *e1, *e2;    // e1, e2: laid out as out, or nullptr
    bool p_kmajor, q_kmajor;
    bool symmetric;                           // the tiles on and above the diagonal, and their mirror images
    uint32_t k;
    uint32_t chunk;                           // blocks of 64 terms that the tensor cores sum by themselves
    float c1, c2, c3;
};

struct OrthoShape {
    int sms = 0;
    bool ready = false;
};

cudaError_t prepare_ortho(OrthoShape* shape);
cudaError_t map_ortho(OrthoBuf* b, uint32_t items);
// What a list of products is thought to take, in microseconds.
double ortho_cost(const OrthoProduct* p, uint32_t n, uint32_t items, uint32_t sms);
// n <= kOrthoOps products one after the other, of `items` items each.  done: [items], counts of what
// is done of an item, zero before its first product; *count: what they are when these begin, and then
// when they are done.
cudaError_t launch_ortho_products(const OrthoProduct* p, uint32_t n, uint32_t items, uint32_t* done, uint32_t* count,
                                  const OrthoShape& shape, unsigned int* err, bool test_expire, cudaStream_t stream, uint64_t* launches);

// The first pass and the last.  Items are `step` elements apart.
struct OrthoMat {
    const void* p;
    uint64_t ld, step;
    int dtype;
};
struct OrthoEnds {
    OrthoMat update, momentum, momentum_out, residual, out;
    uint32_t items, rows, cols, blocks;       // blocks per item
    float3* part;                             // [items][blocks] sums of squares, by size
    uint32_t* done;                           // [items], set to 0 by the first pass
    uint16_t* x;                              // planes of the scaled update, or of the result
    uint64_t ld;
    double eps;
    float mu, alpha, beta;                    // alpha: times the result's scale
    int shift;                                // the scaled update's, in powers of two
    bool nesterov;
};
// The whole step in one kernel: a short side of up to 64, in fp32, each matrix in the shared memory
// of a cluster.  False where it does not fit.
struct OrthoSmall {
    uint32_t steps, parts;                    // in so many segments, the first ones longer by one at most
    float a, b, c;
};
bool ortho_small_fits(uint64_t items, uint32_t rows, uint32_t cols);
cudaError_t launch_ortho_small(const OrthoEnds& e, const OrthoSmall& s, cudaStream_t stream);

uint32_t ortho_blocks(uint32_t items, uint32_t rows, uint32_t cols, uint32_t sms);
cudaError_t launch_ortho_norm(const OrthoEnds& a, cudaStream_t stream);
cudaError_t launch_ortho_scale(const OrthoEnds& a, cudaStream_t stream);
cudaError_t launch_ortho_finish(const OrthoEnds& a, cudaStream_t stream);

}  // namespace fa
