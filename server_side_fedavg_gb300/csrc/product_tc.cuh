// Tensor-core products: launch interface (internal to the library).
#pragma once

#include <cuda.h>

#include "product.cuh"

namespace fa {

constexpr int kTcMaxStages = 8;
constexpr int kTcMaxSlots = 4;
constexpr int kTcConfigs = 7;

// Kernel configurations (rows x columns of a tile of the output).
enum TcConfig {
    kTcPair256 = 0,     // 256 x 256 on two SMs
    kTc128 = 1,         // 128 x 128
    kTc64 = 2,          // 128 x 64
    kTcSwap64 = 3,      // 64 x 128, tokens in the MMA's columns
    kTcSwap32 = 4,      // 32 x 128
    kTcSwap16 = 5,      // 16 x 128
    kTcPair128 = 6,     // 256 x 128 on two SMs
};

// An operand the kernel can read: bf16, base and row stride multiples of 16 bytes.
struct TcOperand {
    const void* p;
    uint64_t ld;        // elements
    uint64_t plane;     // elements between planes
    uint32_t planes;    // 1, or 3 (an fp32 operand's terms)
    bool kmajor;
};

struct TcProduct {
    uint32_t m, n, k;   // each >= 1
    TcOperand a, b;
    ProdEpilogue e;
    int cfg;
    bool drain;         // fp32 results: sums rounded to nearest
    uint32_t splits;    // of the summed index: 1..8
};

struct TcShape {
    int sms = 0;
    int split_ctas[9] = {};   // [i]: CTAs at one time in clusters of i, one CTA per SM
};

struct TcArgs {
    CUtensorMap map_p, map_q;
    CUtensorMap map_out, map_res, map_pre;    // boxes of 32 rows x 128 bytes; with `vec` and splits == 1
    ProdEpilogue e;
    unsigned int* err;
    uint32_t rows, cols, k;                   // of the output and the sum
    uint32_t sub, kblocks;                    // blocks of 64 terms per stage (1 or 2); stages of a sum
    uint32_t tiles, tiles_p, tiles_q;
    uint32_t splits, stages, chunk_kb, planes_p, planes_q;
    uint32_t grain;                           // output elements a store may cover: 1, 2, 4 (without vec)
    uint32_t slots;                           // 4 KB epilogue buffers per drain warp: 2..kTcMaxSlots
    bool p_kmajor, q_kmajor, vec, test_expire;
};

struct TcTile {
    uint32_t p, q;
};

// Tiles in bands of kTcBand tiles of P, down the band first: the CTAs at work at one time share
// few rows of either operand, which stay in L2.  A walker is asked for ascending tiles, and
// keeps its band: divisions would cost each of its users some 200 cycles a tile.
constexpr uint32_t kTcBand = 8;
struct TcWalk {
    uint32_t p0 = 0, start = 0;       // the band's first tile of P, and its first tile
    __device__ __forceinline__ TcTile at(const TcArgs& a, uint32_t t) {
        const uint32_t full = kTcBand * a.tiles_q;
        while (t - start >= full) {
            start += full;
            p0 += kTcBand;
        }
        const uint32_t r = t - start, height = a.tiles_p - p0;
        if (height >= kTcBand) return {p0 + r % kTcBand, r / kTcBand};
        return {p0 + r % height, r / height};
    }
};

cudaError_t prepare_product_tc(TcShape* shape);
cudaError_t launch_product_tc(const TcProduct& p, const TcShape& shape, unsigned int* err, bool test_expire,
                              cudaStream_t stream);

}  // namespace fa
