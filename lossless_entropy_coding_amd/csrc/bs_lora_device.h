// bs_lora_device.h -- structures shared by the host side of the library and
// the kernels of the low-rank adapters (gfx950).  Not part of the public C
// ABI.
#pragma once
#include <stdint.h>

namespace bsd {

constexpr uint32_t kLoraTile = 16;           // tokens of one adapter that are taken together
constexpr uint32_t kLoraAdapters = 4096;     // adapters of a pack
constexpr uint32_t kLoraHead = 4;            // words before a batch's tiles: tiles, tokens, bad indices, 0
constexpr uint32_t kLoraSplits = 8;          // shares of the columns at most

struct LoraArgs {
    const uint16_t* a;          // [adapters][rank / 16][cols_pad / 32][64][8] (bs.h)
    const uint16_t* b;          // [adapters][rows][rank]
    const int32_t* ranks;       // each adapter's own rank
    const float* factor;
    // head, tiles of 4 words (adapter, first, count, 0), the tokens in tile
    // order, then each token's adapter and place in that order
    const int32_t* batch;
    const uint16_t* x;
    uint64_t x_stride;
    const void* y_in;           // BF16 or fp32
    void* y_out;
    const float* part;          // nparts more shares of y (fp32, part_stride apart) to be added
    uint64_t part_stride;
    uint32_t nparts;
    float* t;                   // inner products: [ksplit][tokens][rank], in tile order
    uint64_t y_stride;          // elements between tokens (in and out)
    uint32_t adapters, rank, rows, cols, cols_pad;
    uint32_t tokens, max_tiles, ksplit;
    // where the inner product leaves x for the product beside it (x_tiles 0:
    // nowhere): [x_tiles][cols / 32][64][8], the operand of 16 tokens and 32
    // columns in lane order, zeros for tokens past the last
    uint16_t* x_ops;
    uint32_t x_tiles;
    int x_aligned;              // rows of x can be read 16 B at a time
    int y32;
    int y_vec;                  // y (and part) can be read and written 16 B at a time
};

// the first word of a batch's per-token pairs (16-B aligned)
inline constexpr uint32_t lora_pairs(uint32_t max_tiles, uint32_t tokens) { return (kLoraHead + 4 * max_tiles + tokens + 3) / 4 * 4; }

}  // namespace bsd

// Launchers (bs_lora.hip).  All return a hipError_t as int.
extern "C" {
int bsk_lora_batch(const int32_t* idx, uint32_t tokens, uint32_t adapters, uint32_t max_tiles, int32_t* batch, void* stream);
int bsk_lora_inner(const bsd::LoraArgs* a, void* stream);
int bsk_lora_outer(const bsd::LoraArgs* a, void* stream);
}
