// bs_lora.cpp -- host side of the low-rank adapters: argument checks, the
// choice of launch shapes, and the entry points of bs.h.
#include <hip/hip_runtime.h>
#include <string.h>

#include <algorithm>

#include "bs_device.h"
#include "bs_internal.h"
#include "bs_lora_device.h"

using namespace bs;

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bs_status launched(int e, const char* what) {
    if (e == 0) return BS_OK;
    set_error("%s launch: %s", what, hipGetErrorString((hipError_t)e));
    return BS_E_HIP;
}

// tiles of 16 tokens at most: one for each 16 tokens, and one begun for each
// adapter in use (tokens without one count as an adapter of their own)
uint32_t max_tiles(uint32_t tokens, uint32_t adapters) {
    return tokens / bsd::kLoraTile + std::min<uint32_t>(tokens, adapters + 1);
}

bs_status check_pack(const bs_lora_pack* p) {
    if (!p) { set_error("NULL pack"); return BS_E_INVAL; }
    if (p->adapters == 0 || p->adapters > bsd::kLoraAdapters) {
        set_error("%u adapters (1..%u)", p->adapters, bsd::kLoraAdapters);
        return BS_E_INVAL;
    }
    if (p->rank != 16 && p->rank != 32 && p->rank != 64 && p->rank != 128) {
        set_error("rank %u: 16, 32, 64 or 128 (smaller adapters are padded)", p->rank);
        return BS_E_INVAL;
    }
    if (p->rows == 0 || p->cols == 0 || p->rows >= (1u << 26) || p->cols >= (1u << 26)) {
        set_error("a %u x %u projection", p->rows, p->cols);
        return BS_E_INVAL;
    }
    if (!p->d_a || !p->d_b || !p->d_ranks || !p->d_factor) { set_error("NULL buffer in the pack"); return BS_E_INVAL; }
    if (!aligned(p->d_a, 16) || !aligned(p->d_b, 16) || !aligned(p->d_ranks, 4) || !aligned(p->d_factor, 4)) {
        set_error("a misaligned buffer in the pack");
        return BS_E_INVAL;
    }
    return BS_OK;
}

bool check_tokens(uint64_t tokens) {
    if (tokens <= (1u << 24)) return true;
    set_error("%llu tokens in one call (at most 2^24)", (unsigned long long)tokens);
    return false;
}

// the outer product's grid: tiles times blocks of up to 1024 rows (with as
// many tiles as this), 256 threads each, below 2^32 in all
bool check_grid(const bs_lora_pack* p, uint32_t tokens) {
    if ((uint64_t)max_tiles(tokens, p->adapters) * ((p->rows + 1023) / 1024) < (1u << 24)) return true;
    set_error("%u tokens of %u rows are too many for one call", tokens, p->rows);
    return false;
}

// Workgroups that share the columns of a tile: about eight workgroups per CU
// in all, with 128 columns or more for each of their 4 waves.
uint32_t share_rule(const bs_lora_pack* p, uint32_t tiles) {
    int cus = 0;
    if (bsk_device_cus(&cus) != 0 || cus <= 0) cus = 256;
    const uint32_t want = std::min(std::max<uint32_t>(1, 8u * (uint32_t)cus / std::max(tiles, 1u)), bsd::kLoraSplits);
    const uint32_t blocks = (p->cols + 511) / 512, turns = (blocks + want - 1) / want;
    return (blocks + turns - 1) / turns;         // as many turns of 512 columns with the fewest workgroups
}

// Shares of the columns' panels (of 2048) in the product beside adapters.  A
// CU takes one workgroup (32 rows and a share) at a time, so the time goes by
// rounds of workgroups times the panels of a share (and a quarter of a panel to
// start each): the shares that make it least, the fewest of these, at most 8
// (each is a pass over Y in the last launch).  In all, 8 adapters of rank 16,
// us: 54 tokens on 163 x 14336 take 51 with two shares, 36 with four, 32 with
// seven; 26 on 5182 x 12288 66 with two, 54 with three, 70 with four; 64 on
// 3584 x 14336 54 with two and 65, a second round, with three.  From 8 tokens
// on at least two, as in the plain product; below, one wherever that is as
// fast, since the product's epilogue then adds the adapters (4 tokens on 2000
// x 4096: 17.0 with one, 18.2 with two).
uint32_t panel_shares(uint64_t rows, uint64_t cols, uint32_t tokens) {
    int cus = 0;
    if (bsk_device_cus(&cus) != 0 || cus <= 0) cus = 256;
    const uint64_t panels = cols / 2048, groups = (rows + 31) / 32;
    if (panels < 2 || (tokens < 8 && (panels < 4 || (rows + 15) / 16 * 2 >= (uint64_t)cus))) return 1;
    uint64_t best = 0, least = ~0ull;
    for (uint64_t shares = 2; shares <= std::min<uint64_t>(panels, 8); shares++) {
        const uint64_t rounds = (groups * shares + cus - 1) / cus, turns = (panels + shares - 1) / shares;
        const uint64_t cost = rounds * (4 * turns + 1);
        if (cost < least) { least = cost; best = shares; }
    }
    return (uint32_t)best;
}

// the partial sums of the shares after the first
uint64_t shares_bytes(uint64_t rows, uint64_t cols, uint32_t tokens) {
    return 4ull * (panel_shares(rows, cols, tokens) - 1) * tokens * rows;
}

// X as the product's operand, in batch tiles as its kernels take them; up to
// 16 tokens in one share read X as it is
uint32_t x_tiles(uint64_t rows, uint64_t cols, uint32_t tokens) {
    const uint32_t nt = (tokens + 15) / 16;
    if (nt == 1 && panel_shares(rows, cols, tokens) == 1) return 0;
    return nt == 3 ? 4 : nt;
}

uint64_t x_bytes(uint64_t rows, uint64_t cols, uint32_t tokens) { return 32ull * x_tiles(rows, cols, tokens) * cols; }

uint64_t inner_bytes(const bs_lora_pack* p, uint32_t tokens) {
    return align_up(4ull * share_rule(p, max_tiles(tokens, p->adapters)) * tokens * p->rank, 256);
}

void fill(const bs_lora_pack* p, const int32_t* d_batch, uint32_t tokens, const void* d_x, uint64_t x_stride, float* t,
          bsd::LoraArgs& a) {
    memset(&a, 0, sizeof a);
    a.a = (const uint16_t*)p->d_a;
    a.b = (const uint16_t*)p->d_b;
    a.ranks = p->d_ranks;
    a.factor = p->d_factor;
    a.batch = d_batch;
    a.x = (const uint16_t*)d_x;
    a.x_stride = x_stride;
    a.t = t;
    a.adapters = p->adapters;
    a.rank = p->rank;
    a.rows = p->rows;
    a.cols = p->cols;
    a.cols_pad = (uint32_t)align_up(p->cols, 32);
    a.tokens = tokens;
    a.max_tiles = max_tiles(tokens, p->adapters);
    a.ksplit = share_rule(p, a.max_tiles);
    a.x_aligned = aligned(d_x, 16) && x_stride % 8 == 0;
}

}  // namespace

extern "C" {

uint64_t bs_lora_batch_bytes(uint32_t tokens, uint32_t adapters) {
    if (!check_tokens(tokens) || adapters == 0 || adapters > bsd::kLoraAdapters) return 0;
    return align_up(4ull * (bsd::lora_pairs(max_tiles(tokens, adapters), tokens) + 2ull * tokens), 16);
}

bs_status bs_lora_batch_async(const int32_t* d_adapter_of, uint32_t tokens, uint32_t adapters, int32_t* d_batch,
                              uint64_t batch_bytes, void* stream) {
    if (!check_tokens(tokens)) return BS_E_INVAL;
    if (adapters == 0 || adapters > bsd::kLoraAdapters) {
        set_error("%u adapters (1..%u)", adapters, bsd::kLoraAdapters);
        return BS_E_INVAL;
    }
    if ((tokens && !d_adapter_of) || !d_batch) { set_error("NULL argument"); return BS_E_INVAL; }
    if (!aligned(d_adapter_of, 4) || !aligned(d_batch, 16)) { set_error("a misaligned buffer"); return BS_E_INVAL; }
    if (batch_bytes < bs_lora_batch_bytes(tokens, adapters)) {
        set_error("batch of %llu B, %llu B needed", (unsigned long long)batch_bytes,
                  (unsigned long long)bs_lora_batch_bytes(tokens, adapters));
        return BS_E_INVAL;
    }
    return launched(bsk_lora_batch(d_adapter_of, tokens, adapters, max_tiles(tokens, adapters), d_batch, stream), "adapter batch");
}

uint64_t bs_lora_work_bytes(const bs_lora_pack* pack, uint32_t tokens) {
    if (check_pack(pack) != BS_OK || !check_tokens(tokens) || !check_grid(pack, tokens)) return 0;
    return inner_bytes(pack, tokens);
}

bs_status bs_lora_add_async(const bs_lora_pack* pack, const int32_t* d_batch, uint32_t tokens, const void* d_x,
                            uint64_t x_stride, const void* d_y_in, void* d_y_out, uint64_t y_stride, uint32_t y_type,
                            void* d_work, uint64_t work_bytes, void* stream) {
    const bs_status rc = check_pack(pack);
    if (rc != BS_OK) return rc;
    if (!check_tokens(tokens) || !check_grid(pack, tokens)) return BS_E_INVAL;
    if (y_type != BS_T_BF16 && y_type != BS_T_FP32) { set_error("Y type %u", y_type); return BS_E_INVAL; }
    if (tokens == 0) return BS_OK;
    if (!d_batch || !d_x || !d_y_in || !d_y_out || !d_work) { set_error("NULL argument"); return BS_E_INVAL; }
    const uintptr_t el = y_type == BS_T_FP32 ? 4 : 2;
    if (!aligned(d_batch, 16) || !aligned(d_x, 2) || !aligned(d_y_in, el) || !aligned(d_y_out, el) || !aligned(d_work, 16)) {
        set_error("a misaligned buffer");
        return BS_E_INVAL;
    }
    if (x_stride < pack->cols || y_stride < pack->rows) {
        set_error("token strides %llu and %llu for %u columns and %u rows", (unsigned long long)x_stride,
                  (unsigned long long)y_stride, pack->cols, pack->rows);
        return BS_E_INVAL;
    }
    if (work_bytes < inner_bytes(pack, tokens)) {
        set_error("workspace of %llu B, %llu B needed", (unsigned long long)work_bytes,
                  (unsigned long long)inner_bytes(pack, tokens));
        return BS_E_INVAL;
    }
    const uint64_t need = inner_bytes(pack, tokens), ny = extent(tokens, y_stride, pack->rows, el);
    if (overlap(d_work, need, d_x, extent(tokens, x_stride, pack->cols, 2)) || overlap(d_work, need, d_y_in, ny) ||
        overlap(d_work, need, d_y_out, ny)) {
        set_error("the workspace overlaps X or Y");
        return BS_E_INVAL;
    }
    bsd::LoraArgs a;
    fill(pack, d_batch, tokens, d_x, x_stride, (float*)d_work, a);
    a.y_in = d_y_in;
    a.y_out = d_y_out;
    a.y_stride = y_stride;
    a.y32 = y_type == BS_T_FP32;
    a.y_vec = aligned(d_y_in, 16) && aligned(d_y_out, 16) && y_stride % (16 / el) == 0;
    const bs_status r2 = launched(bsk_lora_inner(&a, stream), "adapters' inner product");
    if (r2 != BS_OK) return r2;
    return launched(bsk_lora_outer(&a, stream), "adapters' outer product");
}

uint64_t bs_fixed_gemm_lora_work_bytes(uint64_t rows, uint64_t cols, uint32_t batch, const bs_lora_pack* pack) {
    if (check_pack(pack) != BS_OK || batch == 0 || batch > 64) return 0;
    if (pack->rows != rows || pack->cols != cols || cols % 2048) return 0;
    return align_up(shares_bytes(rows, cols, batch), 256) + inner_bytes(pack, batch) + x_bytes(rows, cols, batch);
}

bs_status bs_fixed_gemm_lora_async(const bs_fixed_info* info, const void* d_blob, uint64_t rows, uint64_t cols,
                                   uint32_t batch, const void* d_x, float* d_y, uint32_t* d_status,
                                   const bs_lora_pack* pack, const int32_t* d_batch, void* d_work, uint64_t work_bytes,
                                   void* stream) {
    const bs_status rc = check_pack(pack);
    if (rc != BS_OK) return rc;
    if (pack->rows != rows || pack->cols != cols) {
        set_error("adapters of a %u x %u projection beside a %llu x %llu one", pack->rows, pack->cols,
                  (unsigned long long)rows, (unsigned long long)cols);
        return BS_E_INVAL;
    }
    if (batch == 0 || batch > 64) { set_error("batch %u outside 1..64", batch); return BS_E_INVAL; }
    if (!d_batch || !d_work) { set_error("NULL argument"); return BS_E_INVAL; }
    if (!aligned(d_batch, 16) || !aligned(d_work, 256) || !aligned(d_y, 4)) { set_error("a misaligned buffer"); return BS_E_INVAL; }
    const uint64_t need = bs_fixed_gemm_lora_work_bytes(rows, cols, batch, pack);
    if (work_bytes < need) {
        set_error("workspace of %llu B, %llu B needed", (unsigned long long)work_bytes, (unsigned long long)need);
        return BS_E_INVAL;
    }
    // all of it: the shares, the inner products and X in operand order
    if (overlap(d_work, need, d_y, 4ull * batch * rows) || overlap(d_work, need, d_x, 2ull * batch * cols)) {
        set_error("the workspace overlaps X or Y");
        return BS_E_INVAL;
    }
    const uint64_t split = shares_bytes(rows, cols, batch);
    void* part = split ? d_work : nullptr;
    bsd::LoraArgs a;
    fill(pack, d_batch, batch, d_x, cols, (float*)((uint8_t*)d_work + align_up(split, 256)), a);
    a.y_in = d_y;
    a.y_out = d_y;
    a.y_stride = rows;
    a.y32 = 1;
    a.y_vec = aligned(d_y, 16) && rows % 4 == 0;
    a.part = (const float*)part;
    a.part_stride = (uint64_t)batch * rows;
    a.nparts = panel_shares(rows, cols, batch) - 1;
    a.x_tiles = x_tiles(rows, cols, batch);
    a.x_ops = (uint16_t*)((uint8_t*)a.t + inner_bytes(pack, batch));
    // the projection's arguments are checked before anything is enqueued
    const bs_status r0 = fixed_gemm(info, d_blob, rows, cols, batch, d_x, d_y, d_status, part, split, &a, true, stream);
    if (r0 != BS_OK) return r0;
    const bs_status r1 = launched(bsk_lora_inner(&a, stream), "adapters' inner product");
    if (r1 != BS_OK) return r1;
    // without the split, the projection's own epilogue adds the outer product
    const bs_status r2 = fixed_gemm(info, d_blob, rows, cols, batch, d_x, d_y, d_status, part, split, &a, false, stream);
    if (r2 != BS_OK || !split) return r2;
    return launched(bsk_lora_outer(&a, stream), "adapters' outer product");
}

}  // extern "C"
