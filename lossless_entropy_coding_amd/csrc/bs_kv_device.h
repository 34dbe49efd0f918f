// bs_kv_device.h -- structures shared by the host side of the library and the
// kernels of the paged 8-bit key/value cache (gfx950).  Not part of the
// public C ABI.
#pragma once
#include <stdint.h>

namespace bsd {

constexpr uint32_t kKvCounters = 1024;       // words before a workspace's partial results
constexpr uint32_t kKvTile = 64;             // tokens that a wave takes at a time (4 chunks of 16)

// one cache as a kernel sees it (layouts in bs.h)
struct KvView {
    uint8_t* k;
    uint8_t* v;
    float* scale;
    int32_t* refs;
    int32_t* table;
    int32_t* lens;
    uint32_t* status;
    uint64_t side_bytes;        // one page's keys (or values): kv_heads * page * wide
    uint32_t layers, n_pages, max_seqs, max_pages;
    uint32_t kv_heads, dim, wide, page, lp;   // lp = log2 page
    uint32_t type;
};

struct KvAppend {
    KvView c;
    uint32_t layer, n_seqs, total, max_new;
    const int32_t* seqs;
    const int32_t* starts;      // null: one token per sequence
    const void* xk;
    const void* xv;
    uint64_t k_stride, v_stride;   // elements between tokens
    int f32;                    // inputs in fp32 (else BF16)
    int vec;                    // 8 channels of a token can be read 16 B at a time
};

struct KvAttend {
    KvView c;
    const uint8_t* k;           // the layer's keys, values and scales
    const uint8_t* v;
    const float* scale;
    uint32_t n_seqs, heads, group, total, max_new;
    const int32_t* seqs;
    const int32_t* starts;
    const uint16_t* q;
    uint16_t* out;
    float* lse;
    uint64_t q_stride, out_stride;
    float qscale;               // softmax scale
    float softcap;
    uint32_t window, sinks;
    int aligned;                // q can be read 16 B at a time
    int out8;                   // four channels of out can be written at a time
    int many;                   // the kernel for many rows
    uint32_t chunk;             // tiles of a split
    uint32_t splits;            // 1: no partial results
    uint32_t* counters;         // splits > 1: workgroups done of each tile of rows and key head
    float* part;                // splits > 1: [total * heads][splits][wide + 4]: the result, its maximum and sum, 2 unused
};

struct KvPages {
    KvView c;
    uint32_t n;                 // rows or pairs
    const int32_t* a;           // rows (extend, free), sources (fork), source pages (copy)
    const int32_t* b;           // counts (extend), children (fork), destination pages (copy)
    int32_t* work;
    int32_t* table_out;         // compact
    int32_t* refs_out;
};

}  // namespace bsd

// Launchers (bs_kv.hip, bs_kv_attend.hip).  All return a hipError_t as int.
extern "C" {
int bsk_kv_append(const bsd::KvAppend* a, void* stream);
int bsk_kv_attend(const bsd::KvAttend* a, void* stream);
int bsk_kv_extend(const bsd::KvPages* p, void* stream);
int bsk_kv_fork(const bsd::KvPages* p, void* stream);
int bsk_kv_free(const bsd::KvPages* p, void* stream);
int bsk_kv_copy(const bsd::KvPages* p, void* stream);
int bsk_kv_compact(const bsd::KvPages* p, void* stream);
}
