// bs_kv.cpp -- host side of the paged 8-bit key/value cache: argument checks,
// the choice of launch shapes, and the entry points of bs.h.
#include <hip/hip_runtime.h>
#include <string.h>

#include <algorithm>

#include "bs_device.h"
#include "bs_internal.h"
#include "bs_kv_device.h"

using namespace bs;

namespace {

constexpr uint64_t kGridYZ = 65535, kThreads = 0xFFFFFFFFull;   // workgroups of a grid's y and z, threads of its x

bs_status launched(int e, const char* what) {
    if (e == 0) return BS_OK;
    set_error("%s launch: %s", what, hipGetErrorString((hipError_t)e));
    return BS_E_HIP;
}

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// a checked view of the caller's cache
bs_status view(const bs_kv_cache* c, bsd::KvView& v) {
    if (!c) { set_error("NULL cache"); return BS_E_INVAL; }
    if (!c->d_k || !c->d_v || !c->d_scale || !c->d_refs || !c->d_table || !c->d_lens) {
        set_error("NULL buffer in the cache");
        return BS_E_INVAL;
    }
    if (c->type != BS_KV_E4M3 && c->type != BS_KV_INT8) { set_error("cache type %u", c->type); return BS_E_INVAL; }
    if (c->head_dim == 0 || c->head_dim > 256) { set_error("head size %u outside 1..256", c->head_dim); return BS_E_INVAL; }
    if (c->page_tokens < 16 || c->page_tokens > 256 || (c->page_tokens & (c->page_tokens - 1))) {
        set_error("page of %u tokens: 16, 32, 64, 128 or 256", c->page_tokens);
        return BS_E_INVAL;
    }
    if (c->layers == 0 || c->layers > 4096 || c->kv_heads == 0 || c->kv_heads > 1024) {
        set_error("%u layers (1..4096), %u key heads (1..1024)", c->layers, c->kv_heads);
        return BS_E_INVAL;
    }
    if (c->n_pages == 0 || c->n_pages > (1u << 28) || c->max_seqs == 0 || c->max_seqs > (1u << 24) || c->max_pages == 0 ||
        (uint64_t)c->max_pages * c->page_tokens > 0x7FFFFF00ull) {
        set_error("%u pages, %u rows of %u pages", c->n_pages, c->max_seqs, c->max_pages);
        return BS_E_INVAL;
    }
    if (!aligned(c->d_k, 16) || !aligned(c->d_v, 16)) { set_error("keys and values must be 16-B aligned"); return BS_E_INVAL; }
    if (!aligned(c->d_scale, 8) || !aligned(c->d_refs, 16) || !aligned(c->d_table, 4) || !aligned(c->d_lens, 4) ||
        !aligned(c->d_status, 4)) {
        set_error("a misaligned buffer in the cache");
        return BS_E_INVAL;
    }
    v.k = (uint8_t*)c->d_k;
    v.v = (uint8_t*)c->d_v;
    v.scale = c->d_scale;
    v.refs = c->d_refs;
    v.table = c->d_table;
    v.lens = c->d_lens;
    v.status = c->d_status;
    v.layers = c->layers;
    v.n_pages = c->n_pages;
    v.max_seqs = c->max_seqs;
    v.max_pages = c->max_pages;
    v.kv_heads = c->kv_heads;
    v.dim = c->head_dim;
    v.wide = (uint32_t)align_up(c->head_dim, 64);
    v.page = c->page_tokens;
    v.lp = (uint32_t)__builtin_ctz(c->page_tokens);
    v.type = c->type;
    v.side_bytes = (uint64_t)c->kv_heads * c->page_tokens * v.wide;
    return BS_OK;
}

// The tiles that a split takes, and how many splits there are.
void split_rule(const bsd::KvAttend& a, uint32_t max_len, uint32_t& chunk, uint32_t& splits) {
    int cus = 0;
    if (bsk_device_cus(&cus) != 0 || cus <= 0) cus = 256;
    const uint64_t rows = (uint64_t)a.max_new * a.group;
    const uint64_t block_rows = a.many ? (a.c.wide <= 128 ? 256 : 128) : 16, row_tiles = (rows + block_rows - 1) / block_rows;
    uint64_t tiles = ((uint64_t)max_len + bsd::kKvTile - 1) / bsd::kKvTile;
    if (a.window) {
        const uint64_t span = (uint64_t)a.window + a.max_new + bsd::kKvTile;
        tiles = std::min<uint64_t>(tiles, span / bsd::kKvTile + 1 + ((uint64_t)a.sinks + bsd::kKvTile - 1) / bsd::kKvTile);
    }
    const uint64_t groups = std::max<uint64_t>(1, (uint64_t)a.n_seqs * row_tiles * a.c.kv_heads);
    // workgroups per CU that are aimed at (4 of the few-row kernel: 8 and 16
    // made 4 x 131071 tokens 2 and 9% slower), and the fewest tiles of one:
    // one to a wave, so that short rows are read by many CUs
    const uint64_t per = a.many ? 1 : 4, least = a.many ? 8 : 4;
    const uint64_t want = std::max<uint64_t>(1, per * (uint64_t)cus / groups);
    uint64_t ch = std::max<uint64_t>(least, (tiles + want - 1) / want);
    splits = (uint32_t)std::max<uint64_t>(1, (tiles + ch - 1) / ch);
    if (splits > kGridYZ) {
        ch = (tiles + kGridYZ - 1) / kGridYZ;
        splits = (uint32_t)((tiles + ch - 1) / ch);
    }
    chunk = (uint32_t)ch;
    if (groups > bsd::kKvCounters && !a.many) { splits = 1; chunk = (uint32_t)std::max<uint64_t>(1, tiles); }
}

bs_status attend_args(const bs_kv_cache* cache, const bs_kv_attend_args* x, bsd::KvAttend& a, uint32_t& chunk,
                      uint32_t& splits) {
    memset(&a, 0, sizeof a);
    const bs_status rc = view(cache, a.c);
    if (rc != BS_OK) return rc;
    if (!x) { set_error("NULL argument"); return BS_E_INVAL; }
    if (x->layer >= a.c.layers) { set_error("layer %u of %u", x->layer, a.c.layers); return BS_E_INVAL; }
    if (x->heads == 0 || x->heads % a.c.kv_heads || x->heads > kGridYZ) {
        set_error("%u query heads over %u key heads", x->heads, a.c.kv_heads);
        return BS_E_INVAL;
    }
    if (x->n_seqs && x->max_new == 0) { set_error("max_new 0"); return BS_E_INVAL; }
    if (!x->d_starts && x->total_q != x->n_seqs) {
        set_error("%u queries for %u sequences without starts", x->total_q, x->n_seqs);
        return BS_E_INVAL;
    }
    if (!x->d_starts && x->max_new > 1) { set_error("max_new %u without starts", x->max_new); return BS_E_INVAL; }
    if (x->total_q > 0x7FFFFFFFu || (x->total_q && x->n_seqs && x->max_new > x->total_q)) {
        set_error("max_new %u of %u queries", x->max_new, x->total_q);
        return BS_E_INVAL;
    }
    if (!(x->softcap >= 0.f) || !(x->scale == x->scale)) { set_error("softcap %g, scale %g", x->softcap, x->scale); return BS_E_INVAL; }
    const uint64_t row = (uint64_t)x->heads * a.c.dim;
    if (x->q_stride < row || x->out_stride < row) {
        set_error("token strides %llu and %llu below %llu", (unsigned long long)x->q_stride,
                  (unsigned long long)x->out_stride, (unsigned long long)row);
        return BS_E_INVAL;
    }
    const uint64_t layer_off = (uint64_t)x->layer * a.c.n_pages;
    a.k = a.c.k + layer_off * a.c.side_bytes;
    a.v = a.c.v + layer_off * a.c.side_bytes;
    a.scale = a.c.scale + layer_off * a.c.kv_heads * 2;
    a.n_seqs = x->n_seqs;
    a.heads = x->heads;
    a.group = x->heads / a.c.kv_heads;
    a.total = x->total_q;
    a.max_new = x->max_new;
    a.seqs = x->d_seqs;
    a.starts = x->d_starts;
    a.q = (const uint16_t*)x->d_q;
    a.out = (uint16_t*)x->d_out;
    a.lse = x->d_lse;
    a.q_stride = x->q_stride;
    a.out_stride = x->out_stride;
    a.qscale = x->scale > 0.f || x->scale < 0.f ? x->scale : 1.f / __builtin_sqrtf((float)a.c.dim);
    // above 2^100 (infinity, too) c tanh(x / c) is x to fp32's precision, and
    // below 2^-100 every capped logit is 0 to it: neither overflows a constant
    a.softcap = x->softcap > 0x1p100f ? 0.f : x->softcap > 0.f ? std::max(x->softcap, 0x1p-100f) : 0.f;
    a.window = x->window;
    a.sinks = x->sinks;
    a.aligned = aligned(x->d_q, 16) && x->q_stride % 8 == 0 && a.c.dim % 8 == 0;
    const uint64_t row_tiles = ((uint64_t)a.max_new * a.group + 15) / 16;
    a.out8 = aligned(x->d_out, 8) && x->out_stride % 4 == 0 && a.c.dim % 4 == 0;
    a.many = (uint64_t)a.max_new * a.group >= 64;
    // workgroups of the kernel for few rows, of the one for many, and of its join
    const uint64_t block = a.c.wide <= 128 ? 256 : 128, row_blocks = ((uint64_t)a.max_new * a.group + block - 1) / block;
    const uint64_t few = row_tiles * a.n_seqs, many = ((uint64_t)a.n_seqs * a.c.kv_heads + 7) / 8 * 8 * row_blocks;
    if ((uint64_t)a.max_new * a.group > 0x7FFFFFFFull ||
        (a.many ? many > kThreads / 512 || (uint64_t)a.n_seqs * a.max_new > kThreads / 64 : few > kThreads / 256)) {
        set_error("%u sequences of up to %u new tokens are too many for one call (max_new: the most of one row)", a.n_seqs, a.max_new);
        return BS_E_INVAL;
    }
    const uint32_t cap = a.c.max_pages * a.c.page;
    split_rule(a, x->max_len && x->max_len < cap ? x->max_len : cap, chunk, splits);
    return BS_OK;
}

uint64_t part_bytes(const bsd::KvAttend& a, uint32_t splits) {
    return splits > 1 ? 4ull * (bsd::kKvCounters + (uint64_t)a.total * a.heads * splits * (a.c.wide + 4)) : 0;
}

uint64_t page_work(const bsd::KvView& v, uint64_t n) {
    const uint64_t blocks = ((uint64_t)v.n_pages + 4095) / 4096;
    return align_up(4 * std::max<uint64_t>(1 + (uint64_t)v.n_pages + 2 * n, 4 + blocks + 2ull * v.n_pages), 256);
}

bs_status page_call(const bs_kv_cache* cache, uint32_t n, const void* a, bool two, const void* b, bool need_work,
                    void* d_work, uint64_t work_bytes, bsd::KvPages& p) {
    memset(&p, 0, sizeof p);
    const bs_status rc = view(cache, p.c);
    if (rc != BS_OK) return rc;
    if (n && (!a || (two && !b))) { set_error("NULL argument"); return BS_E_INVAL; }
    if (n > kGridYZ) { set_error("%u rows or pages in one call (at most 65535)", n); return BS_E_INVAL; }
    if (need_work) {
        if (!d_work || !aligned(d_work, 16)) { set_error("a 16-B aligned workspace is needed"); return BS_E_INVAL; }
        if (work_bytes < page_work(p.c, n)) {
            set_error("workspace of %llu B, %llu B needed", (unsigned long long)work_bytes,
                      (unsigned long long)page_work(p.c, n));
            return BS_E_INVAL;
        }
    }
    p.n = n;
    p.a = (const int32_t*)a;
    p.b = (const int32_t*)b;
    p.work = (int32_t*)d_work;
    return BS_OK;
}

}  // namespace

extern "C" {

bs_status bs_kv_sizes_get(const bs_kv_cache* cache, bs_kv_sizes* out) {
    if (!cache || !out) { set_error("NULL argument"); return BS_E_INVAL; }
    bs_kv_cache c = *cache;
    // only the shape is looked at
    static const uint64_t dummy[2] __attribute__((aligned(16))) = {0, 0};
    void* d = (void*)dummy;
    c.d_k = c.d_v = d;
    c.d_scale = (float*)d;
    c.d_refs = c.d_table = c.d_lens = (int32_t*)d;
    c.d_status = nullptr;
    bsd::KvView v;
    const bs_status rc = view(&c, v);
    if (rc != BS_OK) return rc;
    memset(out, 0, sizeof *out);
    const uint64_t pages = (uint64_t)v.layers * v.n_pages;
    out->wide = v.wide;
    out->side_bytes = pages * v.side_bytes;
    out->scale_bytes = pages * v.kv_heads * 8;
    out->page_bytes = 2 * v.side_bytes + 8ull * v.kv_heads;
    return BS_OK;
}

bs_status bs_kv_append_async(const bs_kv_cache* cache, uint32_t layer, uint32_t n_seqs, const int32_t* d_seqs,
                             const int32_t* d_starts, uint32_t total, uint32_t max_new, const void* d_k, uint64_t k_stride,
                             const void* d_v, uint64_t v_stride, uint32_t dtype, void* stream) {
    bsd::KvAppend a;
    memset(&a, 0, sizeof a);
    const bs_status rc = view(cache, a.c);
    if (rc != BS_OK) return rc;
    if (layer >= a.c.layers) { set_error("layer %u of %u", layer, a.c.layers); return BS_E_INVAL; }
    if (dtype != BS_T_BF16 && dtype != BS_T_FP32) { set_error("input type %u", dtype); return BS_E_INVAL; }
    if (n_seqs == 0 || total == 0) return BS_OK;
    if (!d_seqs || !d_k || !d_v) { set_error("NULL argument"); return BS_E_INVAL; }
    if (n_seqs > kGridYZ) { set_error("%u sequences in one call (at most 65535)", n_seqs); return BS_E_INVAL; }
    if (total > 0x7FFFFFFFu || max_new == 0 || max_new > total) { set_error("max_new %u of %u tokens", max_new, total); return BS_E_INVAL; }
    const uint64_t touch = ((uint64_t)max_new + 2ull * a.c.page - 2) >> a.c.lp;
    if (touch * 2 * a.c.kv_heads > kThreads / 256) { set_error("max_new %u is too many tokens for one call", max_new); return BS_E_INVAL; }
    if (!d_starts && (total != n_seqs || max_new != 1)) {
        set_error("%u tokens for %u sequences without starts", total, n_seqs);
        return BS_E_INVAL;
    }
    const uint64_t row = (uint64_t)a.c.kv_heads * a.c.dim;
    if (k_stride < row || v_stride < row) {
        set_error("token strides %llu and %llu below %llu", (unsigned long long)k_stride, (unsigned long long)v_stride,
                  (unsigned long long)row);
        return BS_E_INVAL;
    }
    const uintptr_t el = dtype == BS_T_FP32 ? 4 : 2;
    if (!aligned(d_k, el) || !aligned(d_v, el)) { set_error("misaligned input"); return BS_E_INVAL; }
    a.layer = layer;
    a.n_seqs = n_seqs;
    a.total = total;
    a.max_new = max_new;
    a.seqs = d_seqs;
    a.starts = d_starts;
    a.xk = d_k;
    a.xv = d_v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.f32 = dtype == BS_T_FP32;
    const uint64_t unit = 16 / el;
    a.vec = aligned(d_k, 16) && aligned(d_v, 16) && k_stride % unit == 0 && v_stride % unit == 0 && a.c.dim % 8 == 0;
    return launched(bsk_kv_append(&a, stream), "append");
}

uint64_t bs_kv_attend_work_bytes(const bs_kv_cache* cache, const bs_kv_attend_args* args) {
    bsd::KvAttend a;
    uint32_t chunk, splits;
    if (attend_args(cache, args, a, chunk, splits) != BS_OK || args->n_seqs == 0 || args->total_q == 0) return 0;
    return part_bytes(a, splits);
}

bs_status bs_kv_attend_async(const bs_kv_cache* cache, const bs_kv_attend_args* args, void* d_work, uint64_t work_bytes,
                             void* stream) {
    bsd::KvAttend a;
    uint32_t chunk = 1, splits = 1;
    const bs_status rc = attend_args(cache, args, a, chunk, splits);
    if (rc != BS_OK) return rc;
    if (args->n_seqs == 0 || args->total_q == 0) return BS_OK;
    if (!a.seqs || !a.q || !a.out) { set_error("NULL argument"); return BS_E_INVAL; }
    if (!aligned(a.q, 2) || !aligned(a.out, 2) || !aligned(a.lse, 4)) { set_error("misaligned queries or results"); return BS_E_INVAL; }
    a.chunk = chunk;
    a.splits = 1;
    if (d_work && splits > 1) {
        if (!aligned(d_work, 16)) { set_error("the workspace must be 16-B aligned"); return BS_E_INVAL; }
        if (work_bytes < part_bytes(a, splits)) {
            set_error("workspace of %llu B, %llu B needed", (unsigned long long)work_bytes,
                      (unsigned long long)part_bytes(a, splits));
            return BS_E_INVAL;
        }
        const uint64_t need = part_bytes(a, splits), row = (uint64_t)a.heads * a.c.dim;
        if (overlap(d_work, need, a.out, extent(a.total, a.out_stride, row, 2)) ||
            overlap(d_work, need, a.q, extent(a.total, a.q_stride, row, 2)) ||
            (a.lse && overlap(d_work, need, a.lse, 4ull * a.total * a.heads))) {
            set_error("the workspace overlaps queries or results");
            return BS_E_INVAL;
        }
        a.splits = splits;
        a.counters = (uint32_t*)d_work;
        a.part = (float*)d_work + bsd::kKvCounters;
    }
    return launched(bsk_kv_attend(&a, stream), "attention");
}

uint64_t bs_kv_pages_work_bytes(const bs_kv_cache* cache, uint32_t n) {
    bsd::KvView v;
    if (view(cache, v) != BS_OK || n > kGridYZ) return 0;
    return page_work(v, n);
}

bs_status bs_kv_extend_async(const bs_kv_cache* cache, uint32_t n, const int32_t* d_seqs, const int32_t* d_counts,
                             void* d_work, uint64_t work_bytes, void* stream) {
    bsd::KvPages p;
    const bs_status rc = page_call(cache, n, d_seqs, true, d_counts, true, d_work, work_bytes, p);
    if (rc != BS_OK || n == 0) return rc;
    return launched(bsk_kv_extend(&p, stream), "extend");
}

bs_status bs_kv_fork_async(const bs_kv_cache* cache, uint32_t n, const int32_t* d_parents, const int32_t* d_children,
                           void* d_work, uint64_t work_bytes, void* stream) {
    bsd::KvPages p;
    const bs_status rc = page_call(cache, n, d_parents, true, d_children, true, d_work, work_bytes, p);
    if (rc != BS_OK || n == 0) return rc;
    return launched(bsk_kv_fork(&p, stream), "fork");
}

bs_status bs_kv_free_async(const bs_kv_cache* cache, uint32_t n, const int32_t* d_seqs, void* stream) {
    bsd::KvPages p;
    const bs_status rc = page_call(cache, n, d_seqs, false, nullptr, false, nullptr, 0, p);
    if (rc != BS_OK || n == 0) return rc;
    return launched(bsk_kv_free(&p, stream), "free");
}

bs_status bs_kv_copy_pages_async(const bs_kv_cache* cache, uint32_t n, const int32_t* d_from, const int32_t* d_to,
                                 void* stream) {
    bsd::KvPages p;
    const bs_status rc = page_call(cache, n, d_from, true, d_to, false, nullptr, 0, p);
    if (rc != BS_OK || n == 0) return rc;
    return launched(bsk_kv_copy(&p, stream), "page copy");
}

bs_status bs_kv_compact_async(const bs_kv_cache* cache, int32_t* d_table_out, int32_t* d_refs_out, void* d_work,
                              uint64_t work_bytes, void* stream) {
    bsd::KvPages p;
    const bs_status rc = page_call(cache, 0, nullptr, false, nullptr, true, d_work, work_bytes, p);
    if (rc != BS_OK) return rc;
    if (!d_table_out || !d_refs_out) { set_error("NULL argument"); return BS_E_INVAL; }
    if (p.c.max_seqs > kThreads / 256) { set_error("%u rows (at most 2^24 - 1)", p.c.max_seqs); return BS_E_INVAL; }
    const uint64_t tb = 4ull * p.c.max_seqs * p.c.max_pages, rb = 4ull * p.c.n_pages;
    if (overlap(d_table_out, tb, p.c.table, tb) || overlap(d_refs_out, rb, p.c.refs, rb) ||
        overlap(d_table_out, tb, d_refs_out, rb)) {
        set_error("the new table and counts need buffers of their own");
        return BS_E_INVAL;
    }
    if (!aligned(d_table_out, 4) || !aligned(d_refs_out, 16)) { set_error("a misaligned buffer"); return BS_E_INVAL; }
    p.table_out = d_table_out;
    p.refs_out = d_refs_out;
    return launched(bsk_kv_compact(&p, stream), "compact");
}

}  // extern "C"
