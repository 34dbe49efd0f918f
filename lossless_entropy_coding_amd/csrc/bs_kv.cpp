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
constexpr uint32_t kBatchRows = 16384;       // of a plan, whose every workgroup adds up the counts before its own

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

bs_status check_batch(const bs_kv_batch* b);

// attention of a plan's tokens: `plain` is what it is as attention of rows by themselves
struct Shared {
    bs_kv_attend_args plain;
    bsd::KvShared s;
    uint32_t chunk, splits;     // of the attention of rows by themselves
    uint64_t need;              // bytes of workspace
};

uint64_t part_bytes(const bsd::KvAttend& a, uint32_t splits);

bs_status shared_args(const bs_kv_cache* cache, const bs_kv_attend_args* x, const bs_kv_batch* b, Shared& y) {
    memset(&y, 0, sizeof y);
    const bs_status rc = check_batch(b);
    if (rc != BS_OK) return rc;
    if (!x) { set_error("NULL argument"); return BS_E_INVAL; }
    y.plain = *x;
    y.plain.n_seqs = b->n_seqs;
    y.plain.total_q = b->total;
    y.plain.max_new = b->max_new;
    y.plain.d_seqs = b->d_rows;
    y.plain.d_starts = b->d_starts;
    bsd::KvShared& s = y.s;
    const bs_status at = attend_args(cache, &y.plain, s.a, y.chunk, y.splits);
    if (at != BS_OK || b->n_seqs == 0 || b->total == 0) return at;
    if (s.a.many) {
        y.need = part_bytes(s.a, y.splits);
        return BS_OK;
    }
    s.places = b->d_places;
    s.info = b->d_info;
    s.groups = b->n_groups;
    // row blocks: of 16 rows, or 32 in stacks of kKvStack or more with head_dim
    // up to 128 (a smaller stack has at most two more than it would have then)
    const uint64_t rows = (uint64_t)b->total * s.a.group, groups = b->n_groups;
    uint64_t blocks = (rows + 15 * groups) / 16;
    if (s.a.c.wide <= 128) blocks = std::min(blocks, (rows + 31 * groups) / 32 + 2 * groups);
    s.blocks = groups ? (uint32_t)blocks : 0;
    s.row_blocks = (uint32_t)(((uint64_t)b->max_new * s.a.group + 15) / 16);
    // splits: two workgroups to a CU of each kind, and a tile at least to each
    // of their four waves.  How long the common tokens are is the GPU's to know:
    // either kind may have all of them.  The groups are taken to be alike.  Where
    // the rows alone fill the GPU, the common tokens are split half as often
    // (128 rows in 4 groups: 4 splits 96 us, 2 91).
    int cus = 0;
    if (bsk_device_cus(&cus) != 0 || cus <= 0) cus = 256;
    const uint32_t cap = s.a.c.max_pages * s.a.c.page, len = x->max_len && x->max_len < cap ? x->max_len : cap;
    const uint64_t most = std::max<uint64_t>(1, ((uint64_t)len + 4 * bsd::kKvTile - 1) / (4 * bsd::kKvTile));
    const uint64_t stack = (rows + std::max<uint64_t>(1, groups) - 1) / std::max<uint64_t>(1, groups);
    const uint64_t tall = s.a.c.wide <= 128 && stack >= bsd::kKvStack ? 32 : 16;
    const uint64_t pre = std::max<uint64_t>(1, groups * ((stack + tall - 1) / tall) * s.a.c.kv_heads), own = (uint64_t)b->n_seqs * s.row_blocks * s.a.c.kv_heads;
    s.pre = groups ? (uint32_t)std::min(most, std::max<uint64_t>(1, (own >= 2 * (uint64_t)cus ? 1 : 2) * (uint64_t)cus / pre)) : 0;
    s.own = (uint32_t)std::min(most, std::max<uint64_t>(1, 2 * (uint64_t)cus / own));
    if ((((uint64_t)s.a.c.kv_heads * s.pre + 7) / 8 * 8 * s.blocks + own * s.own) > kThreads / 256 ||
        (uint64_t)b->n_seqs * b->max_new > kThreads / 64) {
        set_error("%u rows of up to %u new tokens are too many for one call (max_new: the most of one row)", b->n_seqs, b->max_new);
        return BS_E_INVAL;
    }
    y.need = 4ull * (bsd::kKvCounters + (uint64_t)b->total * s.a.heads * (s.pre + s.own) * (s.a.c.wide + 4));
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

uint64_t reorder_work(const bsd::KvView& v, uint64_t n) { return align_up(4 * (2 + 6 * n + v.max_seqs), 256); }

// a plan's sizes and buffers
bs_status check_batch(const bs_kv_batch* b) {
    if (!b) { set_error("NULL plan"); return BS_E_INVAL; }
    if (b->n_seqs > kBatchRows || b->n_groups > kBatchRows) {
        set_error("%u rows in %u groups (at most %u)", b->n_seqs, b->n_groups, kBatchRows);
        return BS_E_INVAL;
    }
    if (b->total > 0x7FFFFFFFu || (b->n_seqs == 0 && b->total) || (b->total && (b->max_new == 0 || b->max_new > b->total))) {
        set_error("%u tokens of %u rows, at most %u of one", b->total, b->n_seqs, b->max_new);
        return BS_E_INVAL;
    }
    if (b->reserved) { set_error("reserved must be 0"); return BS_E_INVAL; }
    if (b->n_seqs == 0) return BS_OK;
    if (!b->d_rows || !b->d_starts || (b->total && (!b->d_places || !b->d_slots)) || (b->width && !b->d_table) || !b->d_lead || !b->d_shared ||
        !b->d_info) {
        set_error("NULL buffer in the plan");
        return BS_E_INVAL;
    }
    if (!aligned(b->d_rows, 4) || !aligned(b->d_starts, 4) || !aligned(b->d_places, 4) || !aligned(b->d_slots, 8) || !aligned(b->d_table, 4) ||
        !aligned(b->d_lead, 4) || !aligned(b->d_shared, 4) || !aligned(b->d_info, 16)) {
        set_error("a misaligned buffer in the plan");
        return BS_E_INVAL;
    }
    return BS_OK;
}

struct Range {
    const void* p;
    uint64_t bytes;
};

bool over(const Range& a, const Range& b) { return a.p && b.p && overlap(a.p, a.bytes, b.p, b.bytes); }

// a plan's buffers, its rows first
struct Plan {
    static constexpr int kBuffers = 8;
    Range at[kBuffers];
    explicit Plan(const bs_kv_batch& b)
        : at{{b.d_rows, 4ull * b.n_seqs}, {b.d_starts, 4ull * b.n_seqs + 4}, {b.d_places, 4ull * b.total}, {b.d_slots, 8ull * b.total},
             {b.d_table, 4ull * b.n_seqs * b.width}, {b.d_lead, 4ull * b.n_seqs}, {b.d_shared, 4ull * b.n_seqs},
             {b.d_info, 16 + 32 * ((uint64_t)b.n_groups + b.n_seqs)}} {}
};

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

uint64_t bs_kv_attend_shared_work_bytes(const bs_kv_cache* cache, const bs_kv_attend_args* args, const bs_kv_batch* batch) {
    Shared y;
    return shared_args(cache, args, batch, y) == BS_OK ? y.need : 0;
}

bs_status bs_kv_attend_shared_async(const bs_kv_cache* cache, const bs_kv_attend_args* args, const bs_kv_batch* batch,
                                    void* d_work, uint64_t work_bytes, void* stream) {
    Shared y;
    const bs_status rc = shared_args(cache, args, batch, y);
    if (rc != BS_OK) return rc;
    if (batch->n_seqs == 0 || batch->total == 0) return BS_OK;
    bsd::KvAttend& a = y.s.a;
    for (const Range& x : Plan(*batch).at)
        if (over(x, Range{d_work, y.need})) { set_error("the workspace overlaps the plan"); return BS_E_INVAL; }
    if (a.many) return bs_kv_attend_async(cache, &y.plain, d_work, work_bytes, stream);
    if (!a.q || !a.out) { set_error("NULL argument"); return BS_E_INVAL; }
    if (!aligned(a.q, 2) || !aligned(a.out, 2) || !aligned(a.lse, 4)) { set_error("misaligned queries or results"); return BS_E_INVAL; }
    if (!d_work || !aligned(d_work, 16)) { set_error("a 16-B aligned workspace is needed"); return BS_E_INVAL; }
    if (work_bytes < y.need) {
        set_error("workspace of %llu B, %llu B needed", (unsigned long long)work_bytes, (unsigned long long)y.need);
        return BS_E_INVAL;
    }
    const uint64_t row = (uint64_t)a.heads * a.c.dim;
    if (overlap(d_work, y.need, a.out, extent(a.total, a.out_stride, row, 2)) || overlap(d_work, y.need, a.q, extent(a.total, a.q_stride, row, 2)) ||
        (a.lse && overlap(d_work, y.need, a.lse, 4ull * a.total * a.heads))) {
        set_error("the workspace overlaps queries or results");
        return BS_E_INVAL;
    }
    a.part = (float*)d_work + bsd::kKvCounters;
    return launched(bsk_kv_shared(&y.s, stream), "attention of groups");
}

uint64_t bs_kv_reorder_work_bytes(const bs_kv_cache* cache, uint32_t n) {
    bsd::KvView v;
    if (view(cache, v) != BS_OK || n > bsd::kKvReorder) return 0;
    return reorder_work(v, n);
}

bs_status bs_kv_reorder_async(const bs_kv_cache* cache, uint32_t n, const int32_t* d_rows, const int32_t* d_parents,
                              void* d_work, uint64_t work_bytes, void* stream) {
    bsd::KvPages p;
    memset(&p, 0, sizeof p);
    const bs_status rc = view(cache, p.c);
    if (rc != BS_OK) return rc;
    if (n > bsd::kKvReorder) { set_error("%u rows in one call (at most %u)", n, bsd::kKvReorder); return BS_E_INVAL; }
    if (n == 0) return BS_OK;
    if (!d_rows || !d_parents || !aligned(d_rows, 4) || !aligned(d_parents, 4)) { set_error("NULL or misaligned rows or parents"); return BS_E_INVAL; }
    if (!d_work || !aligned(d_work, 16)) { set_error("a 16-B aligned workspace is needed"); return BS_E_INVAL; }
    if (work_bytes < reorder_work(p.c, n)) {
        set_error("workspace of %llu B, %llu B needed", (unsigned long long)work_bytes, (unsigned long long)reorder_work(p.c, n));
        return BS_E_INVAL;
    }
    if (overlap(d_work, reorder_work(p.c, n), d_rows, 4ull * n) || overlap(d_work, reorder_work(p.c, n), d_parents, 4ull * n)) {
        set_error("the workspace overlaps rows or parents");
        return BS_E_INVAL;
    }
    p.n = n;
    p.a = d_rows;
    p.b = d_parents;
    p.work = (int32_t*)d_work;
    return launched(bsk_kv_reorder(&p, stream), "reorder");
}

bs_status bs_kv_batch_async(const bs_kv_cache* cache, const bs_kv_batch* batch, const int32_t* d_seqs,
                            const int32_t* d_counts, const int32_t* d_groups, void* stream) {
    bsd::KvBatch b;
    memset(&b, 0, sizeof b);
    const bs_status rc = view(cache, b.c);
    if (rc != BS_OK) return rc;
    const bs_status at = check_batch(batch);
    if (at != BS_OK) return at;
    if (batch->n_seqs == 0) return BS_OK;
    if (!d_seqs || !aligned(d_seqs, 4) || !aligned(d_counts, 4) || !aligned(d_groups, 4)) { set_error("NULL or misaligned rows, counts or groups"); return BS_E_INVAL; }
    if (!d_counts && batch->total != batch->n_seqs) {
        set_error("%u tokens for %u rows without counts", batch->total, batch->n_seqs);
        return BS_E_INVAL;
    }
    if (!d_groups && batch->n_groups != 1) { set_error("%u groups without their offsets", batch->n_groups); return BS_E_INVAL; }
    const uint64_t n = batch->n_seqs;
    const Range in[] = {{d_seqs, 4 * n}, {d_counts, 4 * n}, {d_groups, 4ull * batch->n_groups + 4},
                        {cache->d_table, 4ull * b.c.max_seqs * b.c.max_pages}, {cache->d_lens, 4ull * b.c.max_seqs}};
    const Plan out(*batch);
    for (int i = 0; i < Plan::kBuffers; i++) {
        bool bad = false;
        for (const Range& x : in)                                // a plan's own rows may be given
            bad = bad || (over(x, out.at[i]) && !(&x == in && i == 0 && d_seqs == batch->d_rows));
        for (int j = 0; j < i; j++) bad = bad || over(out.at[j], out.at[i]);
        if (bad) { set_error("a buffer of the plan overlaps another of the call, or the cache's"); return BS_E_INVAL; }
    }
    b.n = batch->n_seqs;
    b.groups = batch->n_groups;
    b.total = batch->total;
    b.max_new = batch->max_new;
    b.width = batch->width;
    b.seqs = d_seqs;
    b.counts = d_counts;
    b.offs = d_groups;
    b.rows = batch->d_rows;
    b.starts = batch->d_starts;
    b.places = batch->d_places;
    b.slots = batch->d_slots;
    b.table = batch->d_table;
    b.lead = batch->d_lead;
    b.shared = batch->d_shared;
    b.info = batch->d_info;
    return launched(bsk_kv_batch(&b, stream), "batch");
}

}  // extern "C"
