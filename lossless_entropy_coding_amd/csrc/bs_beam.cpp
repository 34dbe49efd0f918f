// bs_beam.cpp -- host side of the choice of continuations: argument checks,
// launch shapes, and the entry points of bs.h.
#include <hip/hip_runtime.h>
#include <string.h>

#include <algorithm>

#include "bs_beam_device.h"
#include "bs_internal.h"

using namespace bs;

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

constexpr uint64_t kOne = 320;

// the call's sizes, checked; pointers are not looked at.  one: a single launch.
bs_status shape(const bs_beam_args* x, bsd::BeamArgs& a, bool& one) {
    memset(&a, 0, sizeof a);
    if (!x) { set_error("NULL argument"); return BS_E_INVAL; }
    if (x->beams == 0 || x->beams > 64 || x->keep == 0 || x->keep > 128) {
        set_error("%u beams (1..64), the best %u (1..128)", x->beams, x->keep);
        return BS_E_INVAL;
    }
    if ((uint64_t)x->batch * x->beams > 65535) { set_error("%u requests of %u beams (65535 beams in all)", x->batch, x->beams); return BS_E_INVAL; }
    if (x->vocab == 0 || x->vocab > 1000000) { set_error("%u tokens (1..1000000)", x->vocab); return BS_E_INVAL; }
    if (x->type != BS_T_BF16 && x->type != BS_T_FP32) { set_error("logits of type %u", x->type); return BS_E_INVAL; }
    if (x->row_stride < x->vocab || x->row_stride > (1ull << 40)) { set_error("row stride %llu", (unsigned long long)x->row_stride); return BS_E_INVAL; }
    if (!(x->softcap >= 0.f)) { set_error("softcap %g", x->softcap); return BS_E_INVAL; }
    if (x->reserved) { set_error("reserved must be 0"); return BS_E_INVAL; }
    a.batch = x->batch;
    a.beams = x->beams;
    a.keep = x->keep;
    a.vocab = x->vocab;
    a.best = std::min(x->keep, x->vocab);
    a.half = x->type == BS_T_BF16;
    a.eos = x->eos;
    // above 2^100 (infinity, too) c tanh(x / c) is x to 64 bits' precision, and
    // below 2^-100 every capped logit is 0: neither overflows a constant
    a.softcap = x->softcap > 0x1p100f ? 0.f : x->softcap > 0.f ? std::max(x->softcap, 0x1p-100f) : 0.f;
    a.stride = x->row_stride;
    // A part of a row is 512 threads times 1, 2 or 4 vectors (8 of fp32 where 64
    // parts of 4 do not hold a row).  Small parts spread few rows over the GPU,
    // large ones cost less per logit (a part's reductions and list are the same
    // for all).  Up to kOne parts one launch does all (see beam_both_kernel);
    // above, small parts as long as there are no more than five workgroups to a
    // CU.
    const uint32_t per = a.half ? 8 : 4;
    auto cut = [&](uint64_t most) {
        for (a.vectors = 1;; a.vectors *= 2) {
            a.chunks = (x->vocab + per - 1 + bsd::kBeamThreads * per * a.vectors - 1) / (bsd::kBeamThreads * per * a.vectors);
            const uint64_t all = (uint64_t)a.chunks * a.batch * a.beams;
            if (a.chunks <= bsd::kBeamChunks && (all <= most || a.vectors >= 4)) return all <= most && a.vectors <= 2;
        }
    };
    one = cut(kOne);
    if (!one) cut(1280);
    return BS_OK;
}

uint64_t parts_bytes(const bsd::BeamArgs& a) { return align_up((uint64_t)a.batch * a.beams * a.chunks * sizeof(bsd::BeamPart), 256); }

uint64_t work_bytes_of(const bsd::BeamArgs& a) {
    return 4 * bsd::kBeamCounters + align_up(parts_bytes(a) + (uint64_t)a.batch * a.beams * a.chunks * a.best * sizeof(bsd::BeamBest), 256);
}

}  // namespace

extern "C" {

uint64_t bs_beam_work_bytes(const bs_beam_args* args) {
    bsd::BeamArgs a;
    bool one;
    return shape(args, a, one) == BS_OK ? work_bytes_of(a) : 0;
}

bs_status bs_beam_select_async(const bs_beam_args* args, void* d_work, uint64_t work_bytes, void* stream) {
    bsd::BeamArgs a;
    bool one;
    const bs_status rc = shape(args, a, one);
    if (rc != BS_OK) return rc;
    if (a.batch == 0) return BS_OK;
    const bs_beam_args& x = *args;
    if (!x.d_logits || !x.d_scores || !x.d_scores_out || !x.d_tokens || !x.d_parents || !x.d_done_out || !d_work) {
        set_error("NULL argument");
        return BS_E_INVAL;
    }
    if (x.d_done && x.eos < 0) { set_error("beams that are done need the token that ends them"); return BS_E_INVAL; }
    const uint64_t el = a.half ? 2 : 4, rows = (uint64_t)a.batch * a.beams, kept = 4ull * a.batch * a.keep, need = work_bytes_of(a);
    if (!aligned(x.d_logits, el) || !aligned(x.d_scores, 4) || !aligned(x.d_done, 4) || !aligned(x.d_scores_out, 4) ||
        !aligned(x.d_tokens, 4) || !aligned(x.d_parents, 4) || !aligned(x.d_done_out, 4) || !aligned(d_work, 16)) {
        set_error("a misaligned buffer");
        return BS_E_INVAL;
    }
    if (work_bytes < need) {
        set_error("workspace of %llu B, %llu B needed", (unsigned long long)work_bytes, (unsigned long long)need);
        return BS_E_INVAL;
    }
    const struct { const void* p; uint64_t n; } in[] = {{x.d_logits, extent(rows, a.stride, a.vocab, el)}, {x.d_scores, 4 * rows}, {x.d_done, 4 * rows}},
        out[] = {{d_work, need}, {x.d_scores_out, kept}, {x.d_tokens, kept}, {x.d_parents, kept}, {x.d_done_out, kept}};
    for (int i = 0; i < 5; i++) {
        bool bad = false;
        for (const auto& y : in) bad = bad || (y.p && overlap(out[i].p, out[i].n, y.p, y.n));
        for (int j = 0; j < i; j++) bad = bad || overlap(out[i].p, out[i].n, out[j].p, out[j].n);
        if (bad) { set_error("the workspace or a result overlaps another buffer of the call"); return BS_E_INVAL; }
    }
    a.logits = x.d_logits;
    a.scores = x.d_scores;
    a.done = x.d_done;
    a.scores_out = x.d_scores_out;
    a.tokens = x.d_tokens;
    a.parents = x.d_parents;
    a.done_out = x.d_done_out;
    a.counters = one ? (uint32_t*)d_work : nullptr;
    a.parts = (bsd::BeamPart*)((uint32_t*)d_work + bsd::kBeamCounters);
    a.bests = (bsd::BeamBest*)((uint8_t*)a.parts + parts_bytes(a));
    const int e = bsk_beam_select(&a, stream);
    if (e == 0) return BS_OK;
    set_error("selection launch: %s", hipGetErrorString((hipError_t)e));
    return BS_E_HIP;
}

}  // extern "C"
