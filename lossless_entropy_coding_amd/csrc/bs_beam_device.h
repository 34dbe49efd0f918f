// bs_beam_device.h -- structures shared by the host side of the library and
// the kernels that choose continuations (gfx950).  Not part of the public C
// ABI.
#pragma once
#include <stdint.h>

namespace bsd {

constexpr uint32_t kBeamThreads = 512;       // of a workgroup
constexpr uint32_t kBeamCounters = 1024;     // words before a workspace's parts
constexpr uint32_t kBeamChunks = 64;         // parts of a row at most: one to a lane of the second launch

// what the first launch leaves of a part of a row, before its best logits
struct BeamPart {
    float max;       // the largest logit, uncapped
    float sum;       // of the exponentials against it (see bs_beam.hip); not finite where a logit is not
    uint32_t n;      // how many of the best follow
    uint32_t unused;
};

struct BeamBest {
    float logit;
    uint32_t token;
};

struct BeamArgs {
    uint32_t batch, beams, keep, vocab;
    uint32_t best;              // of a row: min(keep, vocab)
    uint32_t chunks, vectors;   // parts of a row; 16-B vectors of a thread
    int half;                   // BF16 (else fp32)
    int32_t eos;
    float softcap;              // 0: none
    uint64_t stride;            // elements between rows
    const void* logits;
    const float* scores;
    const int32_t* done;
    float* scores_out;
    int32_t* tokens;
    int32_t* parents;
    int32_t* done_out;
    uint32_t* counters;         // of the requests, where one launch does all; else null
    BeamPart* parts;            // [batch * beams][chunks]
    BeamBest* bests;            // [batch * beams][chunks][best], best first
};

}  // namespace bsd

// Launcher (bs_beam.hip): a hipError_t as int.
extern "C" int bsk_beam_select(const bsd::BeamArgs* a, void* stream);
