// bs_beam.hip -- the best continuations of a request's beams (gfx950).
//
// Of all tokens v of all beams w of a request, the `keep` with the largest
//
//   score_w + y_wv - log sum_v exp(y_wv),   y = logit, or c tanh(logit / c).
//
// Within a beam that order is the logits' own, so only a beam's `keep` largest
// logits can be among them, and nothing needs to be sorted but these.
//
// Launch 1, a workgroup per part of a row: the part is read once, 16 B to a
// load, and stays in registers.  A first pass finds its maximum, a second adds
// the exponentials against it, and those logits that are no smaller than the
// K-th largest of the threads' maxima (of 64 groups of threads, if K <= 16) go
// to a list in LDS: at least K logits are that large, and few more than K.
// Their ranks follow by counting.  Where a part has more of them than the list
// holds (rows of one value, say), the K-th largest is found bit by bit.
//
// Launch 2, a workgroup per request: a wave per beam joins the parts' sums and
// takes the best from the heads of their lists, in turn; then one wave does the
// same with the beams' lists.  Scores and what they are made of have 64 bits:
// 16 bits of a logit or 24 of a sum would decide between beams by their
// rounding.  The exponentials are fp32 ones (their rounding is 2^-24 of t in
// exp t, weighted by exp t itself), except under a soft cap, where 2^-24 of the
// cap is lost in the reciprocal of tanh: there the terms of a beam's best
// tokens, those that its sum is made of, are put right in 64 bits.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bs_beam_device.h"

using namespace bsd;

namespace {

typedef unsigned int v4u __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kList = 1024;             // logits that a part's list holds
constexpr uint32_t kHeads = 8;               // of a part's best that launch 2 keeps in LDS

__device__ __forceinline__ float minus_inf() { return -__builtin_inff(); }

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}

// the maximum (sum) over a wave, in every lane
__device__ __forceinline__ float wave_max(float x) {
    x = fmaxf(x, dpp<0x128>(x));             // rotations of a row of 16 by 8, 4, 2, 1
    x = fmaxf(x, dpp<0x124>(x));
    x = fmaxf(x, dpp<0x122>(x));
    x = fmaxf(x, dpp<0x121>(x));
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}

__device__ __forceinline__ float wave_sum(float x) {
    x += dpp<0x128>(x);
    x += dpp<0x124>(x);
    x += dpp<0x122>(x);
    x += dpp<0x121>(x);
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
    for (int s = 32; s; s >>= 1) x += __shfl_xor(x, s);
    return x;
}

__device__ __forceinline__ double wave_max(double x) {
#pragma unroll
    for (int s = 32; s; s >>= 1) {
        const double y = __shfl_xor(x, s);
        x = y > x ? y : x;
    }
    return x;
}

// The exponential of a logit against a part's reference.  Without a cap (CAP
// 0) the reference is the largest logit.  With one of up to 256 (CAP 1), y =
// c - 2 c r, r = 1 / (e^(2 x / c) + 1), and exp(y - y_ref) = 2^(ref - B r) with
// B = 2 c log2 e and ref = B r of the largest logit: one rounding, and what ref
// loses to it is the same in every term.  Its error grows with the cap, so
// above (CAP 2) the series of tanh to the seventh power takes over where x is
// below c / 4 (the next term is 2^-21.5 of it there), and ref is y of the
// largest logit.
constexpr float kShortCap = 256.f;

struct Capped {
    float c, in, b;
    __device__ __forceinline__ Capped(float cap) : c(cap), in(cap > 0.f ? 2.f * kLog2e / cap : 0.f), b(2.f * cap * kLog2e) {}
    __device__ __forceinline__ float r(float x) const { return __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(x * in) + 1.f); }
    __device__ __forceinline__ float y(float x) const {
        const float u = x / c, u2 = u * u;
        const float p = x * (1.f + u2 * (-1.f / 3 + u2 * (2.f / 15 + u2 * (-17.f / 315))));
        return fabsf(u) < 0.25f ? p : c - 2.f * c * r(x);
    }
    template <int CAP>
    __device__ __forceinline__ float ref(float top) const { return CAP == 0 ? top : CAP == 1 ? b * r(top) : y(top); }
};

template <int CAP>
__device__ __forceinline__ float against(const Capped& k, float x, float ref) {
    if (CAP == 0) return __builtin_amdgcn_exp2f((x - ref) * kLog2e);
    const float t = CAP == 1 ? __builtin_fmaf(-k.b, k.r(x), ref) : (k.y(x) - ref) * kLog2e;
    return x == minus_inf() ? 0.f : __builtin_amdgcn_exp2f(t);
}

// larger logits first, of equal ones the lower token
__device__ __forceinline__ bool better(const BeamBest& a, const BeamBest& b) {
    return a.logit > b.logit || (a.logit == b.logit && a.token < b.token);
}

// a whole number that grows with the logit (both zeros alike)
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// grid: (parts, rows)
template <bool HALF, int NV, int CAP>
__global__ __launch_bounds__(kBeamThreads) void beam_rows_kernel(BeamArgs a) {
    constexpr uint32_t VE = HALF ? 8 : 4, E = NV * VE, CH = kBeamThreads * E, NW = kBeamThreads / 64;
    __shared__ __attribute__((aligned(16))) float maxima[kBeamThreads];
    __shared__ float sums[NW];
    __shared__ float bound;
    __shared__ uint32_t count, total[2];
    __shared__ BeamBest list[kList];

    const uint32_t t = threadIdx.x, lane = t & 63u, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const uint32_t row = blockIdx.y, chunk = blockIdx.x;
    if (a.done && a.done[row] != 0) return;
    if (!(fabsf(a.scores[row]) < __builtin_inff())) return;          // such beams have no continuations
    if (t == 0) count = total[0] = total[1] = 0;

    // p counts from the 16-B boundary at or before the row's first logit
    constexpr uint32_t esize = HALF ? 2 : 4;
    const uint8_t* base = (const uint8_t*)a.logits + (uint64_t)row * a.stride * esize;
    const uint32_t skip = ((uint32_t)(uintptr_t)base & 15u) / esize, stop = a.vocab + skip;
    base -= skip * esize;
    const uint32_t p0 = chunk * CH + t * VE;
    v4u x[NV];
#pragma unroll
    for (uint32_t j = 0; j < NV; j++) {
        const uint32_t p = p0 + j * kBeamThreads * VE;
        if (p >= skip && p + VE <= stop) {
            x[j] = *(const v4u*)(base + (uint64_t)p * esize);
            continue;
        }
#pragma unroll
        for (uint32_t w = 0; w < 4; w++) {                           // the ends of a row, and what is past it
            if (HALF) {
                const uint32_t e = p + 2 * w;
                const uint32_t lo = e >= skip && e < stop ? ((const uint16_t*)base)[e] : 0xFF80u;
                const uint32_t hi = e + 1 >= skip && e + 1 < stop ? ((const uint16_t*)base)[e + 1] : 0xFF80u;
                x[j][w] = lo | hi << 16;
            } else {
                const uint32_t e = p + w;
                x[j][w] = e >= skip && e < stop ? ((const uint32_t*)base)[e] : 0xFF800000u;
            }
        }
    }
    auto logit = [&](uint32_t e) {                                   // e-th of the thread's
        const uint32_t w = HALF ? x[e / 8][e % 8 / 2] : x[e / 4][e % 4];
        return __builtin_bit_cast(float, HALF ? (e & 1 ? w & 0xFFFF0000u : w << 16) : w);
    };
    auto token = [&](uint32_t e) { return p0 + (e / VE) * kBeamThreads * VE + e % VE - skip; };

    float mine = minus_inf();
#pragma unroll
    for (uint32_t e = 0; e < E; e++) mine = fmaxf(mine, logit(e));
    maxima[t] = mine;
    __syncthreads();
    float group = maxima[lane];
#pragma unroll
    for (uint32_t w = 1; w < NW; w++) group = fmaxf(group, maxima[64 * w + lane]);
    const float top = wave_max(group);
    // the bound of the list: of equal maxima the lower place counts as the larger
    if (a.best <= 16) {
        if (wave == 0) {
            uint32_t rank = 0;
#pragma unroll
            for (uint32_t i = 0; i < 64; i++) {
                const float o = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, group), i));
                rank += o > group || (o == group && i < lane);
            }
            if (rank == a.best - 1) bound = group;
        }
    } else {
        uint32_t rank = 0;
        for (uint32_t i = 0; i < kBeamThreads; i += 4) {
            const float4 o = *(const float4*)(maxima + i);
            rank += (o.x > mine || (o.x == mine && i < t)) + (o.y > mine || (o.y == mine && i + 1 < t)) +
                    (o.z > mine || (o.z == mine && i + 2 < t)) + (o.w > mine || (o.w == mine && i + 3 < t));
        }
        if (rank == a.best - 1) bound = mine;
    }
    const Capped k(a.softcap);
    const float ref = k.ref<CAP>(top);
    float sum = 0.f;
    if (top > minus_inf()) {
#pragma unroll
        for (uint32_t e = 0; e < E; e++) sum += against<CAP>(k, logit(e), ref);
    } else {                                                         // nothing is left, or all of it is NaN
#pragma unroll
        for (uint32_t e = 0; e < E; e++) sum += logit(e) == minus_inf() ? 0.f : __builtin_nanf("");
    }
    sum = wave_sum(sum);
    if (lane == 0) sums[wave] = sum;
    __syncthreads();
    const float least = bound;
    if (mine >= least && mine > minus_inf()) {
#pragma unroll
        for (uint32_t e = 0; e < E; e++) {
            const float f = logit(e);
            if (f >= least && f > minus_inf()) {
                const uint32_t at = atomicAdd(&count, 1u);
                if (at < kList) list[at] = BeamBest{f, token(e)};
            }
        }
    }
    __syncthreads();
    uint32_t n = count;
    if (n > kList) {
        // more than the list holds: the K-th largest logit bit by bit, then
        // among those equal to it the last token that is taken
        uint32_t turn = 0;
        auto how_many = [&](auto test) {                             // of the part's logits; every thread takes part
            uint32_t c = 0;
#pragma unroll
            for (uint32_t e = 0; e < E; e++) {
                const float f = logit(e);
                c += f > minus_inf() && test(ordered(f), token(e));
            }
#pragma unroll
            for (int s = 32; s; s >>= 1) c += __shfl_xor(c, s);
            if (lane == 0) atomicAdd(&total[turn & 1], c);
            __syncthreads();
            const uint32_t all = total[turn & 1];
            turn++;
            if (t == 0) total[turn & 1] = 0;
            __syncthreads();
            return all;
        };
        uint32_t key = 0, last = 0;
        for (uint32_t bit = 1u << 31; bit; bit >>= 1)
            if (how_many([&](uint32_t o, uint32_t) { return o >= (key | bit); }) >= a.best) key |= bit;
        const uint32_t equal = a.best - how_many([&](uint32_t o, uint32_t) { return o > key; });
        for (uint32_t bit = 1u << 20; bit; bit >>= 1)
            if (how_many([&](uint32_t o, uint32_t v) { return o == key && v < (last | bit); }) < equal) last |= bit;
        if (t == 0) count = 0;
        __syncthreads();
#pragma unroll
        for (uint32_t e = 0; e < E; e++) {
            const float f = logit(e);
            const uint32_t o = ordered(f), v = token(e);
            if (f > minus_inf() && (o > key || (o == key && v <= last))) list[atomicAdd(&count, 1u)] = BeamBest{f, v};
        }
        __syncthreads();
        n = count;
    }
    const uint64_t at = (uint64_t)row * a.chunks + chunk;
    for (uint32_t i = t; i < n; i += kBeamThreads) {
        const BeamBest b = list[i];
        uint32_t rank = 0;
        for (uint32_t j = 0; j < n; j++) rank += better(list[j], b);
        if (rank < a.best) a.bests[at * a.best + rank] = b;
    }
    if (t == 0) {
        float s = 0.f;
#pragma unroll
        for (uint32_t w = 0; w < NW; w++) s += sums[w];
        a.parts[at] = BeamPart{top, ref, s, min(n, a.best)};
    }
}

// grid: requests.  LDS: beams * best scores, then as many tokens
template <int CAP>
__global__ __launch_bounds__(kBeamThreads) void beam_merge_kernel(BeamArgs a) {
    constexpr uint32_t NW = kBeamThreads / 64;
    extern __shared__ __attribute__((aligned(16))) uint8_t dynamic[];
    __shared__ uint32_t found[64];
    __shared__ BeamBest heads[NW][64][kHeads + 1];                   // one more: lanes on banks of their own
    const uint32_t t = threadIdx.x, lane = t & 63u, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const uint32_t row0 = blockIdx.x * a.beams;
    double* scores = (double*)dynamic;
    uint32_t* tokens = (uint32_t*)(scores + a.beams * a.best);
    const Capped k(a.softcap);
    const double c = a.softcap;
    auto cap = [&](double x) { return CAP ? c * tanh(x / c) : x; };

    for (uint32_t w = wave; w < a.beams; w += NW) {
        const uint32_t row = row0 + w;
        const float score = a.scores[row];
        double* list = scores + w * a.best;
        uint32_t* ids = tokens + w * a.best;
        uint32_t n = 0;
        if (!(fabsf(score) < __builtin_inff())) {
        } else if (a.done && a.done[row] != 0) {
            if (lane == 0) {
                list[0] = score;
                ids[0] = (uint32_t)a.eos;
            }
            n = 1;
        } else {
            BeamPart p{minus_inf(), 0.f, 0.f, 0u};
            const BeamBest* from = a.bests + ((uint64_t)row * a.chunks + lane) * a.best;
            if (lane < a.chunks) {
                p = a.parts[(uint64_t)row * a.chunks + lane];
                for (uint32_t i = 0; i < min(p.n, kHeads); i++) heads[wave][lane][i] = from[i];
            }
            const float top = wave_max(p.max);
            const bool sound = fabsf(p.sum) < __builtin_inff() && p.max < __builtin_inff();
            if (__builtin_amdgcn_ballot_w64(!sound) == 0 && top > minus_inf()) {
                const double ytop = cap(top), ref = CAP == 1 ? c - 2. * c * ((double)p.ref / (double)k.b) : (double)p.ref;
                const double part = p.max > minus_inf() ? exp(ref - ytop) : 0.;
                double sum = wave_sum((double)p.sum * part);
                // the best of all parts: a lane's own next one, `at` of its list
                uint32_t at = 0;
                float head = p.n ? heads[wave][lane][0].logit : minus_inf();
                float mine[2] = {0.f, 0.f};                          // best `lane` and `lane + 64`, their tokens and parts
                uint32_t id[2] = {0, 0}, of[2] = {0, 0};
                for (n = 0; n < a.best; n++) {
                    const float m = wave_max(head);
                    if (m == minus_inf()) break;
                    const uint32_t who = (uint32_t)__builtin_ctzll(__builtin_amdgcn_ballot_w64(head == m));   // lower lanes, lower tokens
                    uint32_t v = 0;
                    if (lane == who) {
                        v = (at < kHeads ? heads[wave][lane][at] : from[at]).token;
                        at++;
                        head = at < p.n ? (at < kHeads ? heads[wave][lane][at] : from[at]).logit : minus_inf();
                    }
                    v = (uint32_t)__builtin_amdgcn_readlane((int)v, who);
                    if (lane == n) {
                        mine[0] = m;
                        id[0] = v;
                        of[0] = who;
                    } else if (lane + 64 == n) {
                        mine[1] = m;
                        id[1] = v;
                        of[1] = who;
                    }
                }
                double y[2];
#pragma unroll
                for (uint32_t h = 0; h < 2; h++) {
                    y[h] = cap(mine[h]);
                    if (CAP) {
                        const float rf = __shfl(p.ref, of[h]);
                        const double f = __shfl(part, of[h]);
                        const double more = exp(y[h] - ytop) - (double)against<CAP>(k, mine[h], rf) * f;
                        sum += wave_sum(64 * h + lane < n ? more : 0.);
                    }
                }
                const double base = (double)score - ytop - log(sum);
#pragma unroll
                for (uint32_t h = 0; h < 2; h++)
                    if (64 * h + lane < n) {
                        list[64 * h + lane] = base + y[h];
                        ids[64 * h + lane] = id[h];
                    }
            }
        }
        if (lane == 0) found[w] = n;
    }
    __syncthreads();
    if (wave != 0) return;
    // the beams' lists, a lane each
    const uint32_t n = lane < a.beams ? found[lane] : 0u;
    const double inf = __builtin_inf();
    uint32_t at = 0;
    double head = n ? scores[lane * a.best] : -inf;
    for (uint32_t i = 0; i < a.keep; i++) {
        const double m = wave_max(head);
        const uint64_t to = (uint64_t)blockIdx.x * a.keep + i;
        if (!(m > -inf)) {
            if (lane == 0) {
                a.scores_out[to] = minus_inf();
                a.tokens[to] = a.parents[to] = -1;
                a.done_out[to] = 0;
            }
            continue;
        }
        const uint32_t who = (uint32_t)__builtin_ctzll(__builtin_amdgcn_ballot_w64(head == m));
        if (lane == who) {
            const int32_t v = (int32_t)tokens[lane * a.best + at];
            at++;
            head = at < n ? scores[lane * a.best + at] : -inf;
            a.scores_out[to] = (float)m;
            a.tokens[to] = v;
            a.parents[to] = (int32_t)(row0 + lane);
            a.done_out[to] = v == a.eos || (a.done && a.done[row0 + lane] != 0);
        }
    }
}

template <bool HALF, int CAP>
void rows(const BeamArgs& a, hipStream_t st) {
    const dim3 grid(a.chunks, a.batch * a.beams), block(kBeamThreads);
    switch (a.vectors) {
        case 1: hipLaunchKernelGGL((beam_rows_kernel<HALF, 1, CAP>), grid, block, 0, st, a); break;
        case 2: hipLaunchKernelGGL((beam_rows_kernel<HALF, 2, CAP>), grid, block, 0, st, a); break;
        case 4: hipLaunchKernelGGL((beam_rows_kernel<HALF, 4, CAP>), grid, block, 0, st, a); break;
        default: hipLaunchKernelGGL((beam_rows_kernel<HALF, 8, CAP>), grid, block, 0, st, a); break;
    }
}

template <int CAP>
void both(const BeamArgs& a, hipStream_t st) {
    a.half ? rows<true, CAP>(a, st) : rows<false, CAP>(a, st);
    hipLaunchKernelGGL(beam_merge_kernel<CAP>, dim3(a.batch), dim3(kBeamThreads), a.beams * a.best * 12, st, a);
}

}  // namespace

extern "C" int bsk_beam_select(const BeamArgs* a, void* stream) {
    hipStream_t st = (hipStream_t)stream;
    if (!(a->softcap > 0.f)) both<0>(*a, st);
    else if (a->softcap <= kShortCap) both<1>(*a, st);
    else both<2>(*a, st);
    return (int)hipGetLastError();
}
