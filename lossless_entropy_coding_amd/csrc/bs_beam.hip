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
// load.  Of each load the largest logit is kept, of each thread the sum of
// exponentials against its largest so far.  Those logits that are no smaller
// than the K-th largest of the threads' maxima (of 64 groups of threads, if
// K <= 16) go to a list in LDS, read again for it: at least K are that large,
// and few more than K.
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
//
// 512 beams, a tenth of them done, 256000 BF16 logits, a soft cap: 73 us, of
// which launch 1 is 64 (3.7 TB/s; at a copy's rate it would take 50).  Vector
// instructions issue 88% of a busy CU's time: 13 to a logit, of which three
// transcendentals take the time of six.  Few rows are bound by the launches;
// one user's four beams take one launch (beam_both_kernel) and 12 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

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

// x of this lane and of the one 32 (16) away, in either order
struct Pair {
    float a, b;
};

__device__ __forceinline__ Pair swap32(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const uint32_t a = r[0], b = r[1];
    return Pair{__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)};
}

__device__ __forceinline__ Pair swap16(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t a = r[0], b = r[1];
    return Pair{__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)};
}

// the maximum (sum) over a wave, in every lane
__device__ __forceinline__ float wave_max(float x) {
    x = fmaxf(x, dpp<0x128>(x));             // rotations of a row of 16 by 8, 4, 2, 1
    x = fmaxf(x, dpp<0x124>(x));
    x = fmaxf(x, dpp<0x122>(x));
    x = fmaxf(x, dpp<0x121>(x));
    Pair p = swap16(x);
    p = swap32(fmaxf(p.a, p.b));
    return fmaxf(p.a, p.b);
}

__device__ __forceinline__ float wave_sum(float x) {
    x += dpp<0x128>(x);
    x += dpp<0x124>(x);
    x += dpp<0x122>(x);
    x += dpp<0x121>(x);
    Pair p = swap16(x);
    p = swap32(p.a + p.b);
    return p.a + p.b;
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

// The exponential of a logit against a part's reference.
//   CAP 0 (no cap): 2^((x - m) L), L = log2 e in fp32, m the largest logit.
//   CAP 1 (c up to 40): y = c - 2 c r, r = 1 / (e^(2 x / c) + 1); 2^(-B r), B = 2
//     c log2 e in fp32, which is e^(y - c): no less than 2^-116, so that it
//     needs no maximum.
//   CAP 2: 2^((y - y(m)) L).  Where x is below c / 4 y is the series of tanh to
//     the seventh power (the next term is 2^-21.5 of it there): the other
//     form's error is 2^-22 of the cap, whatever the logit.
// reference() is, in 64 bits, what the exponential of the part's largest logit
// was taken against, with what B lost to rounding: the loss is then none
// there, and small near it.
constexpr float kShortCap = 40.f;

struct Capped {
    float c, in, b;
    __device__ __forceinline__ Capped(float cap) : c(cap), in(cap > 0.f ? 2.f * kLog2e / cap : 0.f), b(2.f * cap * kLog2e) {}
    __device__ __forceinline__ float r(float x) const { return __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(x * in) + 1.f); }
    __device__ __forceinline__ float y(float x) const {
        const float u = x / c, u2 = u * u;
        const float p = x * (1.f + u2 * (-1.f / 3 + u2 * (2.f / 15 + u2 * (-17.f / 315))));
        return fabsf(u) < 0.25f ? p : c - 2.f * c * r(x);
    }
};

// what against() takes of the largest logit
template <int CAP>
__device__ __forceinline__ float ref_of(const Capped& k, float top) {
    return CAP == 0 ? top : CAP == 1 ? 0.f : k.y(top);
}

template <int CAP>
__device__ __forceinline__ float against(const Capped& k, float x, float ref) {
    if (CAP == 1) return __builtin_amdgcn_exp2f(k.r(x) * -k.b);
    return __builtin_amdgcn_exp2f(((CAP == 0 ? x : k.y(x)) - ref) * kLog2e);
}

// a capped logit in 64 bits, and r of CAP 1 (whose c is small: c - 2 c r loses
// nothing to speak of near 0)
struct Exact {
    double y, r;
};

template <int CAP>
__device__ __forceinline__ Exact exact(const Capped& k, float x) {
    if (CAP == 0) return Exact{(double)x, 0.};
    const double c = k.c, r = 1. / (exp(2. / c * (double)x) + 1.);
    return Exact{CAP == 1 ? c - 2. * c * r : c * tanh((double)x / c), r};
}

template <int CAP>
__device__ __forceinline__ double reference(const Capped& k, float top, const Exact& e) {
    return CAP == 1 ? e.y + (double)k.b * 0.6931471805599453 * e.r : (double)ref_of<CAP>(k, top);
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

// the logit of such a number (what would be below -infinity is -infinity)
__device__ __forceinline__ float unordered(uint32_t o) {
    const uint32_t u = o & 0x80000000u ? o ^ 0x80000000u : ~o;
    return fmaxf(__builtin_bit_cast(float, u), minus_inf());
}

template <bool THROUGH, typename T>
__device__ __forceinline__ void put(T* to, const T& v) {
    static_assert(sizeof(T) % 8 == 0, "in words of 8 B");
    if (!THROUGH) {
        *to = v;
        return;
    }
    uint64_t w[sizeof(T) / 8];
    __builtin_memcpy(w, &v, sizeof(T));
#pragma unroll
    for (uint32_t i = 0; i < sizeof(T) / 8; i++) __hip_atomic_store((uint64_t*)to + i, w[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Part `chunk` of a row.  THROUGH: its results go through the L2, to be read by
// another workgroup of the same launch.
template <bool HALF, int NV, int CAP, bool THROUGH>
__device__ __forceinline__ void read_part(const BeamArgs& a, uint32_t row, uint32_t chunk) {
    constexpr uint32_t VE = HALF ? 8 : 4, CH = kBeamThreads * NV * VE, NW = kBeamThreads / 64, NL = NV < 4 ? NV : 4;
    __shared__ __attribute__((aligned(16))) float maxima[kBeamThreads];
    __shared__ float sums[NW];
    __shared__ float bound;
    __shared__ uint32_t count, total[2], vectors, low;
    __shared__ uint16_t some[kBeamThreads * NV];
    __shared__ BeamBest list[kList];

    const uint32_t t = threadIdx.x, lane = t & 63u, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    if (a.done && a.done[row] != 0) return;
    if (!(fabsf(a.scores[row]) < __builtin_inff())) return;          // such beams have no continuations
    if (t == 0) count = total[0] = total[1] = vectors = 0;

    // p counts from the 16-B boundary at or before the row's first logit
    constexpr uint32_t esize = HALF ? 2 : 4;
    const uint64_t from = (uint64_t)row * a.stride * esize;
    const uint32_t skip = ((uint32_t)((uintptr_t)a.logits + from) & 15u) / esize, stop = a.vocab + skip;
    const uint8_t* const base = (const uint8_t*)a.logits + from - skip * esize;
    const bool inside = chunk * CH >= skip && chunk * CH + CH <= stop;
    uint32_t again = 0;                                              // 0, but see forget()
    auto place = [&](uint32_t j) { return chunk * CH + (j * kBeamThreads + t) * VE + again; };
    auto load = [&](uint32_t j) { return *(const v4u*)(base + (uint64_t)place(j) * esize); };
    // the same where the part reaches past the row: -infinity there
    auto load_edge = [&](uint32_t j) {
        const uint32_t p = place(j);
        if (p >= skip && p + VE <= stop) return load(j);
        v4u x;
#pragma unroll
        for (uint32_t w = 0; w < 4; w++) {
            if (HALF) {
                const uint32_t e = p + 2 * w;
                const uint32_t lo = e >= skip && e < stop ? ((const uint16_t*)base)[e] : 0xFF80u;
                const uint32_t hi = e + 1 >= skip && e + 1 < stop ? ((const uint16_t*)base)[e + 1] : 0xFF80u;
                x[w] = lo | hi << 16;
            } else {
                const uint32_t e = p + w;
                x[w] = e >= skip && e < stop ? ((const uint32_t*)base)[e] : 0xFF800000u;
            }
        }
        return x;
    };
    // The compiler is not to keep what it has read for when it is read again:
    // it would take the registers of the waves that hide the loads.
    auto forget = [&]() { asm volatile("" : "+v"(again)); };
    auto logit = [&](const v4u& x, uint32_t e) {                     // e-th of a vector
        const uint32_t w = HALF ? x[e / 2] : x[e];
        return __builtin_bit_cast(float, HALF ? (e & 1 ? w & 0xFFFF0000u : w << 16) : w);
    };

    // One pass: each vector's largest logit, the thread's, and its sum against
    // it.  What was read is not kept: few logits are needed again.
    const Capped k(a.softcap);
    float sum = 0.f, best[NV], mine = minus_inf(), ref = 0.f;
    auto take = [&](const v4u& x) {
        float most = minus_inf();
#pragma unroll
        for (uint32_t e = 0; e < VE; e += 2) most = fmaxf(fmaxf(logit(x, e), logit(x, e + 1)), most);
        if (CAP != 1) {
            const float now = fmaxf(mine, most), to = now > minus_inf() ? ref_of<CAP>(k, now) : 0.f;
            sum *= mine > minus_inf() ? __builtin_amdgcn_exp2f((ref - to) * kLog2e) : 1.f;   // nothing yet, or NaN
            ref = to;
        }
        mine = fmaxf(mine, most);
#pragma unroll
        for (uint32_t e = 0; e < VE; e++) {
            const float v = logit(x, e), f = against<CAP>(k, v, ref);
            sum += CAP == 2 && v == minus_inf() ? 0.f : f;
        }
        return most;
    };
    if (inside) {
        v4u x[NL], y[NL];
#pragma unroll
        for (uint32_t j = 0; j < NL; j++) x[j] = load(j);
#pragma unroll
        for (uint32_t j0 = 0; j0 < NV; j0 += NL) {
            if (j0 + NL < NV) {
#pragma unroll
                for (uint32_t j = 0; j < NL; j++) y[j] = load(j0 + NL + j);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (uint32_t j = 0; j < NL; j++) {
                best[j0 + j] = take(x[j]);
                __builtin_amdgcn_sched_barrier(0);                   // few logits at a time: registers for more waves
            }
#pragma unroll
            for (uint32_t j = 0; j < NL; j++) x[j] = y[j];
        }
    } else {
        // whole vectors together, as above, then the one or two that are cut (one
        // after the other: 512 rows of 256000 75 us, 73)
        v4u x[NL];
        auto whole = [&](uint32_t j) { return place(j) >= skip && place(j) + VE <= stop; };
#pragma unroll 1
        for (uint32_t j0 = 0; j0 < NV; j0 += NL) {
#pragma unroll
            for (uint32_t j = 0; j < NL; j++)
                if (whole(j0 + j)) x[j] = load(j0 + j);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (uint32_t j = 0; j < NL; j++) {
                if (whole(j0 + j)) take(x[j]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll 1
        for (uint32_t j = 0; j < NV; j++)
            if (!whole(j) && place(j) < stop && place(j) + VE > skip) take(load_edge(j));
    }
    maxima[t] = mine;
    __syncthreads();
    float group = 0.f, top = 0.f;
    if (CAP != 1 || wave == 0) {
        group = maxima[lane];
#pragma unroll
        for (uint32_t w = 1; w < NW; w++) group = fmaxf(group, maxima[64 * w + lane]);
        top = wave_max(group);
    }
    // The bound of the list: the K-th largest maximum.  Of 64 groups, its upper
    // 26 bits as a whole number that grows with it, the others 0: with the lane
    // in their place no two are equal, and a comparison is one instruction.
    if (a.best <= 16) {
        if (wave == 0) {
            __shared__ __attribute__((aligned(16))) uint32_t keys[64];
            const uint32_t key = (ordered(group) & ~63u) | lane;
            keys[lane] = key;
            uint32_t rank = 0;
#pragma unroll
            for (uint32_t i = 0; i < 64; i += 4) {
                const uint4 o = *(const uint4*)(keys + i);
                rank += (o.x > key) + (o.y > key) + (o.z > key) + (o.w > key);
            }
            if (rank == a.best - 1) bound = unordered(key & ~63u);
        }
    } else if (wave == 0) {
        // of all threads', the upper 22 bits, one after the other
        uint32_t keys[NW], key = 0;
#pragma unroll
        for (uint32_t w = 0; w < NW; w++) keys[w] = ordered(maxima[64 * w + lane]);
        for (uint32_t bit = 1u << 31; bit >= 1u << 10; bit >>= 1) {
            uint32_t n = 0;
#pragma unroll
            for (uint32_t w = 0; w < NW; w++) n += (uint32_t)__builtin_popcountll(__builtin_amdgcn_ballot_w64(keys[w] >= (key | bit)));
            if (n >= a.best) key |= bit;
        }
        if (lane == 0) bound = unordered(key);
    }
    if (CAP != 1) {
        if (mine > minus_inf()) sum *= __builtin_amdgcn_exp2f((ref - ref_of<CAP>(k, top)) * kLog2e);
    } else if (t == 0) {
        low = 2.f * k.c * (1.f - k.r(top)) < 32.f;
    }
    sum = wave_sum(sum);
    if (lane == 0) sums[wave] = sum;
    __syncthreads();
    const float least = bound;
    forget();
    if (CAP == 1 && low) {
        // A logit of -infinity has counted as e^(-2 c).  Where the largest is no
        // more than e^32 of that, a part of 32768 of them would show (2^-30).
        sum = 0.f;
#pragma unroll 1
        for (uint32_t j = 0; j < NV; j++) {
            const v4u x = load_edge(j);
#pragma unroll
            for (uint32_t e = 0; e < VE; e++) {
                const float v = logit(x, e), f = against<1>(k, v, 0.f);
                sum += v == minus_inf() ? 0.f : f;
            }
        }
        sum = wave_sum(sum);
        if (lane == 0) sums[wave] = sum;
        forget();
    }
    auto pick = [&](const v4u& x, uint32_t first) {
#pragma unroll
        for (uint32_t e = 0; e < VE; e++) {
            const float f = logit(x, e);
            if (f >= least && f > minus_inf()) {
                const uint32_t at = atomicAdd(&count, 1u);
                if (at < kList) list[at] = BeamBest{f, first + e - skip};
            }
        }
    };
    if (inside) {
        // The few vectors with such logits side by side first, so that one wave
        // looks through them all (with each by its own wave they took a tenth
        // of the kernel's instructions).
#pragma unroll
        for (uint32_t j = 0; j < NV; j++)
            if (best[j] >= least && best[j] > minus_inf()) some[atomicAdd(&vectors, 1u)] = (uint16_t)(j * kBeamThreads + t);
        __syncthreads();
        for (uint32_t i = t; i < vectors; i += kBeamThreads) {
            const uint32_t p = chunk * CH + some[i] * VE;
            pick(*(const v4u*)(base + (uint64_t)p * esize), p);
        }
    } else if (mine >= least && mine > minus_inf()) {
#pragma unroll 1
        for (uint32_t j = 0; j < NV; j++) pick(load_edge(j), place(j));
    }
    __syncthreads();
    uint32_t n = count;
    if (n > kList) {
        // More than the list holds: the K-th largest logit bit by bit, then
        // among those equal to it the last token that is taken.
        uint32_t turn = 0;
        const uint32_t first = max(chunk * CH, skip), end = min(chunk * CH + CH, stop);
        auto each = [&](auto&& f) {
            for (uint32_t p = first + t; p < end; p += kBeamThreads) {
                const uint32_t w = HALF ? (uint32_t)((const uint16_t*)base)[p] << 16 : ((const uint32_t*)base)[p];
                const float v = __builtin_bit_cast(float, w);
                if (v > minus_inf()) f(v, p - skip);
            }
        };
        auto how_many = [&](auto&& test) {                           // of the part's logits; every thread takes part
            uint32_t c = 0;
            each([&](float v, uint32_t id) { c += test(ordered(v), id); });
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
        each([&](float v, uint32_t id) {
            const uint32_t o = ordered(v);
            if (o > key || (o == key && id <= last)) list[atomicAdd(&count, 1u)] = BeamBest{v, id};
        });
        __syncthreads();
        n = count;
    }
    const uint64_t at = (uint64_t)row * a.chunks + chunk;
    for (uint32_t i = t; i < n; i += kBeamThreads) {
        const BeamBest b = list[i];
        uint32_t rank = 0;
        for (uint32_t j0 = 0; j0 < n; j0 += 8) {                     // (the list's length is a multiple of 8)
            BeamBest o[8];
#pragma unroll
            for (uint32_t j = 0; j < 8; j++) o[j] = list[j0 + j];
#pragma unroll
            for (uint32_t j = 0; j < 8; j++) rank += j0 + j < n && better(o[j], b);
        }
        if (rank < a.best) put<THROUGH>(a.bests + at * a.best + rank, b);
    }
    if (t == 0) {
        float s = 0.f;
#pragma unroll
        for (uint32_t w = 0; w < NW; w++) s += sums[w];
        put<THROUGH>(a.parts + at, BeamPart{top, s, min(n, a.best), 0u});
    }
}

// The best of a request from its beams' parts.  LDS: beams * best scores, then
// as many tokens.
template <int CAP>
__device__ __forceinline__ void choose(const BeamArgs& a, uint32_t request) {
    constexpr uint32_t NW = kBeamThreads / 64;
    extern __shared__ __attribute__((aligned(16))) uint8_t dynamic[];
    __shared__ uint32_t found[64];
    __shared__ BeamBest heads[NW][64][kHeads + 1];                   // one more: lanes on banks of their own
    const uint32_t t = threadIdx.x, lane = t & 63u, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const uint32_t row0 = request * a.beams;
    double* scores = (double*)dynamic;
    uint32_t* tokens = (uint32_t*)(scores + a.beams * a.best);
    const Capped k(a.softcap);

    for (uint32_t w = wave; w < a.beams; w += NW) {
        const uint32_t row = row0 + w;
        // all that the beam may need is asked for at once
        const float score = a.scores[row];
        const int32_t ended = a.done ? a.done[row] : 0;
        const uint64_t mine0 = (uint64_t)row * a.chunks + min(lane, a.chunks - 1);
        BeamPart p = a.parts[mine0];
        const BeamBest* from = a.bests + mine0 * a.best;
        BeamBest early[kHeads];
#pragma unroll
        for (uint32_t i = 0; i < kHeads; i++) early[i] = from[min(i, a.best - 1)];
        double* list = scores + w * a.best;
        uint32_t* ids = tokens + w * a.best;
        uint32_t n = 0;
        if (!(fabsf(score) < __builtin_inff())) {
        } else if (ended != 0) {
            if (lane == 0) {
                list[0] = score;
                ids[0] = (uint32_t)a.eos;
            }
            n = 1;
        } else {
            if (lane >= a.chunks) p = BeamPart{minus_inf(), 0.f, 0u, 0u};
#pragma unroll
            for (uint32_t i = 0; i < kHeads; i++) heads[wave][lane][i] = early[i];
            const float top = wave_max(p.max);
            const bool sound = fabsf(p.sum) < __builtin_inff() && p.max < __builtin_inff();
            if (__builtin_amdgcn_ballot_w64(!sound) == 0 && top > minus_inf()) {
                const Exact best = exact<CAP>(k, p.max > minus_inf() ? p.max : top);
                const double ytop = wave_max(best.y);
                const double part = p.max > minus_inf() ? exp(reference<CAP>(k, p.max, best) - ytop) : 0.;
                double sum = wave_sum((double)p.sum * part);
                // the best of all parts: a lane's own next one, `at` of its list
                uint32_t at = 0;
                BeamBest next = early[0];
                float head = p.n ? next.logit : minus_inf();
                float mine[2] = {0.f, 0.f};                          // best `lane` and `lane + 64`, their tokens and parts
                uint32_t id[2] = {0, 0}, of[2] = {0, 0};
                for (n = 0; n < a.best; n++) {
                    const float m = wave_max(head);
                    if (m == minus_inf()) break;
                    const uint32_t who = (uint32_t)__builtin_ctzll(__builtin_amdgcn_ballot_w64(head == m));   // lower lanes, lower tokens
                    const uint32_t v = (uint32_t)__builtin_amdgcn_readlane((int)next.token, who);
                    if (lane == who) {
                        at++;
                        next = heads[wave][lane][min(at, kHeads - 1)];
                        if (at >= kHeads && at < p.n) next = from[at];
                        head = at < p.n ? next.logit : minus_inf();
                    }
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
                    if (64 * h >= n) break;
                    y[h] = exact<CAP>(k, mine[h]).y;
                    if (CAP) {
                        const float rf = ref_of<CAP>(k, __shfl(p.max, of[h]));
                        const double f = __shfl(part, of[h]);
                        const double more = exp(y[h] - ytop) - (double)against<CAP>(k, mine[h], rf) * f;
                        sum += wave_sum(64 * h + lane < n ? more : 0.);
                    }
                }
                // (differences of logits first: a row may hold the type's lowest
                // value everywhere, beside which a score would be lost)
                const double base = (double)score - log(sum);
#pragma unroll
                for (uint32_t h = 0; h < 2; h++)
                    if (64 * h + lane < n) {
                        list[64 * h + lane] = base + (y[h] - ytop);
                        ids[64 * h + lane] = id[h];
                    }
            }
        }
        for (uint32_t i = n + lane; i < a.best; i += 64) list[i] = -__builtin_inf();
        if (lane == 0) found[w] = n;
    }
    __syncthreads();
    const double inf = __builtin_inf();
    auto write = [&](uint32_t rank, double score, int32_t v, uint32_t w) {
        const uint64_t to = (uint64_t)request * a.keep + rank;
        a.scores_out[to] = (float)score;
        a.tokens[to] = v;
        a.parents[to] = (int32_t)(row0 + w);
        a.done_out[to] = v == a.eos || (a.done && a.done[row0 + w] != 0);
    };
    auto nothing = [&](uint32_t rank) {
        const uint64_t to = (uint64_t)request * a.keep + rank;
        a.scores_out[to] = minus_inf();
        a.tokens[to] = a.parents[to] = -1;
        a.done_out[to] = 0;
    };
    const uint32_t all = a.beams * a.best;
    if (all <= kBeamThreads) {
        // few: each finds its place by counting those before it, shared out
        // over some threads side by side
        uint32_t ls = 0;
        while (ls < 6 && all << (ls + 1) <= kBeamThreads) ls++;
        const uint32_t i = t >> ls, each = (all + (1u << ls) - 1) >> ls, from = (t & ((1u << ls) - 1)) * each, to = min(all, from + each);
        const double mine = i < all ? scores[i] : -inf;
        uint32_t rank = 0, total = 0;
        for (uint32_t j0 = from; j0 < to; j0 += 4) {
            double o[4];
#pragma unroll
            for (uint32_t j = 0; j < 4; j++) o[j] = scores[min(j0 + j, all - 1)];
#pragma unroll
            for (uint32_t j = 0; j < 4; j++) {
                rank += j0 + j < to && (o[j] > mine || (o[j] == mine && j0 + j < i));
                total += j0 + j < to && o[j] > -inf;
            }
        }
        for (uint32_t d = 1; d < 1u << ls; d <<= 1) {
            rank += (uint32_t)__shfl_xor((int)rank, (int)d);
            total += (uint32_t)__shfl_xor((int)total, (int)d);
        }
        if (i >= all || from) return;
        if (mine > -inf && rank < a.keep) write(rank, mine, (int32_t)tokens[i], i / a.best);
        for (uint32_t x = total + i; x < a.keep; x += all) nothing(x);
        return;
    }
    if (wave != 0) return;
    // the beams' lists, a lane each
    const uint32_t n = lane < a.beams ? found[lane] : 0u;
    uint32_t at = 0;
    double head = n ? scores[lane * a.best] : -inf;
    for (uint32_t i = 0; i < a.keep; i++) {
        const double m = wave_max(head);
        if (!(m > -inf)) {
            if (lane == 0) nothing(i);
            continue;
        }
        const uint32_t who = (uint32_t)__builtin_ctzll(__builtin_amdgcn_ballot_w64(head == m));
        if (lane == who) {
            write(i, m, (int32_t)tokens[lane * a.best + at], lane);
            at++;
            head = at < n ? scores[lane * a.best + at] : -inf;
        }
    }
}

// grid: (parts, rows)
template <bool HALF, int NV, int CAP>
__global__ __launch_bounds__(kBeamThreads, CAP == 2 ? 4 : 6) void beam_rows_kernel(BeamArgs a) {
    // Workgroups go to the eight XCDs in turn, and a row's last part, which
    // reaches past the row's end, takes longest: rows begin at different parts,
    // so that those are dealt evenly, whatever power of two their number holds
    // (512 rows of 16 parts: 86 us where one XCD had all last parts, 75).
    const uint32_t step = min(a.chunks & (0u - a.chunks), 8u);
    read_part<HALF, NV, CAP, false>(a, blockIdx.y, (blockIdx.x + blockIdx.y * step / 8) % a.chunks);
}

// grid: requests
template <int CAP>
__global__ __launch_bounds__(kBeamThreads) void beam_choose_kernel(BeamArgs a) {
    choose<CAP>(a, blockIdx.x);
}

// Both in one launch: the workgroup that ends last of a request chooses
// (counters are 0 between calls).  The choice's registers leave room for half
// the waves, so this is for about one workgroup to a CU: 4 beams of 256000
// fp32 (252 of them) 12.9 -> 11.9 us, 80 beams of 50257 (560) 13.6 -> 19.7.
// grid: (parts, rows)
template <bool HALF, int NV, int CAP>
__global__ __launch_bounds__(kBeamThreads, 4) void beam_both_kernel(BeamArgs a) {
    __shared__ uint32_t last;
    read_part<HALF, NV, CAP, true>(a, blockIdx.y, blockIdx.x);
    const uint32_t request = blockIdx.y / a.beams;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (threadIdx.x == 0)
        last = __hip_atomic_fetch_add(a.counters + request, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.beams * a.chunks - 1;
    __syncthreads();
    if (!last) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    if (threadIdx.x == 0) __hip_atomic_store(a.counters + request, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    choose<CAP>(a, request);
}

template <bool HALF, int CAP>
void both(const BeamArgs& a, hipStream_t st) {
    const dim3 grid(a.chunks, a.batch * a.beams), block(kBeamThreads);
    const uint32_t lds = a.beams * a.best * 12;
    if (a.counters) {
        switch (a.vectors) {
            case 1: hipLaunchKernelGGL((beam_both_kernel<HALF, 1, CAP>), grid, block, lds, st, a); break;
            default: hipLaunchKernelGGL((beam_both_kernel<HALF, 2, CAP>), grid, block, lds, st, a); break;
        }
        return;
    }
    switch (a.vectors) {
        case 1: hipLaunchKernelGGL((beam_rows_kernel<HALF, 1, CAP>), grid, block, 0, st, a); break;
        case 2: hipLaunchKernelGGL((beam_rows_kernel<HALF, 2, CAP>), grid, block, 0, st, a); break;
        case 4: hipLaunchKernelGGL((beam_rows_kernel<HALF, 4, CAP>), grid, block, 0, st, a); break;
        default: hipLaunchKernelGGL((beam_rows_kernel<false, 8, CAP>), grid, block, 0, st, a); break;   // fp32
    }
    hipLaunchKernelGGL(beam_choose_kernel<CAP>, dim3(a.batch), block, lds, st, a);
}

}  // namespace

extern "C" int bsk_beam_select(const BeamArgs* a, void* stream) {
    hipStream_t st = (hipStream_t)stream;
    if (!(a->softcap > 0.f)) a->half ? both<true, 0>(*a, st) : both<false, 0>(*a, st);
    else if (a->softcap <= kShortCap) a->half ? both<true, 1>(*a, st) : both<false, 1>(*a, st);
    else a->half ? both<true, 2>(*a, st) : both<false, 2>(*a, st);
    return (int)hipGetLastError();
}
