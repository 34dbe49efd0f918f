// bs_kv_attend_device.h -- what the attention kernels over the paged 8-bit
// key/value cache have in common (gfx950): operands from codes, sums over a
// wave's lane groups, what a row sees, partial results.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bs_kv_device.h"

namespace {

using namespace bsd;

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 1024.f;              // sum of a lane's exponentials above which a new maximum is looked for

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Soft cap: top tanh(y), y = t ln2 / 2, top the cap in powers of 2.  The
// kernels' own form, top - 2 top / (2^t + 1), is right to 2^-22 of the cap,
// whatever the logit: up to a cap of 256 that is 2^-14, far below the BF16
// rounding of a probability.  Above (CAP), the series to y^7 takes over below
// 1/4 (the next term is 2^-21.5 of it there), so that the error is 2^-20 of
// the logit.  Where rows are many it costs a third more (2 prompts of 2048
// tokens over 8000, 40 heads on 8 of 128 channels, e4m3: 827 us with a cap of
// 256 or less, 1112 above; 4 x 131071 tokens of int8: 208 either way), and in
// one kernel with the other form it would slow that down, too (827 us to
// 875): hence kernels of their own.
constexpr float kShortCap = 256.f;

__device__ __forceinline__ float capped(float t, float top) {
    const float e = top - 2.f * top * __builtin_amdgcn_rcpf(exp2_fast(t) + 1.f);
    const float y = t * (0.5f * kLn2), y2 = y * y;
    const float p = top * y * (1.f + y2 * (-1.f / 3 + y2 * (2.f / 15 + y2 * (-17.f / 315))));
    return fabsf(y) < 0.25f ? p : e;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2 r = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, r);
}

// four 8-bit codes times a power of two to four BF16 (exact)
template <bool E4M3>
__device__ __forceinline__ v2u widen4(uint32_t c, float scale) {
    if (E4M3) {
        const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, scale, false);
        const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, scale, true);
        return v2u{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
    }
    const float a = (float)(int8_t)c, b = (float)(int8_t)(c >> 8), d = (float)(int8_t)(c >> 16), e = (float)(int8_t)(c >> 24);
    return v2u{pack_bf16(a * scale, b * scale), pack_bf16(d * scale, e * scale)};
}

template <bool E4M3>
__device__ __forceinline__ bf16x8 widen8(uint32_t a, uint32_t b, float scale = 1.f) {
    const v2u x = widen4<E4M3>(a, scale), y = widen4<E4M3>(b, scale);
    return __builtin_bit_cast(bf16x8, v4u{x.x, x.y, y.x, y.y});
}

// x of this lane and of the lane 32 (16) away, in either order: the swap
// exchanges halves (rows) between two copies.  (The elements go through
// variables of their own: a bit cast of a vector's element reads element 0.)
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

// maximum and sum over the four lane groups (lanes l, l + 16, l + 32, l + 48)
__device__ __forceinline__ float max_groups(float x) {
    Pair p = swap32(x);
    p = swap16(fmaxf(p.a, p.b));
    return fmaxf(p.a, p.b);
}

__device__ __forceinline__ float sum_groups(float x) {
    Pair p = swap32(x);
    p = swap16(p.a + p.b);
    return p.a + p.b;
}

// One sequence's part of a call, checked.
struct Seq {
    int32_t row, s0, count, len;    // cache row, first query token, query tokens, length
    bool ok;
};

__device__ __forceinline__ Seq get_seq(const KvAttend& a, uint32_t i) {
    Seq s;
    s.row = a.seqs[i];
    s.s0 = a.starts ? a.starts[i] : (int32_t)i;
    const int32_t s1 = a.starts ? a.starts[i + 1] : (int32_t)i + 1;
    s.count = s1 - s.s0;
    s.ok = s.s0 >= 0 && s1 >= s.s0 && (uint32_t)s1 <= a.total && (uint32_t)s.count <= a.max_new;
    if (!s.ok) s.count = 0;
    s.len = 0;
    if (s.row >= 0 && (uint32_t)s.row < a.c.max_seqs)
        s.len = (int32_t)min((uint64_t)(uint32_t)max(a.c.lens[s.row], 0), (uint64_t)a.c.max_pages << a.c.lp);
    else s.ok = false;
    return s;
}

// the tiles that rows at places lo .. hi (lo may be negative) of a sequence see:
// tiles 0 .. ns - 1 and t0 .. t1 - 1
struct Tiles {
    uint32_t ns, t0, n;             // n: how many in all
    __device__ __forceinline__ uint32_t at(uint32_t i) const { return i < ns ? i : t0 + (i - ns); }
};

__device__ __forceinline__ Tiles get_tiles(const KvAttend& a, int32_t lo, int32_t hi) {
    Tiles t{0, 0, 0};
    if (hi < 0) return t;
    const uint32_t t1 = (uint32_t)hi / kKvTile + 1;
    if (a.window) {
        const int64_t first = max((int64_t)max(lo, 0) - (int64_t)a.window + 1, (int64_t)0);
        t.t0 = (uint32_t)first / kKvTile;
        t.ns = min((uint32_t)(((uint64_t)a.sinks + kKvTile - 1) / kKvTile), t.t0);
    }
    t.n = t.ns + (t1 - t.t0);
    return t;
}

// a query's channels 64 x + 16 g + 8 y ..: 8 values, zeros past head_dim.
// Every load goes out at once, from a place inside the row.
template <int DW>
__device__ __forceinline__ void load_q(const KvAttend& a, uint32_t tok, uint32_t qh, uint32_t g, bf16x8 (&q)[DW][2]) {
    const uint32_t dim = a.c.dim;
    const uint16_t* qp = a.q + (uint64_t)tok * a.q_stride + (uint64_t)qh * dim;
    if (a.aligned) {                                                // dim is a multiple of 8
        v4u w[2 * DW];
#pragma unroll
        for (uint32_t x = 0; x < 2 * DW; x++) w[x] = *(const v4u*)(qp + min(64 * (x >> 1) + 16 * g + 8 * (x & 1u), dim - 8));
#pragma unroll
        for (uint32_t x = 0; x < 2 * DW; x++) {
            const bool in = 64 * (x >> 1) + 16 * g + 8 * (x & 1u) < dim;
            q[x >> 1][x & 1u] = __builtin_bit_cast(bf16x8, v4u{in ? w[x].x : 0u, in ? w[x].y : 0u, in ? w[x].z : 0u, in ? w[x].w : 0u});
        }
        return;
    }
#pragma unroll
    for (uint32_t x = 0; x < 2 * DW; x++) {
        uint32_t u[8];
        const uint32_t d = 64 * (x >> 1) + 16 * g + 8 * (x & 1u);
#pragma unroll
        for (uint32_t e = 0; e < 8; e++) u[e] = qp[min(d + e, dim - 1)];
#pragma unroll
        for (uint32_t e = 0; e < 8; e++) u[e] = d + e < dim ? u[e] : 0u;
        q[x >> 1][x & 1u] = __builtin_bit_cast(bf16x8, v4u{u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16});
    }
}

__device__ __forceinline__ void store_through(float* p, float a, float b) {
    const uint64_t v = (uint64_t)__builtin_bit_cast(uint32_t, a) | (uint64_t)__builtin_bit_cast(uint32_t, b) << 32;
    __hip_atomic_store((uint64_t*)p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Four channels of a row's result from channel ch, the row's maximum and the
// sum of its exponentials: to the workspace, or divided to the output.
// THROUGH: stores that other XCDs see once they are done.
template <int DW, bool THROUGH>
__device__ __forceinline__ void part_write(const KvAttend& a, uint32_t tok, uint32_t qh, uint32_t split, uint32_t ch, float top,
                                           float total, f32x4 v) {
    constexpr uint32_t D = 64 * DW;
    float* pp = a.part + (((uint64_t)tok * a.heads + qh) * a.splits + split) * (D + 4);
    if (THROUGH) {
        store_through(pp + ch, v[0], v[1]);
        store_through(pp + ch + 2, v[2], v[3]);
        if (ch == 0) store_through(pp + D, top, total);
        return;
    }
    *(f32x4*)(pp + ch) = v;
    if (ch == 0) {
        pp[D] = top;
        pp[D + 1] = total;
    }
}

__device__ __forceinline__ void out_write(const KvAttend& a, uint32_t tok, uint32_t qh, uint32_t ch, float top, float total, f32x4 v) {
    const uint32_t dim = a.c.dim;
    const float inv = total == 0.f ? 0.f : 1.f / total;             // a sum of NaN is no empty row's: NaN stays
    uint16_t* op = a.out + (uint64_t)tok * a.out_stride + (uint64_t)qh * dim;
    const uint32_t lo = pack_bf16(v[0] * inv, v[1] * inv), hi = pack_bf16(v[2] * inv, v[3] * inv);
    if (a.out8 && ch + 4 <= dim) {
        *(v2u*)(op + ch) = v2u{lo, hi};
    } else {
        if (ch < dim) op[ch] = (uint16_t)lo;
        if (ch + 1 < dim) op[ch + 1] = (uint16_t)(lo >> 16);
        if (ch + 2 < dim) op[ch + 2] = (uint16_t)hi;
        if (ch + 3 < dim) op[ch + 3] = (uint16_t)(hi >> 16);
    }
    if (a.lse && ch == 0) a.lse[(uint64_t)tok * a.heads + qh] = total == 0.f ? -__builtin_inff() : (top + __builtin_amdgcn_logf(total)) * kLn2;
}

// Four channels of a row from its n parts, in order, 8 loads at a time.
template <int DW>
__device__ __forceinline__ void join_row(const KvAttend& a, uint32_t tok, uint32_t qh, uint32_t ch, uint32_t n) {
    constexpr uint32_t D = 64 * DW;
    const float* pp = a.part + ((uint64_t)tok * a.heads + qh) * a.splits * (D + 4);
    float top = -__builtin_inff();
    for (uint32_t s0 = 0; s0 < n; s0 += 8) {
        float f[8];
#pragma unroll
        for (uint32_t u = 0; u < 8; u++) f[u] = pp[min(s0 + u, n - 1) * (D + 4) + D];
#pragma unroll
        for (uint32_t u = 0; u < 8; u++) top = fmaxf(top, f[u]);
    }
    const float sub = top == -__builtin_inff() ? 0.f : top;
    float total = 0.f;
    f32x4 o = f32x4{0.f, 0.f, 0.f, 0.f};
    for (uint32_t s0 = 0; s0 < n; s0 += 8) {
        f32x4 v[8];
        float f[8], l[8];
#pragma unroll
        for (uint32_t u = 0; u < 8; u++) {
            const float* ps = pp + min(s0 + u, n - 1) * (D + 4);
            v[u] = *(const f32x4*)(ps + ch);
            f[u] = ps[D];
            l[u] = ps[D + 1];
        }
#pragma unroll
        for (uint32_t u = 0; u < 8; u++) {
            const float w = s0 + u < n ? exp2_fast(f[u] - sub) : 0.f;
            total += w * l[u];
            o += w * v[u];
        }
    }
    out_write(a, tok, qh, ch, top, total, o);
}

}  // namespace
