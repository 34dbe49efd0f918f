// bs_kv.hip -- the paged 8-bit key/value cache (gfx950): storing new tokens,
// and the upkeep of its pages.  Layouts and rules are in bs.h.
//
// append: one workgroup per (touched page, head, side).  The scale of a page
// is a power of two, so x / scale and the change from an old scale to a new
// one are exact in fp32 and each stored value is rounded once (ties to even),
// whatever the order of the tokens.
//
// Pages: a page is free when its count is 0, and the lowest free page is
// taken first, so the state after any sequence of calls is one value and no
// list of free pages has to be kept.  extend and fork allocate in a single
// workgroup (a scan over the counts, 4096 at a time, that ends with the last
// page wanted); the copies and the rows of the table are filled by as many
// workgroups as they need.
//
// Measured: copies run at a large copy's rate (compaction of 42 layers, 0.7 GB
// read and as much written: 290 us, 4.8 TB/s; fork's copies of 42 layers, 32
// children: 29 us).  A scan of 1000 pages' counts takes 3 to 6 us, a chain of
// loads and barriers, so one workgroup: calls on few rows are bound by that
// and by their launches.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "bs_kv_device.h"

using namespace bsd;

namespace {

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));

enum : uint32_t {
    kStPages = 1, kStRow = 2, kStId = 4, kStBusy = 8, kStValue = 16, kStCount = 32
};

__device__ __forceinline__ void flag(uint32_t* status, uint32_t bit) {
    if (status) atomicOr(status, bit);
}

__device__ __forceinline__ float load_x(const void* x, uint64_t i, int f32) {
    if (f32) return ((const float*)x)[i];
    return __builtin_bit_cast(float, (uint32_t)((const uint16_t*)x)[i] << 16);
}

// the least exponent e >= -60 with amax <= Q 2^e: with amax = m 2^x, m in
// [1, 2), Q = 1.75 2^8 (e4m3) or 127/64 2^6 (int8); amax 0 gives -60
__device__ __forceinline__ int need_exp(float amax, bool e4m3) {
    if (!(amax > 0.f)) return -60;
    const uint32_t b = __builtin_bit_cast(uint32_t, amax);
    const int x = (int)(b >> 23) - 127;
    const uint32_t m = b & 0x7FFFFFu;
    const int e = e4m3 ? x - 8 + (m > 0x600000u) : x - 6 + (m > 0x7E0000u);
    return e < -60 ? -60 : e;
}

__device__ __forceinline__ float pow2(int e) { return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23); }

// nearest code (ties to even) of y, |y| within the type's range
__device__ __forceinline__ uint32_t to_code(float y, bool e4m3) {
    if (e4m3) {
        y = fminf(fmaxf(y, -448.f), 448.f);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y, y, 0, false) & 0xFFu;
    }
    y = fminf(fmaxf(rintf(y), -127.f), 127.f);
    return (uint32_t)(int)y & 0xFFu;
}

__device__ __forceinline__ float of_code(uint32_t c, bool e4m3) {
    if (e4m3) return __builtin_amdgcn_cvt_f32_fp8((int)c, 0);
    return (float)(int)(int8_t)(c & 0xFFu);
}

// four codes times f (a power of two, at most 1), rounded again; bytes past
// the first n stay as they are
template <bool E4M3>
__device__ __forceinline__ uint32_t again4(uint32_t c, float f, int32_t n) {
    if (n <= 0) return c;
    uint32_t r = 0;
#pragma unroll
    for (int b = 0; b < 4; b++) r |= to_code(of_code(c >> (8 * b), E4M3) * f, E4M3) << (8 * b);
    const uint32_t keep = n >= 4 ? 0u : ~0u << (8 * n);
    return (r & ~keep) | (c & keep);
}

// 8 values of the input from element i
template <bool F32>
__device__ __forceinline__ void load8(const void* x, uint64_t i, float* v) {
    if (F32) {
        const v4f a = *(const v4f*)((const float*)x + i), b = *(const v4f*)((const float*)x + i + 4);
#pragma unroll
        for (int e = 0; e < 4; e++) {
            v[e] = a[e];
            v[4 + e] = b[e];
        }
    } else {
        const v4u a = *(const v4u*)((const uint16_t*)x + i);
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const uint32_t w = a[e];
            v[2 * e] = __builtin_bit_cast(float, w << 16);
            v[2 * e + 1] = __builtin_bit_cast(float, w & 0xFFFF0000u);
        }
    }
}

template <bool E4M3>
__device__ __forceinline__ uint32_t code_of(float v, float inv) {
    return to_code(v != v ? 0.f : v * inv, E4M3);
}

// four codes as the bytes of a word
template <bool E4M3>
__device__ __forceinline__ uint32_t codes4(float a, float b, float d, float e, float inv) {
    if (!E4M3)
        return code_of<false>(a, inv) | code_of<false>(b, inv) << 8 | code_of<false>(d, inv) << 16 | code_of<false>(e, inv) << 24;
    auto in = [&](float v) { return v != v ? 0.f : fminf(fmaxf(v * inv, -448.f), 448.f); };
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(in(a), in(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(in(d), in(e), lo, true);
}

// 8 values of the input as they are in memory
template <bool F32>
struct Raw {
    v4u w[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* x, uint64_t i) {
        const v4u* p = (const v4u*)((const uint8_t*)x + i * (F32 ? 4 : 2));
#pragma unroll
        for (int k = 0; k < (F32 ? 2 : 1); k++) w[k] = p[k];
    }
    __device__ __forceinline__ float at(int e) const {
        const uint32_t u = F32 ? w[F32 ? e >> 2 : 0][e & 3] : w[0][e >> 1];
        return __builtin_bit_cast(float, F32 ? u : (e & 1) ? u & 0xFFFF0000u : u << 16);
    }
};

constexpr uint32_t kHeld = 8;                // 8-channel loads that a thread keeps

// grid: (pages a sequence can touch x 2 kv_heads, sequences), the heads and
// sides of a page next to each other: together they read whole rows of the
// input.  The page's new tokens are needed twice, for the largest magnitude
// and for the codes.  VEC: rows of the input can be read 16 B at a time; a
// thread then takes 8 channels of a token at a time, and keeps them in
// registers where a page fits (up to 16384 values: 64 tokens of 256 channels).
// Values go out channel by channel: a thread takes four tokens on end, whose
// codes are a word of each channel, and the words pass through LDS so that 16
// tokens of a channel are stored at once.  Larger pages and other inputs are
// read twice (the second time from the L2).
//
// Memory bounds it: 4 prompts of up to 8191 tokens (8 heads of 128 channels,
// e4m3), 158 MB, in 40 us, 3.9 TB/s; read twice, with a page's heads far
// apart, it took 46.  A decode step of 64 sequences is a chain of dependent
// loads (row, length, page, scale): 6.8 us.
template <bool E4M3, bool VEC, bool F32>
__global__ __launch_bounds__(256) void append_kernel(KvAppend a) {
    const KvView& c = a.c;
    const uint32_t t = threadIdx.x, seq_i = blockIdx.y, page_i = blockIdx.x / (2 * c.kv_heads);
    const uint32_t head = (blockIdx.x - page_i * 2 * c.kv_heads) >> 1, side = blockIdx.x & 1u;
    const int32_t row = a.seqs[seq_i];
    const int32_t s0 = a.starts ? a.starts[seq_i] : (int32_t)seq_i;
    const int32_t s1 = a.starts ? a.starts[seq_i + 1] : (int32_t)seq_i + 1;
    if (row < 0 || (uint32_t)row >= c.max_seqs) {
        if (t == 0) flag(c.status, kStId);
        return;
    }
    const int32_t len = c.lens[row];
    if (s0 < 0 || s1 < s0 || (uint32_t)s1 > a.total || s1 - s0 > len || (uint32_t)(s1 - s0) > a.max_new) {
        if (t == 0) flag(c.status, kStId);
        return;
    }
    if (s1 == s0) return;
    const uint32_t begin = (uint32_t)(len - (s1 - s0));      // the first new token's place
    const uint32_t pg = (begin >> c.lp) + page_i;
    if ((uint64_t)pg << c.lp >= (uint32_t)len) return;
    if (pg >= c.max_pages) {
        if (t == 0) flag(c.status, kStRow);
        return;
    }
    const int32_t pid = c.table[(uint64_t)row * c.max_pages + pg];             // looked at after the first pass
    const uint32_t lo = max(begin, pg << c.lp) - (pg << c.lp);                 // the page's new slots
    const uint32_t hi = min((uint32_t)len - (pg << c.lp), c.page);
    const void* x = side ? a.xv : a.xk;
    const uint64_t xs = side ? a.v_stride : a.k_stride;
    // the input's element of slot 0, channel 0 of the page (slots below lo are not read)
    const int64_t x0 = ((int64_t)s0 + (int64_t)(pg << c.lp) - (int64_t)begin) * (int64_t)xs + (int64_t)head * c.dim;
    const uint32_t nt = hi - lo, d8 = c.dim / 8, w8 = c.wide / 8;
    const bool there = pid >= 0 && (uint32_t)pid < c.n_pages;
    float* sp = c.scale + (((uint64_t)a.layer * c.n_pages + (there ? (uint32_t)pid : 0u)) * c.kv_heads + head) * 2 + side;
    const float old = lo && there ? *sp : 0.f;
    const bool held = VEC && c.page * d8 <= 256 * kHeld;
    const uint32_t q0 = lo / 4, nq = (hi + 3) / 4 - q0;                        // quads of slots
    const bool quads = side && nt >= 4;
    const uint32_t most = quads ? 4 * ((nq * d8 + 255) / 256) : (nt * d8 + 255) / 256;   // accesses of a thread
    Raw<F32> raw[kHeld];

    // the largest finite magnitude
    float m = 0.f;
    bool odd = false;
    // access u of the thread: its slot and its channels 8 g ..
    auto access = [&](uint32_t u, uint32_t& slot, uint32_t& g) {
        if (quads) {
            const uint32_t i = t + 256 * (u >> 2), q = i / d8;
            slot = 4 * (q0 + q) + (u & 3u);
            g = i - q * d8;
            return q < nq && slot >= lo && slot < hi;
        }
        const uint32_t i = t + 256 * u, tk = i / d8;
        slot = lo + tk;
        g = i - tk * d8;
        return tk < nt;
    };
    if (held) {
#pragma unroll
        for (uint32_t u = 0; u < kHeld; u++) {
            if (u >= most) break;
            uint32_t slot, g;
#pragma unroll
            for (int k = 0; k < (F32 ? 2 : 1); k++) raw[u].w[k] = v4u{0, 0, 0, 0};
            if (access(u, slot, g)) raw[u].load(x, (uint64_t)(x0 + (int64_t)((uint64_t)slot * xs + 8 * g)));
        }
#pragma unroll
        for (uint32_t u = 0; u < kHeld; u++) {
            if (u >= most) break;
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float v = fabsf(raw[u].at(e));
                if (v < __builtin_inff()) m = fmaxf(m, v);
                else odd = true;
            }
        }
    } else if (VEC) {
        for (uint32_t i = t; i < nt * d8; i += 256) {
            const uint32_t tk = i / d8, g = i - tk * d8;
            float v[8];
            load8<F32>(x, (uint64_t)(x0 + (int64_t)((uint64_t)(lo + tk) * xs + 8 * g)), v);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float u = fabsf(v[e]);
                if (u < __builtin_inff()) m = fmaxf(m, u);
                else odd = true;
            }
        }
    } else {
        for (uint32_t i = t; i < nt * c.dim; i += 256) {
            const uint32_t tk = i / c.dim, d = i - tk * c.dim;
            const float v = fabsf(load_x(x, (uint64_t)(x0 + (int64_t)((uint64_t)(lo + tk) * xs + d)), F32));
            if (v < __builtin_inff()) m = fmaxf(m, v);
            else odd = true;
        }
    }
    if (odd) flag(c.status, kStValue);
    if (!there) {
        if (t == 0) flag(c.status, kStId);
        return;
    }
    __shared__ float red[4];
#pragma unroll
    for (int s = 32; s; s >>= 1) m = fmaxf(m, __shfl_xor(m, s));
    if ((t & 63u) == 0) red[t >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float now = fmaxf(old, pow2(need_exp(m, E4M3)));
    const float inv = 1.f / now;                                               // exact: a power of two
    uint8_t* base = (side ? c.v : c.k) + ((uint64_t)a.layer * c.n_pages + (uint32_t)pid) * c.side_bytes +
                    (uint64_t)head * c.page * c.wide;
    if (lo && old < now) {                                                     // older tokens: rounded again
        const float f = old * inv;
        // 16 B at a time: lo rows of keys on end; of each channel of values the chunks that begin below lo
        const uint32_t per = side ? (lo + 15) / 16 : 0, n = side ? c.wide * per : lo * c.wide / 16;
        for (uint32_t i = t; i < n; i += 256) {
            const uint32_t ch = side ? i / per : 0, q = side ? i - ch * per : 0;
            v4u* p = (v4u*)(base + (side ? ch * c.page + 16 * q : 16 * i));
            const int32_t keep = side ? (int32_t)(lo - 16 * q) : 16;
            v4u w = *p;
#pragma unroll
            for (int e = 0; e < 4; e++) w[e] = again4<E4M3>(w[e], f, keep - 4 * e);
            *p = w;
        }
        __syncthreads();                                                       // before new tokens of the same chunks
    }
    if (held && !quads) {
#pragma unroll
        for (uint32_t u = 0; u < kHeld; u++) {
            if (u >= most) break;
            uint32_t slot, g;
            if (!access(u, slot, g)) continue;
            uint32_t r[2];
#pragma unroll
            for (int e = 0; e < 2; e++)
                r[e] = codes4<E4M3>(raw[u].at(4 * e), raw[u].at(4 * e + 1), raw[u].at(4 * e + 2), raw[u].at(4 * e + 3), inv);
            if (side == 0) *(v2u*)(base + slot * c.wide + 8 * g) = v2u{r[0], r[1]};
            else
#pragma unroll
                for (int e = 0; e < 8; e++) base[(8 * g + e) * c.page + slot] = (uint8_t)(r[e >> 2] >> (8 * (e & 3)));
        }
        for (uint32_t i = t; i < nt * (w8 - d8); i += 256) {                   // zeros past dim
            const uint32_t tk = i / (w8 - d8), g = d8 + i - tk * (w8 - d8);
            if (side == 0) *(v2u*)(base + (lo + tk) * c.wide + 8 * g) = v2u{0u, 0u};
            else
                for (uint32_t e = 0; e < 8; e++) base[(8 * g + e) * c.page + lo + tk] = 0;
        }
    } else if (held) {
        // word q of channel n at n (nq + 1) + q: at most 32 quads more than the page's words
        __shared__ uint32_t words[64 * kHeld * 8 + 256];
#pragma unroll
        for (uint32_t u = 0; u < kHeld; u += 4) {
            const uint32_t i = t + 64 * u, q = i / d8, g = i - q * d8;
            if (q < nq) {
#pragma unroll
                for (int e = 0; e < 8; e++)
                    words[(8 * g + e) * (nq + 1) + q] =
                        codes4<E4M3>(raw[u].at(e), raw[u + 1].at(e), raw[u + 2].at(e), raw[u + 3].at(e), inv);
            }
        }
        __syncthreads();
        const uint32_t c0 = lo / 16, nc = (hi + 15) / 16 - c0;                 // 16 slots of a channel at a time
        for (uint32_t i = t; i < c.wide * nc; i += 256) {
            const uint32_t n = i / nc, first = 16 * (c0 + i - n * nc);
            uint8_t* p = base + n * c.page + first;
            uint32_t w[4];
#pragma unroll
            for (uint32_t k = 0; k < 4; k++) {
                const uint32_t q = first / 4 + k - q0;                         // wraps where the chunk begins before lo
                w[k] = n < c.dim && q < nq ? words[n * (nq + 1) + q] : 0u;
            }
            if (first >= lo && first + 16 <= hi) {
                *(v4u*)p = v4u{w[0], w[1], w[2], w[3]};
            } else {
#pragma unroll
                for (uint32_t b = 0; b < 16; b++)
                    if (first + b >= lo && first + b < hi) p[b] = (uint8_t)(w[b / 4] >> (8 * (b & 3u)));
            }
        }
    } else if (VEC && side == 0) {
        for (uint32_t i = t; i < nt * w8; i += 256) {
            const uint32_t tk = i / w8, g = i - tk * w8;
            uint32_t r[2] = {0u, 0u};
            if (g < d8) {
                float v[8];
                load8<F32>(x, (uint64_t)(x0 + (int64_t)((uint64_t)(lo + tk) * xs + 8 * g)), v);
#pragma unroll
                for (int e = 0; e < 8; e++) r[e >> 2] |= code_of<E4M3>(v[e], inv) << (8 * (e & 3));
            }
            *(v2u*)(base + (lo + tk) * c.wide + 8 * g) = v2u{r[0], r[1]};
        }
    } else if (VEC) {
        for (uint32_t i = t; i < nq * w8; i += 256) {
            const uint32_t g = i / nq, q = q0 + (i - g * nq);
            uint32_t r[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
            for (uint32_t k = 0; k < 4; k++) {
                const uint32_t slot = 4 * q + k;
                if (g < d8 && slot >= lo && slot < hi) {
                    float v[8];
                    load8<F32>(x, (uint64_t)(x0 + (int64_t)((uint64_t)slot * xs + 8 * g)), v);
#pragma unroll
                    for (int e = 0; e < 8; e++) r[e] |= code_of<E4M3>(v[e], inv) << (8 * k);
                }
            }
            uint8_t* p = base + 8 * g * c.page + 4 * q;
            if (4 * q >= lo && 4 * q + 4 <= hi) {
#pragma unroll
                for (int e = 0; e < 8; e++) *(uint32_t*)(p + e * c.page) = r[e];
            } else {
                for (uint32_t k = 0; k < 4; k++)
                    if (4 * q + k >= lo && 4 * q + k < hi) {
#pragma unroll
                        for (int e = 0; e < 8; e++) p[e * c.page + k] = (uint8_t)(r[e] >> (8 * k));
                    }
            }
        }
    } else {
        for (uint32_t i = t; i < nt * c.wide; i += 256) {
            const uint32_t d = side ? i / nt : i % c.wide, s = lo + (side ? i - d * nt : i / c.wide);
            uint32_t r = 0;
            if (d < c.dim) r = code_of<E4M3>(load_x(x, (uint64_t)(x0 + (int64_t)((uint64_t)s * xs + d)), F32), inv);
            base[side ? d * c.page + s : s * c.wide + d] = (uint8_t)r;
        }
    }
    if (t == 0) *sp = now;
}

// ------------------------------------------------------------------ pages
constexpr uint32_t kScan = 1024;             // threads of the allocating workgroup

// exclusive prefix over the workgroup of v, and its total.  CAP: sums stop at
// `cap` (at most 2^28 + 1; less than cap is exact, and so are its prefixes):
// 1024 rows of up to 2^27 pages each would pass 32 bits
template <bool CAP = false>
__device__ __forceinline__ uint32_t block_prefix(uint32_t v, uint32_t* sums, uint32_t& total, uint32_t cap = 0) {
    const uint32_t t = threadIdx.x, lane = t & 63u, w = t >> 6;
    if (CAP) v = min(v, cap);
    uint32_t x = v;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
        const uint32_t y = __shfl_up(x, s);
        if (lane >= (uint32_t)s) x = CAP ? min(x + y, cap) : x + y;
    }
    __syncthreads();
    if (lane == 63) sums[w] = x;
    __syncthreads();
    uint32_t before = 0;                         // of up to 15 waves
    std::conditional_t<CAP, uint64_t, uint32_t> all = 0;
    for (uint32_t i = 0; i < blockDim.x / 64; i++) {
        const uint32_t y = sums[i];
        if (i < w) before += y;
        all += y;
    }
    total = CAP ? (uint32_t)min((uint64_t)all, (uint64_t)cap) : (uint32_t)all;
    return before + x - v;
}

// The lowest `want` free pages, in order, to list; returns how many there
// are (at most want).
__device__ uint32_t find_free(const KvView& c, uint32_t want, int32_t* list, uint32_t* sums) {
    uint32_t got = 0;
    for (uint32_t base = 0; base < c.n_pages && got < want; base += 4 * kScan) {
        const uint32_t i = base + 4 * threadIdx.x;
        uint32_t f[4], n = 0;
#pragma unroll
        for (uint32_t k = 0; k < 4; k++) {
            f[k] = i + k < c.n_pages && c.refs[i + k] == 0;
            n += f[k];
        }
        uint32_t total;
        uint32_t at = got + block_prefix(n, sums, total);
#pragma unroll
        for (uint32_t k = 0; k < 4; k++)
            if (f[k]) {
                if (at < want) list[at] = (int32_t)(i + k);
                at++;
            }
        got += total;
    }
    return min(got, want);
}

__device__ __forceinline__ uint32_t pages_of(const KvView& c, uint32_t tokens) { return (tokens + c.page - 1) >> c.lp; }

// work: [0] 1 if the call goes through, [1..] the free pages found, then for
// each row the first of them that is its own, then its length before the
// call (read once: a row that is named twice cannot take a page that was not
// counted)
// extend: rows a[i] grow by b[i] tokens
// fork: children b[i] of rows a[i]
template <bool FORK>
__global__ __launch_bounds__(kScan) void alloc_kernel(KvPages p) {
    const KvView& c = p.c;
    __shared__ uint32_t sums[kScan / 64];
    __shared__ uint32_t bad;
    const uint32_t t = threadIdx.x;
    if (t == 0) bad = 0;
    __syncthreads();
    int32_t* list = p.work + 1;
    int32_t* offs = list + c.n_pages;
    int32_t* lens = offs + p.n;
    uint32_t total = 0;
    for (uint32_t base = 0; base < p.n; base += kScan) {
        const uint32_t i = base + t;
        uint32_t need = 0, err = 0;
        int32_t had = 0;
        if (i < p.n) {
            const int32_t r = p.a[i], x = p.b[i];
            if (r < 0 || (uint32_t)r >= c.max_seqs) err = kStId;
            else if (FORK) {
                if (x < 0 || (uint32_t)x >= c.max_seqs || x == r) err = kStId;
                else if (c.lens[x] != 0) err = kStBusy;
                else {
                    had = max(c.lens[r], 0);
                    if (pages_of(c, (uint32_t)had) > c.max_pages) err = kStRow;
                    else need = ((uint32_t)had & (c.page - 1)) != 0;
                }
            } else {
                had = max(c.lens[r], 0);
                const int64_t to = (int64_t)had + x;
                if (x < 0) err = kStId;
                else if (to > (int64_t)c.max_pages << c.lp) err = kStRow;
                else need = pages_of(c, (uint32_t)to) - pages_of(c, (uint32_t)had);
            }
        }
        if (err) atomicOr(&bad, err);
        uint32_t sum;
        const uint32_t at = block_prefix<true>(need, sums, sum, c.n_pages + 1);
        if (i < p.n) {
            offs[i] = (int32_t)(total + at);
            lens[i] = had;
        }
        total += sum;
        if (total > c.n_pages) {               // the same in every thread
            if (t == 0) atomicOr(&bad, (uint32_t)kStPages);
            break;
        }
    }
    __syncthreads();
    const bool early = bad != 0;
    const uint32_t got = early ? 0 : find_free(c, total, list, sums);
    __syncthreads();
    const bool ok = !early && got == total;
    if (t == 0) {
        p.work[0] = ok;
        if (!ok) flag(c.status, early ? bad : (uint32_t)kStPages);
    }
    if (!ok) return;
    if (FORK) {
        for (uint32_t i = t; i < p.n; i += kScan) {
            const uint32_t dst = (uint32_t)p.b[i], len = (uint32_t)lens[i];
            if (len & (c.page - 1)) {
                const int32_t pg = list[offs[i]];
                c.refs[pg] = 1;
                c.table[(uint64_t)dst * c.max_pages + (len >> c.lp)] = pg;
            }
            c.lens[dst] = (int32_t)len;
        }
    } else {
        // page j of the list goes to the last row whose first page is not after j
        for (uint32_t j = t; j < total; j += kScan) {
            uint32_t lo = 0, hi = p.n;
            while (hi - lo > 1) {
                const uint32_t mid = (lo + hi) / 2;
                if ((uint32_t)offs[mid] <= j) lo = mid;
                else hi = mid;
            }
            const uint32_t r = (uint32_t)p.a[lo];
            const uint32_t col = pages_of(c, (uint32_t)lens[lo]) + (j - (uint32_t)offs[lo]);
            c.table[(uint64_t)r * c.max_pages + col] = list[j];
            c.refs[list[j]] = 1;
        }
        __syncthreads();
        for (uint32_t i = t; i < p.n; i += kScan) {
            c.lens[p.a[i]] = lens[i] + p.b[i];
        }
    }
}

// copies part of one page (keys, values, scales) of one layer
__device__ __forceinline__ void copy_page(const KvView& c, uint64_t layer, uint32_t from, uint32_t to, uint32_t part,
                                          uint32_t parts) {
    const uint64_t n16 = c.side_bytes / 16;
    const v4u* ks = (const v4u*)(c.k + (layer * c.n_pages + from) * c.side_bytes);
    const v4u* vs = (const v4u*)(c.v + (layer * c.n_pages + from) * c.side_bytes);
    v4u* kd = (v4u*)(c.k + (layer * c.n_pages + to) * c.side_bytes);
    v4u* vd = (v4u*)(c.v + (layer * c.n_pages + to) * c.side_bytes);
    const uint64_t step = (uint64_t)parts * 256;
    for (uint64_t i = (uint64_t)part * 256 + threadIdx.x; i < n16; i += step) {
        const v4u x = ks[i], y = vs[i];
        kd[i] = x;
        vd[i] = y;
    }
    if (part == 0)
        for (uint32_t i = threadIdx.x; i < 2 * c.kv_heads; i += 256)
            c.scale[(layer * c.n_pages + to) * c.kv_heads * 2 + i] = c.scale[(layer * c.n_pages + from) * c.kv_heads * 2 + i];
}

// fork's second half: x < parts copies of the last page per layer, then the
// rows of the table.  grid: (layers * parts + 1, pairs)
__global__ __launch_bounds__(256) void fork_fill_kernel(KvPages p, uint32_t parts) {
    const KvView& c = p.c;
    if (!p.work[0]) return;
    const uint32_t i = blockIdx.y;
    const uint32_t src = (uint32_t)p.a[i], dst = (uint32_t)p.b[i];
    const uint32_t len = (uint32_t)c.lens[dst], whole = len >> c.lp;
    const int32_t* from = c.table + (uint64_t)src * c.max_pages;
    int32_t* to = c.table + (uint64_t)dst * c.max_pages;
    if (blockIdx.x == c.layers * parts) {
        for (uint32_t j = threadIdx.x; j < whole; j += 256) {
            const int32_t pid = from[j];
            to[j] = pid;
            if (pid >= 0 && (uint32_t)pid < c.n_pages) atomicAdd(c.refs + pid, 1);
            else flag(c.status, kStId);
        }
        return;
    }
    if ((len & (c.page - 1)) == 0) return;
    const int32_t s = from[whole], d = to[whole];
    if (s < 0 || (uint32_t)s >= c.n_pages || d < 0 || (uint32_t)d >= c.n_pages) {
        if (threadIdx.x == 0) flag(c.status, kStId);
        return;
    }
    copy_page(c, blockIdx.x / parts, (uint32_t)s, (uint32_t)d, blockIdx.x % parts, parts);
}

// grid: rows
__global__ __launch_bounds__(256) void free_kernel(KvPages p) {
    const KvView& c = p.c;
    __shared__ int32_t len;
    const int32_t r = p.a[blockIdx.x];
    if (r < 0 || (uint32_t)r >= c.max_seqs) {
        if (threadIdx.x == 0) flag(c.status, kStId);
        return;
    }
    if (threadIdx.x == 0) len = atomicExch(c.lens + r, 0);   // a row named twice is freed once
    __syncthreads();
    const uint32_t n = min(pages_of(c, (uint32_t)max(len, 0)), c.max_pages);
    for (uint32_t j = threadIdx.x; j < n; j += 256) {
        const int32_t pid = c.table[(uint64_t)r * c.max_pages + j];
        if (pid < 0 || (uint32_t)pid >= c.n_pages) {
            flag(c.status, kStId);
        } else if (atomicSub(c.refs + pid, 1) <= 0) {
            atomicAdd(c.refs + pid, 1);
            flag(c.status, kStCount);
        }
    }
}

// grid: (layers * parts, pages)
__global__ __launch_bounds__(256) void copy_kernel(KvPages p, uint32_t parts) {
    const KvView& c = p.c;
    const int32_t s = p.a[blockIdx.y], d = p.b[blockIdx.y];
    if (s < 0 || (uint32_t)s >= c.n_pages || d < 0 || (uint32_t)d >= c.n_pages) {
        if (threadIdx.x == 0) flag(c.status, kStId);
        return;
    }
    if (s != d) copy_page(c, blockIdx.x / parts, (uint32_t)s, (uint32_t)d, blockIdx.x % parts, parts);
}

// ---------------------------------------------------------------- compact
// work: [0] pages in use, [1] pages to move, [4 ..] block counts, then the list
// of movers and the list of holes
constexpr uint32_t kCompactBlock = 4096;

__device__ __forceinline__ uint32_t live_count(const KvView& c, uint32_t lo, uint32_t hi, uint32_t* sums) {
    uint32_t n = 0;
    for (uint32_t i = lo + threadIdx.x; i < hi; i += 256) n += c.refs[i] > 0;
    uint32_t total;
    block_prefix(n, sums, total);
    return total;
}

__global__ __launch_bounds__(256) void compact_count_kernel(KvPages p) {
    __shared__ uint32_t sums[4];
    const uint32_t lo = blockIdx.x * kCompactBlock, hi = min(lo + kCompactBlock, p.c.n_pages);
    const uint32_t n = live_count(p.c, lo, hi, sums);
    if (threadIdx.x == 0) p.work[4 + blockIdx.x] = (int32_t)n;
}

__global__ __launch_bounds__(256) void compact_rank_kernel(KvPages p, uint32_t blocks) {
    const KvView& c = p.c;
    __shared__ uint32_t sums[4];
    uint32_t n = 0, before = 0;
    for (uint32_t b = threadIdx.x; b < blocks; b += 256) {
        const uint32_t x = (uint32_t)p.work[4 + b];
        n += x;
        if (b < blockIdx.x) before += x;
    }
    uint32_t live, mine, low = 0;
    block_prefix(n, sums, live);
    block_prefix(before, sums, mine);
    // pages in use below `live`
    const uint32_t bl = live / kCompactBlock;
    for (uint32_t b = threadIdx.x; b < min(bl, blocks); b += 256) low += (uint32_t)p.work[4 + b];
    uint32_t below;
    block_prefix(low, sums, below);
    below += live_count(c, min(bl * kCompactBlock, live), live, sums);
    int32_t* movers = p.work + 4 + blocks;
    int32_t* holes = movers + c.n_pages;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.work[0] = (int32_t)live;
        p.work[1] = (int32_t)(live - below);
    }
    uint32_t seen = mine;                    // pages in use before this step
    const uint32_t lo = blockIdx.x * kCompactBlock, hi = min(lo + kCompactBlock, c.n_pages);
    for (uint32_t base = lo; base < hi; base += 256) {
        const uint32_t i = base + threadIdx.x;
        const int32_t r = i < hi ? c.refs[i] : 0;
        uint32_t total;
        const uint32_t at = seen + block_prefix(r > 0, sums, total);
        if (i < hi) {
            if (i >= live) p.refs_out[i] = 0;
            if (r > 0 && i >= live) movers[at - below] = (int32_t)i;
            if (r > 0 && i < live) p.refs_out[i] = r;
            if (r <= 0 && i < live) holes[i - at] = (int32_t)i;
        }
        seen += total;
    }
}

// the place of page i after the move: movers is ascending
__device__ __forceinline__ int32_t new_place(int32_t i, uint32_t live, uint32_t moves, const int32_t* movers,
                                             const int32_t* holes) {
    if ((uint32_t)i < live) return i;
    uint32_t lo = 0, hi = moves;
    while (lo < hi) {
        const uint32_t mid = (lo + hi) / 2;
        if (movers[mid] < i) lo = mid + 1;
        else hi = mid;
    }
    return lo < moves && movers[lo] == i ? holes[lo] : -1;
}

// grid: (layers * parts + 1, max moves at most): the copies and the movers' counts
__global__ __launch_bounds__(256) void compact_move_kernel(KvPages p, uint32_t blocks, uint32_t parts) {
    const KvView& c = p.c;
    const uint32_t moves = (uint32_t)p.work[1];
    const int32_t* movers = p.work + 4 + blocks;
    const int32_t* holes = movers + c.n_pages;
    for (uint32_t m = blockIdx.y; m < moves; m += gridDim.y) {
        const uint32_t s = (uint32_t)movers[m], d = (uint32_t)holes[m];
        if (blockIdx.x == c.layers * parts) {
            if (threadIdx.x == 0) p.refs_out[d] = c.refs[s];
        } else {
            copy_page(c, blockIdx.x / parts, s, d, blockIdx.x % parts, parts);
        }
    }
}

// grid: rows
__global__ __launch_bounds__(256) void compact_table_kernel(KvPages p, uint32_t blocks) {
    const KvView& c = p.c;
    const uint32_t live = (uint32_t)p.work[0], moves = (uint32_t)p.work[1];
    const int32_t* movers = p.work + 4 + blocks;
    const int32_t* holes = movers + c.n_pages;
    const uint64_t at = (uint64_t)blockIdx.x * c.max_pages;
    const uint32_t n = min(pages_of(c, (uint32_t)max(c.lens[blockIdx.x], 0)), c.max_pages);
    for (uint32_t j = threadIdx.x; j < c.max_pages; j += 256) {
        int32_t to = -1;
        if (j < n) {
            const int32_t pid = c.table[at + j];
            if (pid >= 0 && (uint32_t)pid < c.n_pages) to = new_place(pid, live, moves, movers, holes);
            if (to < 0) flag(c.status, kStId);
        }
        p.table_out[at + j] = to;
    }
}

// workgroups per page and layer: 16 B per thread and side, at most 8 of them
uint32_t copy_parts(const KvView& c) {
    return (uint32_t)std::max<uint64_t>(1, std::min<uint64_t>(8, c.side_bytes / 16 / 256));
}

}  // namespace

extern "C" int bsk_kv_append(const KvAppend* a, void* stream) {
    const uint32_t touch = (a->max_new + 2 * a->c.page - 2) >> a->c.lp;
    const dim3 grid(touch * 2 * a->c.kv_heads, a->n_seqs);
    hipStream_t st = (hipStream_t)stream;
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, *a); };
    auto typed = [&](auto vec, auto f32) {
        if (a->c.type == 1) go(append_kernel<true, decltype(vec)::value, decltype(f32)::value>);
        else go(append_kernel<false, decltype(vec)::value, decltype(f32)::value>);
    };
    if (a->vec && a->f32) typed(std::true_type{}, std::true_type{});
    else if (a->vec) typed(std::true_type{}, std::false_type{});
    else if (a->f32) typed(std::false_type{}, std::true_type{});
    else typed(std::false_type{}, std::false_type{});
    return (int)hipGetLastError();
}

extern "C" int bsk_kv_extend(const KvPages* p, void* stream) {
    hipLaunchKernelGGL(alloc_kernel<false>, dim3(1), dim3(kScan), 0, (hipStream_t)stream, *p);
    return (int)hipGetLastError();
}

extern "C" int bsk_kv_fork(const KvPages* p, void* stream) {
    hipLaunchKernelGGL(alloc_kernel<true>, dim3(1), dim3(kScan), 0, (hipStream_t)stream, *p);
    const uint32_t parts = copy_parts(p->c);
    hipLaunchKernelGGL(fork_fill_kernel, dim3(p->c.layers * parts + 1, p->n), dim3(256), 0, (hipStream_t)stream, *p, parts);
    return (int)hipGetLastError();
}

extern "C" int bsk_kv_free(const KvPages* p, void* stream) {
    hipLaunchKernelGGL(free_kernel, dim3(p->n), dim3(256), 0, (hipStream_t)stream, *p);
    return (int)hipGetLastError();
}

extern "C" int bsk_kv_copy(const KvPages* p, void* stream) {
    const uint32_t parts = copy_parts(p->c);
    hipLaunchKernelGGL(copy_kernel, dim3(p->c.layers * parts, p->n), dim3(256), 0, (hipStream_t)stream, *p, parts);
    return (int)hipGetLastError();
}

extern "C" int bsk_kv_compact(const KvPages* p, void* stream) {
    const uint32_t blocks = (p->c.n_pages + kCompactBlock - 1) / kCompactBlock, parts = copy_parts(p->c);
    hipStream_t st = (hipStream_t)stream;
    hipLaunchKernelGGL(compact_count_kernel, dim3(blocks), dim3(256), 0, st, *p);
    hipLaunchKernelGGL(compact_rank_kernel, dim3(blocks), dim3(256), 0, st, *p, blocks);
    const uint32_t most = std::min<uint32_t>((p->c.n_pages + 1) / 2, 1024);
    hipLaunchKernelGGL(compact_move_kernel, dim3(p->c.layers * parts + 1, most), dim3(256), 0, st, *p, blocks, parts);
    hipLaunchKernelGGL(compact_table_kernel, dim3(p->c.max_seqs), dim3(256), 0, st, *p, blocks);
    return (int)hipGetLastError();
}
