// bs_lora.hip -- low-rank adapters of many requests (gfx950):
//   y[t] += s_a B_a (A_a x_t),  a = the adapter of token t.
//
// batch: sorts the tokens by adapter and cuts each adapter's into tiles of
// 16, once for all projections that the batch goes through.
// inner: t = A x for a tile, on v_mfma_f32_16x16x32_bf16 (A operand: 16 rows
// of the adapter, B operand: the tile's 16 tokens), the columns split over
// workgroups and over the waves of each; the shares' sums are left in a
// workspace and added, in order, by
// outer: y += s B t (or the epilogue of the product that makes y, for a few
// tokens).  t is kept to fp32's precision: it enters the product
// as the sum of three BF16 numbers (8 + 8 + 8 significant bits), since the
// product is a few MFMAs beside the loads of B and y.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "bs_device.h"
#include "bs_lora_device.h"

using namespace bsd;

namespace {

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf(uint32_t w) { return __builtin_bit_cast(float, w << 16); }

__global__ __launch_bounds__(1024) void batch_kernel(const int32_t* idx, uint32_t tokens, uint32_t adapters,
                                                     uint32_t max_tiles, int32_t* out) {
    // bin 0: no adapter, bin a + 1: adapter a
    __shared__ uint32_t cnt[kLoraAdapters + 1], cur[kLoraAdapters + 1];
    __shared__ uint32_t wt[16], wl[16];
    __shared__ uint32_t bad;
    const uint32_t t = threadIdx.x, lane = t & 63u, wave = t >> 6, bins = adapters + 1;
    for (uint32_t i = t; i < bins; i += 1024) cnt[i] = 0;
    if (t == 0) bad = 0;
    __syncthreads();
    for (uint32_t i = t; i < tokens; i += 1024) {
        int32_t a = idx[i];
        if (a < -1 || a >= (int32_t)adapters) {
            atomicAdd(&bad, 1u);
            a = -1;
        }
        atomicAdd(&cnt[a + 1], 1u);
    }
    __syncthreads();
    // exclusive prefixes of tokens and tiles, 1024 bins at a time
    uint32_t tok = 0, til = 0;
    for (uint32_t b0 = 0; b0 < bins; b0 += 1024) {
        const uint32_t b = b0 + t, c = b < bins ? cnt[b] : 0, l = (c + kLoraTile - 1) / kLoraTile;
        uint32_t x = c, y = l;
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const uint32_t px = __shfl_up(x, s), py = __shfl_up(y, s);
            if (lane >= (uint32_t)s) { x += px; y += py; }
        }
        __syncthreads();
        if (lane == 63) { wt[wave] = x; wl[wave] = y; }
        __syncthreads();
        uint32_t bx = tok, by = til;
        for (uint32_t w = 0; w < 16; w++) {
            if (w < wave) { bx += wt[w]; by += wl[w]; }
            tok += wt[w];
            til += wl[w];
        }
        if (b < bins) {
            const uint32_t first = bx + x - c, tile = by + y - l;
            cur[b] = first;
            for (uint32_t k = 0; k < l; k++) {
                int32_t* e = out + kLoraHead + 4 * (tile + k);
                e[0] = (int32_t)b - 1;
                e[1] = (int32_t)(first + kLoraTile * k);
                e[2] = (int32_t)min(kLoraTile, c - kLoraTile * k);
                e[3] = 0;
            }
        }
    }
    __syncthreads();
    // a token's result does not depend on its place among its adapter's
    for (uint32_t i = t; i < tokens; i += 1024) {
        int32_t a = idx[i];
        if (a < -1 || a >= (int32_t)adapters) a = -1;
        const uint32_t at = atomicAdd(&cur[a + 1], 1u);
        out[kLoraHead + 4 * max_tiles + at] = (int32_t)i;
        int32_t* pair = out + lora_pairs(max_tiles, tokens) + 2 * i;
        pair[0] = a;
        pair[1] = (int32_t)at;
    }
    if (t == 0) {
        out[0] = (int32_t)til;
        out[1] = (int32_t)tokens;
        out[2] = (int32_t)bad;
        out[3] = 0;
    }
}

// One tile of a batch, checked against this call's sizes.
struct Tile {
    int32_t adapter;
    uint32_t first, count;
};

__device__ __forceinline__ bool get_tile(const LoraArgs& p, uint32_t i, Tile& tl) {
    // both loads go out together (tile i lies inside the batch's buffer)
    const int32_t tiles = p.batch[0];
    const v4u e = *(const v4u*)(p.batch + kLoraHead + 4 * i);
    tl.adapter = (int32_t)e[0];
    tl.first = e[1];
    tl.count = e[2];
    return i < (uint32_t)tiles && tl.adapter >= -1 && tl.adapter < (int32_t)p.adapters && tl.count >= 1 && tl.count <= kLoraTile &&
           tl.first < p.tokens && tl.count <= p.tokens - tl.first;
}

__device__ __forceinline__ uint32_t token_at(const LoraArgs& p, uint32_t i) {
    return min((uint32_t)p.batch[kLoraHead + 4 * p.max_tiles + i], p.tokens - 1);
}

// Both kernels are bounded to 256 registers (two waves per SIMD), so that the
// products' accumulators stay out of the AGPRs: with them there, the compiler
// here reads a product's later elements at a block's join without the wait
// that it puts before the first, and they come back stale.

// 8 elements of a row of x from column c, zeros past the last
__device__ __forceinline__ bf16x8 load_x(const LoraArgs& p, const uint16_t* xp, uint32_t c) {
    if (p.x_aligned && c + 8 <= p.cols) return *(const bf16x8*)(xp + c);
    uint32_t w[4];
#pragma unroll
    for (uint32_t e = 0; e < 4; e++) {
        const uint32_t lo = c + 2 * e < p.cols ? xp[c + 2 * e] : 0u, hi = c + 2 * e + 1 < p.cols ? xp[c + 2 * e + 1] : 0u;
        w[e] = lo | hi << 16;
    }
    return __builtin_bit_cast(bf16x8, v4u{w[0], w[1], w[2], w[3]});
}

// grid: (tiles, shares of the columns), and before the tiles the workgroups that
// lay x out for the product beside it; RT: 16-row tiles of the rank.  A wave
// takes 128 columns at a time, all their loads issued before the first
// product.  A is kept in the order of the product's operand, so a wave reads
// 4 KiB on end of each 16 rows.  A's bytes bound it: 64 tokens, each with an
// adapter of up to 64 ranks of its own, on 14336 columns: 82 MB in 19 us, 4.4
// TB/s (21 us with x laid out for the product).  4097 tokens with 5 adapters on 3584 columns: 29 MB of x in 10.5 us.
template <int RT>
__global__ __launch_bounds__(256, 2) void inner_kernel(LoraArgs p) {
    const uint32_t t = threadIdx.x, lane = t & 63u, m = lane & 15u, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const uint32_t packs = gridDim.x - p.max_tiles;
    if (blockIdx.x < packs) {
        const uint32_t steps = p.cols / 32, all = p.x_tiles * steps;
        const uint32_t w = (blockIdx.y * packs + blockIdx.x) * 4 + wave, waves = packs * gridDim.y * 4;
        for (uint32_t u = w; u < all; u += waves) {
            const uint32_t tile = u / steps, tok = 16 * tile + m;
            v4u v = {0, 0, 0, 0};
            if (tok < p.tokens) v = *(const v4u*)(p.x + (uint64_t)tok * p.x_stride + 32 * (u - tile * steps) + 8 * g);
            *(v4u*)(p.x_ops + ((uint64_t)u * 64 + lane) * 8) = v;
        }
        return;
    }
    Tile tl;
    if (!get_tile(p, blockIdx.x - packs, tl) || tl.adapter < 0) return;
    __shared__ f32x4 red[3][RT][64];
    const uint32_t rank = (uint32_t)p.ranks[tl.adapter], nr = min((rank + 15) / 16, (uint32_t)RT);
    const uint32_t tok = token_at(p, tl.first + min(m, tl.count - 1));
    const uint16_t* xp = p.x + (uint64_t)tok * p.x_stride;
    const uint32_t steps = p.cols_pad / 32;
    const uint16_t* ap = p.a + (uint64_t)tl.adapter * p.rank * p.cols_pad + 8 * lane;
    f32x4 acc[RT];
#pragma unroll
    for (int r = 0; r < RT; r++) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
    const uint32_t step = 4 * p.ksplit;
    constexpr uint32_t U = RT == 8 ? 2 : 4;      // 64 columns at rank 128, where 128 would not fit the registers
    for (uint32_t k = blockIdx.y * 4 + wave; 32 * U * k < p.cols_pad; k += step) {
        const uint32_t c0 = 32 * U * k + 8 * g;
        bf16x8 xv[U], av[U][RT];
#pragma unroll
        for (uint32_t u = 0; u < U; u++) {
            const uint32_t c = c0 + 32 * u;
            const uint32_t st = min(U * k + u, steps - 1);
            xv[u] = load_x(p, xp, c);
#pragma unroll
            for (uint32_t r = 0; r < RT; r++)
                if (r < nr) av[u][r] = *(const bf16x8*)(ap + ((uint64_t)r * steps + st) * 512);
        }
#pragma unroll
        for (uint32_t u = 0; u < U; u++) {
            if (U * k + u >= steps) break;       // 0 of x times an infinity of the last step's A would be NaN
#pragma unroll
            for (uint32_t r = 0; r < RT; r++)
                if (r < nr) acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[u][r], xv[u], acc[r], 0, 0, 0);
        }
    }
    if (wave > 0) {
#pragma unroll
        for (int r = 0; r < RT; r++) red[wave - 1][r][lane] = acc[r];
    }
    __syncthreads();
    if (wave > 0) return;
    // rows 16 r + 4 g .. of the adapter, token m of the tile
    if (m < tl.count) {
        float* tp = p.t + ((uint64_t)blockIdx.y * p.tokens + tl.first + m) * p.rank;
#pragma unroll
        for (int r = 0; r < RT; r++) {
            f32x4 s = acc[r];
#pragma unroll
            for (int w = 0; w < 3; w++) s += red[w][r][lane];
            // past the adapter's rank A's zeros times an infinity of x are NaN
#pragma unroll
            for (uint32_t e = 0; e < 4; e++) s[e] = 16 * r + 4 * g + e < rank ? s[e] : 0.f;
            *(f32x4*)(tp + 16 * r + 4 * g) = s;
        }
    }
}

// a float as the sum of three BF16 numbers
__device__ __forceinline__ void three(float v, __bf16& a, __bf16& b, __bf16& c) {
    a = (__bf16)v;
    const float r = fabsf((float)a) < __builtin_inff() ? v - (float)a : 0.f;   // an infinity or NaN is in a alone
    b = (__bf16)r;
    c = (__bf16)(r - (float)b);
}

// y of 4 (fp32) or 8 (BF16) rows from element `at`, n of them inside, as it
// is in memory (FROM: y or one of the parts)
template <bool Y32>
__device__ __forceinline__ v4u load_some(const void* from, uint64_t at, uint32_t n) {
    v4u v = {0, 0, 0, 0};
#pragma unroll
    for (uint32_t e = 0; e < (Y32 ? 4u : 8u); e++)
        if (e < n) {
            if (Y32) v[e] = ((const uint32_t*)from)[at + e];
            else v[e / 2] |= (uint32_t)((const uint16_t*)from)[at + e] << (16 * (e & 1u));
        }
    return v;
}

template <bool Y32>
__device__ __forceinline__ v4u load_all(const void* from, uint64_t at) {
    return *(const v4u*)((const uint8_t*)from + at * (Y32 ? 4 : 2));
}

template <bool Y32>
__device__ __forceinline__ void store_y(const LoraArgs& p, uint64_t at, uint32_t n, const float* y) {
    constexpr uint32_t N = Y32 ? 4 : 8;
    if (p.y_vec && n >= N) {
        if (Y32) *(f32x4*)((float*)p.y_out + at) = f32x4{y[0], y[1], y[2], y[3]};
        else {
            v4u v;
#pragma unroll
            for (uint32_t e = 0; e < 4; e++) {
                const bf16x2 w = {(__bf16)y[2 * e], (__bf16)y[2 * e + 1]};
                v[e] = __builtin_bit_cast(uint32_t, w);
            }
            *(v4u*)((uint16_t*)p.y_out + at) = v;
        }
        return;
    }
#pragma unroll
    for (uint32_t e = 0; e < N; e++)
        if (e < n) {
            if (Y32) ((float*)p.y_out)[at + e] = y[e];
            else ((uint16_t*)p.y_out)[at + e] = __builtin_bit_cast(uint16_t, (__bf16)y[e]);
        }
}

// x of lane l ^ 1
__device__ __forceinline__ float from_neighbour(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), 0xB1, 0xF, 0xF, true));
}

// grid: blocks of rows x tiles, the blocks of a tile side by side, so that
// neighbouring workgroups fill whole rows of y; a workgroup's waves take
// `strips` strips of 64 rows in turn.  The workgroup first adds the shares of
// t and leaves its three BF16 parts in LDS, in the order of the product's
// operand.  The 64 rows of a strip are dealt to the four 16-row products such
// that a lane ends up with rows that lie side by side in y: 4 (fp32, 16 j +
// 4 g ..) or 8 (BF16, 32 j + 8 g ..) to each 16-B access, and the four lane
// groups fill 64 B of a token's row.  In BF16 two neighbouring lanes then swap
// halves, so that each access fills whole lines of 128 B (62.7 instead of 64.8
// us on the case below; in fp32 it gained nothing).
//
// y's traffic bounds it: 235 MB of 4097 tokens x 14336 rows in BF16 in 50.5 us,
// 4.7 TB/s, as fast as a large copy.  What is read ahead stays as it is in
// memory until it is added (a conversion beside the load made every load wait
// for the one before: 62.7 us).  Four waves per SIMD: 64 tokens of a decode
// batch are 3.5 waves per SIMD on 3584 rows, one more round with less.
template <int RT, bool Y32>
__global__ __launch_bounds__(256, RT <= 4 ? 4 : 2) void outer_kernel(LoraArgs p, uint32_t strips, uint32_t blocks) {
    constexpr int KC = (RT + 1) / 2;             // steps of 32 ranks
    constexpr int NB = RT == 1 ? 2 : 3;
    // part n of step k, lane's 8 ranks
    __shared__ __attribute__((aligned(16))) __bf16 tb[NB][KC][64][8];
    Tile tl;
    const uint32_t tile = blockIdx.x / blocks, rb = blockIdx.x % blocks;
    if (!get_tile(p, tile, tl)) return;
    if (tl.adapter < 0 && p.y_in == p.y_out && p.nparts == 0) return;
    const uint32_t t = threadIdx.x, lane = t & 63u, m = lane & 15u, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const uint32_t begin = (rb * 4 * strips + wave) * 64;
    // lanes 2 q and 2 q + 1 go to tokens 2 q and 2 q + 1 in turn, half a line each
    constexpr bool kPairs = !Y32;
    constexpr uint32_t N = Y32 ? 4 : 8, NY = 16 / N;
    const uint32_t odd = m & 1u, q0 = kPairs ? m - odd : m, q1 = kPairs ? q0 + 1 : m;
    const uint64_t yrow[2] = {(uint64_t)token_at(p, tl.first + min(q0, tl.count - 1)) * p.y_stride,
                              (uint64_t)token_at(p, tl.first + min(q1, tl.count - 1)) * p.y_stride};
    const bool mine[2] = {q0 < tl.count, q1 < tl.count};
    // rows of the lane's access i of the strip at s0, and how many are inside
    auto row_of = [&](uint32_t s0, uint32_t i) { return s0 + 4 * N * (kPairs ? (i & ~1u) + odd : i) + N * g; };
    auto left_of = [&](uint32_t r, uint32_t i) { return mine[i & 1u] && r < p.rows ? p.rows - r : 0u; };
    // what is read ahead stays as it is in memory until it is added: a
    // conversion beside the load waits for each load before the next
    v4u next[NY];
    auto load_y = [&](uint32_t s0) {
        const bool whole = p.y_vec && s0 + 64 <= p.rows;
        if (whole) {
#pragma unroll
            for (uint32_t i = 0; i < NY; i++)
                if (mine[i & 1u]) next[i] = load_all<Y32>(p.y_in, yrow[i & 1u] + row_of(s0, i));
        } else {
#pragma unroll
            for (uint32_t i = 0; i < NY; i++) {
                const uint32_t r = row_of(s0, i), n = left_of(r, i);
                next[i] = load_some<Y32>(p.y_in, yrow[i & 1u] + r, n);
            }
        }
    };
    load_y(begin);
    bf16x8 a[4][KC];
    uint32_t nk = 0;
    auto load_b = [&](uint32_t s0) {
        const uint32_t in = min(s0, p.rows - 1), left = p.rows - 1 - in;
        const uint16_t* base = p.b + ((uint64_t)(uint32_t)tl.adapter * p.rows + in) * p.rank;
#pragma unroll
        for (uint32_t j = 0; j < 4; j++) {
            // row m of product j: lane group m / 4, element m % 4
            const uint32_t r = Y32 ? 16 * j + m : 32 * (j >> 1) + 8 * (m >> 2) + 4 * (j & 1u) + (m & 3u);
            const uint16_t* bp = base + min(r, left) * p.rank;
#pragma unroll
            for (uint32_t k = 0; k < KC; k++)
                if (k < nk) a[j][k] = *(const bf16x8*)(bp + (RT == 1 ? 8 * (g & 1u) : 32 * k + 8 * g));
        }
    };
    if (tl.adapter >= 0) {
        nk = min((uint32_t)(p.ranks[tl.adapter] + 31) / 32, (uint32_t)KC);
        const float f = p.factor[tl.adapter];
        load_b(begin);
        // t[token q][rank r] for the tile's 16 tokens; all loads go out together
        float w[RT][kLoraSplits];
#pragma unroll
        for (uint32_t i = 0; i < RT; i++) {
            const uint32_t q = (t + 256 * i) / (16 * RT), r = (t + 256 * i) % (16 * RT);
            const uint32_t at = q * p.rank + r;
#pragma unroll
            for (uint32_t s = 0; s < kLoraSplits; s++)
                if (s < p.ksplit && q < tl.count) w[i][s] = (p.t + ((uint64_t)s * p.tokens + tl.first) * p.rank)[at];
        }
#pragma unroll
        for (uint32_t i = 0; i < RT; i++) {
            const uint32_t q = (t + 256 * i) / (16 * RT), r = (t + 256 * i) % (16 * RT);
            float v = 0.f;
#pragma unroll
            for (uint32_t s = 0; s < kLoraSplits; s++)
                if (s < p.ksplit) v += w[i][s];
            if (q >= tl.count) v = 0.f;
            __bf16 x, y, z;
            three(v * f, x, y, z);
            const uint32_t l = 16 * ((r >> 3) & 3u) + q, e = r & 7u;
            tb[0][r >> 5][l][e] = x;
            if (RT == 1) {
                // a rank of 16 fills half of a step: lane groups 2 and 3
                // take the second parts of the same ranks
                tb[0][0][l + 32][e] = y;
                tb[1][0][l][e] = z;
                tb[1][0][l + 32][e] = (__bf16)0.f;
            } else {
                tb[1][r >> 5][l][e] = y;
                tb[NB - 1][r >> 5][l][e] = z;
            }
        }
        __syncthreads();
    }
    for (uint32_t s = 0; s < strips; s++) {
        const uint32_t s0 = begin + 256 * s;
        if (s0 >= p.rows) break;
        float y[16], add[16];
        const bool more = s + 1 < strips && s0 + 256 < p.rows;
        auto take_y = [&]() {
#pragma unroll
            for (uint32_t i = 0; i < NY; i++)
#pragma unroll
                for (uint32_t e = 0; e < 4; e++) {
                    const uint32_t w = next[i][e];
                    if (Y32) y[4 * i + e] = __builtin_bit_cast(float, w);
                    else {
                        y[8 * i + 2 * e] = bf(w & 0xFFFFu);
                        y[8 * i + 2 * e + 1] = __builtin_bit_cast(float, w & 0xFFFF0000u);
                    }
                }
            for (uint32_t k = 0; Y32 && k < p.nparts; k++) {
                const float* from = p.part + k * p.part_stride;
                v4u w[NY];
#pragma unroll
                for (uint32_t i = 0; i < NY; i++) {
                    const uint32_t r = row_of(s0, i);
                    if (p.y_vec && s0 + 64 <= p.rows) {
                        if (mine[i & 1u]) w[i] = load_all<true>(from, yrow[i & 1u] + r);
                    } else w[i] = load_some<true>(from, yrow[i & 1u] + r, left_of(r, i));
                }
#pragma unroll
                for (uint32_t i = 0; i < NY; i++)
#pragma unroll
                    for (uint32_t e = 0; e < 4; e++) {
                        const uint32_t u = w[i][e];
                        y[4 * i + e] += __builtin_bit_cast(float, u);
                    }
            }
            if (more) load_y(s0 + 256);
        };
        auto multiply = [&]() {
            if (tl.adapter >= 0) {
                // t is read again for each strip: kept in registers it would cost a wave of each SIMD
                asm volatile("" ::: "memory");
                bf16x8 b[NB][KC];
#pragma unroll
                for (int n = 0; n < NB; n++)
#pragma unroll
                    for (int k = 0; k < KC; k++) b[n][k] = *(const bf16x8*)tb[n][k][lane];
#pragma unroll
                for (uint32_t j = 0; j < 4; j++) {
                    f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (uint32_t k = 0; k < KC; k++)
                        if (k < nk) {
#pragma unroll
                            for (int n = NB - 1; n >= 0; n--)
                                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[j][k], b[n][k], acc, 0, 0, 0);
                        }
#pragma unroll
                    for (uint32_t e = 0; e < 4; e++) add[4 * j + e] = acc[e];
                }
            }
        };
        // the next strip's y is asked for as early as the registers allow: in
        // fp32, before the products, it would spill
        if (!Y32) take_y();
        multiply();
        if (Y32) take_y();
        if (more && tl.adapter >= 0) load_b(s0 + 256);
        if (tl.adapter >= 0) {
            if (kPairs) {
#pragma unroll
                for (uint32_t e = 0; e < 8; e++) {
                    const float keep = odd ? add[8 + e] : add[e], other = from_neighbour(odd ? add[e] : add[8 + e]);
                    y[e] += odd ? other : keep;
                    y[8 + e] += odd ? keep : other;
                }
            } else {
#pragma unroll
                for (uint32_t e = 0; e < 16; e++) y[e] += add[e];
            }
        }
#pragma unroll
        for (uint32_t i = 0; i < NY; i++) {
            const uint32_t r = row_of(s0, i), n = left_of(r, i);
            if (n) store_y<Y32>(p, yrow[i & 1u] + r, n, y + N * i);
        }
    }
}

template <int RT>
int outer(const LoraArgs& a, hipStream_t st) {
    // strips of a wave: each workgroup first finds its tile and joins t, so up
    // to four where 16 workgroups per CU are left (4097 tokens x 14336 rows in
    // BF16: 58.4 us with 1, 52.6, 51.8 and 50.5 with 2, 3 and 4, 54.1 with 5)
    int cus = 0;
    if (bsk_device_cus(&cus) != 0 || cus <= 0) cus = 256;
    const uint64_t all = (uint64_t)a.max_tiles * ((a.rows + 255) / 256);
    const uint32_t strips = (uint32_t)std::min<uint64_t>(4, std::max<uint64_t>(1, all / (16ull * (uint64_t)cus)));
    const uint32_t blocks = (a.rows + 256 * strips - 1) / (256 * strips);
    const dim3 grid(blocks * a.max_tiles);
    if (a.y32) hipLaunchKernelGGL((outer_kernel<RT, true>), grid, dim3(256), 0, st, a, strips, blocks);
    else hipLaunchKernelGGL((outer_kernel<RT, false>), grid, dim3(256), 0, st, a, strips, blocks);
    return (int)hipGetLastError();
}

}  // namespace

extern "C" int bsk_lora_batch(const int32_t* idx, uint32_t tokens, uint32_t adapters, uint32_t max_tiles, int32_t* batch,
                              void* stream) {
    hipLaunchKernelGGL(batch_kernel, dim3(1), dim3(1024), 0, (hipStream_t)stream, idx, tokens, adapters, max_tiles, batch);
    return (int)hipGetLastError();
}

extern "C" int bsk_lora_inner(const LoraArgs* a, void* stream) {
    const uint32_t units = a->x_tiles * (a->cols / 32), four = 16 * a->ksplit;   // four units to a wave
    const dim3 grid(a->max_tiles + (units + four - 1) / four, a->ksplit);
    hipStream_t st = (hipStream_t)stream;
    switch (a->rank / 16) {
        case 1: hipLaunchKernelGGL(inner_kernel<1>, grid, dim3(256), 0, st, *a); break;
        case 2: hipLaunchKernelGGL(inner_kernel<2>, grid, dim3(256), 0, st, *a); break;
        case 4: hipLaunchKernelGGL(inner_kernel<4>, grid, dim3(256), 0, st, *a); break;
        case 8: hipLaunchKernelGGL(inner_kernel<8>, grid, dim3(256), 0, st, *a); break;
        default: return (int)hipErrorInvalidValue;
    }
    return (int)hipGetLastError();
}

extern "C" int bsk_lora_outer(const LoraArgs* a, void* stream) {
    hipStream_t st = (hipStream_t)stream;
    switch (a->rank / 16) {
        case 1: return outer<1>(*a, st);
        case 2: return outer<2>(*a, st);
        case 4: return outer<4>(*a, st);
        case 8: return outer<8>(*a, st);
        default: return (int)hipErrorInvalidValue;
    }
}
