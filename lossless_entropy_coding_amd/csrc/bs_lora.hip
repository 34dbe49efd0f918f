// bs_lora.hip -- low-rank adapters of many requests (gfx950):
//   y[t] += s_a B_a (A_a x_t),  a = the adapter of token t.
//
// batch: sorts the tokens by adapter and cuts each adapter's into tiles of
// 16, once for all projections that the batch goes through.
// inner: t = A x for a tile, on v_mfma_f32_16x16x32_bf16 (A operand: 16 rows
// of the adapter, B operand: the tile's 16 tokens), the columns split over
// workgroups and over the waves of each; the shares' sums are left in a
// workspace and added, in order, by
// outer: y += s B t.  t is kept to fp32's precision: it enters the product
// as the sum of three BF16 numbers (8 + 8 + 8 significant bits), since the
// product is a few MFMAs beside the loads of B and y.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "bs_lora_device.h"

using namespace bsd;

namespace {

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
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
        out[kLoraHead + 4 * max_tiles + atomicAdd(&cur[a + 1], 1u)] = (int32_t)i;
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
    if (i >= p.max_tiles || i >= (uint32_t)p.batch[0]) return false;
    const int32_t* e = p.batch + kLoraHead + 4 * i;
    tl.adapter = e[0];
    tl.first = (uint32_t)e[1];
    tl.count = (uint32_t)e[2];
    return tl.adapter >= -1 && tl.adapter < (int32_t)p.adapters && tl.count >= 1 && tl.count <= kLoraTile &&
           tl.first < p.tokens && tl.count <= p.tokens - tl.first;
}

__device__ __forceinline__ uint32_t token_at(const LoraArgs& p, uint32_t i) {
    return min((uint32_t)p.batch[kLoraHead + 4 * p.max_tiles + i], p.tokens - 1);
}

// Both kernels are bounded to 256 registers (two waves per SIMD), so that the
// products' accumulators stay out of the AGPRs: with them there, the compiler
// here reads a product's later elements at a block's join without the wait
// that it puts before the first, and they come back stale.

// grid: (tiles, shares of the columns); RT: 16-row tiles of the rank
template <int RT>
__global__ __launch_bounds__(256, 2) void inner_kernel(LoraArgs p) {
    Tile tl;
    if (!get_tile(p, blockIdx.x, tl) || tl.adapter < 0) return;
    __shared__ f32x4 red[3][RT][64];
    const uint32_t t = threadIdx.x, lane = t & 63u, m = lane & 15u, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const uint32_t nr = min((uint32_t)(p.ranks[tl.adapter] + 15) / 16, (uint32_t)RT);
    const uint32_t tok = token_at(p, tl.first + min(m, tl.count - 1));
    const uint16_t* xp = p.x + (uint64_t)tok * p.x_stride;
    const uint16_t* ap = p.a + ((uint64_t)tl.adapter * p.rank + m) * p.cols_pad;
    f32x4 acc[RT];
#pragma unroll
    for (int r = 0; r < RT; r++) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
    const uint32_t steps = p.cols_pad / 32, step = 4 * p.ksplit;
    for (uint32_t k = blockIdx.y * 4 + wave; k < steps; k += step) {
        const uint32_t c = 32 * k + 8 * g;
        bf16x8 xv;
        if (p.x_aligned && c + 8 <= p.cols) {
            xv = *(const bf16x8*)(xp + c);
        } else {
            uint32_t w[4];
#pragma unroll
            for (uint32_t e = 0; e < 4; e++) {
                const uint32_t lo = c + 2 * e < p.cols ? xp[c + 2 * e] : 0u, hi = c + 2 * e + 1 < p.cols ? xp[c + 2 * e + 1] : 0u;
                w[e] = lo | hi << 16;
            }
            xv = __builtin_bit_cast(bf16x8, v4u{w[0], w[1], w[2], w[3]});
        }
#pragma unroll
        for (uint32_t r = 0; r < RT; r++)
            if (r < nr) {
                const bf16x8 av = *(const bf16x8*)(ap + (uint64_t)(16 * r) * p.cols_pad + c);
                acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, xv, acc[r], 0, 0, 0);
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

// grid: (tiles, row blocks of 64 R); a wave takes R steps of 16 rows
template <int RT, bool Y32>
__global__ __launch_bounds__(256, 2) void outer_kernel(LoraArgs p, uint32_t rows_per_wave) {
    Tile tl;
    if (!get_tile(p, blockIdx.x, tl)) return;
    const uint32_t t = threadIdx.x, lane = t & 63u, m = lane & 15u, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const uint32_t tok = token_at(p, tl.first + min(m, tl.count - 1));
    constexpr int KC = (RT + 1) / 2;             // steps of 32 ranks
    bf16x8 b0[KC], b1[KC], b2[KC];
    if (tl.adapter >= 0) {
        const float f = p.factor[tl.adapter];
#pragma unroll
        for (int k = 0; k < KC; k++) {
            const uint32_t r0 = 32 * k + 8 * g;
#pragma unroll
            for (uint32_t e = 0; e < 8; e++) {
                float v = 0.f;
                if (r0 + e < 16 * RT && m < tl.count) {
                    const float* tp = p.t + ((uint64_t)tl.first + m) * p.rank + r0 + e;
                    for (uint32_t s = 0; s < p.ksplit; s++) v += tp[(uint64_t)s * p.tokens * p.rank];
                }
                __bf16 x, y, z;
                three(v * f, x, y, z);
                b0[k][e] = x;
                b1[k][e] = y;
                b2[k][e] = z;
            }
        }
    }
    const uint32_t r_begin = (blockIdx.y * 4 + wave) * rows_per_wave;
    for (uint32_t r0 = r_begin; r0 < min(r_begin + rows_per_wave, p.rows); r0 += 16) {
        f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
        if (tl.adapter >= 0) {
            const uint32_t row = min(r0 + m, p.rows - 1);
            const uint16_t* bp = p.b + ((uint64_t)tl.adapter * p.rows + row) * p.rank;
#pragma unroll
            for (int k = 0; k < KC; k++) {
                const uint32_t c = 32 * k + 8 * g;
                const bf16x8 bv = *(const bf16x8*)(bp + (c < 16 * RT ? c : 0u));
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv, b2[k], acc, 0, 0, 0);
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv, b1[k], acc, 0, 0, 0);
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv, b0[k], acc, 0, 0, 0);
            }
        }
        if (m < tl.count) {
            const uint64_t at = (uint64_t)tok * p.y_stride + r0 + 4 * g;
#pragma unroll
            for (uint32_t e = 0; e < 4; e++) {
                if (r0 + 4 * g + e >= p.rows) continue;
                float y = Y32 ? ((const float*)p.y_in)[at + e] : bf(((const uint16_t*)p.y_in)[at + e]);
                if (p.part) y += p.part[at + e];
                y += acc[e];
                if (Y32) ((float*)p.y_out)[at + e] = y;
                else ((uint16_t*)p.y_out)[at + e] = __builtin_bit_cast(uint16_t, (__bf16)y);
            }
        }
    }
}

template <int RT>
int outer(const LoraArgs& a, hipStream_t st) {
    // rows of a wave: 16 for few tiles, more where the tiles fill the GPU
    const uint32_t rw = a.max_tiles >= 64 ? 64 : 16;
    const dim3 grid(a.max_tiles, (a.rows + 4 * rw - 1) / (4 * rw));
    if (a.y32) hipLaunchKernelGGL((outer_kernel<RT, true>), grid, dim3(256), 0, st, a, rw);
    else hipLaunchKernelGGL((outer_kernel<RT, false>), grid, dim3(256), 0, st, a, rw);
    return (int)hipGetLastError();
}

}  // namespace

extern "C" int bsk_lora_batch(const int32_t* idx, uint32_t tokens, uint32_t adapters, uint32_t max_tiles, int32_t* batch,
                              void* stream) {
    hipLaunchKernelGGL(batch_kernel, dim3(1), dim3(1024), 0, (hipStream_t)stream, idx, tokens, adapters, max_tiles, batch);
    return (int)hipGetLastError();
}

extern "C" int bsk_lora_inner(const LoraArgs* a, void* stream) {
    const dim3 grid(a->max_tiles, a->ksplit);
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
