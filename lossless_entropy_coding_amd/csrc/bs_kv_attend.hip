// bs_kv_attend.hip -- attention over the paged 8-bit key/value cache (gfx950).
//
// Rows are the queries that share a key head: row r of a sequence is token
// r / group, head r % group of the key head's group.  A wave takes 64 tokens
// of one sequence and key head at a time against 16 rows:
//
//   S^T = K Q^T     v_mfma_f32_16x16x32_bf16, A = 16 tokens x 32 channels,
//                   B = 32 channels x 16 rows.  An 8-bit code is exact in
//                   BF16 (e4m3 has 4 significant bits, int8 7), so the
//                   products are exact and summed in fp32; the page's scale
//                   multiplies the sum.
//   O^T += V^T P^T  A = 16 channels x 32 tokens, B = 32 tokens x 16 rows.
//                   P (times the scale of V's page, a power of two) enters
//                   as two BF16 numbers, 16 significant bits, where rows are
//                   few: the products are exact and the result is the fp32
//                   form's to its own rounding (1e-4 of it apart or less on
//                   777, 64 x 4096 and 4 x 131071 tokens, where one BF16
//                   number gave 1e-3 to 2e-3).  It costs up to 1.5% where HBM
//                   or drafts bound it and 0.2 us of a lone short row's 10.5.
//                   Where rows are many the matrix products would take half
//                   as long again and the registers do not hold the second
//                   part: P is rounded to BF16, the type of the result.  The
//                   tokens' rounding errors are independent, and their sum is
//                   about as large as the result's own rounding (two prompts
//                   of up to 2048 tokens over 8000: 2.3e-3 from the 64-bit
//                   result, the fp32 form 1.7e-3).  The sum of P is kept in
//                   fp32 from the unrounded values.
//
// The tokens of a 64-token tile are dealt to the four 16-token steps of S^T
// such that lane group g (lanes 16 g ..) ends up with tokens 16 g .. 16 g +
// 15 of its row, four of each step.  These are the tokens that the lane has
// to hold for the second product, in the order in which it reads V (kept
// with a channel's tokens side by side), so P goes from one product to the
// other without leaving the lane, and one lane's tokens are always of one
// page.  Keys and values are read 16 B per lane.
//
// The running maximum and sum of a row's softmax are held per row (a lane's
// column), the result is scaled when the maximum grows.  The waves of a
// workgroup take the tiles in turn and are joined in wave order; where there
// are too few rows to fill the GPU, a row's tiles are also split over
// workgroups, and the one that ends last joins their results in order.
//
// What bounds it, measured:
// few rows: the cache's bytes.  4 sequences of 131071 tokens (40 heads on 8 of
//   128 channels, int8): 1.07 GB in 203 us, 5.3 TB/s.  64 ragged sequences
//   with a window of 4096 (16 heads on 8 of 256 channels, e4m3): 750 MB in 159
//   us, 4.7 TB/s.  A large copy moves 4.8 TB/s here.  A lone short row is a
//   chain of dependent loads (row, page, keys, values, join): 777 tokens, 11 us.
// many rows (attend_rows_kernel): 2 prompts of up to 2048 new tokens over 8000
//   (40 heads on 8 of 128 channels, e4m3): 536 us, 827 TFLOP/s; a large
//   library product reaches 1430.  See there.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "bs_kv_attend_device.h"

using namespace bsd;

namespace {

// grid: (sequences * row tiles, key heads, splits); four waves.  The bound of
// two waves per SIMD keeps the kernel within 256 registers and so the
// products' accumulators out of the AGPRs: with them there, the compiler here
// reads a product's later elements at a block's join without the wait that
// it puts before the first, and they come back stale.
template <int DW, bool E4M3, bool CAP>
__global__ __launch_bounds__(256, 2) void attend_kernel(KvAttend a, uint32_t row_tiles) {
    const KvView& c = a.c;
    constexpr uint32_t D = 64 * DW, NW = 4;
    // values loaded with the keys; the rest follow when the keys' registers
    // are free (all at once, head_dim 256 spills registers)
    constexpr uint32_t kFirst = DW >= 3 ? 2 * DW : 4 * DW;
    __shared__ float ml[NW][2][16];
    __shared__ __attribute__((aligned(16))) float os[NW][16][D + 4];
    // Q as operands of the product: in registers it would leave too few for
    // a tile's keys and values in flight at head_dim 256
    __shared__ __attribute__((aligned(16))) uint8_t qs[2 * DW][1024];

    const uint32_t t = threadIdx.x, lane = t & 63u, m = lane & 15u, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const uint32_t split = blockIdx.z, head = blockIdx.y;
    const uint32_t seq_i = blockIdx.x / row_tiles, rt = blockIdx.x % row_tiles;
    const Seq sq = get_seq(a, seq_i);
    if (!sq.ok && t == 0 && split == 0) {
        if (c.status) atomicOr(c.status, 4u);
    }
    const uint32_t rows = (uint32_t)sq.count * a.group;
    if (16 * rt >= rows) return;
    const uint32_t nrows = min(16u, rows - 16 * rt);
    const int32_t base = sq.len - sq.count;                         // the first query's place
    const int32_t lo = base + (int32_t)(16 * rt / a.group), hi = base + (int32_t)((16 * rt + nrows - 1) / a.group);
    const Tiles tl = get_tiles(a, lo, hi);
    const uint32_t i0 = split * a.chunk;
    if (split > 0 && i0 >= tl.n) return;
    const uint32_t i1 = split + 1 < a.splits ? min(tl.n, i0 + a.chunk) : tl.n;   // the last takes what is left
    const int32_t* trow = c.table + (uint64_t)(uint32_t)max(sq.row, 0) * c.max_pages;
    const uint64_t hoff = (uint64_t)head * c.page * c.wide;
    const uint32_t end = (uint32_t)(hi + 1);                        // tokens past it are seen by no row
    // pages of the lane's 16-token chunks of tile i: its keys' (by step row m)
    // and its own tokens' (by group); -1 past the end
    auto pages = [&](uint32_t i, int32_t& pk, int32_t& pv) {
        pk = pv = -1;
        if (i >= i1) return;
        const uint32_t tile0 = tl.at(i) * kKvTile, ck = tile0 + 16 * (m >> 2), cv = tile0 + 16 * g;
        if (ck < end) pk = trow[ck >> c.lp];
        if (cv < end) pv = trow[cv >> c.lp];
    };
    int32_t pk1, pv1;
    pages(i0 + wave, pk1, pv1);

    // this lane's row
    const uint32_t r = 16 * rt + min(m, nrows - 1);
    const uint32_t tok = (uint32_t)sq.s0 + r / a.group, qh = head * a.group + r % a.group;
    const int32_t pos = base + (int32_t)(r / a.group);
    if (wave == 0) {
        bf16x8 q[DW][2];
        load_q<DW>(a, tok, qh, g, q);
#pragma unroll
        for (uint32_t x = 0; x < 2 * DW; x++) *(bf16x8*)(qs[x] + 16 * lane) = q[x >> 1][x & 1];
    }
    __syncthreads();
    const float sc = a.softcap > 0.f ? a.qscale : a.qscale * kLog2e;
    const float cap_in = a.softcap > 0.f ? 2.f * kLog2e / a.softcap : 0.f, cap_out = a.softcap * kLog2e;

    f32x4 o[4 * DW];
#pragma unroll
    for (int d = 0; d < 4 * DW; d++) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
    float mx = -__builtin_inff(), sum = 0.f;
    uint32_t bad = 0;

    for (uint32_t i = i0 + wave; i < i1; i += NW) {
        const uint32_t tile0 = tl.at(i) * kKvTile;
        const uint32_t ck = tile0 + 16 * (m >> 2), cv = tile0 + 16 * g;
        const bool okk = (uint32_t)pk1 < c.n_pages, okv = (uint32_t)pv1 < c.n_pages;
        if (cv < end && !okv) bad = 1;
        const uint32_t ipk = okk ? (uint32_t)pk1 : 0u, ipv = okv ? (uint32_t)pv1 : 0u;
        const uint8_t* kp = a.k + (uint64_t)ipk * c.side_bytes + hoff + (uint64_t)((ck + (m & 3u)) & (c.page - 1)) * D + 16 * g;
        const uint8_t* vp = a.v + (uint64_t)ipv * c.side_bytes + hoff + (uint64_t)m * c.page + (cv & (c.page - 1));
        v4u kr[4][DW], vr[4 * DW];
#pragma unroll
        for (uint32_t h = 0; h < 4; h++)
#pragma unroll
            for (uint32_t x = 0; x < DW; x++) kr[h][x] = *(const v4u*)(kp + 4 * h * D + 64 * x);
        const float* sp = a.scale + ((uint64_t)ipv * c.kv_heads + head) * 2;
        const float ks = sp[0] * sc, vs = okv ? sp[1] : 0.f;
#pragma unroll
        for (uint32_t d = 0; d < kFirst; d++) vr[d] = *(const v4u*)(vp + (uint64_t)(16 * d) * c.page);
        pages(i + NW, pk1, pv1);

        f32x4 s[4];
#pragma unroll
        for (uint32_t h = 0; h < 4; h++) {
            s[h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (uint32_t x = 0; x < DW; x++) {
                const bf16x8 q0 = *(const bf16x8*)(qs[2 * x] + 16 * lane), q1 = *(const bf16x8*)(qs[2 * x + 1] + 16 * lane);
                s[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<E4M3>(kr[h][x].x, kr[h][x].y), q0, s[h], 0, 0, 0);
                s[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<E4M3>(kr[h][x].z, kr[h][x].w), q1, s[h], 0, 0, 0);
            }
        }
        if (kFirst < 4 * DW) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (uint32_t d = kFirst; d < 4 * DW; d++) vr[d] = *(const v4u*)(vp + (uint64_t)(16 * d) * c.page);
        // step h's element e is token cv + 4 h + e
        float p[16];
        float top = -__builtin_inff();
#pragma unroll
        for (uint32_t h = 0; h < 4; h++)
#pragma unroll
            for (uint32_t e = 0; e < 4; e++) {
                float x = s[h][e] * ks;
                if (CAP) x = capped(x * cap_in, cap_out);
                else if (a.softcap > 0.f) x = cap_out * (1.f - 2.f * __builtin_amdgcn_rcpf(exp2_fast(x * cap_in) + 1.f));
                const int32_t tk = (int32_t)(cv + 4 * h + e);
                const bool seen = okv && tk <= pos &&
                                  (a.window == 0 || (int64_t)tk > (int64_t)pos - (int64_t)a.window || (uint32_t)tk < a.sinks);
                x = seen ? x : -__builtin_inff();
                p[4 * h + e] = x;
                top = fmaxf(top, x);
            }
        // what no row sees may hold anything: its values count as 0
        if (cv + 16 > end || !okv) {
            const int32_t left = okv ? (int32_t)(end - cv) : 0;      // tokens of the chunk that are kept
#pragma unroll
            for (int d = 0; d < 4 * DW; d++)
#pragma unroll
                for (int w = 0; w < 4; w++) {
                    const int32_t nb = left - 4 * w;
                    const uint32_t mask = nb >= 4 ? ~0u : nb <= 0 ? 0u : (1u << (8 * nb)) - 1u;
                    vr[d][w] &= mask;
                }
        }
        top = fmaxf(max_groups(top), mx);
        const float sub = top == -__builtin_inff() ? 0.f : top;
        if (__builtin_amdgcn_ballot_w64(top > mx) != 0) {
            const float alpha = exp2_fast(mx - sub);
            mx = top;
            sum *= alpha;
#pragma unroll
            for (int d = 0; d < 4 * DW; d++) o[d] *= alpha;
        }
        float part = 0.f;
#pragma unroll
        for (int e = 0; e < 16; e++) {
            p[e] = exp2_fast(p[e] - sub);
            part += p[e];
        }
        sum += part;
        // P in two BF16 parts
        bf16x8 pb[2], pl[2];
#pragma unroll
        for (int y = 0; y < 2; y++) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const float u = p[8 * y + 2 * e] * vs, v = p[8 * y + 2 * e + 1] * vs;
                hi[e] = pack_bf16(u, v);
                lo[e] = pack_bf16(u - __builtin_bit_cast(float, hi[e] << 16), v - __builtin_bit_cast(float, hi[e] & 0xFFFF0000u));
            }
            pb[y] = __builtin_bit_cast(bf16x8, v4u{hi[0], hi[1], hi[2], hi[3]});
            pl[y] = __builtin_bit_cast(bf16x8, v4u{lo[0], lo[1], lo[2], lo[3]});
        }
#pragma unroll
        for (int d = 0; d < 4 * DW; d++) {
            const bf16x8 v0 = widen8<E4M3>(vr[d].x, vr[d].y), v1 = widen8<E4M3>(vr[d].z, vr[d].w);
            o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, pl[0], o[d], 0, 0, 0);
            o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, pl[1], o[d], 0, 0, 0);
            o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, pb[0], o[d], 0, 0, 0);
            o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, pb[1], o[d], 0, 0, 0);
        }
    }
    if (bad && c.status) atomicOr(c.status, 4u);

    // join the waves, in wave order: every wave leaves its rows, its maxima
    // and sums in LDS, then each thread adds four channels of a row
    sum = sum_groups(sum);
    if (g == 0) {
        ml[wave][0][m] = mx;
        ml[wave][1][m] = sum;
    }
    if (m < nrows) {
#pragma unroll
        for (int d = 0; d < 4 * DW; d++) *(f32x4*)&os[wave][m][16 * d + 4 * g] = o[d];
    }
    __syncthreads();
    const uint32_t parts = min(max(1u, (tl.n + a.chunk - 1) / a.chunk), a.splits);   // workgroups of these rows
    for (uint32_t i = t; i < nrows * (D / 4); i += 64 * NW) {
        const uint32_t n = i / (D / 4), ch = 4 * (i % (D / 4));
        float top = -__builtin_inff(), total = 0.f;
#pragma unroll
        for (uint32_t w = 0; w < NW; w++) top = fmaxf(top, ml[w][0][n]);
        const float sub = top == -__builtin_inff() ? 0.f : top;
        f32x4 v = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (uint32_t w = 0; w < NW; w++) {
            const float f = exp2_fast(ml[w][0][n] - sub);
            total += f * ml[w][1][n];
            v += f * *(const f32x4*)&os[w][n][ch];
        }
        const uint32_t rr = 16 * rt + n, tk = (uint32_t)sq.s0 + rr / a.group, h = head * a.group + rr % a.group;
        if (parts > 1) part_write<DW, true>(a, tk, h, split, ch, top, total, v);
        else out_write(a, tk, h, ch, top, total, v);
    }
    if (parts == 1) return;

    // The workgroup that ends last joins them all, in split order; counters are
    // 0 between calls.  The parts are stored through the L2 (the XCDs' L2s do
    // not see each other's lines) and waited for before the workgroup counts
    // itself.  A release at the GPU's scope would write back the whole L2 each
    // time: with it, 4 x 131071 tokens took 388 us instead of 201 with a
    // second launch for the join.
    __shared__ uint32_t last;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    uint32_t* counter = a.counters + blockIdx.x * c.kv_heads + head;
    if (t == 0) last = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == parts - 1;
    __syncthreads();
    if (!last) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    for (uint32_t i = t; i < nrows * (D / 4); i += 64 * NW) {
        const uint32_t n = i / (D / 4), ch = 4 * (i % (D / 4));
        const uint32_t rr = 16 * rt + n, tk = (uint32_t)sq.s0 + rr / a.group, h = head * a.group + rr % a.group;
        join_row<DW>(a, tk, h, ch, parts);
    }
    if (t == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ---------------------------------------------------------------- many rows
//
// From 64 rows on (prompts, long drafts) a workgroup of 8 waves takes 128 NR
// rows of one key head, 16 NR to a wave, and all of them use one copy of a
// tile's keys and values: each wave loads a quarter of a side of the tile
// ahead while the current one is multiplied, widens it to BF16 once and
// leaves it in LDS as the operands of the products, 1 KiB to each, so that
// every read of them is 16 B per lane on end.  Two tiles are in LDS.
//
// Codes times their page's scale, a power of two, are exact in BF16, so the
// scales go into the operands.  The exponentials are taken against the
// maximum of earlier tiles, as long as a lane's 16 of them sum to 2^10 or
// less (as exact in fp32 and BF16 as below 1); then neither the tile's
// maximum nor a scaling of the result is needed.  Neither unit is full: of the
// SIMDs' time in CUs that have work, matrix instructions take 41% and issued
// vector instructions (an exponential as long as four others) 56%, LDS reads
// 26% of the CUs', with no bank conflicts.  The first two nearly add up to the
// whole, so the halves of the waves overlap less than they are meant to; why
// is not found.  Dealing tiles evenly to one workgroup per CU, 8-bit operands
// in LDS and reading two tiles ahead were 2 to 15% slower.
template <int DW, bool E4M3, int NR, bool CAP>
__global__ __launch_bounds__(512, 2) void attend_rows_kernel(KvAttend a, uint32_t row_blocks, uint32_t combos) {
    const KvView& c = a.c;
    constexpr uint32_t D = 64 * DW, kFrags = 8 * DW;                // 1-KiB operands of a side of a tile
    __shared__ __attribute__((aligned(16))) uint8_t buf[2][2 * kFrags][1024];
    __shared__ float least[8][NR][16];                              // of each row: -infinity, NaN where its query is not finite

    const uint32_t t = threadIdx.x, lane = t & 63u, m = lane & 15u, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(t >> 6);
    // workgroups of one sequence and key head share an XCD's L2 (consecutive
    // workgroups go to the 8 XCDs in turn), the longest rows first
    const uint32_t xcd = blockIdx.x & 7u, j = blockIdx.x >> 3;
    const uint32_t combo = xcd + 8 * (j / row_blocks), rb = row_blocks - 1 - j % row_blocks, split = blockIdx.y;
    if (combo >= combos) return;
    const uint32_t seq_i = combo / c.kv_heads, head = combo % c.kv_heads;
    const Seq sq = get_seq(a, seq_i);
    if (!sq.ok && t == 0 && split == 0 && c.status) atomicOr(c.status, 4u);
    const uint32_t rows = (uint32_t)sq.count * a.group, wg0 = 128 * NR * rb;
    if (wg0 >= rows) return;
    const int32_t base = sq.len - sq.count;
    const uint32_t wg1 = min(wg0 + 128 * NR, rows);                 // the workgroup's rows
    const Tiles tl = get_tiles(a, base + (int32_t)(wg0 / a.group), base + (int32_t)((wg1 - 1) / a.group));
    const uint32_t i0 = split * a.chunk;
    if (split > 0 && i0 >= tl.n) return;
    const uint32_t i1 = split + 1 < a.splits ? min(tl.n, i0 + a.chunk) : tl.n;   // the last takes what is left
    const uint32_t end = (uint32_t)(base + (int32_t)((wg1 - 1) / a.group) + 1);   // (only read where tiles exist)

    const uint32_t w0 = wg0 + 16 * NR * wave;                       // the wave's first row
    int32_t pos[NR];
    uint32_t tok[NR], qh[NR];
    bf16x8 q[NR][DW][2];
#pragma unroll
    for (uint32_t n = 0; n < NR; n++) {
        const uint32_t r = min(w0 + 16 * n + m, rows - 1);
        tok[n] = (uint32_t)sq.s0 + r / a.group;
        qh[n] = head * a.group + r % a.group;
        pos[n] = base + (int32_t)(r / a.group);
        load_q<DW>(a, tok[n], qh[n], g, q[n]);
        if (a.qscale < 0.f) {                                       // the scale's sign goes into Q
#pragma unroll
            for (uint32_t x = 0; x < 2 * DW; x++) {
                v4u w = __builtin_bit_cast(v4u, q[n][x >> 1][x & 1]);
                w ^= 0x80008000u;
                q[n][x >> 1][x & 1] = __builtin_bit_cast(bf16x8, w);
            }
        }
    }
    const bool active = w0 < rows;
    const int32_t wlo = base + (int32_t)(min(w0, rows - 1) / a.group);
    const int32_t whi = base + (int32_t)(min(w0 + 16 * NR - 1, rows - 1) / a.group);
    // to powers of 2 (at least 2^-120: a masked logit times it stays -infinity)
    const float mul = a.softcap > 0.f ? 1.f : fmaxf(kLog2e * fabsf(a.qscale), 0x1p-120f);
    const float cap_in = a.softcap > 0.f ? 2.f * kLog2e / a.softcap * fabsf(a.qscale) : 0.f, cap_out = a.softcap * kLog2e;

    f32x4 o[NR][4 * DW];
    float mx[NR], sum[NR];
#pragma unroll
    for (uint32_t n = 0; n < NR; n++) {
#pragma unroll
        for (int d = 0; d < 4 * DW; d++) o[n][d] = f32x4{0.f, 0.f, 0.f, 0.f};
        mx[n] = -__builtin_inff();
        sum[n] = 0.f;
        // 0, or NaN for a query that holds a NaN or an infinity (0 times it)
        f32x4 z = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (uint32_t x = 0; x < 2 * DW; x++)
            z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, v4u{0u, 0u, 0u, 0u}), q[n][x >> 1][x & 1], z, 0, 0, 0);
        if (g == 0) least[wave][n][m] = z[0] == 0.f ? -__builtin_inff() : z[0];
    }
    const int32_t* trow = c.table + (uint64_t)(uint32_t)max(sq.row, 0) * c.max_pages;
    const uint64_t hoff = (uint64_t)head * c.page * c.wide;

    // What a wave stages of a tile: waves 0..3 keys (the 16 tokens of step
    // `wave`), waves 4..7 values (channel blocks (wave - 4) DW ..).
    const bool vside = wave >= 4;
    const uint32_t part = wave & 3u;
    struct Next {
        v4u r[DW];
        float scale;
        uint32_t keep;          // tokens of the lane's chunk that count (keys: 0 or 16)
    };
    uint32_t bad = 0;
    // the table's entry for chunk ch of tile i, -1 past the end
    auto entry = [&](uint32_t i, uint32_t ch) {
        if (i >= i1) return -1;
        const uint32_t at = tl.at(i) * kKvTile + 16 * ch;
        return at < end ? trow[at >> c.lp] : -1;
    };
    // an entry's page (0 where there is none: nothing of it is used)
    auto page_of = [&](uint32_t i, uint32_t ch, int32_t e, bool& ok) {
        ok = (uint32_t)e < c.n_pages;
        if (!ok && i < i1 && tl.at(i) * kKvTile + 16 * ch < end) bad = 1;
        return ok ? (uint32_t)e : 0u;
    };
    const uint32_t chst = vside ? g : m >> 2;                       // the lane's chunk of what it stages
    auto stage_load = [&](uint32_t i, int32_t e, Next& x) {
        x.keep = 0;
        if (i >= i1) return;
        const uint32_t tile0 = tl.at(i) * kKvTile, at = tile0 + 16 * chst;
        bool ok;
        const uint32_t p = page_of(i, chst, e, ok);
        x.scale = a.scale[((uint64_t)p * c.kv_heads + head) * 2 + (vside ? 1 : 0)];
        x.keep = ok ? (vside ? min(end - at, 16u) : 16u) : 0u;
        if (vside) {
            const uint8_t* vp = a.v + (uint64_t)p * c.side_bytes + hoff + (uint64_t)(16 * part * DW + m) * c.page + (at & (c.page - 1));
#pragma unroll
            for (uint32_t d = 0; d < DW; d++) x.r[d] = *(const v4u*)(vp + (uint64_t)(16 * d) * c.page);
        } else {
            const uint8_t* kp = a.k + (uint64_t)p * c.side_bytes + hoff + (uint64_t)((at + 4 * part + (m & 3u)) & (c.page - 1)) * D + 16 * g;
#pragma unroll
            for (uint32_t d = 0; d < DW; d++) x.r[d] = *(const v4u*)(kp + 64 * d);
        }
    };
    // operand 2 (part DW + d) of its side, and the next one.  Keys that have no
    // page become NaN, and with them their logits: the softmax leaves these out.
    auto stage_store = [&](uint32_t i, Next& x, uint32_t d) {
        if (i >= i1) return;
        if (x.keep < 16) {
#pragma unroll
            for (int w = 0; w < 4; w++) {
                const int32_t nb = (int32_t)x.keep - 4 * w;
                x.r[d][w] &= nb >= 4 ? ~0u : nb <= 0 ? 0u : (1u << (8 * nb)) - 1u;
                if (E4M3 && !vside) x.r[d][w] = 0x7F7F7F7Fu;         // the code of NaN
            }
        }
        uint8_t* to = buf[(i - i0) & 1u][(vside ? kFrags : 0) + 2 * (part * DW + d)] + 16 * lane;
        const float f = x.keep ? x.scale : E4M3 || vside ? 1.f : __builtin_nanf("");
        *(bf16x8*)to = widen8<E4M3>(x.r[d].x, x.r[d].y, f);
        *(bf16x8*)(to + 1024) = widen8<E4M3>(x.r[d].z, x.r[d].w, f);
    };

    // Ahead of the tile that is multiplied: its successor's operands wait in
    // registers, the one after that is being loaded, and the table's entries
    // are read one more tile ahead, so that no load waits for another.  A wave
    // of the first half stages keys of tile i + 1, one of the second half
    // values of tile i, in its products' phase of tile i.
    const uint32_t off = vside ? 0u : 1u;
    Next nx;
    {
        const int32_t e0 = entry(i0, chst), e1 = entry(i0 + off, chst);
        if (!vside) {
            stage_load(i0, e0, nx);
#pragma unroll
            for (uint32_t d = 0; d < DW; d++) stage_store(i0, nx, d);
        }
        stage_load(i0 + off, e1, nx);
    }
    int32_t est = entry(i0 + off + 1, chst);
    bf16x8 pb[NR][2];
    f32x4 s[NR][4];
    bool prev = false;                                              // pb holds the last tile's probabilities
    // Operands are read from LDS four at a time, a group ahead of the products
    // (left to itself, the compiler reads two and waits for them).
    // Between the groups of the first product, in the shadow of its
    // instructions, a wave does a step of its staging (for tile i1 nothing).
    auto stage_step = [&](uint32_t i, uint32_t b) {
        if (b < DW) stage_store(i + off, nx, b);
        if (b + 1 == DW) stage_load(i + off + 1, est, nx);
        if (b == DW) est = entry(i + off + 2, chst);
    };
    auto pv_product = [&](uint32_t i) {
        const uint8_t* vb = buf[(i - i0) & 1u][kFrags] + 16 * lane;
        bf16x8 f[2][4];
#pragma unroll
        for (uint32_t u = 0; u < 4; u++) f[0][u] = *(const bf16x8*)(vb + 1024 * u);
#pragma unroll
        for (uint32_t b = 0; b < kFrags / 4; b++) {
            if (b + 1 < kFrags / 4) {
#pragma unroll
                for (uint32_t u = 0; u < 4; u++) f[(b + 1) & 1][u] = *(const bf16x8*)(vb + 1024 * (4 * b + 4 + u));
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (uint32_t u = 0; u < 4; u++)
#pragma unroll
                for (uint32_t n = 0; n < NR; n++)
                    o[n][2 * b + (u >> 1)] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[b & 1][u], pb[n][u & 1], o[n][2 * b + (u >> 1)], 0, 0, 0);
            stage_step(i + 1, b);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto qk_product = [&](uint32_t i) {
        const uint8_t* kb = buf[(i - i0) & 1u][0] + 16 * lane;
        bf16x8 f[2][4];
#pragma unroll
        for (uint32_t u = 0; u < 4; u++) f[0][u] = *(const bf16x8*)(kb + 1024 * u);
#pragma unroll
        for (uint32_t h = 0; h < 4; h++)
#pragma unroll
            for (uint32_t n = 0; n < NR; n++) s[n][h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (uint32_t b = 0; b < kFrags / 4; b++) {
            if (b + 1 < kFrags / 4) {
#pragma unroll
                for (uint32_t u = 0; u < 4; u++) f[(b + 1) & 1][u] = *(const bf16x8*)(kb + 1024 * (4 * b + 4 + u));
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (uint32_t u = 0; u < 4; u++)
#pragma unroll
                for (uint32_t n = 0; n < NR; n++) {
                    const uint32_t x = 4 * b + u, h = x / (2 * DW), y = x % (2 * DW);
                    s[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[b & 1][u], q[n][y >> 1][y & 1], s[n][h], 0, 0, 0);
                }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // The two waves of a SIMD are half a tile apart: while one multiplies (O
    // += V P of the last tile, S = K Q of this one), the other takes its
    // exponentials.  Barriers part the phases; in phase 2 i (2 i + 1 for the
    // second half) tile i's keys and tile i - 1's values are read, so keys of
    // tile i + 1 and values of tile i can be written to the buffers that
    // tiles i - 1 and i - 2 have left.
    __syncthreads();
    if (vside) __syncthreads();
    for (uint32_t i = i0; i < i1; i++) {
        const uint32_t tile0 = tl.at(i) * kKvTile;
        // does the wave see any of the tile, or all of it?
        bool any = active && (int32_t)tile0 <= whi;
        bool all = (int32_t)(tile0 + kKvTile - 1) <= wlo;
        if (a.window) {
            any = any && ((int64_t)tile0 + kKvTile - 1 > (int64_t)wlo - a.window || tile0 < a.sinks);
            all = all && ((int64_t)tile0 > (int64_t)whi - a.window || tile0 + kKvTile <= a.sinks);
        }
        __builtin_amdgcn_s_setprio(1);
        if (prev) {
            pv_product(i - 1);
        } else {
#pragma unroll
            for (uint32_t b = 0; b <= DW; b++) stage_step(i, b);
        }
        if (any) qk_product(i);
        __builtin_amdgcn_s_setprio(0);
        __syncthreads();
        if (any) {
#pragma unroll
            for (uint32_t n = 0; n < NR; n++) {
                float p[16];
#pragma unroll
                for (uint32_t e = 0; e < 16; e++) p[e] = s[n][e >> 2][e & 3];
                if (CAP) {
#pragma unroll
                    for (uint32_t e = 0; e < 16; e++) p[e] = capped(p[e] * cap_in, cap_out);
                } else if (a.softcap > 0.f) {
#pragma unroll
                    for (uint32_t e = 0; e < 16; e++)
                        p[e] = cap_out - 2.f * cap_out * __builtin_amdgcn_rcpf(exp2_fast(p[e] * cap_in) + 1.f);
                }
                if (!all) {
#pragma unroll
                    for (uint32_t e = 0; e < 16; e++) {
                        const int32_t tk = (int32_t)(tile0 + 16 * g + e);
                        const bool seen = tk <= pos[n] &&
                                          (a.window == 0 || (int64_t)tk > (int64_t)pos[n] - (int64_t)a.window || (uint32_t)tk < a.sinks);
                        p[e] = seen ? p[e] : -__builtin_inff();
                    }
                }
                // against the maximum so far; only where a row's sum shows
                // that it has been passed by far (or there is none yet: the
                // sum is then infinite or NaN) is the new one looked for
                float x[16], tot = 0.f;
#pragma unroll
                for (uint32_t e = 0; e < 16; e++) {
                    x[e] = exp2_fast(p[e] * mul - mx[n]);
                    tot += x[e];
                }
                if (__builtin_amdgcn_ballot_w64(!(tot <= kGrow)) != 0) {
                    // NaN of a finite query: a token without a page (the larger of two NaN is NaN)
                    const float low = least[wave][n][m];
#pragma unroll
                    for (uint32_t e = 0; e < 16; e++) p[e] = fmaxf(p[e], low);
                    float top = p[0];
#pragma unroll
                    for (uint32_t e = 1; e < 16; e++) top = fmaxf(top, p[e]);
                    const float now = fmaxf(max_groups(top * mul), mx[n]), sub = now == -__builtin_inff() ? 0.f : now;
                    const float alpha = exp2_fast(mx[n] - sub);
                    mx[n] = now;
                    sum[n] *= alpha;
#pragma unroll
                    for (int d = 0; d < 4 * DW; d++) o[n][d] *= alpha;
                    tot = 0.f;
#pragma unroll
                    for (uint32_t e = 0; e < 16; e++) {
                        x[e] = exp2_fast(p[e] * mul - sub);
                        tot += x[e];
                    }
                }
                sum[n] += tot;
#pragma unroll
                for (int y = 0; y < 2; y++)
                    pb[n][y] = __builtin_bit_cast(bf16x8, v4u{pack_bf16(x[8 * y], x[8 * y + 1]), pack_bf16(x[8 * y + 2], x[8 * y + 3]),
                                                              pack_bf16(x[8 * y + 4], x[8 * y + 5]), pack_bf16(x[8 * y + 6], x[8 * y + 7])});
            }
        }
        prev = any;
        __syncthreads();
    }
    if (prev) pv_product(i1 - 1);
    if (!vside) __syncthreads();
    if (bad && c.status) atomicOr(c.status, 4u);
    if (!active) return;
#pragma unroll
    for (uint32_t n = 0; n < NR; n++) {
        const float total = sum_groups(sum[n]);
        if (w0 + 16 * n + m >= rows) continue;
#pragma unroll
        for (uint32_t d = 0; d < 4 * DW; d++) {
            if (a.splits > 1) part_write<DW, false>(a, tok[n], qh[n], split, 16 * d + 4 * g, mx[n], total, o[n][d]);
            else out_write(a, tok[n], qh[n], 16 * d + 4 * g, mx[n], total, o[n][d]);
        }
    }
}

// Joins the splits of attend_rows_kernel: four channels to a thread.  grid:
// (sequences * max_new, blocks of 64 / (16 DW) heads)
template <int DW>
__global__ __launch_bounds__(64) void join_kernel(KvAttend a, uint32_t block_rows) {
    constexpr uint32_t kLanes = 16 * DW, kHeads = 64 / kLanes > 0 ? 64 / kLanes : 1;   // 3: 48 lanes of 64
    const uint32_t seq_i = blockIdx.x / a.max_new, j = blockIdx.x % a.max_new;
    const uint32_t qh = blockIdx.y * kHeads + threadIdx.x / kLanes, ch = 4 * (threadIdx.x % kLanes);
    const Seq sq = get_seq(a, seq_i);
    if (j >= (uint32_t)sq.count || qh >= a.heads || threadIdx.x >= kHeads * kLanes) return;
    const uint32_t r0 = (j * a.group + qh % a.group) / block_rows * block_rows;
    const int32_t base = sq.len - sq.count;
    const uint32_t r1 = min(r0 + block_rows, (uint32_t)sq.count * a.group) - 1;
    const Tiles tl = get_tiles(a, base + (int32_t)(r0 / a.group), base + (int32_t)(r1 / a.group));
    join_row<DW>(a, (uint32_t)sq.s0 + j, qh, ch, min(max(1u, (tl.n + a.chunk - 1) / a.chunk), a.splits));
}

// rows of a workgroup of attend_rows_kernel: two row tiles to a wave where
// the accumulators leave room (head_dim up to 128)
template <int DW>
constexpr int kRowTiles = DW <= 2 ? 2 : 1;

template <int DW, bool E4M3, bool CAP>
int launch(const KvAttend& a, hipStream_t st) {
    if (a.many) {
        constexpr int NR = kRowTiles<DW>;
        const uint32_t row_blocks = (uint32_t)(((uint64_t)a.max_new * a.group + 128 * NR - 1) / (128 * NR));
        const uint32_t combos = a.n_seqs * a.c.kv_heads;
        const dim3 grid((combos + 7) / 8 * 8 * row_blocks, a.splits);
        hipLaunchKernelGGL((attend_rows_kernel<DW, E4M3, NR, CAP>), grid, dim3(512), 0, st, a, row_blocks, combos);
        constexpr uint32_t heads = 64 / (16 * DW) > 0 ? 64 / (16 * DW) : 1;
        if (a.splits > 1) hipLaunchKernelGGL(join_kernel<DW>, dim3(a.n_seqs * a.max_new, (a.heads + heads - 1) / heads), dim3(64), 0, st, a, 128u * NR);
        return (int)hipGetLastError();
    }
    const uint32_t row_tiles = (a.max_new * a.group + 15) / 16;
    const dim3 grid(a.n_seqs * row_tiles, a.c.kv_heads, a.splits);
    hipLaunchKernelGGL((attend_kernel<DW, E4M3, CAP>), grid, dim3(256), 0, st, a, row_tiles);
    return (int)hipGetLastError();
}

template <int DW>
int launch(const KvAttend& a, hipStream_t st) {
    const bool cap = a.softcap > kShortCap;
    if (a.c.type == 1) return cap ? launch<DW, true, true>(a, st) : launch<DW, true, false>(a, st);
    return cap ? launch<DW, false, true>(a, st) : launch<DW, false, false>(a, st);
}

}  // namespace

extern "C" int bsk_kv_attend(const KvAttend* a, void* stream) {
    switch (a->c.wide / 64) {
        case 1: return launch<1>(*a, (hipStream_t)stream);
        case 2: return launch<2>(*a, (hipStream_t)stream);
        case 3: return launch<3>(*a, (hipStream_t)stream);
        case 4: return launch<4>(*a, (hipStream_t)stream);
        default: return (int)hipErrorInvalidValue;
    }
}
