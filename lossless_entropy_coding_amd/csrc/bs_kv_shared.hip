// bs_kv_shared.hip -- attention of rows in groups whose first tokens are on the
// same pages of the 8-bit key/value cache (gfx950).
//
// The softmax over a row's tokens is split in two: the tokens that its group
// has in common, and its own.  For the first, the queries of all rows of a
// group that share a key head are stacked and read the tokens together; for the
// second each row's queries stand alone.  Both leave a part, the result against
// a maximum of its own and the sum of its exponentials, and a second launch
// adds a row's parts:
//
//   o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i,   m = max_i m_i.
//
// A workgroup takes 32 stacked rows and some tiles of 64 tokens, its eight
// waves one tile each in turn.  Products and the lanes' tokens are those of the
// kernel for few rows (bs_kv_attend.hip): S^T = K Q^T, O^T += V^T P^T, keys and
// values straight from memory to the registers of the wave that multiplies
// them.  Here an operand made of 8-bit codes meets two row tiles of 16.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "bs_kv_attend_device.h"

using namespace bsd;

namespace {

constexpr uint32_t kWaves = 8;
constexpr uint32_t kRowTiles = kKvBlock / 16;

// the tiles of a part: a0 .. a0 + na - 1, then b0 ..
struct Part {
    uint32_t a0, na, b0, n;
    __device__ __forceinline__ uint32_t at(uint32_t i) const { return i < na ? a0 + i : b0 + (i - na); }
};

// of the tiles that rows at places lo .. hi see, those before tile `cut`, or those from it on
__device__ __forceinline__ Part get_part(const KvAttend& a, int32_t lo, int32_t hi, uint32_t cut, bool before) {
    const Tiles t = get_tiles(a, lo, hi);
    const uint32_t t1 = t.t0 + (t.n - t.ns);
    Part p;
    p.a0 = before ? 0u : min(t.ns, cut);
    p.na = (before ? min(t.ns, cut) : t.ns) - p.a0;
    p.b0 = before ? min(t.t0, cut) : max(t.t0, cut);
    p.n = p.na + (before ? min(t1, cut) : max(t1, cut)) - p.b0;
    return p;
}

__device__ __forceinline__ int32_t row_min(int32_t x) {
#pragma unroll
    for (int s = 8; s; s >>= 1) x = min(x, __shfl_xor(x, s));
    return x;
}

__device__ __forceinline__ int32_t row_max(int32_t x) {
#pragma unroll
    for (int s = 8; s; s >>= 1) x = max(x, __shfl_xor(x, s));
    return x;
}

// a workgroup's rows and tokens
struct Job {
    uint32_t first, rows, r0;       // first token of the stack, its rows, the block's first
    uint32_t head, split, splits, slot;
    uint32_t cut;                   // tiles in common
    int32_t row;                    // of the table
    bool before, valid;
};

// which group and block of 32 rows: the blocks of the groups one after the other
__device__ __forceinline__ bool find_block(const KvShared& s, uint32_t block, Job& j) {
    const uint32_t lane = threadIdx.x & 63u;
    uint32_t seen = 0;
    for (uint32_t base = 0; base < s.groups; base += 64) {
        const uint32_t g = base + lane;
        int4 x = make_int4(0, 0, 0, -1);
        if (g < s.groups) x = *(const int4*)(s.info + 4 * (g + 1));
        const bool ok = x.x >= 0 && x.y >= x.x && (uint32_t)x.y <= s.a.total && x.z > 0 && x.w >= 0 && (uint32_t)x.w < s.a.c.max_seqs;
        const uint32_t rows = ok ? (uint32_t)(x.y - x.x) * s.a.group : 0u;
        uint32_t n = (rows + kKvBlock - 1) / kKvBlock;
        const uint32_t mine = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t y = __shfl_up(n, d);
            if (lane >= (uint32_t)d) n += y;
        }
        const uint64_t in = __builtin_amdgcn_ballot_w64(block < seen + n);
        if (in) {
            const int who = (int)__builtin_ctzll(in);
            j.first = (uint32_t)__shfl(x.x, who);
            j.rows = (uint32_t)__shfl((int)rows, who);
            j.r0 = (block - seen - (uint32_t)__shfl((int)(n - mine), who)) * kKvBlock;
            j.cut = (uint32_t)__shfl(x.z, who) / kKvTile;
            j.row = __shfl(x.w, who);
            return true;
        }
        seen += (uint32_t)__shfl((int)n, 63);
    }
    return false;
}

// grid: workgroups of the groups' common tokens (row blocks of a key head and
// split follow each other on one XCD, whose L2 they share), then those of the
// rows' own tokens
template <int DW, bool E4M3, bool CAP>
__global__ __launch_bounds__(64 * kWaves, 2) void shared_kernel(KvShared s, uint32_t common) {
    const KvAttend& a = s.a;
    const KvView& c = a.c;
    constexpr uint32_t D = 64 * DW, NR = kRowTiles;
    // steps of keys and channel blocks of values that are loaded at a time: all
    // at once, beside the results of 32 rows, head_dim 256 spills registers
    constexpr uint32_t KS = DW >= 3 ? 2 : 4, VS = DW >= 3 ? 2 * DW : 4 * DW;
    __shared__ __attribute__((aligned(16))) uint8_t qs[NR][2 * DW][1024];
    __shared__ __attribute__((aligned(16))) f32x4 os[kWaves / 2][NR][4 * DW][64];
    __shared__ float ml[kWaves / 2][NR][2][64];

    const uint32_t t = threadIdx.x, lane = t & 63u, m = lane & 15u, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(t >> 6);
    Job j;
    if (blockIdx.x < common) {
        const uint32_t at = blockIdx.x >> 3, combo = (blockIdx.x & 7u) + 8 * (at / s.blocks);
        j.head = combo % c.kv_heads;
        j.split = combo / c.kv_heads;
        j.splits = s.pre;
        j.slot = 0;
        j.before = true;
        j.valid = j.split < s.pre && find_block(s, at % s.blocks, j);
    } else {
        uint32_t x = blockIdx.x - common;
        j.head = x % c.kv_heads;
        x /= c.kv_heads;
        j.r0 = x % s.row_blocks * kKvBlock;
        x /= s.row_blocks;
        const uint32_t seq = x % a.n_seqs;
        j.split = x / a.n_seqs;
        j.splits = s.own;
        j.slot = s.pre;
        j.before = false;
        const int32_t s0 = a.starts[seq], s1 = a.starts[seq + 1];
        j.row = a.seqs[seq];
        j.cut = (uint32_t)max(s.shared[seq], 0) / kKvTile;
        j.valid = s0 >= 0 && s1 >= s0 && (uint32_t)s1 <= a.total && (uint32_t)(s1 - s0) <= a.max_new;
        if (!j.valid && t == 0 && j.r0 == 0 && j.split == 0 && c.status) atomicOr(c.status, 4u);
        j.first = (uint32_t)s0;
        j.rows = j.valid ? (uint32_t)(s1 - s0) * a.group : 0u;
        if (j.row < 0 || (uint32_t)j.row >= c.max_seqs) {           // the plan has given its tokens no place
            if (t == 0 && j.r0 == 0 && j.split == 0 && c.status) atomicOr(c.status, 4u);
            j.row = 0;
        }
        j.valid = j.valid && j.r0 < j.rows;
    }
    if (!j.valid) return;
    const uint32_t nrows = min(kKvBlock, j.rows - j.r0);
    const bool two = nrows > 16;

    // this lane's rows: row m of each row tile
    uint32_t tok[NR], qh[NR];
    int32_t pos[NR];
    const int32_t cap = (int32_t)(c.max_pages << c.lp);
#pragma unroll
    for (uint32_t n = 0; n < NR; n++) {
        const uint32_t r = j.r0 + min(16 * n + m, nrows - 1);
        tok[n] = j.first + r / a.group;
        qh[n] = j.head * a.group + r % a.group;
        pos[n] = min(s.places[tok[n]], cap - 1);
    }
    int32_t lo = 0x7FFFFFFF, hi = -1;
#pragma unroll
    for (uint32_t n = 0; n < NR; n++) {
        if (pos[n] >= 0) lo = min(lo, pos[n]);
        hi = max(hi, pos[n]);
    }
    const bool every = __builtin_amdgcn_ballot_w64(pos[0] < 0 || pos[NR - 1] < 0) == 0;
    lo = __builtin_amdgcn_readfirstlane(row_min(lo));
    hi = __builtin_amdgcn_readfirstlane(row_max(hi));
    const Part pt = get_part(a, lo, hi, j.cut, j.before);
    const uint32_t chunk = max(kWaves, (pt.n + j.splits - 1) / j.splits);
    const uint32_t i0 = j.split * chunk;
    if (j.split > 0 && i0 >= pt.n) return;
    const uint32_t i1 = min(pt.n, i0 + chunk), parts = (pt.n + chunk - 1) / chunk;
    const int32_t* trow = c.table + (uint64_t)(uint32_t)j.row * c.max_pages;
    const uint64_t hoff = (uint64_t)j.head * c.page * c.wide;
    const uint32_t end = (uint32_t)(hi + 1);                        // tokens past it are seen by no row
    auto pages = [&](uint32_t i, int32_t& pk, int32_t& pv) {
        pk = pv = -1;
        if (i >= i1) return;
        const uint32_t tile0 = pt.at(i) * kKvTile, ck = tile0 + 16 * (m >> 2), cv = tile0 + 16 * g;
        if (ck < end) pk = trow[ck >> c.lp];
        if (cv < end) pv = trow[cv >> c.lp];
    };
    int32_t pk1, pv1;
    pages(i0 + wave, pk1, pv1);
    if (wave < NR && (wave == 0 || two)) {
        bf16x8 q[DW][2];
        load_q<DW>(a, wave ? tok[NR - 1] : tok[0], wave ? qh[NR - 1] : qh[0], g, q);
#pragma unroll
        for (uint32_t x = 0; x < 2 * DW; x++) *(bf16x8*)(qs[wave][x] + 16 * lane) = q[x >> 1][x & 1];
    }
    __syncthreads();
    const float sc = a.softcap > 0.f ? a.qscale : a.qscale * kLog2e;
    const float cap_in = a.softcap > 0.f ? 2.f * kLog2e / a.softcap : 0.f, cap_out = a.softcap * kLog2e;

    f32x4 o[NR][4 * DW];
    float mx[NR], sum[NR];
#pragma unroll
    for (uint32_t n = 0; n < NR; n++) {
#pragma unroll
        for (int d = 0; d < 4 * DW; d++) o[n][d] = f32x4{0.f, 0.f, 0.f, 0.f};
        mx[n] = -__builtin_inff();
        sum[n] = 0.f;
    }
    uint32_t bad = 0;

    auto tile = [&](uint32_t i, auto count) {
        constexpr uint32_t N = decltype(count)::value;
        const uint32_t tile0 = pt.at(i) * kKvTile;
        const uint32_t ck = tile0 + 16 * (m >> 2), cv = tile0 + 16 * g;
        const bool okk = (uint32_t)pk1 < c.n_pages, okv = (uint32_t)pv1 < c.n_pages;
        if (cv < end && !okv) bad = 1;
        const uint32_t ipk = okk ? (uint32_t)pk1 : 0u, ipv = okv ? (uint32_t)pv1 : 0u;
        const uint8_t* kp = a.k + (uint64_t)ipk * c.side_bytes + hoff + (uint64_t)((ck + (m & 3u)) & (c.page - 1)) * D + 16 * g;
        const uint8_t* vp = a.v + (uint64_t)ipv * c.side_bytes + hoff + (uint64_t)m * c.page + (cv & (c.page - 1));
        v4u kr[KS][DW], vr[VS];
        auto load_keys = [&](uint32_t h0) {
#pragma unroll
            for (uint32_t h = 0; h < KS; h++)
#pragma unroll
                for (uint32_t x = 0; x < DW; x++) kr[h][x] = *(const v4u*)(kp + 4 * (h0 + h) * D + 64 * x);
        };
        auto load_values = [&](uint32_t d0) {
#pragma unroll
            for (uint32_t d = 0; d < VS; d++) vr[d] = *(const v4u*)(vp + (uint64_t)(16 * (d0 + d)) * c.page);
        };
        load_keys(0);
        const float* sp = a.scale + ((uint64_t)ipv * c.kv_heads + j.head) * 2;
        const float ks = sp[0] * sc, vs = okv ? sp[1] : 0.f;
        if (VS == 4 * DW) load_values(0);
        pages(i + kWaves, pk1, pv1);

        f32x4 sx[N][4];
#pragma unroll
        for (uint32_t h = 0; h < 4; h++) {
            if (KS < 4 && h == KS) {
                __builtin_amdgcn_sched_barrier(0);
                load_keys(h);
            }
#pragma unroll
            for (uint32_t n = 0; n < N; n++) sx[n][h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (uint32_t x = 0; x < DW; x++) {
                const v4u kc = kr[h % KS][x];
                const bf16x8 k0 = widen8<E4M3>(kc.x, kc.y), k1 = widen8<E4M3>(kc.z, kc.w);
#pragma unroll
                for (uint32_t n = 0; n < N; n++) {
                    const bf16x8 q0 = *(const bf16x8*)(qs[n][2 * x] + 16 * lane), q1 = *(const bf16x8*)(qs[n][2 * x + 1] + 16 * lane);
                    sx[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, q0, sx[n][h], 0, 0, 0);
                    sx[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, q1, sx[n][h], 0, 0, 0);
                }
            }
        }
        if (VS < 4 * DW) {
            __builtin_amdgcn_sched_barrier(0);
            load_values(0);
        }
        // what every row sees needs no mask
        bool all = every && (int32_t)(tile0 + kKvTile - 1) <= lo && __builtin_amdgcn_ballot_w64(!okv) == 0;
        if (a.window) all = all && ((int64_t)tile0 > (int64_t)hi - (int64_t)a.window || tile0 + kKvTile <= a.sinks);
        bf16x8 pb[N][2], pl[N][2];
#pragma unroll
        for (uint32_t n = 0; n < N; n++) {
            // step h's element e is token cv + 4 h + e
            float p[16];
            float top = -__builtin_inff();
#pragma unroll
            for (uint32_t e = 0; e < 16; e++) {
                float x = sx[n][e >> 2][e & 3] * ks;
                if (CAP) x = capped(x * cap_in, cap_out);
                else if (a.softcap > 0.f) x = cap_out * (1.f - 2.f * __builtin_amdgcn_rcpf(exp2_fast(x * cap_in) + 1.f));
                p[e] = x;
            }
            if (!all) {
#pragma unroll
                for (uint32_t e = 0; e < 16; e++) {
                    const int32_t tk = (int32_t)(cv + e);
                    const bool seen = okv && tk <= pos[n] &&
                                      (a.window == 0 || (int64_t)tk > (int64_t)pos[n] - (int64_t)a.window || (uint32_t)tk < a.sinks);
                    p[e] = seen ? p[e] : -__builtin_inff();
                }
            }
#pragma unroll
            for (uint32_t e = 0; e < 16; e++) top = fmaxf(top, p[e]);
            top = fmaxf(max_groups(top), mx[n]);
            const float sub = top == -__builtin_inff() ? 0.f : top;
            if (__builtin_amdgcn_ballot_w64(top > mx[n]) != 0) {
                const float alpha = exp2_fast(mx[n] - sub);
                mx[n] = top;
                sum[n] *= alpha;
#pragma unroll
                for (int d = 0; d < 4 * DW; d++) o[n][d] *= alpha;
            }
            float part = 0.f;
#pragma unroll
            for (int e = 0; e < 16; e++) {
                p[e] = exp2_fast(p[e] - sub);
                part += p[e];
            }
            sum[n] += part;
            // P in two BF16 parts
#pragma unroll
            for (int y = 0; y < 2; y++) {
                uint32_t up[4], low[4];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float u = p[8 * y + 2 * e] * vs, v = p[8 * y + 2 * e + 1] * vs;
                    up[e] = pack_bf16(u, v);
                    low[e] = pack_bf16(u - __builtin_bit_cast(float, up[e] << 16), v - __builtin_bit_cast(float, up[e] & 0xFFFF0000u));
                }
                pb[n][y] = __builtin_bit_cast(bf16x8, v4u{up[0], up[1], up[2], up[3]});
                pl[n][y] = __builtin_bit_cast(bf16x8, v4u{low[0], low[1], low[2], low[3]});
            }
        }
#pragma unroll
        for (uint32_t d0 = 0; d0 < 4 * DW; d0 += VS) {
            if (d0) {
                __builtin_amdgcn_sched_barrier(0);
                load_values(d0);
            }
            // what no row sees may hold anything: its values count as 0
            if (cv + 16 > end || !okv) {
                const int32_t left = okv ? (int32_t)(end - cv) : 0;  // tokens of the chunk that are kept
#pragma unroll
                for (uint32_t d = 0; d < VS; d++)
#pragma unroll
                    for (int w = 0; w < 4; w++) {
                        const int32_t nb = left - 4 * w;
                        const uint32_t mask = nb >= 4 ? ~0u : nb <= 0 ? 0u : (1u << (8 * nb)) - 1u;
                        vr[d][w] &= mask;
                    }
            }
#pragma unroll
            for (uint32_t d = 0; d < VS; d++) {
                const bf16x8 v0 = widen8<E4M3>(vr[d].x, vr[d].y), v1 = widen8<E4M3>(vr[d].z, vr[d].w);
#pragma unroll
                for (uint32_t n = 0; n < N; n++) {
                    f32x4& to = o[n][d0 + d];
                    to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, pl[n][0], to, 0, 0, 0);
                    to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, pl[n][1], to, 0, 0, 0);
                    to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, pb[n][0], to, 0, 0, 0);
                    to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, pb[n][1], to, 0, 0, 0);
                }
            }
        }
    };
    if (two) {
        for (uint32_t i = i0 + wave; i < i1; i += kWaves) tile(i, std::integral_constant<uint32_t, NR>{});
    } else {
        for (uint32_t i = i0 + wave; i < i1; i += kWaves) tile(i, std::integral_constant<uint32_t, 1>{});
    }
    if (bad && c.status) atomicOr(c.status, 4u);

    // join the waves that had tiles, always in the same pairs
    const uint32_t busy = min(kWaves, i1 - i0);
    const uint32_t tiles = two ? NR : 1;
#pragma unroll
    for (uint32_t half = kWaves / 2; half; half >>= 1) {
        if (busy <= half) continue;
        if (wave >= half && wave < 2 * half && wave < busy) {
#pragma unroll
            for (uint32_t n = 0; n < NR; n++) {
                if (n >= tiles) break;
                ml[wave - half][n][0][lane] = mx[n];
                ml[wave - half][n][1][lane] = sum[n];
#pragma unroll
                for (int d = 0; d < 4 * DW; d++) os[wave - half][n][d][lane] = o[n][d];
            }
        }
        __syncthreads();
        if (wave < half && wave + half < busy) {
#pragma unroll
            for (uint32_t n = 0; n < NR; n++) {
                if (n >= tiles) break;
                const float other = ml[wave][n][0][lane], top = fmaxf(mx[n], other), sub = top == -__builtin_inff() ? 0.f : top;
                const float f = exp2_fast(mx[n] - sub), h = exp2_fast(other - sub);
                mx[n] = top;
                sum[n] = f * sum[n] + h * ml[wave][n][1][lane];
#pragma unroll
                for (int d = 0; d < 4 * DW; d++) o[n][d] = f * o[n][d] + h * os[wave][n][d][lane];
            }
        }
        __syncthreads();
    }
    if (wave != 0) return;
    const uint32_t slots = s.pre + s.own;
#pragma unroll
    for (uint32_t n = 0; n < NR; n++) {
        const float total = sum_groups(sum[n]);
        if (16 * n + m >= nrows) continue;
        float* pp = a.part + (((uint64_t)tok[n] * a.heads + qh[n]) * slots + j.slot + j.split) * (D + 4);
#pragma unroll
        for (int d = 0; d < 4 * DW; d++) *(f32x4*)(pp + 16 * d + 4 * g) = o[n][d];
        if (g == 0) *(f32x4*)(pp + D) = f32x4{mx[n], total, __builtin_bit_cast(float, parts), 0.f};
    }
}

// Adds a row's parts: those of its group's common tokens, then its own; four
// channels to a thread.  grid: (sequences * max_new, blocks of heads)
template <int DW>
__global__ __launch_bounds__(64) void shared_join_kernel(KvShared s) {
    const KvAttend& a = s.a;
    constexpr uint32_t D = 64 * DW, kLanes = 16 * DW, kHeads = 64 / kLanes > 0 ? 64 / kLanes : 1;
    const uint32_t seq = blockIdx.x / a.max_new, i = blockIdx.x % a.max_new;
    const uint32_t qh = blockIdx.y * kHeads + threadIdx.x / kLanes, ch = 4 * (threadIdx.x % kLanes);
    const int32_t s0 = a.starts[seq], s1 = a.starts[seq + 1];
    if (s0 < 0 || s1 < s0 || (uint32_t)s1 > a.total || (uint32_t)(s1 - s0) > a.max_new) return;
    if (i >= (uint32_t)(s1 - s0) || qh >= a.heads || threadIdx.x >= kHeads * kLanes) return;
    const uint32_t tok = (uint32_t)s0 + i;
    const float* pp = a.part + ((uint64_t)tok * a.heads + qh) * (s.pre + s.own) * (D + 4);
    const bool grouped = s.shared[seq] >= (int32_t)kKvTile;
    const float n0 = pp[D + 2], n1 = pp[s.pre * (D + 4) + D + 2];
    const uint32_t pre = grouped ? min(__builtin_bit_cast(uint32_t, n0), s.pre) : 0u;
    const uint32_t n = pre + min(__builtin_bit_cast(uint32_t, n1), s.own);
    auto part = [&](uint32_t x) { return pp + (x < pre ? x : s.pre + (x - pre)) * (D + 4); };
    float top = -__builtin_inff(), total = 0.f;
    f32x4 o = f32x4{0.f, 0.f, 0.f, 0.f};
    for (uint32_t x0 = 0; x0 < n; x0 += 8) {
        f32x4 v[8], h[8];
        float most = top;
#pragma unroll
        for (uint32_t u = 0; u < 8; u++) {
            const float* px = part(min(x0 + u, n - 1));
            v[u] = *(const f32x4*)(px + ch);
            h[u] = *(const f32x4*)(px + D);
        }
#pragma unroll
        for (uint32_t u = 0; u < 8; u++) most = fmaxf(most, h[u][0]);
        const float sub = most == -__builtin_inff() ? 0.f : most, f = exp2_fast(top - sub);
        top = most;
        total *= f;
        o *= f;
#pragma unroll
        for (uint32_t u = 0; u < 8; u++) {
            const float w = x0 + u < n ? exp2_fast(h[u][0] - sub) : 0.f;
            total += w * h[u][1];
            o += w * v[u];
        }
    }
    out_write(a, tok, qh, ch, top, total, o);
}

template <int DW, bool E4M3, bool CAP>
void launch(const KvShared& s, hipStream_t st) {
    const uint32_t common = (s.a.c.kv_heads * s.pre + 7) / 8 * 8 * s.blocks, own = s.a.n_seqs * s.row_blocks * s.a.c.kv_heads * s.own;
    hipLaunchKernelGGL((shared_kernel<DW, E4M3, CAP>), dim3(common + own), dim3(64 * kWaves), 0, st, s, common);
    constexpr uint32_t heads = 64 / (16 * DW) > 0 ? 64 / (16 * DW) : 1;
    hipLaunchKernelGGL(shared_join_kernel<DW>, dim3(s.a.n_seqs * s.a.max_new, (s.a.heads + heads - 1) / heads), dim3(64), 0, st, s);
}

template <int DW>
int launch(const KvShared& s, hipStream_t st) {
    const bool cap = s.a.softcap > kShortCap;
    if (s.a.c.type == 1) cap ? launch<DW, true, true>(s, st) : launch<DW, true, false>(s, st);
    else cap ? launch<DW, false, true>(s, st) : launch<DW, false, false>(s, st);
    return (int)hipGetLastError();
}

}  // namespace

extern "C" int bsk_kv_shared(const KvShared* s, void* stream) {
    switch (s->a.c.wide / 64) {
        case 1: return launch<1>(*s, (hipStream_t)stream);
        case 2: return launch<2>(*s, (hipStream_t)stream);
        case 3: return launch<3>(*s, (hipStream_t)stream);
        case 4: return launch<4>(*s, (hipStream_t)stream);
        default: return (int)hipErrorInvalidValue;
    }
}
