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
// A workgroup takes 16 stacked rows, 32 in stacks of 64 rows or more with
// head_dim up to 128, and some tiles of 64 tokens, its four waves one tile each
// in turn.  Products and the lanes' tokens are those of the kernel for few
// rows (bs_kv_attend.hip): S^T = K Q^T, O^T += V^T P^T, keys and values straight
// from memory to the registers of the wave that multiplies them.  With 32 rows
// an operand made of 8-bit codes meets two row tiles, and P is rounded to BF16,
// as in the kernel for many rows; else it enters in two BF16 parts.
//
// Measured, join included, beside the kernel for few rows with each row alone:
//   4 x 32 rows on 4099 tokens and up to 1021 more, a window of 4096, 16 query
//     heads on 8 of 256, e4m3: 90 us, 241 (bytes: most are the rows' own)
//   32 rows on 8000 and up to 600 more, 40 heads on 8 of 128, int8: 33 us, 83
//   8 rows of 4 new tokens on 100003, 40 heads on 8 of 128, e4m3: 107 us, 342
//     (a busy CU's matrix instructions take 32% of its SIMDs' time, the vector
//     ones 57%, and they hardly overlap)
// A row's parts joined in this launch by the workgroup that ends last took
// longer: its stores and the others' wait cost 1 to 38 us, the second launch 4.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "bs_kv_attend_device.h"

using namespace bsd;

namespace {

constexpr uint32_t kWaves = 4;

// row tiles of a workgroup of a large stack: two where the accumulators leave
// room for a tile's keys and values in flight (head_dim up to 128)
template <int DW>
constexpr uint32_t kRowTiles = DW <= 2 ? 2 : 1;

// rows of a workgroup of a stack
template <uint32_t NR>
__device__ __forceinline__ uint32_t block_rows(uint32_t rows) {
    return NR > 1 && rows >= kKvStack ? 16 * NR : 16;
}

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

// a workgroup's rows and tokens
struct Job {
    uint32_t first, rows, r0;       // first token of the stack, its rows, the block's first
    uint32_t head, split, splits, slot;
    uint32_t cut;                   // tiles in common
    int32_t row;                    // of the table
    int32_t lo, hi;                 // places of the stack
    bool before, valid;
};

// a record of the plan, checked: its rows, 0 for one that does not hold
__device__ __forceinline__ uint32_t record_rows(const KvShared& s, int4 x, uint32_t most) {
    const bool ok = x.x >= 0 && x.y >= x.x && (uint32_t)x.y <= s.a.total && (uint32_t)(x.y - x.x) <= most && x.z >= 0 && x.w >= 0 &&
                    (uint32_t)x.w < s.a.c.max_seqs;
    return ok ? (uint32_t)(x.y - x.x) * s.a.group : 0u;
}

// which group and block of rows: the blocks of the groups one after the other
template <uint32_t NR>
__device__ __forceinline__ bool find_block(const KvShared& s, uint32_t block, Job& j) {
    const uint32_t lane = threadIdx.x & 63u;
    uint32_t seen = 0;
    for (uint32_t base = 0; base < s.groups; base += 64) {
        const uint32_t g = base + lane;
        int4 x = make_int4(0, 0, 0, -1);
        int2 y = make_int2(0, -1);
        if (g < s.groups) {
            x = *(const int4*)(s.info + 4 + 8 * g);
            y = *(const int2*)(s.info + 8 + 8 * g);
        }
        const uint32_t rows = x.z >= (int32_t)kKvTile ? record_rows(s, x, s.a.total) : 0u;
        const uint32_t mine = NR > 1 && rows >= kKvStack ? (rows + 16 * NR - 1) / (16 * NR) : (rows + 15) / 16;
        uint32_t n = mine;
        if (s.groups > 1) {
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const uint32_t z = __shfl_up(n, d);
                if (lane >= (uint32_t)d) n += z;
            }
        }
        const uint64_t in = __builtin_amdgcn_ballot_w64(g < s.groups && block < seen + n);
        if (in) {
            const int who = (int)__builtin_ctzll(in);
            auto of = [&](int32_t v) { return __builtin_amdgcn_readlane(v, who); };
            j.first = (uint32_t)of(x.x);
            j.rows = (uint32_t)of((int32_t)rows);
            j.r0 = (block - seen - (uint32_t)of((int32_t)(n - mine))) * block_rows<NR>(j.rows);
            j.cut = (uint32_t)of(x.z) / kKvTile;
            j.row = of(x.w);
            j.lo = of(y.x);
            j.hi = of(y.y);
            return true;
        }
        seen += (uint32_t)__shfl((int)n, 63);
    }
    return false;
}

// grid: workgroups of the groups' common tokens (row blocks of a key head and
// split follow each other on one XCD, whose L2 they share), then those of the
// rows' own tokens.  Two waves to a SIMD: 256 registers, and no AGPRs.
template <int DW, bool E4M3, bool CAP>
__global__ __launch_bounds__(64 * kWaves, 2) void shared_kernel(KvShared s, uint32_t common) {
    const KvAttend& a = s.a;
    const KvView& c = a.c;
    constexpr uint32_t D = 64 * DW, NR = kRowTiles<DW>;
    // Q as operands of the product, later the waves' results
    __shared__ __attribute__((aligned(16))) f32x4 os[kWaves / 2][NR][4 * DW][64];
    __shared__ float ml[kWaves / 2][NR][2][64];
    static_assert(sizeof os >= NR * 2 * DW * 1024, "Q fits");
    uint8_t* qs = (uint8_t*)os;

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
        j.valid = j.split < s.pre && find_block<NR>(s, at % s.blocks, j);
    } else {
        uint32_t x = blockIdx.x - common;
        j.head = x % c.kv_heads;
        x /= c.kv_heads;
        j.r0 = x % s.row_blocks * 16;
        x /= s.row_blocks;
        const uint32_t seq = x % a.n_seqs;
        j.split = x / a.n_seqs;
        j.splits = s.own;
        j.slot = s.pre;
        j.before = false;
        const int32_t* at = s.info + 4 + 8 * (s.groups + seq);
        const int4 r = *(const int4*)at;
        const int2 y = *(const int2*)(at + 4);
        j.first = (uint32_t)r.x;
        j.rows = record_rows(s, r, a.max_new);
        j.cut = (uint32_t)r.z / kKvTile;
        j.row = r.w;
        j.lo = y.x;
        j.hi = y.y;
        j.valid = j.r0 < j.rows;
    }
    if (!j.valid) return;
    const bool tall = NR > 1 && j.before && j.rows >= kKvStack;
    const uint32_t nrows = min(tall ? 16 * NR : 16u, j.rows - j.r0);
    j.hi = min(j.hi, (int32_t)(c.max_pages << c.lp) - 1);
    j.lo = min(j.lo, max(j.hi, 0));
    const Part pt = get_part(a, j.lo, j.hi, j.cut, j.before);
    const uint32_t chunk = max(kWaves, (pt.n + j.splits - 1) / j.splits);
    const uint32_t i0 = j.split * chunk;
    if (j.split > 0 && i0 >= pt.n) return;
    const uint32_t i1 = min(pt.n, i0 + chunk), parts = (pt.n + chunk - 1) / chunk;
    const int32_t* trow = c.table + (uint64_t)(uint32_t)j.row * c.max_pages;
    const uint64_t hoff = (uint64_t)j.head * c.page * c.wide;
    const uint32_t end = (uint32_t)(j.hi + 1);                      // tokens past it are seen by no row

    // Entries of the table, then keys, then values are loaded a step ahead:
    // keys of the wave's next tile when this one's are multiplied, its values
    // when this one's are, into the same registers.
    // (Always the same loads in the same order, so that waiting for keys never
    // waits for values: entries come before those, and where there is no tile
    // or token the last one is read again.)
    int32_t pk = -1, pv = -1;                                       // entries of the tile to be loaded
    auto entries = [&](uint32_t i) {
        const uint32_t tile0 = pt.at(min(i, i1 - 1)) * kKvTile, last = (end - 1) >> c.lp;
        pk = trow[min((tile0 + 16 * (m >> 2)) >> c.lp, last)];
        pv = trow[min((tile0 + 16 * g) >> c.lp, last)];
    };
    if (i0 < i1) entries(i0 + wave);

    // this lane's rows: row m of each row tile
    uint32_t tok[NR], qh[NR];
    int32_t pos[NR];
#pragma unroll
    for (uint32_t n = 0; n < NR; n++) {
        const uint32_t r = j.r0 + min(16 * n + m, nrows - 1);
        tok[n] = j.first + r / a.group;
        qh[n] = j.head * a.group + r % a.group;
        pos[n] = s.places[tok[n]];
    }
    if (wave < NR) {
        bf16x8 q[DW][2];
        load_q<DW>(a, wave ? tok[NR - 1] : tok[0], wave ? qh[NR - 1] : qh[0], g, q);
        const uint32_t sign = a.qscale < 0.f ? 0x80008000u : 0u;    // the scale's sign goes into Q
#pragma unroll
        for (uint32_t x = 0; x < 2 * DW; x++)
            *(v4u*)(qs + (wave * 2 * DW + x) * 1024 + 16 * lane) = __builtin_bit_cast(v4u, q[x >> 1][x & 1]) ^ sign;
    }

    // Above head_dim 192 a whole tile's values do not fit beside its keys: the
    // second half of them takes the registers of keys 0 and 1 of each four
    // between their product and the next tile's.
    constexpr bool HALF = DW >= 4;
    constexpr uint32_t VS = HALF ? 2 * DW : 4 * DW;
    v4u kr[4][DW], vr[VS];
    struct Tile {
        const uint8_t *k, *v;
        float ks, vs;           // scales of the lane's pages
        bool ok;                // its own tokens have a page
    };
    Tile now{}, next{};
    auto locate = [&](uint32_t i) {
        const uint32_t tile0 = pt.at(i) * kKvTile, ck = tile0 + 16 * (m >> 2), cv = tile0 + 16 * g;
        next.ok = cv < end && (uint32_t)pv < c.n_pages;
        const uint32_t ik = (uint32_t)pk < c.n_pages ? (uint32_t)pk : 0u, iv = (uint32_t)pv < c.n_pages ? (uint32_t)pv : 0u;
        next.k = a.k + (uint64_t)ik * c.side_bytes + hoff + (uint64_t)((ck + (m & 3u)) & (c.page - 1)) * D + 16 * g;
        next.v = a.v + (uint64_t)iv * c.side_bytes + hoff + (uint64_t)m * c.page + (cv & (c.page - 1));
        // e4m3: the scale of keys goes into the operand, so it is that of the
        // operand's token; int8: into the product, so that of the product's
        next.ks = a.scale[((uint64_t)(E4M3 ? ik : iv) * c.kv_heads + j.head) * 2];
        next.vs = a.scale[((uint64_t)iv * c.kv_heads + j.head) * 2 + 1];
    };
    auto load_keys = [&](const Tile& from, uint32_t h0, uint32_t h1) {
#pragma unroll
        for (uint32_t h = h0; h < h1; h++)
#pragma unroll
            for (uint32_t x = 0; x < DW; x++) kr[h][x] = *(const v4u*)(from.k + 4 * h * D + 64 * x);
    };
    auto load_values = [&](const Tile& from) {
#pragma unroll
        for (uint32_t d = 0; d < VS; d++) vr[d] = *(const v4u*)(from.v + (uint64_t)(16 * d) * c.page);
    };
    if (i0 + wave < i1) {
        locate(i0 + wave);
        load_keys(next, HALF ? 2 : 0, 4);
        if (HALF) load_keys(next, 0, 2);
        entries(i0 + wave + kWaves);
        load_values(next);
        now = next;
    }
    const bool every = __builtin_amdgcn_ballot_w64(pos[0] < 0 || pos[NR - 1] < 0) == 0;
    __syncthreads();
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
    }
    uint32_t bad = 0;

    // one tile: N row tiles, P in one or two BF16 parts
    auto tile = [&](uint32_t i, auto count, auto twice) {
        constexpr uint32_t N = decltype(count)::value;
        constexpr bool TWO = decltype(twice)::value;
        const uint32_t tile0 = pt.at(i) * kKvTile, cv = tile0 + 16 * g;
        const bool more = i + kWaves < i1;
        f32x4 sx[N][4];
        auto qk = [&](uint32_t h0, uint32_t h1) {
#pragma unroll
            for (uint32_t h = h0; h < h1; h++)
#pragma unroll
                for (uint32_t n = 0; n < N; n++) sx[n][h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (uint32_t x = 0; x < DW; x++) {
                bf16x8 q[N][2];
#pragma unroll
                for (uint32_t n = 0; n < N; n++)
#pragma unroll
                    for (uint32_t y = 0; y < 2; y++) q[n][y] = *(const bf16x8*)(qs + (n * 2 * DW + 2 * x + y) * 1024 + 16 * lane);
#pragma unroll
                for (uint32_t h = h0; h < h1; h++) {
                    v4u kc = kr[h][x];
                    // (left to itself, the compiler takes int8 codes apart where
                    // they are loaded, and spills what it makes of them)
                    if (!E4M3) asm volatile("" : "+v"(kc));
                    const float f = E4M3 ? now.ks : 1.f;
                    const bf16x8 k0 = widen8<E4M3>(kc.x, kc.y, f), k1 = widen8<E4M3>(kc.z, kc.w, f);
#pragma unroll
                    for (uint32_t n = 0; n < N; n++) sx[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, q[n][0], sx[n][h], 0, 0, 0);
#pragma unroll
                    for (uint32_t n = 0; n < N; n++) sx[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, q[n][1], sx[n][h], 0, 0, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        if (HALF) {
            qk(2, 4);
            if (more) {
                locate(i + kWaves);
                load_keys(next, 2, 4);
                entries(i + 2 * kWaves);
            }
            qk(0, 2);
#pragma unroll
            for (uint32_t d = 0; d < VS; d++) kr[d / DW][d % DW] = *(const v4u*)(now.v + (uint64_t)(16 * (VS + d)) * c.page);
        } else {
            qk(0, 4);
            if (more) {
                locate(i + kWaves);
                load_keys(next, 0, 4);
                entries(i + 2 * kWaves);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        const bool okv = now.ok;
        const float kscale = now.ks, vscale = okv ? now.vs : 0.f;
        if (cv < end && !okv) bad = 1;
        // what every row sees needs no mask
        bool all = every && (int32_t)(tile0 + kKvTile - 1) <= j.lo && __builtin_amdgcn_ballot_w64(!okv) == 0;
        if (a.window) all = all && ((int64_t)tile0 > (int64_t)j.hi - (int64_t)a.window || tile0 + kKvTile <= a.sinks);
        bf16x8 pb[N][2], pl[N][2];
#pragma unroll
        for (uint32_t n = 0; n < N; n++) {
            // step h's element e is token cv + 4 h + e
            float p[16];
#pragma unroll
            for (uint32_t e = 0; e < 16; e++) p[e] = E4M3 ? sx[n][e >> 2][e & 3] : sx[n][e >> 2][e & 3] * kscale;
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
                    const int32_t tk = (int32_t)(cv + e);
                    const bool seen = okv && tk <= pos[n] &&
                                      (a.window == 0 || (int64_t)tk > (int64_t)pos[n] - (int64_t)a.window || (uint32_t)tk < a.sinks);
                    p[e] = seen ? p[e] : -__builtin_inff();
                }
            }
            // against the maximum so far; only where a row's sum shows that it
            // has been passed by far (or there is none yet: the sum is then
            // infinite or NaN) is the new one looked for
            float x[16], tot = 0.f;
#pragma unroll
            for (uint32_t e = 0; e < 16; e++) {
                x[e] = exp2_fast(p[e] * mul - mx[n]);
                tot += x[e];
            }
            if (__builtin_amdgcn_ballot_w64(!(tot <= kGrow)) != 0) {
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
            for (int y = 0; y < 2; y++) {
                uint32_t up[4], low[4];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float f = E4M3 ? 1.f : vscale, u = x[8 * y + 2 * e] * f, v = x[8 * y + 2 * e + 1] * f;
                    up[e] = pack_bf16(u, v);
                    if (TWO) low[e] = pack_bf16(u - __builtin_bit_cast(float, up[e] << 16), v - __builtin_bit_cast(float, up[e] & 0xFFFF0000u));
                }
                pb[n][y] = __builtin_bit_cast(bf16x8, v4u{up[0], up[1], up[2], up[3]});
                if (TWO) pl[n][y] = __builtin_bit_cast(bf16x8, v4u{low[0], low[1], low[2], low[3]});
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        // what no row sees may hold anything: its values count as 0
        const int32_t left = okv ? (int32_t)(end - cv) : 0;          // tokens of the chunk that are kept
        if (__builtin_amdgcn_ballot_w64(left < 16) != 0) {
            uint32_t mask[4];
#pragma unroll
            for (int e = 0; e < 4; e++) mask[e] = left >= 4 * e + 4 ? ~0u : left <= 4 * e ? 0u : (1u << (8 * (left - 4 * e))) - 1u;
            const v4u keep = {mask[0], mask[1], mask[2], mask[3]};
#pragma unroll
            for (uint32_t d = 0; d < VS; d++) vr[d] &= keep;
            if (HALF) {
#pragma unroll
                for (uint32_t d = 0; d < VS; d++) kr[d / DW][d % DW] &= keep;
            }
        }
        auto pv_block = [&](v4u w, uint32_t d) {
            const float f = E4M3 ? vscale : 1.f;
            const bf16x8 v0 = widen8<E4M3>(w.x, w.y, f), v1 = widen8<E4M3>(w.z, w.w, f);
            if (TWO) {
#pragma unroll
                for (uint32_t n = 0; n < N; n++) o[n][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, pl[n][0], o[n][d], 0, 0, 0);
#pragma unroll
                for (uint32_t n = 0; n < N; n++) o[n][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, pl[n][1], o[n][d], 0, 0, 0);
            }
#pragma unroll
            for (uint32_t n = 0; n < N; n++) o[n][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, pb[n][0], o[n][d], 0, 0, 0);
#pragma unroll
            for (uint32_t n = 0; n < N; n++) o[n][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, pb[n][1], o[n][d], 0, 0, 0);
            if (d & 1) __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (uint32_t d = 0; d < VS; d++) pv_block(vr[d], d);
        if (more) load_values(next);
        if (HALF) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (uint32_t d = 0; d < VS; d++) pv_block(kr[d / DW][d % DW], VS + d);
            if (more) load_keys(next, 0, 2);
        }
        now = next;
        __builtin_amdgcn_sched_barrier(0);
    };
    // Two row tiles share an operand, and P enters in one part, in large
    // stacks; what would be a third form (two row tiles, P in two parts) makes
    // the compiler spill registers in all of them.
    if (tall) {
        for (uint32_t i = i0 + wave; i < i1; i += kWaves) tile(i, std::integral_constant<uint32_t, NR>{}, std::integral_constant<bool, NR == 1>{});
    } else {
        for (uint32_t i = i0 + wave; i < i1; i += kWaves) tile(i, std::integral_constant<uint32_t, 1>{}, std::true_type{});
    }
    if (bad && c.status) atomicOr(c.status, 4u);

    // join the waves that had tiles, always in the same pairs
    const uint32_t busy = min(kWaves, i1 - i0), high = (nrows + 15) / 16;
    __syncthreads();                                                // Q is not needed any more
#pragma unroll
    for (uint32_t half = kWaves / 2; half; half >>= 1) {
        if (busy <= half) continue;
        if (wave >= half && wave < 2 * half && wave < busy) {
#pragma unroll
            for (uint32_t n = 0; n < NR; n++) {
                if (n >= high) break;
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
                if (n >= high) break;
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
    const int4 r = *(const int4*)(s.info + 4 + 8 * (s.groups + seq));
    if (i * a.group >= record_rows(s, r, a.max_new) || qh >= a.heads || threadIdx.x >= kHeads * kLanes) return;
    const uint32_t tok = (uint32_t)r.x + i;
    const float* pp = a.part + ((uint64_t)tok * a.heads + qh) * (s.pre + s.own) * (D + 4);
    const bool grouped = r.z >= (int32_t)kKvTile && s.places[tok] >= 0;
    const uint32_t slots = s.pre + s.own;
    uint32_t pre = 0, own = 0;
    float top = -__builtin_inff(), total = 0.f;
    f32x4 o = f32x4{0.f, 0.f, 0.f, 0.f};
    // eight places at a time; the first eight are read, used or not, while the
    // numbers of parts are
    const float n0 = pp[D + 2], n1 = pp[s.pre * (D + 4) + D + 2];
    for (uint32_t x0 = 0; x0 < slots; x0 += 8) {
        if (x0 && x0 >= pre && (x0 + 8 <= s.pre || x0 >= s.pre + own)) continue;
        f32x4 v[8];
        float f[8], l[8], most = top;
#pragma unroll
        for (uint32_t u = 0; u < 8; u++) {
            const float* px = pp + min(x0 + u, slots - 1) * (D + 4);
            v[u] = *(const f32x4*)(px + ch);
            f[u] = px[D];
            l[u] = px[D + 1];
        }
        if (x0 == 0) {
            pre = grouped ? min(__builtin_bit_cast(uint32_t, n0), s.pre) : 0u;
            own = min(__builtin_bit_cast(uint32_t, n1), s.own);
        }
#pragma unroll
        for (uint32_t u = 0; u < 8; u++) {
            const uint32_t x = x0 + u;
            const bool used = x < pre || (x >= s.pre && x < s.pre + own);
            f[u] = used ? f[u] : -__builtin_inff();
            l[u] = used ? l[u] : 0.f;
#pragma unroll
            for (int e = 0; e < 4; e++) v[u][e] = used ? v[u][e] : 0.f;
            most = fmaxf(most, f[u]);
        }
        const float sub = most == -__builtin_inff() ? 0.f : most, g = exp2_fast(top - sub);
        top = most;
        total *= g;
        o *= g;
#pragma unroll
        for (uint32_t u = 0; u < 8; u++) {
            const float w = exp2_fast(f[u] - sub);
            total += w * l[u];
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
