// bs_kv_batch.hip -- the plan of a step's tokens over the paged key/value
// cache (gfx950): offsets, places and slots of the tokens, the rows' pages side
// by side, and how many leading tokens the rows of a group have in common.
//
// One launch, some workgroups to a row: each adds up the counts before its
// own (a few thousand at most, from the L2), so no workgroup waits for
// another.  A row is compared with the first of its group, page by page; the
// workgroup that ends last takes the least of each group.  Where a plan is
// small, each row's workgroup compares its whole group instead, and none is
// the last: 64 rows of 127 pages 8.9 -> 6.2 us, chains of dependent loads
// either way; for more pages than kSmall the reads would be repeated too often.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "bs_kv_device.h"

using namespace bsd;

namespace {

constexpr uint32_t kThreads = 256, kWaves = kThreads / 64;
constexpr uint32_t kSlice = 1024;            // tokens, and columns, of a workgroup
constexpr uint32_t kMaxParts = 64;

__device__ __forceinline__ void flag(uint32_t* status, uint32_t bit) {
    if (status) atomicOr(status, bit);
}

__device__ __forceinline__ void store_through(int32_t* p, int32_t v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

constexpr uint32_t kSmall = 8192, kSmallRows = 512;   // pages of all rows, and rows and groups
// Pages that all rows have room for: rows may be longer than the plan's table is
// wide, and their pages are to be counted in 32 bits and read in a few ms.
constexpr uint64_t kSmallRoom = 1ull << 22;

__device__ __forceinline__ int32_t wave_min(int32_t x) {
#pragma unroll
    for (int s = 32; s; s >>= 1) x = min(x, __shfl_xor(x, s));
    return x;
}

// the records that attention reads: see KvShared
__device__ __forceinline__ void record(int32_t* to, int32_t s0, int32_t s1, int32_t shared, int32_t row, int32_t low, int32_t high) {
    *(int4*)to = make_int4(s0, s1, shared, row);
    *(int4*)(to + 4) = make_int4(low, high, 0, 0);
}

// A group's common tokens, as attention takes them: `few`, the least of those
// `members` of its n rows that have a tile or more in common with the first.  A
// row that has not (a beam that was emptied and grew anew) stands alone and
// costs the others nothing, unless most rows do: all rows of a group are
// multiplied with its common tokens.  (32 samples over 8000 tokens, one of them
// ended: attention 34 us, 69 with each row by itself.)
__device__ __forceinline__ int32_t in_common(uint32_t n, uint32_t members, int32_t few) {
    return members == n || (members >= 2 && members >= n - members) ? few : 0;
}

// A small plan's groups: the row's own, `from` .. `to` - 1 (none where from ==
// to); `first` token of row i, `wrong` where the groups do not ascend.
__device__ __forceinline__ void small_groups(const KvBatch& b, uint32_t i, uint32_t from, uint32_t to, uint32_t first, uint32_t end, int32_t row,
                                             int32_t low, int32_t high) {
    const KvView& c = b.c;
    __shared__ int32_t rows[kSmallRows], lens[kSmallRows], least[3][kWaves];
    __shared__ uint32_t many[kWaves];
    const uint32_t t = threadIdx.x, lane = t & 63u, wave = t >> 6, n = to - from, cap = c.max_pages << c.lp;
    int wrong = 0;
    for (uint32_t g = t; b.offs && g < b.groups; g += kThreads) wrong |= b.offs[g] < 0 || b.offs[g + 1] < b.offs[g] || b.offs[g + 1] > (int32_t)b.n;
    // the least of the waves' numbers, in every thread
    auto join = [&](int32_t few, int32_t lo, int32_t hi) {
        few = wave_min(few);
        lo = wave_min(lo);
        hi = wave_min(-hi);
        if (lane == 0) {
            least[0][wave] = few;
            least[1][wave] = lo;
            least[2][wave] = hi;
        }
        __syncthreads();
        if (t < 3) least[t][0] = min(min(least[t][0], least[t][1]), min(least[t][2], least[t][3]));
        __syncthreads();
    };
    // the group's rows, their lengths and places
    int32_t few = 0x7FFFFFFF, lo = 0x7FFFFFFF, hi = -1;
    uint32_t tokens = 0;
    for (uint32_t j = t; j < n; j += kThreads) {
        const int32_t r = b.seqs[from + j];
        const uint32_t cnt = b.counts ? (uint32_t)max(b.counts[from + j], 0) : 1u;
        const bool known = r >= 0 && (uint32_t)r < c.max_seqs;
        const uint32_t len = known ? min((uint32_t)max(c.lens[r], 0), cap) : 0u;
        rows[j] = known ? r : 0;
        lens[j] = (int32_t)len;
        few = min(few, (int32_t)len);
        tokens += min(cnt, b.total);
        if (cnt && len) {
            lo = min(lo, (int32_t)(len - min(cnt, len)));
            hi = max(hi, (int32_t)len - 1);
        }
    }
    wrong = __syncthreads_or(wrong);
    const uint32_t pages = n ? ((uint32_t)lens[0] + c.page - 1) >> c.lp : 0u;
    const int32_t* lead = c.table + (uint64_t)(uint32_t)(n ? rows[0] : 0) * c.max_pages;
    // (past a shorter row's end the entry may be anything: its length says less already)
    auto differ = [&](uint32_t j, uint32_t col) {
        const int32_t a = lead[col], d = c.table[(uint64_t)(uint32_t)rows[j] * c.max_pages + col];
        return a != d || a < 0 || (uint32_t)a >= c.n_pages;
    };
    for (uint32_t x = t; x < n * pages; x += kThreads)
        if (differ(x / pages, x % pages)) few = min(few, (int32_t)(x % pages << c.lp));
#pragma unroll
    for (int s = 32; s; s >>= 1) tokens += __shfl_xor(tokens, s);
    if (lane == 0) many[wave] = tokens;
    join(few, lo, hi);
    const int32_t shared = n && !wrong ? least[0][0] & ~(int32_t)(kKvTile - 1) : 0;
    int32_t most = shared, mine = shared;
    if (__builtin_expect(n > 1 && !wrong && shared == 0, 0)) {
        // some row has no tile in common with the first: again, a wave to a row
        __shared__ int32_t own;
        __shared__ uint32_t some[kWaves];
        uint32_t members = 0;
        few = lo = 0x7FFFFFFF, hi = -1;
        for (uint32_t j = wave; j < n; j += kWaves) {
            const int32_t len = lens[j];
            int32_t s = min(len, lens[0]);
            for (uint32_t col = lane; col < pages; col += 64)
                if (differ(j, col)) s = min(s, (int32_t)(col << c.lp));
            s = wave_min(s) & ~(int32_t)(kKvTile - 1);
            if (lane == 0 && j == i - from) own = s;
            if (s == 0) continue;
            members++;
            few = min(few, s);
            const int32_t cnt = b.counts ? max(b.counts[from + j], 0) : 1;
            if (cnt) {
                lo = min(lo, len - min(cnt, len));
                hi = max(hi, len - 1);
            }
        }
        if (lane == 0) some[wave] = members;
        join(few, lo, hi);
        most = in_common(n, some[0] + some[1] + some[2] + some[3], least[0][0]);
        mine = own ? most : 0;
    }
    if (t == 0) {
        b.rows[i] = b.seqs[i];
        b.lead[i] = (int32_t)(n ? from : i);
        b.shared[i] = shared;
        b.starts[i] = (int32_t)first;
        if (i + 1 == b.n) b.starts[b.n] = (int32_t)end;
        record(b.info + 4 + 8 * (b.groups + i), (int32_t)first, (int32_t)end, mine, row, low, high);
        if (i == 0 && wrong) flag(c.status, 4u);
    }
    // records of the groups: their first rows write them, the first row of all
    // those that have none
    const uint64_t stop = (uint64_t)first + many[0] + many[1] + many[2] + many[3];
    for (uint32_t g = t; g < b.groups; g += kThreads) {
        const int32_t f = b.offs ? b.offs[g] : 0, e = b.offs ? b.offs[g + 1] : (int32_t)b.n;
        int32_t* to4 = b.info + 4 + 8 * g;
        if (wrong || f == e) {
            if (i == 0) record(to4, 0, 0, 0, -1, 0x7FFFFFFF, -1);
        } else if (f == (int32_t)i) {
            record(to4, (int32_t)first, (int32_t)min(stop, (uint64_t)b.total), most, rows[0], least[1][0], -least[2][0]);
        }
    }
}

// grid: (rows, parts)
__global__ __launch_bounds__(kThreads) void batch_kernel(KvBatch b, int small) {
    const KvView& c = b.c;
    __shared__ uint64_t sums[kWaves];
    __shared__ uint32_t least[kWaves], last;
    const uint32_t t = threadIdx.x, lane = t & 63u, wave = t >> 6, i = blockIdx.x, part = blockIdx.y;
    const int32_t r = b.seqs[i];
    const bool known = r >= 0 && (uint32_t)r < c.max_seqs;
    const int32_t* trow = c.table + (uint64_t)(known ? (uint32_t)r : 0u) * c.max_pages;
    const uint32_t cap = c.max_pages << c.lp;
    const uint32_t len = known ? min((uint32_t)max(c.lens[r], 0), cap) : 0u;
    const uint32_t held = (len + c.page - 1) >> c.lp;

    // the tokens before the row's own; what is negative counts as none
    const int32_t given = b.counts ? b.counts[i] : 1;
    uint64_t before = i;
    if (b.counts) {
        uint64_t x = 0;
        for (uint32_t j = t; j < i; j += kThreads) x += (uint32_t)max(b.counts[j], 0);
#pragma unroll
        for (int s = 32; s; s >>= 1) x += __shfl_xor(x, s);
        if (lane == 0) sums[wave] = x;
        __syncthreads();
        before = sums[0] + sums[1] + sums[2] + sums[3];
    }
    const uint32_t count = (uint32_t)max(given, 0);
    const uint32_t s0 = (uint32_t)min(before, (uint64_t)b.total), s1 = (uint32_t)min(before + count, (uint64_t)b.total);
    uint32_t err = !known || given < 0 || count > b.max_new || count > len || before + count > b.total || (i + 1 == b.n && s1 != b.total) ? 4u : 0u;

    for (uint32_t s = s0 + part * kThreads + t; s < s1; s += gridDim.y * kThreads) {
        const int64_t place = (int64_t)len - (int64_t)count + (int64_t)(s - s0);
        const bool has = place >= 0 && count <= b.max_new;           // (attention leaves longer rows out)
        int64_t slot = -1;
        if (has) {
            const int32_t pg = trow[place >> c.lp];
            if (pg >= 0 && (uint32_t)pg < c.n_pages) slot = ((int64_t)pg << c.lp) + (place & (c.page - 1));
            else err = 4u;
        }
        b.places[s] = has ? (int32_t)place : -1;
        b.slots[s] = slot;
    }
    if (i + 1 == b.n)                                               // tokens of no row
        for (uint32_t s = s1 + part * kThreads + t; s < b.total; s += gridDim.y * kThreads) {
            b.places[s] = -1;
            b.slots[s] = -1;
        }
    for (uint32_t j = part * kThreads + t; j < b.width; j += gridDim.y * kThreads)
        b.table[(uint64_t)i * b.width + j] = j < held ? trow[j] : -1;
    if (err) flag(c.status, err);
    if (part != 0) return;

    // the row's group: the last that begins at i or before
    uint32_t lo = 0, hi = b.groups, first = 0;
    bool grouped = true;
    if (b.offs) {
        while (lo < hi) {
            const uint32_t mid = (lo + hi) / 2;
            if (b.offs[mid] <= (int32_t)i) lo = mid + 1;
            else hi = mid;
        }
        const int32_t f = lo ? b.offs[lo - 1] : -1;
        grouped = lo && f >= 0 && f <= (int32_t)i && (int32_t)i < b.offs[lo];
        first = grouped ? (uint32_t)f : i;
    }
    if (small) {
        const bool any = known && count && len;
        const uint32_t to = !grouped ? first : b.offs ? (uint32_t)min(b.offs[lo], (int32_t)b.n) : b.n;
        small_groups(b, i, first, to, s0, s1, known ? r : 0, any ? (int32_t)(len - min(count, len)) : 0x7FFFFFFF, any ? (int32_t)len - 1 : -1);
        return;
    }
    const int32_t fr = b.seqs[first];
    uint32_t same = 0;
    if (grouped && known && fr >= 0 && (uint32_t)fr < c.max_seqs) {
        const int32_t* frow = c.table + (uint64_t)(uint32_t)fr * c.max_pages;
        const uint32_t both = min(len, min((uint32_t)max(c.lens[fr], 0), cap)), pages = (both + c.page - 1) >> c.lp;
        uint32_t stop = pages;                                      // the first page that differs
        for (uint32_t j0 = 0; j0 < pages; j0 += 4 * kThreads) {
            int32_t x[4], y[4];
#pragma unroll
            for (uint32_t u = 0; u < 4; u++) {
                const uint32_t j = min(j0 + u * kThreads + t, pages - 1);
                x[u] = trow[j];
                y[u] = frow[j];
            }
#pragma unroll
            for (uint32_t u = 0; u < 4; u++)
                if (x[u] != y[u] || x[u] < 0 || (uint32_t)x[u] >= c.n_pages) stop = min(stop, min(j0 + u * kThreads + t, pages - 1));
        }
#pragma unroll
        for (int s = 32; s; s >>= 1) stop = min(stop, (uint32_t)__shfl_xor((int)stop, s));
        if (lane == 0) least[wave] = stop;
        __syncthreads();
        stop = min(min(least[0], least[1]), min(least[2], least[3]));
        same = (uint32_t)min((uint64_t)both, (uint64_t)stop << c.lp) & ~(kKvTile - 1);
    }
    int32_t* mine = b.info + 4 + 8 * (b.groups + i);
    if (t == 0) {
        b.rows[i] = r;
        b.lead[i] = (int32_t)first;
        store_through(b.shared + i, (int32_t)same);
        store_through(b.starts + i, (int32_t)s0);
        if (i + 1 == b.n) store_through(b.starts + b.n, (int32_t)s1);
        const bool any = known && count && len;
        store_through(mine, (int32_t)s0);
        store_through(mine + 1, (int32_t)s1);
        store_through(mine + 2, (int32_t)same);
        store_through(mine + 3, known ? r : 0);                     // its tokens have no place
        store_through(mine + 4, any ? (int32_t)(len - min(count, len)) : 0x7FFFFFFF);
        store_through(mine + 5, any ? (int32_t)len - 1 : -1);
    }
    // the last of the rows' workgroups; the counter is 0 between calls
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (t == 0) last = __hip_atomic_fetch_add((uint32_t*)b.info, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == b.n - 1;
    __syncthreads();
    if (!last) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    // groups that overlap have nothing in common: a token is to be in one at most
    int wrong = 0;
    for (uint32_t g = t; b.offs && g < b.groups; g += kThreads) wrong |= b.offs[g] < 0 || b.offs[g + 1] < b.offs[g] || b.offs[g + 1] > (int32_t)b.n;
    wrong = __syncthreads_or(wrong);
    if (wrong && t == 0) flag(c.status, 4u);
    for (uint32_t g = wave; g < b.groups; g += kWaves) {
        const int32_t f = b.offs ? b.offs[g] : 0, e = b.offs ? b.offs[g + 1] : (int32_t)b.n;
        const uint32_t from = (uint32_t)min(max(f, 0), (int32_t)b.n), to = (uint32_t)min(max(e, (int32_t)from), (int32_t)b.n);
        const int32_t* rec = b.info + 4 + 8 * b.groups;
        const uint32_t n = to - from;
        int32_t few = 0x7FFFFFFF, low = 0x7FFFFFFF, high = -1;
        // of the rows that have `least` tokens in common with the first: how
        // many they all have, and the places of their new ones
        auto join = [&](int32_t least) {
            few = low = 0x7FFFFFFF, high = -1;
            uint32_t members = 0;
            for (uint32_t j = from + lane; j < to; j += 64) {
                const int32_t s = rec[8 * j + 2], l = rec[8 * j + 4], h = rec[8 * j + 5];
                const bool in = s >= least;
                members += in;
                few = min(few, in ? s : 0x7FFFFFFF);
                low = min(low, in ? l : 0x7FFFFFFF);
                high = max(high, in ? h : -1);
            }
#pragma unroll
            for (int s = 32; s; s >>= 1) {
                few = min(few, __shfl_xor(few, s));
                low = min(low, __shfl_xor(low, s));
                high = max(high, __shfl_xor(high, s));
            }
            return members;
        };
        join(0);
        if (n == 0 || wrong) few = 0;
        const int32_t all = few;
        const bool apart = n > 1 && !wrong && few == 0;              // some row has no tile in common with the first
        if (__builtin_expect(apart, 0)) {
            uint32_t members = join(kKvTile);
#pragma unroll
            for (int s = 32; s; s >>= 1) members += __shfl_xor(members, s);
            few = in_common(n, members, few);
        }
        for (uint32_t j = from + lane; j < to; j += 64) {
            b.shared[j] = all;
            if (!apart || rec[8 * j + 2]) b.info[4 + 8 * (b.groups + j) + 2] = few;
        }
        if (lane == 0)
            record(b.info + 4 + 8 * g, b.starts[from], b.starts[to], few, from < to ? max(b.seqs[from], 0) : -1, low, high);
    }
    if (t == 0) __hip_atomic_store((uint32_t*)b.info, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

}  // namespace

extern "C" int bsk_kv_batch(const KvBatch* b, void* stream) {
    const uint32_t most = std::max(std::min(b->max_new, b->total), b->width);
    const uint32_t parts = std::min(kMaxParts, std::max(1u, (most + kSlice - 1) / kSlice));
    const int small = (uint64_t)b->n * b->width <= kSmall && b->width && b->n <= kSmallRows && b->groups <= kSmallRows &&
                      (uint64_t)b->n * b->c.max_pages <= kSmallRoom;
    hipLaunchKernelGGL(batch_kernel, dim3(b->n, parts), dim3(kThreads), 0, (hipStream_t)stream, *b, small);
    return (int)hipGetLastError();
}
