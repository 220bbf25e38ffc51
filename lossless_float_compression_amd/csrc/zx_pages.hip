// zx_pages.hip -- who holds which page of a paged K/V cache: rows of the table that go on from other
// rows, pages given out and taken back, pages brought together at the front of the pool.
//
// All there is to keep is refs[page], the number of rows that hold a page; a page with none is free, and free
// pages are given out from the lowest up.  So nothing has to be kept in step with refs, and what a call does follows from its
// arguments alone: counts are added up with atomics on whole numbers, whose order does not show, and ranks come
// from prefix sums over the pool, which a launch ahead has counted by segments of kSegment pages.
//
// Bound by launches (one or two of 3 to 6 us) for the pools and tables of a serving step: each is a chain of trips to memory, lengths -> table ->
// counts -> ranks, so what does not depend on each other is read together, and pools of up to 4096 pages are served by one workgroup in
// one launch.  The bytes are the table's entries in use and refs, read and written once.
// Four beams over 1000 tokens: fork 4.0 us, extend 5.0; 64 x 8 beams over 32768 tokens in pages of 16 (a million
// entries): 9.9 + 2.0 and 4.6 + 5.6; 256 sequences, five tokens each: trim 3.0, extend 4.0 + 4.9; 16 prompts of 20000: 4.5, 3.4 + 5.7;
// 6000 pages brought together: 9.0.
#include "zx_paged.h"

namespace zxg {

using zxk::report;
using zxp::ceil_div;
using zxp::div_up;

constexpr uint32_t kMostPages = 1u << 23;
constexpr uint32_t kMostSeqs = 2048;             // of one call that gives out pages, and beams of a group
constexpr uint32_t kThreads = 1024;
constexpr uint32_t kEach = 4;                    // pages of a thread
constexpr uint32_t kSegment = kThreads * kEach;  // pages whose free ones a workgroup counts

struct Pool {
    int32_t *refs;
    uint32_t n_pages, log_page;
    uint32_t *err;
};

struct Rows {
    int32_t *table, *held;
    uint32_t n, width;
    int32_t cap;                                 // tokens that a row of the table has room for
};

__device__ __forceinline__ uint32_t pages_of(const Pool &p, int32_t tokens) { return ((uint32_t)tokens + (1u << p.log_page) - 1u) >> p.log_page; }

// Sums over the workgroup of two numbers, and over the threads ahead of this one.  `sums` is free again at the next barrier.
struct Two {
    uint32_t a, b;
};
__device__ __forceinline__ Two block_scan(Two v, Two (&sums)[kThreads / 64], Two &total)
{
    Two w;
    Two ex{zxk::wave_excl_scan(v.a, w.a), zxk::wave_excl_scan(v.b, w.b)};
    __syncthreads();
    if ((threadIdx.x & 63u) == 63u) sums[threadIdx.x >> 6] = w;
    __syncthreads();
    total = Two{0, 0};
#pragma unroll
    for (uint32_t i = 0; i < kThreads / 64; ++i) {
        const Two s = sums[i];
        if (i < threadIdx.x >> 6) {
            ex.a += s.a;
            ex.b += s.b;
        }
        total.a += s.a;
        total.b += s.b;
    }
    return ex;
}

// Bit i: page `first` + i is free, of a thread's kEach.
__device__ __forceinline__ uint32_t free_bits(const Pool &p, uint32_t first)
{
    int32_t r[kEach];
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i) r[i] = first + i < p.n_pages ? p.refs[first + i] : 1;
    uint32_t m = 0;
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i) m |= (uint32_t)(r[i] <= 0) << i;
    return m;
}

// ---------------------------------------------------------------- rows go on from other rows

struct ForkArgs {
    Pool p;
    Rows r;
    const int32_t *parents;
    uint32_t beams, log_strip;                   // columns that a workgroup holds at a time
    uint32_t share;                              // workgroups of a group; a single one writes the lengths too
};

// The lengths and parents of a group into LDS, and the most pages that a row has; whether all are in range.
__device__ __forceinline__ bool load_group(const ForkArgs &g, uint32_t group, int32_t *held, int32_t *parent, uint32_t *bad, uint32_t *cols)
{
    if (threadIdx.x == 0) *bad = *cols = 0;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < g.beams; i += blockDim.x) {
        const int32_t h = g.r.held[(uint64_t)group * g.beams + i], q = g.parents[(uint64_t)group * g.beams + i];
        held[i] = h;
        parent[i] = q;
        if (h < 0 || h > g.r.cap || q < -1 || q >= (int32_t)g.beams) *bad = 1;
        else atomicMax(cols, pages_of(g.p, h));
    }
    __syncthreads();
    if (*bad && threadIdx.x == 0) report(g.p.err, ZX_E_CORRUPT);
    return !*bad;
}

// Old rows are read into LDS strip by strip, then written where they go on, so rows may trade places.  A page's
// count changes by (rows that go on from a row that holds it) - 1 for each such row; these are added up over
// neighbouring rows that hold the same page in a column (beams of one prompt mostly do), and most sums are zero.
__global__ __launch_bounds__(1024) void k_pages_fork(ForkArgs g)
{
    extern __shared__ int32_t lds[];
    __shared__ uint32_t bad, cols;
    int32_t *held = lds, *parent = held + g.beams, *children = parent + g.beams, *strip = children + g.beams;
    const uint32_t group = blockIdx.x / g.share, nth = blockIdx.x % g.share, tid = threadIdx.x, ls = g.log_strip, ns = 1u << ls;
    int32_t *table = g.r.table + (uint64_t)group * g.beams * g.r.width;
    int32_t x[4];                                // four entries of a thread under way at once, the first beside the lengths
    auto read = [&](uint32_t c0, uint32_t i0, auto in) {
#pragma unroll
        for (uint32_t u = 0; u < 4; ++u) {
            const uint32_t i = i0 + u * blockDim.x, r = i >> ls, c = c0 + (i & (ns - 1));
            x[u] = 0;
            if (r < g.beams && in(r, c)) x[u] = table[(uint64_t)r * g.r.width + c];
        }
    };
    const uint32_t first = nth * ns;
    read(first, tid, [&](uint32_t, uint32_t c) { return c < g.r.width; });
    if (!load_group(g, group, held, parent, &bad, &cols)) return;
    for (uint32_t i = tid; i < g.beams; i += blockDim.x) children[i] = 0;
    __syncthreads();
    for (uint32_t i = tid; i < g.beams; i += blockDim.x)
        if (parent[i] >= 0) atomicAdd(&children[parent[i]], 1);
    for (uint32_t c0 = first; c0 < cols; c0 += g.share * ns) {
        const uint32_t nc = cols - c0 < ns ? cols - c0 : ns;
        __syncthreads();
        for (uint32_t i0 = tid; i0 < g.beams << ls; i0 += 4 * blockDim.x) {
            if (c0 != first || i0 != tid) read(c0, i0, [&](uint32_t r, uint32_t c) { return c < pages_of(g.p, held[r]); });
#pragma unroll
            for (uint32_t u = 0; u < 4; ++u)
                if (i0 + u * blockDim.x < g.beams << ls) strip[i0 + u * blockDim.x] = x[u];
        }
        __syncthreads();
        for (uint32_t i = tid; i < g.beams << ls; i += blockDim.x) {
            const uint32_t r = i >> ls, c = i & (ns - 1);
            const int32_t q = parent[r];
            if (q >= 0 && q != (int32_t)r && c < nc && c0 + c < pages_of(g.p, held[q]))
                table[(uint64_t)r * g.r.width + c0 + c] = strip[((uint32_t)q << ls) + c];
        }
        // runs of up to 64 neighbouring rows that hold the same page in a column, one thread each
        for (uint32_t i = tid; i < g.beams << ls; i += blockDim.x) {
            const uint32_t r = i >> ls, c = i & (ns - 1), page = (uint32_t)strip[i];
            auto holds = [&](uint32_t q) { return c0 + c < pages_of(g.p, held[q]) && (uint32_t)strip[(q << ls) + c] == page; };
            if (!holds(r) || ((r & 63u) && holds(r - 1))) continue;
            int32_t sum = children[r] - 1;
            for (uint32_t q = r + 1; q < g.beams && (q & 63u) && holds(q); ++q) sum += children[q] - 1;
            if (sum == 0) continue;
            if (page >= g.p.n_pages || atomicAdd(&g.p.refs[page], sum) + sum < 0) report(g.p.err, ZX_E_CORRUPT);
        }
    }
    if (g.share == 1)
        for (uint32_t i = tid; i < g.beams; i += blockDim.x)
            if (parent[i] != (int32_t)i) g.r.held[(uint64_t)group * g.beams + i] = parent[i] < 0 ? 0 : held[parent[i]];
}

// The lengths, where several workgroups of a group had to read them.
__global__ __launch_bounds__(256) void k_pages_fork_held(ForkArgs g)
{
    extern __shared__ int32_t lds[];
    __shared__ uint32_t bad, cols;
    int32_t *held = lds, *parent = held + g.beams;
    if (!load_group(g, blockIdx.x, held, parent, &bad, &cols)) return;
    for (uint32_t i = threadIdx.x; i < g.beams; i += blockDim.x)
        g.r.held[(uint64_t)blockIdx.x * g.beams + i] = parent[i] < 0 ? 0 : held[parent[i]];
}

// ---------------------------------------------------------------- rows give pages back

__global__ __launch_bounds__(1024) void k_pages_trim(Pool p, Rows r, const int32_t *keep)
{
    const uint32_t s = blockIdx.x;
    const int32_t held = r.held[s], want = keep ? keep[s] : 0;
    if (held < 0 || held > r.cap || want < 0) {
        if (threadIdx.x == 0) report(p.err, ZX_E_CORRUPT);
        return;
    }
    if (want >= held) return;
    const uint32_t first = pages_of(p, want), end = pages_of(p, held);
    const int32_t *row = r.table + (uint64_t)s * r.width;
    for (uint32_t c = first + threadIdx.x; c < end; c += blockDim.x) {
        const uint32_t page = (uint32_t)row[c];
        if (page >= p.n_pages) report(p.err, ZX_E_CORRUPT);
        else if (atomicAdd(&p.refs[page], -1) <= 0) report(p.err, ZX_E_CORRUPT);
    }
    __syncthreads();                             // all have read the length
    if (threadIdx.x == 0) r.held[s] = want;
}

// ---------------------------------------------------------------- pages are given out

struct Need {
    uint32_t before;                             // pages that the sequences ahead take
    uint32_t first;                              // first table place that is given a page
    uint32_t pair;                               // bit 31: that place's old page is copied, as this pair
    uint32_t tokens;                             // of it
    int32_t held, kv;                            // lengths after the call
    uint32_t old, left;                          // bit 31 of old: this sequence sets that page's count to `left`
};
constexpr uint32_t kFlag = 1u << 31, kPairBits = 12;

struct ExtendArgs {
    Pool p;
    Rows r;
    const int32_t *q_start;
    int32_t *kv_len, *pairs, *count;
    uint32_t max_q;
    Need *need;                                  // [n]
    uint64_t *total;                             // pages wanted, and pairs
    uint32_t *counted;                           // [segments] free pages
    uint32_t n_segments, log_slots;
};

// What every sequence needs, by one workgroup.  A sequence that goes on in a page which others hold too
// may not write there: it gets a page of its own and a copy of what it has, unless all that hold the page go on
// in this call, when the first of them keeps it.  How many go on in a page, and who is first, is counted in a
// hash table in LDS; neither depends on the order of entry.
__device__ __forceinline__ void find_needs(const ExtendArgs &g, uint32_t *slots, Two (&sums)[kThreads / 64])
{
    // slots: [slot][3]: page + 1, sequences that write it, the first of them
    const uint32_t tid = threadIdx.x;
    Two total;
    constexpr uint32_t kSeqs = kMostSeqs / kThreads;         // sequences of a thread, side by side
    const uint32_t T = 1u << g.p.log_page, per = div_up(g.r.n, kThreads), s0 = tid * per;
    struct Seq {
        int32_t nq, held;
        uint32_t page, refs;                     // refs > 0 where it goes on in a page that has tokens
        bool ok;
    } v[kSeqs];
#pragma unroll
    for (uint32_t i = 0; i < kSeqs; ++i) {
        const uint32_t s = s0 + i;
        v[i] = Seq{0, 0, 0, 0, false};
        if (i >= per || s >= g.r.n) continue;
        const int32_t q0 = g.q_start[s], q1 = g.q_start[s + 1], held = g.r.held[s];
        v[i].held = held;
        // (differences in 64 bits: lengths that are nonsense must not wrap into sense)
        const int64_t nq = (int64_t)q1 - q0, all = nq + held;
        if (q0 < 0 || nq < 0 || nq > (int64_t)g.max_q || held < 0 || all > (int64_t)g.r.cap) continue;
        v[i].nq = (int32_t)nq;
        v[i].ok = true;
        if (nq > 0 && (uint32_t)held & (T - 1)) {
            v[i].page = (uint32_t)g.r.table[(uint64_t)s * g.r.width + ((uint32_t)held >> g.p.log_page)];
            const int32_t refs = v[i].page < g.p.n_pages ? g.p.refs[v[i].page] : 0;
            if (refs <= 0) v[i].ok = false;      // no page, or one that nobody is said to hold
            else v[i].refs = (uint32_t)refs;
        }
    }
    const uint32_t n_slots = 1u << g.log_slots, mask = n_slots - 1;
    for (uint32_t i = tid; i < n_slots; i += kThreads) {
        slots[3 * i] = slots[3 * i + 1] = 0;
        slots[3 * i + 2] = 0xFFFFFFFFu;
    }
    __syncthreads();
    uint32_t slot[kSeqs];
#pragma unroll
    for (uint32_t i = 0; i < kSeqs; ++i) {
        slot[i] = 0;
        if (i >= per || s0 + i >= g.r.n) continue;
        if (!v[i].ok) report(g.p.err, ZX_E_CORRUPT);
        if (!v[i].ok || v[i].refs == 0) continue;
        uint32_t j = (v[i].page * 0x9E3779B1u) >> (32 - g.log_slots);
        for (;;) {                               // (twice as many slots as sequences: one is free)
            const uint32_t was = atomicCAS(&slots[3 * j], 0u, v[i].page + 1);
            if (was == 0 || was == v[i].page + 1) break;
            j = (j + 1) & mask;
        }
        atomicAdd(&slots[3 * j + 1], 1u);
        atomicMin(&slots[3 * j + 2], s0 + i);
        slot[i] = j;
    }
    __syncthreads();
    Need d[kSeqs];
    uint32_t n[kSeqs];
    Two mine{0, 0};
#pragma unroll
    for (uint32_t i = 0; i < kSeqs; ++i) {
        d[i] = Need{};
        n[i] = 0;
        if (!v[i].ok) {
            d[i].held = v[i].held;               // left out: it stays as it is
            continue;
        }
        d[i].held = d[i].kv = v[i].held + v[i].nq;
        d[i].first = pages_of(g.p, v[i].held);
        if (v[i].refs > 0) {
            const uint32_t writers = slots[3 * slot[i] + 1];
            const bool leads = slots[3 * slot[i] + 2] == s0 + i;
            d[i].old = v[i].page;
            if (leads) {
                d[i].old |= kFlag;
                d[i].left = writers >= v[i].refs ? 1 : v[i].refs - writers;
            }
            d[i].tokens = (uint32_t)v[i].held & (T - 1);
            if (!(leads && writers >= v[i].refs)) {
                d[i].pair = kFlag;
                --d[i].first;
            }
        }
        n[i] = v[i].nq > 0 ? pages_of(g.p, d[i].held) - d[i].first : 0;
        if (n[i] > g.p.n_pages) n[i] = g.p.n_pages + 1;
        mine.a += n[i];
        mine.b += (d[i].pair ? 1u : 0u) + (n[i] >> 15 << kPairBits);
    }
    // 2048 times 2^23 pages would not fit 32 bits.  Beside the pairs go the parts' sums in units of 2^15 pages, which do (2^19 above
    // 12 bits), and where these are no more than the pool, the whole sum is below 2^23 + 2048 * 2^15
    const Two ahead = block_scan(mine, sums, total);
    uint32_t before = ahead.a, pair = ahead.b & ((1u << kPairBits) - 1u);
#pragma unroll
    for (uint32_t i = 0; i < kSeqs; ++i) {
        if (i >= per || s0 + i >= g.r.n) continue;
        d[i].before = before;
        if (d[i].pair) d[i].pair = kFlag | pair++;
        before += n[i];
        g.need[s0 + i] = d[i];
    }
    if (tid == 0) {
        g.total[0] = (uint64_t)(total.b >> kPairBits) << 15 > g.p.n_pages ? 0xFFFFFFFFu : total.a;
        g.total[1] = total.b & ((1u << kPairBits) - 1u);
    }
}

// A workgroup gives out the free pages of its segment: the r-th free page of the pool to the sequence whose part holds r.
__device__ __forceinline__ void give_pages(const ExtendArgs &g, uint32_t seg, uint32_t is_free, uint32_t *before, Two (&sums)[kThreads / 64])
{
    const uint32_t tid = threadIdx.x, p0 = seg * kSegment + tid * kEach;
    const uint32_t wanted = (uint32_t)g.total[0], pairs = (uint32_t)g.total[1];
    Two n{0, 0}, total;
    if (g.n_segments == 1)
        n.a = (uint32_t)__builtin_popcount(is_free);
    else
        for (uint32_t i = tid; i < g.n_segments; i += kThreads) {
            const uint32_t c = g.counted[i];
            n.a += c;
            if (i < seg) n.b += c;
        }
    for (uint32_t s = tid; s < g.r.n; s += kThreads) before[s] = g.need[s].before;
    (void)block_scan(n, sums, total);
    const bool enough = wanted <= total.a;
    const uint32_t ahead = total.b;
    if (seg == 0) {
        if (!enough && tid == 0) report(g.p.err, ZX_E_NOSPACE);
        if (tid == 0) *g.count = enough ? (int32_t)pairs : 0;
        for (uint32_t s = tid; s < g.r.n; s += kThreads) {
            const Need d = g.need[s];
            g.kv_len[s] = enough ? d.kv : 0;
            if (!enough) continue;
            g.r.held[s] = d.held;
            // (counts of pages that others hold stay above zero: no one here takes them for free ones)
            if (d.old & kFlag) g.p.refs[d.old & ~kFlag] = (int32_t)d.left;
        }
    }
    if (!enough || wanted <= ahead) return;
    uint32_t r = ahead + block_scan(Two{(uint32_t)__builtin_popcount(is_free), 0}, sums, total).a;
    if (!is_free || r >= wanted) return;
    uint32_t lo = 0, hi = g.r.n;                 // the last sequence with before <= r
    while (hi - lo > 1) {
        const uint32_t m = (lo + hi) / 2;
        if (before[m] <= r) lo = m;
        else hi = m;
    }
    Need d = g.need[lo];
    for (; is_free && r < wanted; is_free &= is_free - 1, ++r) {
        if (lo + 1 < g.r.n && before[lo + 1] <= r) {         // on to the next one that takes any
            while (lo + 1 < g.r.n && before[lo + 1] <= r) ++lo;
            d = g.need[lo];
        }
        const uint32_t page = p0 + (uint32_t)__builtin_ctz(is_free), at = d.first + (r - d.before);
        int32_t *entry = g.r.table + (uint64_t)lo * g.r.width + at;
        if ((d.pair & kFlag) && at == d.first) {
            int32_t *pr = g.pairs + 3 * (uint64_t)(d.pair & ~kFlag);
            pr[0] = (int32_t)(d.old & ~kFlag);
            pr[1] = (int32_t)page;
            pr[2] = (int32_t)d.tokens;
        }
        *entry = (int32_t)page;
        g.p.refs[page] = 1;
    }
}

__global__ __launch_bounds__(kThreads) void k_pages_need(ExtendArgs g)
{
    extern __shared__ uint32_t slots[];
    __shared__ Two sums[kThreads / 64];
    if (blockIdx.x == 0) return find_needs(g, slots, sums);
    const uint32_t seg = blockIdx.x - 1;
    Two total;
    (void)block_scan(Two{(uint32_t)__builtin_popcount(free_bits(g.p, seg * kSegment + threadIdx.x * kEach)), 0}, sums, total);
    if (threadIdx.x == 0) g.counted[seg] = total.a;
}

__global__ __launch_bounds__(kThreads) void k_pages_give(ExtendArgs g)
{
    __shared__ Two sums[kThreads / 64];
    __shared__ uint32_t before[kMostSeqs];
    // a thread's pages lie side by side, so ranks ascend with the page
    give_pages(g, blockIdx.x, free_bits(g.p, blockIdx.x * kSegment + threadIdx.x * kEach), before, sums);
}

// The whole of it by one workgroup, for pools of one segment: 1 x 4 rows 3.0 + 3.4 us in two launches.
__global__ __launch_bounds__(kThreads) void k_pages_extend(ExtendArgs g)
{
    extern __shared__ uint32_t slots[];
    __shared__ Two sums[kThreads / 64];
    __shared__ uint32_t before[kMostSeqs];
    const uint32_t is_free = free_bits(g.p, threadIdx.x * kEach);
    find_needs(g, slots, sums);
    __syncthreads();                             // (what it wrote to memory is read by this workgroup alone)
    give_pages(g, 0, is_free, before, sums);
}

// ---------------------------------------------------------------- pages in use are brought together

struct CompactArgs {
    Pool p;
    Rows r;
    int32_t *remap, *pairs, *count, *nth;        // nth[page]: which pair moves it, or -1
    uint32_t *counted;
    uint32_t n_segments;
};

__global__ __launch_bounds__(kThreads) void k_pages_count(CompactArgs g)
{
    __shared__ Two sums[kThreads / 64];
    Two total;
    (void)block_scan(Two{(uint32_t)__builtin_popcount(free_bits(g.p, blockIdx.x * kSegment + threadIdx.x * kEach)), 0}, sums, total);
    if (threadIdx.x == 0) g.counted[blockIdx.x] = total.a;
}

// With L pages in use, those of them at L or behind go into the free ones ahead of L, in order: the j-th such page into the
// j-th hole.  There are as many of the one as of the other.
__device__ __forceinline__ void pair_pages(const CompactArgs &g, uint32_t seg, Two (&sums)[kThreads / 64])
{
    const uint32_t tid = threadIdx.x;
    const uint32_t p0 = seg * kSegment + tid * kEach, is_free = free_bits(g.p, p0);
    Two n{0, 0}, total;
    if (g.n_segments == 1)
        n.a = (uint32_t)__builtin_popcount(is_free);
    else
        for (uint32_t i = tid; i < g.n_segments; i += kThreads) {
            const uint32_t c = g.counted[i];
            n.a += c;
            if (i < seg) n.b += c;
        }
    (void)block_scan(n, sums, total);
    const uint32_t ahead = total.b, L = g.p.n_pages - total.a;       // free pages of the segments ahead; pages in use
    // holes: free pages ahead of L, of whole segments and of the one that L lies in
    const uint32_t ls = L / kSegment;
    uint32_t holes = 0;
    if (g.n_segments > 1)
        for (uint32_t i = tid; i < ls; i += kThreads) holes += g.counted[i];
    const uint32_t pl = ls * kSegment + tid * kEach;
    if (pl < L) {
        const uint32_t m = L - pl < kEach ? (1u << (L - pl)) - 1u : (1u << kEach) - 1u;
        holes += (uint32_t)__builtin_popcount((ls == seg ? is_free : free_bits(g.p, pl)) & m);
    }
    uint32_t f = block_scan(Two{(uint32_t)__builtin_popcount(is_free), holes}, sums, total).a + ahead;        // free pages ahead
    holes = total.b;
    if (seg == 0 && tid == 0) *g.count = (int32_t)holes;
    const uint32_t most = g.p.n_pages / 2;       // (never more, unless refs is written meanwhile)
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i) {
        const uint32_t page = p0 + i;
        if (page >= g.p.n_pages) break;
        const bool empty = is_free >> i & 1u;
        int32_t to = empty ? -1 : (int32_t)page, j = -1;
        if (empty && page < L && f < most) {
            g.pairs[3 * (uint64_t)f + 1] = (int32_t)page;
            g.pairs[3 * (uint64_t)f + 2] = 1 << g.p.log_page;
        } else if (!empty && page >= L) {
            j = (int32_t)((page - f) - (L - holes));         // pages in use ahead of it, less those ahead of L
            if ((uint32_t)j < most) g.pairs[3 * (uint64_t)j] = (int32_t)page;
            else j = -1;
        }
        g.nth[page] = j;
        if (j < 0) g.remap[page] = to;
        f += empty;
    }
}

// The pairs' counts and new places, shared by `of` workgroups.
__device__ __forceinline__ void move_counts(const CompactArgs &g, uint32_t nth, uint32_t of)
{
    const uint32_t said = (uint32_t)*g.count, n = said < g.p.n_pages / 2 ? said : g.p.n_pages / 2;
    for (uint32_t j = nth * blockDim.x + threadIdx.x; j < n; j += of * blockDim.x) {
        const uint32_t from = (uint32_t)g.pairs[3 * (uint64_t)j], to = (uint32_t)g.pairs[3 * (uint64_t)j + 1];
        if (from >= g.p.n_pages || to >= g.p.n_pages) continue;
        g.remap[from] = (int32_t)to;
        g.p.refs[to] = g.p.refs[from];
        g.p.refs[from] = 0;
    }
}
// Entries c, c + step ... of a row of the table find their new place through nth and the pairs.
__device__ __forceinline__ void move_row(const CompactArgs &g, uint32_t s, uint32_t c, uint32_t step)
{
    const int32_t held = g.r.held[s];
    if (held < 0 || held > g.r.cap) {
        if (c == 0) report(g.p.err, ZX_E_CORRUPT);
        return;
    }
    const uint32_t n = pages_of(g.p, held);
    int32_t *row = g.r.table + (uint64_t)s * g.r.width;
    for (; c < n; c += step) {
        const uint32_t page = (uint32_t)row[c];
        if (page >= g.p.n_pages) {
            report(g.p.err, ZX_E_CORRUPT);
            continue;
        }
        const int32_t j = g.nth[page];
        if (j >= 0) row[c] = g.pairs[3 * (uint64_t)j + 1];
        else if (g.remap[page] < 0) report(g.p.err, ZX_E_CORRUPT);       // a page that nobody is said to hold
    }
}

__global__ __launch_bounds__(kThreads) void k_pages_pair(CompactArgs g)
{
    __shared__ Two sums[kThreads / 64];
    pair_pages(g, blockIdx.x, sums);
}

constexpr uint32_t kMoveThreads = 256;
__global__ __launch_bounds__(kMoveThreads) void k_pages_move(CompactArgs g, uint32_t for_pairs, uint32_t per_row)
{
    if (blockIdx.x < for_pairs) return move_counts(g, blockIdx.x, for_pairs);
    const uint32_t item = blockIdx.x - for_pairs;
    move_row(g, item / per_row, (item % per_row) * kMoveThreads + threadIdx.x, per_row * kMoveThreads);
}

// The whole of it by one workgroup, for pools of one segment and tables of up to 16384 entries; a wave takes a row at a time.
__global__ __launch_bounds__(kThreads) void k_pages_compact(CompactArgs g)
{
    __shared__ Two sums[kThreads / 64];
    pair_pages(g, 0, sums);
    __syncthreads();                             // (what it wrote to memory is read by this workgroup alone)
    move_counts(g, 0, 1);
    for (uint32_t s = threadIdx.x / 64; s < g.r.n; s += kThreads / 64) move_row(g, s, threadIdx.x & 63u, 64);
}

// ---- host side
inline bool al4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

zx_status make_pool(const zx_page_pool *p, uint32_t *err, Pool &o)
{
    if (!p || !p->refs || !al4(p->refs) || !al4(err) || p->n_pages == 0 || !zxp::pow2_in(p->page_tokens, 16, 4096)) return ZX_E_INVAL;
    if (p->n_pages > kMostPages) return ZX_E_LIMIT;
    o = Pool{p->refs, p->n_pages, zxp::log2_of(p->page_tokens), err};
    return ZX_OK;
}

zx_status make_rows(const zx_page_rows *r, const zx_page_pool *p, Rows &o)
{
    if (!r) return ZX_E_INVAL;
    if (r->n_seqs && (!r->held || (r->table_width && !r->page_table) || !al4(r->held) || !al4(r->page_table))) return ZX_E_INVAL;
    const uint64_t room = (uint64_t)r->table_width * p->page_tokens;
    if (room > 0x3FFFFFFFu || r->n_seqs > 65536) return ZX_E_LIMIT;
    o = Rows{r->page_table, r->held, r->n_seqs, r->table_width, (int32_t)room};
    return ZX_OK;
}

inline bool good_copies(const zx_page_copies *c, uint32_t least)
{
    return c && c->count && c->cap >= least && (c->pairs || least == 0) && al4(c->count) && al4(c->pairs);
}

inline zx_status launched() { return hipGetLastError() == hipSuccess ? ZX_OK : ZX_E_HIP; }

}  // namespace zxg

using namespace zxg;

extern "C" zx_status zx_pages_fork(const zx_page_pool *pool, const zx_page_rows *rows, uint32_t beams, const int32_t *parents,
                                   uint32_t *err, hipStream_t stream)
{
    ForkArgs g{};
    zx_status st = make_pool(pool, err, g.p);
    if (st == ZX_OK) st = make_rows(rows, pool, g.r);
    if (st != ZX_OK) return st;
    if (beams == 0 || rows->n_seqs % beams) return ZX_E_INVAL;
    if (beams > kMostSeqs) return ZX_E_LIMIT;
    if (rows->n_seqs == 0) return ZX_OK;
    if (!parents || !al4(parents)) return ZX_E_INVAL;
    g.parents = parents;
    g.beams = beams;
    const uint32_t groups = rows->n_seqs / beams;
    // 4 KB of table entries at a time, four columns at least (16 KB: 10.9 us for 64 x 8 rows of 2068 entries, 4 KB: 9.9)
    const uint32_t width = rows->table_width;
    g.log_strip = 10;
    while (g.log_strip > 2 && (((uint64_t)beams << g.log_strip) > 1024 || 1u << (g.log_strip - 1) >= width)) --g.log_strip;
    // a group with more than two strips is shared by workgroups, about 2048 in all; the lengths are then written by a launch of
    // their own, behind those that read them
    const uint32_t n_strips = ceil_div(width, 1u << g.log_strip), fair = 1 + 2047 / groups;
    g.share = n_strips <= 2 ? 1 : n_strips < fair ? n_strips : fair;
    const uint32_t lds = (3 * beams + (beams << g.log_strip)) * 4, threads = beams << g.log_strip <= 1024 ? 256 : 1024;
    hipLaunchKernelGGL(k_pages_fork, dim3(groups * g.share), dim3(threads), lds, stream, g);
    if (g.share > 1) hipLaunchKernelGGL(k_pages_fork_held, dim3(groups), dim3(256), 2 * beams * 4, stream, g);
    return launched();
}

extern "C" zx_status zx_pages_trim(const zx_page_pool *pool, const zx_page_rows *rows, const int32_t *keep, uint32_t *err,
                                   hipStream_t stream)
{
    Pool p;
    Rows r;
    zx_status st = make_pool(pool, err, p);
    if (st == ZX_OK) st = make_rows(rows, pool, r);
    if (st != ZX_OK || rows->n_seqs == 0) return st;
    if (!al4(keep)) return ZX_E_INVAL;
    hipLaunchKernelGGL(k_pages_trim, dim3(r.n), dim3(r.n <= 256 && r.width > 512 ? 1024 : 256), 0, stream, p, r, keep);
    return launched();
}

extern "C" size_t zx_pages_extend_workspace_bytes(const zx_page_pool *pool, uint32_t n_seqs)
{
    if (!pool || pool->n_pages > kMostPages || n_seqs > kMostSeqs) return 0;
    return 16 + (size_t)n_seqs * sizeof(Need) + (size_t)ceil_div(pool->n_pages, kSegment) * 4;
}

extern "C" zx_status zx_pages_extend(const zx_page_pool *pool, const zx_page_rows *rows, const int32_t *q_start, uint32_t max_q,
                                     uint32_t max_kv, int32_t *kv_len, const zx_page_copies *copies, void *workspace, size_t ws_bytes,
                                     uint32_t *err, hipStream_t stream)
{
    ExtendArgs g{};
    zx_status st = make_pool(pool, err, g.p);
    if (st == ZX_OK) st = make_rows(rows, pool, g.r);
    if (st != ZX_OK) return st;
    if (rows->n_seqs > kMostSeqs) return ZX_E_LIMIT;
    if (!good_copies(copies, rows->n_seqs)) return ZX_E_INVAL;
    if (rows->n_seqs && (!q_start || !kv_len || !al4(q_start) || !al4(kv_len))) return ZX_E_INVAL;
    if (!workspace || ((uintptr_t)workspace & 15u) || ws_bytes < zx_pages_extend_workspace_bytes(pool, rows->n_seqs)) return ZX_E_INVAL;
    if ((uint32_t)g.r.cap > max_kv) g.r.cap = (int32_t)max_kv;
    g.q_start = q_start;
    g.kv_len = kv_len;
    g.pairs = copies->pairs;
    g.count = copies->count;
    g.max_q = max_q;
    g.n_segments = ceil_div(pool->n_pages, kSegment);
    g.total = static_cast<uint64_t *>(workspace);
    g.need = reinterpret_cast<Need *>(g.total + 2);
    g.counted = reinterpret_cast<uint32_t *>(g.need + rows->n_seqs);
    g.log_slots = 6;
    while ((1u << g.log_slots) < 2 * rows->n_seqs) ++g.log_slots;
    const uint32_t lds = (3u << g.log_slots) * 4;
    if (g.n_segments == 1) {
        hipLaunchKernelGGL(k_pages_extend, dim3(1), dim3(kThreads), lds, stream, g);
    } else {
        hipLaunchKernelGGL(k_pages_need, dim3(1 + g.n_segments), dim3(kThreads), lds, stream, g);
        hipLaunchKernelGGL(k_pages_give, dim3(g.n_segments), dim3(kThreads), 0, stream, g);
    }
    return launched();
}

extern "C" size_t zx_pages_compact_workspace_bytes(const zx_page_pool *pool)
{
    if (!pool || pool->n_pages > kMostPages) return 0;
    return (size_t)pool->n_pages * 4 + (size_t)ceil_div(pool->n_pages, kSegment) * 4;
}

extern "C" zx_status zx_pages_compact(const zx_page_pool *pool, const zx_page_rows *rows, int32_t *remap, const zx_page_copies *copies,
                                      void *workspace, size_t ws_bytes, uint32_t *err, hipStream_t stream)
{
    CompactArgs g{};
    zx_status st = make_pool(pool, err, g.p);
    if (st == ZX_OK) st = make_rows(rows, pool, g.r);
    if (st != ZX_OK) return st;
    if (!remap || !al4(remap) || !good_copies(copies, pool->n_pages / 2)) return ZX_E_INVAL;
    if (!workspace || ((uintptr_t)workspace & 15u) || ws_bytes < zx_pages_compact_workspace_bytes(pool)) return ZX_E_INVAL;
    g.remap = remap;
    g.pairs = copies->pairs;
    g.count = copies->count;
    g.nth = static_cast<int32_t *>(workspace);
    g.counted = reinterpret_cast<uint32_t *>(g.nth + pool->n_pages);
    g.n_segments = ceil_div(pool->n_pages, kSegment);
    if (g.n_segments == 1 && (uint64_t)rows->n_seqs * rows->table_width <= 16384) {
        hipLaunchKernelGGL(k_pages_compact, dim3(1), dim3(kThreads), 0, stream, g);
        return launched();
    }
    hipLaunchKernelGGL(k_pages_count, dim3(g.n_segments), dim3(kThreads), 0, stream, g);
    hipLaunchKernelGGL(k_pages_pair, dim3(g.n_segments), dim3(kThreads), 0, stream, g);
    // workgroups for the pairs, and for each row of the table
    const uint32_t pairs = ceil_div(pool->n_pages / 2 + 1, kMoveThreads), for_pairs = pairs < 256 ? pairs : 256;
    const uint32_t most = ceil_div(rows->table_width, kMoveThreads);
    const uint32_t fair = rows->n_seqs ? 1 + 1024 / rows->n_seqs : 1, per_row = most == 0 ? 1 : most < fair ? most : fair;
    hipLaunchKernelGGL(k_pages_move, dim3(for_pairs + rows->n_seqs * per_row), dim3(kMoveThreads), 0, stream, g, for_pairs, per_row);
    return launched();
}
