// zx_paged_select.hip -- which blocks of a paged K/V cache a new token should read.
//
// For a group of G query heads and a block with smallest and largest keys lo, hi per
// channel, no key of the block scores more than
//   sum_g sum_d max(q_gd lo_d, q_gd hi_d) = sum_d up_d hi_d + dn_d lo_d,
//   up_d = sum_g max(q_gd, 0), dn_d = sum_g min(q_gd, 0):
// one dot product of 2 D terms a block, whatever the group's size, over 4 D bytes of
// bounds: bound by those bytes.  Which blocks are taken is a yes or no, and two ways of
// adding up in 32 bits would now and then say differently for blocks next to the border,
// so the sums are taken in 64 bits (the vector units' 64-bit multiply-add has the rate of the 32-bit one).
// With finite bounds and queries the two forms are one sum.  An infinite bound (a key that overflowed) times a part that is
// zero is NaN in the second form only, so a row with a sum that is infinite or NaN has those taken again by the first.
//
//   k_pick   one workgroup for a token and K/V head: a key (the sum, as an integer that orders like it)
//            for each block, in LDS, then the top_k-th largest by radix selection and the
//            taken blocks in ascending order
//   k_score, k_top  the same in two steps, with the keys in memory: for more blocks than LDS holds, or
//            few tokens and so many blocks that one CU alone would read too long
//
// 32 tokens over 65536 and less (8 K/V heads of 128 channels, blocks of 64): k_pick 27 us for 44 MB of bounds (the
// longest row's 512 KB alone pass one CU in 9 us, and the selection takes about as long);
// one token over 32768: k_score 5 us, k_top 6 us, each little more than a launch.
#include "zx_paged.h"

namespace zxp {
namespace {

constexpr uint32_t kThreads = 256;
constexpr int kDigit = 10;              // bits of a radix digit of k_top
constexpr uint32_t kHeld = 4096;        // keys of a row that k_top holds in LDS (32 KB)

struct SelectArgs {
    Cache c;
    Batch b;
    Rows q;
    int32_t *blocks;
    uint64_t *keys;                     // [rows of the slab][heads][nb]
    uint32_t group, top_k, keep_first, keep_last;
    uint32_t nb;                        // blocks of the longest sequence
    uint32_t slab0, slab;               // token groups of this launch: slab0 .. slab0 + slab - 1
    uint32_t per;                       // blocks of a workgroup of k_score
    uint32_t head_dim;
};

// An integer that orders like the double; NaN below everything.
__device__ __forceinline__ uint64_t order_key(double x)
{
    const int64_t b = __double_as_longlong(x);
    if (x != x) return 0;
    return b < 0 ? ~(uint64_t)b : (uint64_t)b | 0x8000000000000000ull;
}

__device__ __forceinline__ bool finite_key(uint64_t x) { return x > 0x000FFFFFFFFFFFFFull && x < 0xFFF0000000000000ull; }

// x of the lane that DPP pattern CTRL names
template <int CTRL>
__device__ __forceinline__ double moved(double x)
{
    const uint64_t b = (uint64_t)__double_as_longlong(x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, true);
    return __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
}

// Sum over the LB neighbouring lanes of a block, in all of them: pairs, pairs of pairs
// (quad_perm), halves of a row of 16 (half_mirror, row_mirror), rows.
template <int LB>
__device__ __forceinline__ double sum_lanes(double x)
{
    x += moved<0xB1>(x);                                 // quad_perm 1 0 3 2
    x += moved<0x4E>(x);                                 // quad_perm 2 3 0 1
    x += moved<0x141>(x);                                // row_half_mirror
    if constexpr (LB >= 16) x += moved<0x140>(x);        // row_mirror
    if constexpr (LB >= 32) x += __shfl_xor(x, 16, 64);
    return x;
}

// The bounds of kUnroll blocks j, j + STEP, ..: eight channels of each for a lane (blocks past j1 - 1 repeat it).
constexpr int kUnroll = 4;
struct Fetched {
    bf8 lo[kUnroll], hi[kUnroll];
    uint32_t none;                                       // blocks of these that have no page
};
template <int D, uint32_t STEP>
__device__ __forceinline__ void fetch(const SelectArgs &g, const int32_t *table, uint32_t h, uint32_t j, uint32_t j1, uint32_t ln, Fetched &f)
{
    const uint32_t lp = g.c.log_page - g.c.log_block, nbp = 1u << lp;
    uint32_t page[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) page[u] = (uint32_t)table[(j + u * STEP < j1 ? j + u * STEP : j1 - 1) >> lp];
    f.none = 0;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const uint32_t ju = j + u * STEP < j1 ? j + u * STEP : j1 - 1;
        if (page[u] >= g.c.n_pages) {
            report(g.b.err, ZX_E_CORRUPT);
            page[u] = 0;
            f.none |= 1u << u;
        }
        const __bf16 *bp = g.c.bounds + (((uint64_t)page[u] * g.c.heads + h) * nbp + (ju & (nbp - 1u))) * (2 * D) + 8 * ln;
        f.lo[u] = *reinterpret_cast<const bf8 *>(bp);
        f.hi[u] = *reinterpret_cast<const bf8 *>(bp + D);
    }
}

// Sums over the group's heads of the positive and of the negative parts of every channel, for nt tokens from packed
// row `row` on, into sh.total.  By a whole workgroup of NT threads, once (every lane for itself would
// take 2 us more with eight heads, and 25 with sixteen and four tokens).  A NaN stays one in both sums.
template <int D, int TT, int NT>
struct Sums {
    static constexpr uint32_t P = NT / D;                // threads of a channel
    double parts[P][2][D], total[TT][2][D];
};
template <int D, int TT, int NT>
__device__ __forceinline__ void group_sums(const SelectArgs &g, int64_t row, uint32_t nt, uint32_t h, Sums<D, TT, NT> &sh)
{
    constexpr uint32_t P = Sums<D, TT, NT>::P;
    const uint32_t ch = threadIdx.x % D, p = threadIdx.x / D;
    const __bf16 *qp = g.q.p + row * g.q.token + (int64_t)(h * g.group) * g.q.head + ch;
#pragma unroll
    for (uint32_t t = 0; t < (uint32_t)TT; ++t) {
        if (t >= nt) break;
        double a = 0.0, b = 0.0;
        for (uint32_t e = p; e < g.group; e += P) {
            const float y = (float)qp[t * g.q.token + (int64_t)e * g.q.head];
            a += (double)(y < 0.0f ? 0.0f : y);
            b += (double)(y > 0.0f ? 0.0f : y);
        }
        sh.parts[p][0][ch] = a;
        sh.parts[p][1][ch] = b;
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < 2 * D; i += NT) {
            a = (&sh.parts[0][0][0])[i];
#pragma unroll
            for (uint32_t j = 1; j < P; ++j) a += (&sh.parts[j][0][0])[i];
            (&sh.total[t][0][0])[i] = a;
        }
        __syncthreads();
    }
}

// Block u of those fetched, for one token: the sum over all lanes of the block, in all of them.
template <int LB>
__device__ __forceinline__ double block_sum(const Fetched &f, int u, const double (&up)[8], const double (&dn)[8])
{
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = __builtin_fma(up[i], (double)(float)f.hi[u][i], __builtin_fma(dn[i], (double)(float)f.lo[u][i], s));
    return sum_lanes<LB>(s);
}

// Tokens of a sequence come in groups of TT that share what is read of the bounds.
template <int D, int TT>
__global__ __launch_bounds__(kThreads) void k_score(SelectArgs g)
{
    constexpr uint32_t LB = D / 8;                       // lanes of a block
    constexpr uint32_t PB = kThreads / LB;               // blocks at a time
    __shared__ __align__(16) Sums<D, TT, kThreads> sums;
    const uint32_t h = blockIdx.x % g.c.heads, grp = blockIdx.x / g.c.heads;
    uint32_t seq, local, unused;
    Seq sv;
    if (!find_item(g.b, g.slab0 + grp, [](const Seq &v) { return div_up((uint32_t)v.nq, TT); }, [](const Seq &) { return 0u; }, seq, sv, local, unused)) return;
    const uint32_t tok = local * TT, nt = (uint32_t)sv.nq - tok < (uint32_t)TT ? (uint32_t)sv.nq - tok : (uint32_t)TT;
    const int32_t p9 = sv.kv - sv.nq + (int32_t)(tok + nt - 1);      // position of the last token
    if (p9 < 0) return;
    const uint32_t seen = ((uint32_t)p9 >> g.c.log_block) + 1;
    if (seen <= g.top_k) return;                                     // every block is taken
    const uint32_t j0 = blockIdx.y * g.per, j1 = j0 + g.per < seen ? j0 + g.per : seen;
    if (j0 >= j1) return;

    const uint32_t ln = threadIdx.x % LB, slot = threadIdx.x / LB;
    const int32_t *table = g.b.table + (uint64_t)seq * g.b.width;
    Fetched f;
    fetch<D, PB>(g, table, h, j0 + slot, j1, ln, f);                 // under way while the queries are added up
    group_sums(g, sv.q0 + (int64_t)tok, nt, h, sums);
    double up[TT][8], dn[TT][8];
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            up[t][i] = sums.total[(uint32_t)t < nt ? t : 0][0][8 * ln + i];
            dn[t][i] = sums.total[(uint32_t)t < nt ? t : 0][1][8 * ln + i];
        }
    for (uint32_t j = j0 + slot; j < j1; j += kUnroll * PB) {
        double s[kUnroll][TT];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int t = 0; t < TT; ++t) s[u][t] = block_sum<(int)LB>(f, u, up[t], dn[t]);
        const uint32_t gone = f.none;
        if (j + kUnroll * PB < j1) fetch<D, PB>(g, table, h, j + kUnroll * PB, j1, ln, f);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (ln < nt && j + u * PB < j1) {
                double x = s[u][0];
#pragma unroll
                for (int t = 1; t < TT; ++t) x = ln == (uint32_t)t ? s[u][t] : x;
                g.keys[((uint64_t)(grp * TT + ln) * g.c.heads + h) * g.nb + j + u * PB] = gone >> u & 1u ? 0 : order_key(x);
            }
    }
}

struct Picking {
    uint32_t hist[1 << kDigit];
    uint64_t wide[2][8];
    uint32_t sums[2][8];
    uint32_t pick[3];
};

// What a row of the result is about: its token's packed row and sequence, its head.
struct Place {
    int64_t row;
    const int32_t *table;
    uint32_t h;
};

// The key of block j from its sum by definition, NaN where any product is; 0 where the block has no page.  By one wave.
__device__ __forceinline__ uint64_t defined_key(const SelectArgs &g, const Place &at, uint32_t j)
{
    const uint32_t lp = g.c.log_page - g.c.log_block, nbp = 1u << lp, D = g.head_dim, page = (uint32_t)at.table[j >> lp];
    if (page >= g.c.n_pages) return 0;
    const __bf16 *bp = g.c.bounds + (((uint64_t)page * g.c.heads + at.h) * nbp + (j & (nbp - 1u))) * (2 * D);
    double s = 0.0;
    for (uint32_t ch = threadIdx.x & 63u; ch < D; ch += 64) {
        const double lo = (double)(float)bp[ch], hi = (double)(float)bp[D + ch];
        const __bf16 *qp = g.q.p + at.row * g.q.token + (int64_t)(at.h * g.group) * g.q.head + ch;
        for (uint32_t e = 0; e < g.group; ++e) {
            const double q = (double)(float)qp[(int64_t)e * g.q.head], a = q * lo, b = q * hi;
            s += a != a ? a : a > b ? a : b;             // (b where it is NaN)
        }
    }
    for (int w = 32; w >= 1; w >>= 1) s += __shfl_xor(s, w, 64);
    return order_key(s);
}

// The smallest and the largest key of all NT threads, in all of them.
template <uint32_t NT>
__device__ __forceinline__ void join_range(uint64_t &least, uint64_t &most, Picking &sh)
{
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    for (int w = 32; w >= 1; w >>= 1) {
        const uint64_t a = __shfl_xor(least, w, 64), b = __shfl_xor(most, w, 64);
        least = a < least ? a : least;
        most = b > most ? b : most;
    }
    if (lane == 0) {
        sh.wide[0][wave] = least;
        sh.wide[1][wave] = most;
    }
    __syncthreads();
    for (uint32_t w = 0; w < NT / 64; ++w) {
        least = sh.wide[0][w] < least ? sh.wide[0][w] : least;
        most = sh.wide[1][w] > most ? sh.wide[1][w] : most;
    }
}

// Blocks f0 .. f0 + n - 1 compete with their keys for `want` < n places of `out`; the rest of
// a row's top_k are the blocks in front of them and behind them.  By all NT threads.
template <uint32_t NT>
__device__ __forceinline__ void pick_row(const SelectArgs &g, const Place &place, uint64_t *keys, uint32_t f0, uint32_t n, uint32_t want, uint64_t least, uint64_t most, int32_t *out, Picking &sh)
{
    constexpr uint32_t NWV = NT / 64;
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6, K = g.top_k;
    auto key = [&](uint32_t i) { return keys[i]; };
    join_range<NT>(least, most, sh);
    if (!finite_key(least) || !finite_key(most)) {
        // some sum is infinite or NaN, or some block has no page
        __syncthreads();
        least = ~0ull;
        most = 0;
        for (uint32_t i0 = 64 * wave; i0 < n; i0 += NT) {
            const bool in = i0 + lane < n;
            uint64_t x = in ? key(i0 + lane) : 0;
            for (uint64_t odd = __ballot(in && !finite_key(x)); odd; odd &= odd - 1) {
                const uint32_t l = (uint32_t)__builtin_ctzll(odd);
                const uint64_t y = defined_key(g, place, f0 + i0 + l);
                if (lane == l) keys[i0 + l] = x = y;
            }
            if (in) {
                least = x < least ? x : least;
                most = x > most ? x : most;
            }
        }
        join_range<NT>(least, most, sh);
    }
    // keys at or above `cut` in the bits of `mask` are taken, but of those equal to it in
    // these bits only the first `want`
    const uint64_t diff = least ^ most;
    int top = diff ? 64 - __builtin_clzll(diff) : 0;     // bits that are not alike in all keys
    uint64_t mask = top == 64 ? 0ull : ~0ull << top, cut = most & mask;
    uint32_t same = n;                                   // keys equal to `cut` in the bits of `mask`
    if (want == 0) {                                     // only the forced blocks
        cut = ~0ull;
        mask = ~0ull;
        same = 0;
        top = 0;
    }
    while (top > 0 && same != want) {
        const int bits = top < kDigit ? top : kDigit, sft = top - bits;
        for (uint32_t i = tid; i < 1u << kDigit; i += NT) sh.hist[i] = 0;
        __syncthreads();
        for (uint32_t i = tid; i < n; i += NT) {
            const uint64_t x = key(i);
            if ((x & mask) == cut) atomicAdd(&sh.hist[(uint32_t)(x >> sft) & ((1u << bits) - 1u)], 1u);
        }
        __syncthreads();
        // thread t has kEach digits, the highest first: the digit at which the count from above reaches `want`
        constexpr uint32_t kEach = (1u << kDigit) / NT;
        uint32_t c[kEach], mine = 0, total;
#pragma unroll
        for (uint32_t i = 0; i < kEach; ++i) {
            c[i] = sh.hist[(1u << kDigit) - 1u - kEach * tid - i];
            mine += c[i];
        }
        uint32_t above = wave_excl_scan(mine, total);
        if (lane == 0) sh.sums[0][wave] = total;
        __syncthreads();
        for (uint32_t w = 0; w < wave; ++w) above += sh.sums[0][w];
#pragma unroll
        for (uint32_t i = 0; i < kEach; ++i) {
            if (above < want && above + c[i] >= want) {
                sh.pick[0] = (1u << kDigit) - 1u - kEach * tid - i;
                sh.pick[1] = above;
                sh.pick[2] = c[i];
            }
            above += c[i];
        }
        __syncthreads();
        cut |= (uint64_t)sh.pick[0] << sft;
        mask |= (uint64_t)((1u << bits) - 1u) << sft;
        want -= sh.pick[1];
        same = sh.pick[2];
        top = sft;
        __syncthreads();
    }

    // every thread takes a run of neighbouring blocks, so that ranks come out of one scan
    const uint32_t run = div_up(n, NT), i0 = tid * run < n ? tid * run : n, i1 = i0 + run < n ? i0 + run : n;
    uint32_t over = 0, equal = 0;
    for (uint32_t i = i0; i < i1; ++i) {
        const uint64_t x = key(i) & mask;
        over += x > cut;
        equal += x == cut;
    }
    uint32_t ta, tb;
    uint32_t ra = wave_excl_scan(over, ta), rb = wave_excl_scan(equal, tb);
    if (lane == 0) {
        sh.sums[0][wave] = ta;
        sh.sums[1][wave] = tb;
    }
    __syncthreads();
    for (uint32_t w = 0; w < wave; ++w) {
        ra += sh.sums[0][w];
        rb += sh.sums[1][w];
    }
    uint32_t at = g.keep_first + ra + (rb < want ? rb : want);
    for (uint32_t i = i0; i < i1; ++i) {
        const uint64_t x = key(i) & mask;
        bool take = x > cut;
        if (x == cut) take = rb++ < want;
        if (take) out[at++] = (int32_t)(f0 + i);
    }
    for (uint32_t i = tid; i < g.keep_first; i += NT) out[i] = (int32_t)i;
    for (uint32_t i = tid; i < g.keep_last; i += NT) out[K - g.keep_last + i] = (int32_t)(f0 + n + i);
}

// Blocks that the new token `tok` of a sequence sees; its row of the result.  True where all of them
// are taken, which is then done.
__device__ __forceinline__ bool all_taken(const SelectArgs &g, const Seq &sv, uint32_t tok, uint32_t h, uint32_t &seen, int32_t *&out)
{
    const int32_t p = sv.kv - sv.nq + (int32_t)tok;
    seen = p < 0 ? 0u : ((uint32_t)p >> g.c.log_block) + 1;
    out = g.blocks + ((uint64_t)(sv.q0 + (int32_t)tok) * g.c.heads + h) * g.top_k;
    if (seen > g.top_k) return false;
    for (uint32_t i = threadIdx.x; i < g.top_k; i += blockDim.x) out[i] = i < seen ? (int32_t)i : -1;
    return true;
}

template <int TT>
__global__ __launch_bounds__(kThreads) void k_top(SelectArgs g)
{
    __shared__ uint64_t held[kHeld];
    __shared__ Picking sh;
    const uint32_t h = blockIdx.x % g.c.heads, row = blockIdx.x / g.c.heads;
    uint32_t seq, local, unused, seen;
    Seq sv;
    int32_t *out;
    if (!find_item(g.b, g.slab0 * TT + row, [](const Seq &v) { return div_up((uint32_t)v.nq, TT) * TT; }, [](const Seq &) { return 0u; }, seq, sv, local, unused))
        return;
    if (local >= (uint32_t)sv.nq || all_taken(g, sv, local, h, seen, out)) return;
    // blocks f0 .. f0 + n - 1 compete; those before and behind are taken anyway
    const uint32_t f0 = g.keep_first, n = seen - g.keep_last - f0;
    uint64_t *src = g.keys + ((uint64_t)row * g.c.heads + h) * g.nb + f0;
    const bool in_lds = n <= kHeld;
    uint64_t least = ~0ull, most = 0;
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t x = src[i];
        if (in_lds) held[i] = x;
        least = x < least ? x : least;
        most = x > most ? x : most;
    }
    const uint32_t want = g.top_k - g.keep_first - g.keep_last;
    const Place place{sv.q0 + (int64_t)local, g.b.table + (uint64_t)seq * g.b.width, h};
    if (in_lds) pick_row<kThreads>(g, place, held, f0, n, want, least, most, out, sh);
    else pick_row<kThreads>(g, place, src, f0, n, want, least, most, out, sh);
}

constexpr uint32_t kPickThreads = 512;

template <int D>
__global__ __launch_bounds__(kPickThreads) void k_pick(SelectArgs g)
{
    constexpr uint32_t LB = D / 8, PB = kPickThreads / LB;
    __shared__ uint64_t held[kHeld];
    __shared__ Picking sh;
    __shared__ __align__(16) Sums<D, 1, kPickThreads> sums;
    const uint32_t h = blockIdx.x % g.c.heads, row = blockIdx.x / g.c.heads;
    uint32_t seq, local, unused, seen;
    Seq sv;
    int32_t *out;
    if (!find_item(g.b, row, [](const Seq &v) { return (uint32_t)v.nq; }, [](const Seq &) { return 0u; }, seq, sv, local, unused)) return;
    if (all_taken(g, sv, local, h, seen, out)) return;
    const uint32_t f0 = g.keep_first, f1 = seen - g.keep_last, n = f1 - f0;
    const uint32_t ln = threadIdx.x % LB, slot = threadIdx.x / LB;
    const int32_t *table = g.b.table + (uint64_t)seq * g.b.width;
    uint64_t least = ~0ull, most = 0;
    Fetched f;
    fetch<D, PB>(g, table, h, f0 + slot, f1, ln, f);                 // under way while the queries are added up
    group_sums(g, sv.q0 + (int64_t)local, 1, h, sums);
    double up[8], dn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        up[i] = sums.total[0][0][8 * ln + i];
        dn[i] = sums.total[0][1][8 * ln + i];
    }
    for (uint32_t j = f0 + slot; j < f1; j += kUnroll * PB) {
        const Fetched now = f;
        if (j + kUnroll * PB < f1) fetch<D, PB>(g, table, h, j + kUnroll * PB, f1, ln, f);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const double s = block_sum<(int)LB>(now, u, up, dn);
            if (j + u * PB < f1) {
                const uint64_t x = now.none >> u & 1u ? 0 : order_key(s);
                if (ln == 0) held[j + u * PB - f0] = x;
                least = x < least ? x : least;
                most = x > most ? x : most;
            }
        }
    }
    __syncthreads();
    pick_row<kPickThreads>(g, Place{sv.q0 + (int64_t)local, table, h}, held, f0, n, g.top_k - g.keep_first - g.keep_last, least, most, out, sh);
}

// Tokens that share a read of the bounds: with one new token a sequence there is nothing to share.
inline uint32_t sharing(const zx_paged_batch *b, uint32_t n) { return (b->max_q < n ? b->max_q : n) > 1 ? 4 : 1; }

struct Slabs {
    uint32_t tt, groups, slab, nb;
    uint64_t bytes;
    bool fused;                  // k_pick
};

// The keys of all tokens at once, or of as many token groups as 256 MB hold.
Slabs make_slabs(const zx_paged_cache *c, const zx_paged_batch *b, uint32_t n)
{
    Slabs s{};
    const uint64_t room = (uint64_t)b->table_width * c->page_tokens, cap = b->max_kv < room ? b->max_kv : room;
    s.nb = ceil_div(cap, c->block_tokens);
    s.tt = sharing(b, n);
    const uint32_t seqs = b->n_seqs < n ? b->n_seqs : n;
    s.groups = s.tt == 1 ? n : n / s.tt + seqs < n ? n / s.tt + seqs : n;
    const uint64_t each = (uint64_t)s.tt * c->kv_heads * s.nb * 8;
    // k_pick saves a launch, reads the bounds of a token and head with one CU (57 bytes a nanosecond) and
    // shares no read between tokens.  Us of selection and attention, k_pick / both steps: one token over 8000
    // tokens (64 KB of bounds a head) 23.6 / 24.7, over 32768 (256 KB) 28.4 / 25.1; 24 and 32 tokens of 8 heads,
    // each of a sequence over 65536, 52 / 54 and 106 / 108.  Where four tokens share reads: 8 over 30000 29.9 / 32.1,
    // 3 x 41 of 2 heads over 17000 32 / 43, but 40 over 60000 61 / 53 and 4 x 30 over 8000 51 / 48.
    const uint64_t read = (uint64_t)s.nb * 4 * c->head_dim, wgs = (uint64_t)n * c->kv_heads;
    const bool pays = s.tt == 1 ? read <= 128 << 10 || wgs >= 192 : read * (wgs < 256 ? 256 : wgs) <= 256ull * (320 << 10);
    s.fused = s.nb <= kHeld && pays;
    if (s.fused) return s;
    // (a launch counts its threads in 32 bits)
    const uint64_t by_bytes = (256ull << 20) / (each ? each : 1), by_threads = 0xFFFFFFFFull / ((uint64_t)kThreads * s.tt * c->kv_heads);
    const uint64_t most = by_bytes < by_threads ? by_bytes : by_threads;
    s.slab = most < 1 ? 1 : most < s.groups ? (uint32_t)most : s.groups;
    s.bytes = each * s.slab;
    return s;
}

template <int TT>
void launch(uint32_t D, const SelectArgs &g, uint32_t pieces, hipStream_t stream)
{
    const dim3 grid(g.slab * g.c.heads, pieces);
    if (D == 64) hipLaunchKernelGGL((k_score<64, TT>), grid, dim3(kThreads), 0, stream, g);
    else if (D == 128) hipLaunchKernelGGL((k_score<128, TT>), grid, dim3(kThreads), 0, stream, g);
    else hipLaunchKernelGGL((k_score<256, TT>), grid, dim3(kThreads), 0, stream, g);
    hipLaunchKernelGGL((k_top<TT>), dim3(g.slab * TT * g.c.heads), dim3(kThreads), 0, stream, g);
}

}  // namespace
}  // namespace zxp

extern "C" size_t zx_paged_select_workspace_bytes(const zx_paged_cache *cache, const zx_paged_batch *batch, uint32_t n_tokens)
{
    using namespace zxp;
    SelectArgs g{};
    if (make_cache(cache, g.c) != ZX_OK || make_batch(batch, cache, n_tokens, nullptr, g.b) != ZX_OK || !cache->block_tokens || n_tokens == 0 ||
        batch->n_seqs == 0)
        return 0;
    return (size_t)make_slabs(cache, batch, n_tokens).bytes;
}

extern "C" zx_status zx_paged_select(const zx_paged_cache *cache, const zx_paged_batch *batch, uint32_t n_tokens, const zx_rows *q,
                                     uint32_t q_heads, uint32_t top_k, uint32_t keep_first, uint32_t keep_last, int32_t *blocks,
                                     void *workspace, size_t ws_bytes, uint32_t *err, hipStream_t stream)
{
    using namespace zxp;
    SelectArgs g{};
    zx_status st = make_cache(cache, g.c);
    if (st == ZX_OK) st = make_batch(batch, cache, n_tokens, err, g.b);
    if (st != ZX_OK) return st;
    if (!cache->block_tokens || q_heads == 0 || q_heads % cache->kv_heads || q_heads > 65536 || top_k == 0 || top_k > 1024 ||
        (uint64_t)keep_first + keep_last > top_k || !blocks)
        return ZX_E_INVAL;
    if (n_tokens == 0 || batch->n_seqs == 0) return ZX_OK;
    if ((st = make_rows(q, g.q)) != ZX_OK) return st;
    const Slabs s = make_slabs(cache, batch, n_tokens);
    if (s.bytes && (!workspace || ws_bytes < s.bytes || !al16(workspace))) return ZX_E_INVAL;
    if (s.nb > (1u << 26)) return ZX_E_LIMIT;
    g.blocks = blocks;
    g.keys = static_cast<uint64_t *>(workspace);
    g.group = q_heads / cache->kv_heads;
    g.top_k = top_k;
    g.keep_first = keep_first;
    g.keep_last = keep_last;
    g.nb = s.nb;
    g.head_dim = cache->head_dim;
    g.slab = s.slab;
    if (s.fused) {
        if ((uint64_t)n_tokens * cache->kv_heads * kPickThreads > 0xFFFFFFFFull) return ZX_E_LIMIT;
        const dim3 grid(n_tokens * cache->kv_heads);
        if (cache->head_dim == 64) hipLaunchKernelGGL((k_pick<64>), grid, dim3(kPickThreads), 0, stream, g);
        else if (cache->head_dim == 128) hipLaunchKernelGGL((k_pick<128>), grid, dim3(kPickThreads), 0, stream, g);
        else hipLaunchKernelGGL((k_pick<256>), grid, dim3(kPickThreads), 0, stream, g);
        return hipGetLastError() == hipSuccess ? ZX_OK : ZX_E_HIP;
    }
    // blocks of a workgroup: few enough to fill the card, many enough to be worth its start
    const uint32_t at_once = 4 * kThreads / (cache->head_dim / 8);
    const uint64_t want = ceil_div(s.tt == 1 ? 1280 : 512, (uint64_t)s.slab * cache->kv_heads);
    uint32_t per = ceil_div(s.nb ? s.nb : 1, want);
    per = ceil_div(per, at_once) * at_once;
    if (ceil_div(s.nb ? s.nb : 1, per) > 65535) per = ceil_div(ceil_div(s.nb, 65535), at_once) * at_once;
    g.per = per;
    const uint32_t pieces = ceil_div(s.nb ? s.nb : 1, per);
    for (uint32_t at = 0; at < s.groups; at += s.slab) {
        g.slab0 = at;
        if (s.groups - at < g.slab) g.slab = s.groups - at;
        if (s.tt == 1) launch<1>(cache->head_dim, g, pieces, stream);
        else launch<4>(cache->head_dim, g, pieces, stream);
    }
    return hipGetLastError() == hipSuccess ? ZX_OK : ZX_E_HIP;
}
