// zx_paged_attend.h -- what the attention kernels over a paged K/V cache share: their
// arguments, how the tokens are split between workgroups, and the kernel that joins the pieces.
#pragma once

#include <type_traits>

#include "zx_paged.h"

namespace zxp {

// global memory by name: an address put together from integers would else be read as one of any kind
typedef __attribute__((address_space(1))) u4 global_u4;
typedef __attribute__((address_space(1))) u2 global_u2;
typedef __attribute__((address_space(1))) uint32_t global_u32;
typedef __attribute__((address_space(1))) uint8_t global_u1;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_huge_valf();
// The running maximum is raised only when a score passes it by more than this (in powers
// of two): until then weights stay below 2^8, which 32-bit sums and BF16 weights hold
// as exactly as weights below one.
constexpr float kSlack = 8.0f;

constexpr uint32_t kStep = 128;               // tokens of a four-wave workgroup's step in k_rows: 32 for each wave

struct AttendArgs {
    Cache c;
    Batch b;
    Rows q, out;
    float *lse;
    const int32_t *blocks;                    // [n_tokens][heads][n_blocks], or null
    float *part;                              // [slot][heads][rows of a tile][D]: sums of weights times values
    float *stat;                              // [slot][heads][rows of a tile][2]: maximum, sum of weights
    float scale;                              // includes log2 e
    int32_t causal, window;
    uint32_t group, q_heads, n_blocks;
    uint32_t lo_rows, hi_rows;                // this kernel takes sequences with lo_rows < rows <= hi_rows
    uint32_t slots;                           // pieces that the workspace has room for
    uint32_t pieces;                          // block lists: pieces of a row tile
    // how sequences are split (chunk_steps): pieces a head to aim at, whether they are to fit one round of
    // the card, and the fewest steps of a piece
    uint32_t goal, one_round, least;
};

// A row at position p sees tokens [max(0, p - window + 1), p + 1) if causal, else up to kv; at a
// negative position (fewer tokens than new ones) none.
__device__ __forceinline__ int32_t first_seen(const AttendArgs &g, int32_t p)
{
    return g.window > 0 && p - g.window + 1 > 0 ? p - g.window + 1 : 0;
}
__device__ __forceinline__ int32_t end_seen(const AttendArgs &g, int32_t p, int32_t kv)
{
    return p < 0 ? 0 : g.causal ? p + 1 : kv;
}

// Steps of UNIT tokens that cover what the sequence's rows see (at least one).
template <int UNIT>
__device__ __forceinline__ uint32_t seq_steps(const AttendArgs &g, const Seq &v)
{
    const int32_t lo = first_seen(g, v.kv - v.nq) & ~15;
    return v.kv > lo ? div_up((uint32_t)(v.kv - lo), UNIT) : 1u;
}

__device__ __forceinline__ bool takes(const AttendArgs &g, const Seq &v)
{
    const uint32_t rows = (uint32_t)v.nq * g.group;
    return rows > g.lo_rows && rows <= g.hi_rows;
}

// How the tokens of long sequences are split: `chunk` steps of UNIT tokens for a
// workgroup, by the same rule in the kernel that does the work and in the one that joins it.
// The host aims at `goal` pieces a head (Split).  Where they are to fit into what the card
// holds at a time, the chunk is raised until they do (steps / chunk rounds up for every
// sequence): a second round of a few workgroups would cost as much as the first.
template <int ROWS, int UNIT>
__device__ __forceinline__ uint32_t chunk_steps(const AttendArgs &g)
{
    if (g.slots == 0) return 0x7FFFFFFFu;        // no sequence is long enough to be split
    const uint32_t lane = threadIdx.x & 63u;
    auto sum = [&](auto of) {
        uint32_t all = 0;
        for (uint32_t s0 = 0; s0 < g.b.n_seqs; s0 += 64) {
            uint32_t w = 0, total;
            if (s0 + lane < g.b.n_seqs) {
                const Seq v = load_seq(g.b, s0 + lane);
                if (takes(g, v)) w = div_up((uint32_t)v.nq * g.group, ROWS) * of(seq_steps<UNIT>(g, v));
            }
            (void)wave_excl_scan(w, total);
            all += total;
        }
        return all;
    };
    uint32_t c = div_up(sum([](uint32_t s) { return s; }), g.goal);
    if (c <= g.least) return g.least;
    for (int i = 0; i < 3 && g.one_round; ++i) {
        const uint32_t n = sum([c](uint32_t s) { return div_up(s, c); });
        if (n <= g.goal) break;
        const uint32_t d = (uint32_t)(((uint64_t)c * n + g.goal - 1) / g.goal);
        c = d > c ? d : c + 1;
    }
    return c;
}

// Items of a sequence: its row tiles times the pieces of each.  A piece of a row tile that is
// split has a slot of the workspace; slots are counted over split sequences only.  (A split
// sequence has more than one piece's steps, so it has fewer than twice steps / chunk pieces,
// and all of them together fewer than twice as many as were aimed at.)
template <int ROWS, int UNIT>
__device__ __forceinline__ uint32_t seq_pieces(const AttendArgs &g, const Seq &v, uint32_t chunk)
{
    return div_up(seq_steps<UNIT>(g, v), chunk);
}
template <int ROWS, int UNIT>
__device__ __forceinline__ bool find_piece(const AttendArgs &g, uint32_t item, uint32_t chunk, uint32_t &seq, Seq &sv, uint32_t &rt, uint32_t &part,
                                           uint32_t &nch, uint32_t &slot)
{
    uint32_t local, before;
    if (!find_item(
            g.b, item, [&](const Seq &v) { return takes(g, v) ? div_up((uint32_t)v.nq * g.group, ROWS) * seq_pieces<ROWS, UNIT>(g, v, chunk) : 0u; },
            [&](const Seq &v) {
                const uint32_t n = takes(g, v) ? seq_pieces<ROWS, UNIT>(g, v, chunk) : 1u;
                return n > 1 ? div_up((uint32_t)v.nq * g.group, ROWS) * n : 0u;
            },
            seq, sv, local, before))
        return false;
    nch = seq_pieces<ROWS, UNIT>(g, sv, chunk);
    rt = local / nch;
    part = local % nch;
    slot = before + local;
    return nch == 1 || slot < g.slots;           // (overlapping sequences may make more than there is room for)
}

__device__ __forceinline__ float max_halves(float x)     // over lanes l and l ^ 32
{
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float sum_halves(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}
__device__ __forceinline__ float max_quarters(float x)   // over lanes l, l ^ 16, l ^ 32, l ^ 48
{
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    return max_halves(fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1])));
}
__device__ __forceinline__ float sum_quarters(float x)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    return sum_halves(__builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]));
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const bf2 r = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, r);
}

// Two E4M3 bytes of w (the low or the high half) as two BF16 values: exact.
template <bool HI>
__device__ __forceinline__ uint32_t fp8_pair(uint32_t w)
{
    const bf2 r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, 1.0f, HI);
    return __builtin_bit_cast(uint32_t, r);
}

// Whether either BF16 value of a pair is infinite or NaN.
__device__ __forceinline__ bool odd_pair(uint32_t w)
{
    return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}
// The pair with such values as zero.
__device__ __forceinline__ uint32_t tame_pair(uint32_t w)
{
    if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
    if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
    return w;
}
// ---------------------------------------------------------------- joining

// One workgroup adds up pieces of rows of one row tile.  UNIT 0: block lists, whose row tiles all have
// g.pieces pieces; else row tiles of split sequences.
template <int D, int ROWS, int UNIT>
static __global__ __launch_bounds__(256) void k_join(AttendArgs g)
{
    constexpr int LN = D / 4;                    // lanes of a row
    constexpr int GR = 256 / LN;                 // rows, or pieces of one, at a time
    __shared__ __align__(16) float xs[GR][D + 4];
    __shared__ float ls[GR];
    const uint32_t h = blockIdx.x % g.c.heads, item = blockIdx.x / g.c.heads;
    const uint32_t G = g.group;
    uint32_t seq, local, before, nch, base_slot, tok0 = 0, row0, nrows;
    Seq sv;
    if constexpr (UNIT == 0) {
        const uint32_t tiles = div_up(G, ROWS);
        nch = g.pieces;
        if (!find_item(g.b, item, [&](const Seq &v) { return (uint32_t)v.nq * tiles; }, [](const Seq &) { return 0u; }, seq, sv, local, before)) return;
        tok0 = local / tiles;
        row0 = (local % tiles) * ROWS;
        nrows = G - row0;
        base_slot = item * nch;
    } else {
        const uint32_t chunk = chunk_steps<ROWS, UNIT>(g);
        auto split = [&](const Seq &v) {         // row tiles of a split sequence
            return takes(g, v) && seq_pieces<ROWS, UNIT>(g, v, chunk) > 1 ? div_up((uint32_t)v.nq * G, ROWS) : 0u;
        };
        if (!find_item(g.b, item, split, [&](const Seq &v) { return split(v) * seq_pieces<ROWS, UNIT>(g, v, chunk); }, seq, sv, local, before)) return;
        nch = seq_pieces<ROWS, UNIT>(g, sv, chunk);
        row0 = local * ROWS;
        nrows = (uint32_t)sv.nq * G - row0;
        base_slot = before + local * nch;
        if (base_slot + nch > g.slots) return;
    }
    if (nrows > (uint32_t)ROWS) nrows = ROWS;
    const uint32_t gr = threadIdx.x / LN, ln = threadIdx.x % LN;
    const float vs = g.c.v_scale ? g.c.v_scale[h] : 1.0f;
    auto where = [&](uint32_t piece, uint32_t row) { return ((uint64_t)(base_slot + piece) * g.c.heads + h) * ROWS + row; };
    auto place = [&](uint32_t row) { return sv.q0 + (int64_t)(tok0 + (row0 + row) / G); };
    auto head = [&](uint32_t row) { return h * G + (row0 + row) % G; };
    // GR rows at a time, a lane adds up its four channels, N pieces under way at once
    auto rows = [&](auto most) {
        constexpr uint32_t N = decltype(most)::value;
        for (uint32_t row = blockIdx.z * GR + gr; row < nrows; row += gridDim.z * GR) {
            f4 x = {0, 0, 0, 0};
            float mm = -kInf, ll = 0.0f;
            for (uint32_t i0 = 0; i0 < nch; i0 += N) {
                // (reads past the last piece repeat it)
                f4 y[N];
                float pm[N], pl[N], nm = mm;
#pragma unroll
                for (uint32_t i = 0; i < N; ++i) {
                    const uint64_t at = where(i0 + i < nch ? i0 + i : nch - 1, row);
                    pm[i] = g.stat[at * 2];
                    pl[i] = g.stat[at * 2 + 1];
                    y[i] = *reinterpret_cast<const f4 *>(g.part + at * D + 4 * ln);
                }
#pragma unroll
                for (uint32_t i = 0; i < N; ++i) nm = fmaxf(nm, pm[i]);
                const float base = nm == -kInf ? 0.0f : nm, old = __builtin_amdgcn_exp2f(mm - base);
                mm = nm;
                ll *= old;
                x *= old;
#pragma unroll
                for (uint32_t i = 0; i < N; ++i) {
                    if (i0 + i >= nch) break;
                    const float f = __builtin_amdgcn_exp2f(pm[i] - base);
                    ll += pl[i] * f;
                    x += y[i] * f;
                }
            }
            const float inv = ll == 0.0f ? 0.0f : vs / ll;
            *reinterpret_cast<u2 *>(g.out.p + place(row) * g.out.token + (int64_t)head(row) * g.out.head + 4 * ln) =
                u2{pack2(x[0] * inv, x[1] * inv), pack2(x[2] * inv, x[3] * inv)};
            if (g.lse && ln == 0) g.lse[place(row) * g.q_heads + head(row)] = ll == 0.0f ? -kInf : (mm + log2f(ll)) * kLn2;
        }
    };
    // (repeated reads are not free: five or six pieces of 13 x 256 rows 22 us at six, 28 at eight)
    if (nch <= 3) return rows(std::integral_constant<uint32_t, 3>{});
    if (nch <= 6) return rows(std::integral_constant<uint32_t, 6>{});
    if (nch <= 8 || gridDim.z < nrows) return rows(std::integral_constant<uint32_t, 8>{});
    // many pieces and a workgroup for every row: its pieces are shared between GR groups of lanes
    for (uint32_t row = blockIdx.z; row < nrows; row += gridDim.z) {
        float mm = -kInf;
        for (uint32_t i = threadIdx.x & 63u; i < nch; i += 64) mm = fmaxf(mm, g.stat[where(i, row) * 2]);
        for (int w = 32; w >= 1; w >>= 1) mm = fmaxf(mm, __shfl_xor(mm, w, 64));
        const float base = mm == -kInf ? 0.0f : mm;
        f4 x = {0, 0, 0, 0};
        float ll = 0.0f;
#pragma unroll 4
        for (uint32_t i = gr; i < nch; i += GR) {
            const uint64_t at = where(i, row);
            const float f = __builtin_amdgcn_exp2f(g.stat[at * 2] - base);
            ll += g.stat[at * 2 + 1] * f;
            x += *reinterpret_cast<const f4 *>(g.part + at * D + 4 * ln) * f;
        }
        __syncthreads();
        *reinterpret_cast<f4 *>(&xs[gr][4 * ln]) = x;
        if (ln == 0) ls[gr] = ll;
        __syncthreads();
        if (threadIdx.x < D / 2) {
            const uint32_t ch = threadIdx.x * 2;
            float a = 0.0f, b = 0.0f;
            ll = 0.0f;
#pragma unroll
            for (int i = 0; i < GR; ++i) {
                a += xs[i][ch];
                b += xs[i][ch + 1];
                ll += ls[i];
            }
            const float inv = ll == 0.0f ? 0.0f : vs / ll;
            *reinterpret_cast<uint32_t *>(g.out.p + place(row) * g.out.token + (int64_t)head(row) * g.out.head + ch) = pack2(a * inv, b * inv);
            if (g.lse && ch == 0) g.lse[place(row) * g.q_heads + head(row)] = ll == 0.0f ? -kInf : (mm + log2f(ll)) * kLn2;
        }
    }
}

// sum over the sequences of ceil(nq * group / rows), bounded by what the host knows
inline uint32_t bound_tiles(uint64_t n, uint64_t seqs, uint64_t group, uint64_t rows)
{
    const uint64_t a = n * ceil_div(group, rows), b = n * group / rows + seqs;
    return (uint32_t)(a < b ? a : b);
}

// How a kernel's row tiles are split, from what the host knows: `tiles` row tiles a head at
// most, `room` workgroups a head that the card holds at a time, `many` rounds of them to
// aim at where the row tiles alone fill more than half of one, and the fewest steps of a
// piece in either case.
inline void plan_split(uint32_t tiles, uint32_t room, uint32_t many, uint32_t least, uint32_t least_many, uint64_t cap, uint32_t unit, AttendArgs &g)
{
    g.one_round = 2 * tiles <= room;
    g.goal = g.one_round ? room : many * room;
    g.least = g.one_round ? least : least_many;
    const uint64_t each = ceil_div(cap, (uint64_t)g.least * unit), all = tiles * each;       // pieces that lengths up to cap may make
    g.slots = each <= 1 ? 0 : all < 2 * g.goal ? (uint32_t)all : 2 * g.goal;
}
// Items of the kernel, and row tiles for its join (0: nothing can be split).  Row tiles that are not split are items
// too but have no slot: steps / chunk, rounded up for each of them, makes at most goal + tiles, and no more than all
// pieces that lengths up to cap may make, which slots holds where that is below 2 * goal (elsewhere goal + tiles is less).
inline uint32_t split_items(uint32_t tiles, const AttendArgs &g)
{
    if (!g.slots) return tiles;
    const uint32_t most = g.goal + tiles;
    return g.slots < 2 * g.goal && g.slots < most ? g.slots : most;
}
inline uint32_t split_tiles(uint32_t tiles, const AttendArgs &g) { return !g.slots ? 0 : tiles < g.goal ? tiles : g.goal; }

// Workgroups of k_join that share the rows of a row tile: about a thousand in all.
inline uint32_t join_depth(uint32_t tiles, uint32_t rows)
{
    const uint32_t z = tiles ? ceil_div(1024, tiles) : 1;
    return z < rows ? z : rows;
}

// The tiled kernel for many rows (zx_paged_chunk.hip) and its join, with how it is to be launched.
struct ChunkPlan {
    uint32_t waves, tiles;           // waves of a workgroup; bound of the row tiles a head
};
// A launch counts its threads in 32 bits.
inline bool launchable(uint64_t workgroups, uint32_t threads) { return workgroups * threads <= 0xFFFFFFFFull; }
ChunkPlan plan_chunk(uint64_t rows, uint32_t head_dim, uint32_t heads, uint64_t tokens, uint64_t seqs, uint64_t group, uint64_t cap, AttendArgs &g);
void run_chunk(int dtype, uint32_t head_dim, const ChunkPlan &p, const AttendArgs &g, hipStream_t stream);

}  // namespace zxp
