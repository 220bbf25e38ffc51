// zx_paged_attend.h -- what the attention kernels over a paged K/V cache share: their
// arguments, how the tokens are split between workgroups, and the kernel that joins the pieces.
#pragma once

#include "zx_paged.h"

namespace zxp {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kInf = __builtin_huge_valf();
// The running maximum is raised only when a score passes it by more than this (in powers
// of two): until then weights stay below 2^8, which 32-bit sums and BF16 weights hold
// as exactly as weights below one.
constexpr float kSlack = 8.0f;

constexpr uint32_t kRowsThreads = 256;        // four waves
constexpr uint32_t kStep = 128;               // tokens of a workgroup's step: 32 for each wave

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
    uint32_t slots;                           // pieces that the workspace has room for (k_rows)
    uint32_t target;                          // k_rows: workgroups wanted for each head; k_chunk and block lists: pieces of a row tile
};

// The new tokens of a sequence see tokens from `lo` on, in all; a row at position p
// sees [max(0, p - window + 1), p + 1) if causal, else up to kv.
__device__ __forceinline__ int32_t first_seen(const AttendArgs &g, int32_t p)
{
    return g.window > 0 && p - g.window + 1 > 0 ? p - g.window + 1 : 0;
}
__device__ __forceinline__ int32_t end_seen(const AttendArgs &g, int32_t p, int32_t kv)
{
    const int32_t e = g.causal ? p + 1 : kv;
    return e < 0 ? 0 : e;
}

// Steps of kStep tokens that cover what the sequence's rows see (at least one).
__device__ __forceinline__ uint32_t seq_steps(const AttendArgs &g, const Seq &v)
{
    const int32_t lo = first_seen(g, v.kv - v.nq) & ~15;
    return v.kv > lo ? div_up((uint32_t)(v.kv - lo), kStep) : 1u;
}

__device__ __forceinline__ bool takes(const AttendArgs &g, const Seq &v)
{
    const uint32_t rows = (uint32_t)v.nq * g.group;
    return rows > g.lo_rows && rows <= g.hi_rows;
}

// How k_rows and k_join split the work of whole sequences: `chunk` steps for a workgroup,
// such that about `target` workgroups a head share all of it.
template <int ROWS>
__device__ __forceinline__ uint32_t chunk_steps(const AttendArgs &g)
{
    const uint32_t lane = threadIdx.x & 63u;
    uint32_t sum = 0;
    for (uint32_t s0 = 0; s0 < g.b.n_seqs; s0 += 64) {
        uint32_t w = 0, total;
        if (s0 + lane < g.b.n_seqs) {
            const Seq v = load_seq(g.b, s0 + lane);
            if (takes(g, v)) w = div_up((uint32_t)v.nq * g.group, ROWS) * seq_steps(g, v);
        }
        (void)wave_excl_scan(w, total);
        sum += total;
    }
    const uint32_t c = div_up(sum, g.target);
    return c ? c : 1u;
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
// The pair with such values as zero, and the pair of ones where a value is +inf or NaN
// (SIGN 0), or -inf or NaN (SIGN 1): what a row that sees the value has to add, times infinity.
__device__ __forceinline__ uint32_t tame_pair(uint32_t w)
{
    if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
    if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
    return w;
}
template <int SIGN>
__device__ __forceinline__ uint32_t wild_pair(uint32_t w)
{
    uint32_t r = 0;
    const uint32_t inf = SIGN ? 0xFF80u : 0x7F80u, a = w & 0xFFFFu, b = w >> 16;
    if (a == inf || (a & 0x7FFFu) > 0x7F80u) r |= 0x3F80u;
    if (b == inf || (b & 0x7FFFu) > 0x7F80u) r |= 0x3F800000u;
    return r;
}

// ---------------------------------------------------------------- joining

enum { JOIN_ROWS, JOIN_LIST, JOIN_CHUNK };

// One workgroup adds up the pieces of one row of a row tile (or of every gridDim.z-th).
template <int D, int ROWS, int MODE>
static __global__ __launch_bounds__(256) void k_join(AttendArgs g)
{
    constexpr int LN = D / 4;                    // lanes of a row
    constexpr int GR = 256 / LN;                 // pieces at a time
    __shared__ __align__(16) float xs[GR][D + 4];
    __shared__ float ls[GR];
    const uint32_t h = blockIdx.x % g.c.heads, item = blockIdx.x / g.c.heads;
    const uint32_t G = g.group;
    uint32_t seq, local, before, nch, base_slot, tok0 = 0, row0, nrows;
    Seq sv;
    if constexpr (MODE == JOIN_LIST) {
        const uint32_t tiles = div_up(G, ROWS);
        nch = g.target;
        if (!find_item(g.b, item, [&](const Seq &v) { return (uint32_t)v.nq * tiles; }, [](const Seq &) { return 0u; }, seq, sv, local, before)) return;
        tok0 = local / tiles;
        row0 = (local % tiles) * ROWS;
        nrows = G - row0;
        base_slot = item * nch;
    } else if constexpr (MODE == JOIN_CHUNK) {
        nch = g.target;
        if (!find_item(g.b, item, [&](const Seq &v) { return takes(g, v) ? div_up((uint32_t)v.nq * G, ROWS) : 0u; }, [](const Seq &) { return 0u; }, seq, sv,
                       local, before))
            return;
        row0 = local * ROWS;
        nrows = (uint32_t)sv.nq * G - row0;
        base_slot = item * nch;
    } else {
        const uint32_t chunk = chunk_steps<ROWS>(g);
        if (!find_item(
                g.b, item, [&](const Seq &v) { return takes(g, v) ? div_up((uint32_t)v.nq * G, ROWS) : 0u; },
                [&](const Seq &v) { return takes(g, v) ? div_up((uint32_t)v.nq * G, ROWS) * div_up(seq_steps(g, v), chunk) : 0u; }, seq, sv, local, before))
            return;
        nch = div_up(seq_steps(g, sv), chunk);
        row0 = local * ROWS;
        nrows = (uint32_t)sv.nq * G - row0;
        base_slot = before + local * nch;
    }
    if (nch == 1) return;                        // written by the kernel itself
    if (MODE == JOIN_ROWS && base_slot + nch > g.slots) return;   // overlapping sequences: more pieces than there is room for
    if (nrows > (uint32_t)ROWS) nrows = ROWS;
    const uint32_t gr = threadIdx.x / LN, ln = threadIdx.x % LN;
    const float vs = g.c.v_scale ? g.c.v_scale[h] : 1.0f;
    for (uint32_t row = blockIdx.z; row < nrows; row += gridDim.z) {
        float mm = -kInf;
        for (uint32_t i = threadIdx.x & 63u; i < nch; i += 64)
            mm = fmaxf(mm, g.stat[((((uint64_t)(base_slot + i) * g.c.heads + h) * ROWS) + row) * 2]);
        for (int w = 32; w >= 1; w >>= 1) mm = fmaxf(mm, __shfl_xor(mm, w, 64));
        const float base = mm == -kInf ? 0.0f : mm;
        f4 x = {0, 0, 0, 0};
        float ll = 0.0f;
        for (uint32_t i = gr; i < nch; i += GR) {
            const uint64_t at = ((uint64_t)(base_slot + i) * g.c.heads + h) * ROWS + row;
            const float pm = g.stat[at * 2], pl = g.stat[at * 2 + 1];
            const f4 y = *reinterpret_cast<const f4 *>(g.part + at * D + 4 * ln);
            const float f = __builtin_amdgcn_exp2f(pm - base);
            ll += pl * f;
            x += y * f;
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
            const uint32_t tok = tok0 + (row0 + row) / G, gh = (row0 + row) % G;
            const int64_t at = sv.q0 + (int32_t)tok;
            const float inv = ll == 0.0f ? 0.0f : vs / ll;
            *reinterpret_cast<uint32_t *>(g.out.p + at * g.out.token + (int64_t)(h * G + gh) * g.out.head + ch) = pack2(a * inv, b * inv);
            if (g.lse && ch == 0) g.lse[at * g.q_heads + h * G + gh] = ll == 0.0f ? -kInf : (mm + log2f(ll)) * kLn2;
        }
    }
}

// The tiled kernel for many rows (zx_paged_chunk.hip): waves of a workgroup for a batch
// whose longest sequence has `rows` rows, and the launch with its join.
uint32_t chunk_waves(uint64_t rows, uint32_t head_dim);
void run_chunk(int dtype, uint32_t head_dim, uint32_t waves, uint32_t items, uint32_t split, const AttendArgs &g, hipStream_t stream);

}  // namespace zxp
