// zx_beam.hip -- the choice of the next beams from the logits.
//
// With lse_b = ln sum_t exp(s x_bt) over the tokens that beam b may take, candidate (b, t) has the total
// score_b + s x_bt - lse_b, and the n_out candidates of a group with the largest weight_b * total are taken.
//
// Bound by reading the logits once.  k_beam_parts: a wave holds one part of a row in registers, 64 * E logits,
// so that the part's maximum is known before the first exponential and none is taken twice.  The n_out largest of
// the part are found without sorting: the n_out-th largest of the 64 lanes' maxima (by bisection of its bits, with
// ballots) is no larger than the n_out-th largest logit, so only logits from there on can be among them, and
// hardly more than n_out are; those few are ranked by counting.  k_beam_pick: one workgroup a group joins the
// parts' sums, turns the parts' candidates into totals, and finds the n_out best of them in the same two steps.
//
// Rounding: a part's sum is taken in 32 bits over a lane's E logits and in 64 bits from there on; totals are
// formed and compared in 64 bits, since which of two beams is taken must not turn on a rounding.
#include "zx_common.h"

namespace zxb {

using zxk::report;

typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr float kInf = __builtin_huge_valf();
constexpr float kLowest = -3.4028234663852886e38f;
constexpr uint32_t kMostOut = 64, kMostBeams = 64;
constexpr uint32_t kMostVocab = 1u << 24;

enum { BF16, F16, F32 };

struct Stat {
    float top;                       // the part's largest logit (-inf: none may be taken)
    uint32_t unused;
    double sum;                      // of exp(s (x - top)) over the part
};
struct Cand {
    float x;                         // -inf: none
    uint32_t token;
};

struct BeamArgs {
    const void *logits;
    int64_t group_stride, beam_stride;           // in elements
    const float *scores, *weights;
    const uint8_t *finished;
    const uint32_t *allowed;
    Stat *stat;                                  // [row][part]
    Cand *cand;                                  // [row][part][n_out], the largest first
    float *out_scores;
    int32_t *parents, *tokens;
    uint8_t *out_finished;
    uint32_t *err;
    double scale;
    uint32_t groups, beams, vocab, n_out, parts, words;
    int32_t end;
};

// Whether a row's logits are needed: the beam lives and is not finished.
__device__ __forceinline__ bool row_runs(const BeamArgs &g, uint32_t row)
{
    const float s = g.scores[row];
    return s > -kInf && s < kInf && !(g.finished && g.finished[row]);
}

__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k)
{
    return __builtin_bit_cast(float, k ^ ((uint32_t)(~(int32_t)k >> 31) | 0x80000000u));
}
__device__ __forceinline__ uint64_t ordered(double x)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}

// The largest t that at least n of the wave's keys reach (0 where there are fewer than n lanes' worth), or, once
// exactly n keys reach it, a smaller one that does as well.
__device__ __forceinline__ uint32_t nth_largest(uint32_t key, uint32_t n)
{
    uint32_t t = 0;
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t u = t | (1u << bit);
        const uint32_t c = (uint32_t)__popcll(__ballot(key >= u));
        if (c >= n) t = u;
        if (c == n) break;
    }
    return t;
}

template <int TY>
struct Type {
    static constexpr int N = TY == F32 ? 4 : 8;  // logits of 16 bytes
    static constexpr int W = TY == F32 ? 4 : 2;  // bytes of one
};

template <int TY>
__device__ __forceinline__ float one_logit(const uint8_t *p)
{
    if constexpr (TY == F32) {
        float x;
        __builtin_memcpy(&x, p, 4);
        return x;
    } else {
        uint16_t h;
        __builtin_memcpy(&h, p, 2);
        return TY == BF16 ? __builtin_bit_cast(float, (uint32_t)h << 16) : (float)__builtin_bit_cast(_Float16, h);
    }
}

template <int TY>
__device__ __forceinline__ void unpack(u4 w, float *x)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t v = w[i];                 // (a bit cast of the element itself takes the vector's first)
        if constexpr (TY == F32) {
            x[i] = __builtin_bit_cast(float, v);
        } else if constexpr (TY == BF16) {
            x[2 * i] = __builtin_bit_cast(float, v << 16);
            x[2 * i + 1] = __builtin_bit_cast(float, v & 0xFFFF0000u);
        } else {
            x[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)v);
            x[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(v >> 16));
        }
    }
}

__device__ __forceinline__ float wave_max(float x)
{
    for (int o = 32; o >= 1; o >>= 1) x = fmaxf(x, __shfl_xor(x, o, 64));
    return x;
}
__device__ __forceinline__ double wave_sum(double x)
{
    for (int o = 32; o >= 1; o >>= 1) x += __shfl_xor(x, o, 64);
    return x;
}

constexpr uint32_t kRoom = 128;                  // logits of a part that are ranked at a time (two a lane)

// Rank of each of a wave's n <= 128 keys (lane l's a is key l, its b key 64 + l): how many are larger.
__device__ __forceinline__ void rank_keys(uint64_t a, uint64_t b, uint32_t n, uint32_t &ra, uint32_t &rb)
{
    ra = rb = 0;
    const uint32_t first = n < 64 ? n : 64;
    auto other = [](uint64_t k, uint32_t j) {
        return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(k >> 32), (int)j) << 32 |
               (uint32_t)__builtin_amdgcn_readlane((int)k, (int)j);
    };
    for (uint32_t j = 0; j < first; ++j) {
        const uint64_t k = other(a, j);
        ra += k > a;
        rb += k > b;
    }
    for (uint32_t j = 64; j < n; ++j) {
        const uint64_t k = other(b, j - 64);
        ra += k > a;
        rb += k > b;
    }
}

template <int TY, int E>
__global__ __launch_bounds__(256) void k_beam_parts(BeamArgs g)
{
    constexpr int N = Type<TY>::N, W = Type<TY>::W, U = E / N;
    __shared__ uint64_t room[4][kRoom];
    const uint32_t lane = threadIdx.x & 63u, wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t item = blockIdx.x * 4 + wave;
    const uint32_t row = item / g.parts, part = item - row * g.parts;
    if (row >= g.groups * g.beams || !row_runs(g, row)) return;
    const uint8_t *p = static_cast<const uint8_t *>(g.logits) +
                       ((int64_t)(row / g.beams) * g.group_stride + (int64_t)(row % g.beams) * g.beam_stride) * W;
    const uint32_t t0 = part * (64 * E) + lane * N;          // the lane's first token
    float x[E];
    {
        u4 raw[U];
        uint32_t bits[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t t = t0 + u * (64 * N);
            raw[u] = u4{0, 0, 0, 0};
            if (t + N <= g.vocab) __builtin_memcpy(&raw[u], p + (uint64_t)t * W, 16);
            bits[u] = t < g.vocab ? 0xFFFFFFFFu : 0;
            if (g.allowed && t < g.vocab) bits[u] = g.allowed[(uint64_t)row * g.words + (t >> 5)] >> (t & 31u);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t t = t0 + u * (64 * N);
            unpack<TY>(raw[u], x + u * N);
            if (t < g.vocab && t + N > g.vocab) {            // a row's last tokens
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (t + i < g.vocab) x[u * N + i] = one_logit<TY>(p + (uint64_t)(t + i) * W);
                    else bits[u] &= ~(1u << i);
            }
            if (g.allowed || t + N > g.vocab) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (!(bits[u] >> i & 1u)) x[u * N + i] = -kInf;
            }
        }
    }
    float mine = -kInf;
#pragma unroll
    for (int i = 0; i < E; ++i) mine = fmaxf(mine, x[i]);    // (NaN is left out here; it shows in the sum)
    const float top = wave_max(mine);
    const float base = top == -kInf ? 0.0f : top, c = (float)(g.scale * 1.4426950408889634);
    float s[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < E; ++i) s[i & 3] += __builtin_amdgcn_exp2f((x[i] - base) * c);
    const double sum = wave_sum((double)(s[0] + s[1]) + (double)(s[2] + s[3]));

    const uint64_t at = (uint64_t)row * g.parts + part;
    if (lane == 0) {
        g.stat[at].top = top;
        g.stat[at].sum = sum;
    }
    // the part's n_out largest: keys that order by logit, then by token, the earlier first
    float edge = fmaxf(unordered(nth_largest(ordered(mine), g.n_out)), kLowest);
    uint32_t edge_token = 0xFFFFFFFFu;           // of logits equal to the edge, those up to this token
    uint32_t n;
    uint64_t ka, kb;
    uint32_t ra, rb;
    for (;;) {
        n = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const uint32_t t = t0 + (i / N) * (64 * N) + i % N;
            const uint64_t m = __ballot(x[i] > edge || (x[i] == edge && t <= edge_token));
            if (m) {
                const uint32_t to = n + (uint32_t)__popcll(m & zxk::lanemask_lt());
                // (+ 0: minus zero is no smaller than zero)
                if ((m >> lane & 1u) && to < kRoom) room[wave][to] = (uint64_t)ordered(x[i] + 0.0f) << 32 | (0xFFFFFFFFu - t);
                n += (uint32_t)__popcll(m);
            }
        }
        zxk::wave_sync();
        const uint32_t some = n < kRoom ? n : kRoom;
        ka = lane < some ? room[wave][lane] : 0;
        kb = lane + 64 < some ? room[wave][lane + 64] : 0;
        rank_keys(ka, kb, some, ra, rb);
        if (n <= kRoom) break;
        // too many: the n_out-th of those that fit is an edge that leaves out kRoom - n_out of them at least
        const uint64_t ma = __ballot(ra == g.n_out - 1), mb = __ballot(rb == g.n_out - 1);
        const uint64_t k = ma ? ka : kb;
        const int l = __builtin_ctzll(ma ? ma : mb);
        edge = unordered((uint32_t)__builtin_amdgcn_readlane((int)(k >> 32), l));
        edge_token = 0xFFFFFFFFu - (uint32_t)__builtin_amdgcn_readlane((int)k, l);
        zxk::wave_sync();
    }
    Cand *o = g.cand + at * g.n_out;
    if (lane < n && ra < g.n_out) o[ra] = Cand{unordered((uint32_t)(ka >> 32)), 0xFFFFFFFFu - (uint32_t)ka};
    if (lane + 64 < n && rb < g.n_out) o[rb] = Cand{unordered((uint32_t)(kb >> 32)), 0xFFFFFFFFu - (uint32_t)kb};
    if (lane >= n && lane < g.n_out) o[lane] = Cand{-kInf, 0};
}

struct Best {
    uint64_t key;                                // orders like weight * total
    uint64_t place;                              // beam << 32 | token
    double total;
};
constexpr uint32_t kList = 1024;

__device__ __forceinline__ bool better(uint64_t ka, uint64_t pa, uint64_t kb, uint64_t pb) { return ka > kb || (ka == kb && pa < pb); }

template <int NT>
__global__ __launch_bounds__(NT) void k_beam_pick(BeamArgs g)
{
    __shared__ Best list[kList];
    __shared__ double base[kMostBeams], tops[kMostBeams], weight[kMostBeams];
    __shared__ uint32_t kind[kMostBeams];        // 0: no candidates, 1: the parts', 2: finished
    __shared__ uint32_t count, edge_hi[NT / 64];
    __shared__ uint64_t edge_key, edge_place;
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
    const uint32_t row0 = blockIdx.x * g.beams;
    for (uint32_t b = wave; b < g.beams; b += NT / 64) {
        const uint32_t row = row0 + b;
        const float sc = g.scores[row], w = g.weights ? g.weights[row] : 1.0f;
        const bool ended = g.finished && g.finished[row];
        uint32_t k = 0;
        double from = sc;
        float top = -kInf;
        const bool there = sc != -kInf;
        bool bad = there && (!(sc < kInf) || !(w > 0.0f && w < kInf));       // (NaN too)
        if (there && !bad) {
            k = 2;
            if (!ended) {
                for (uint32_t i = lane; i < g.parts; i += 64) top = fmaxf(top, g.stat[(uint64_t)row * g.parts + i].top);
                top = wave_max(top);
                double s = 0.0;
                for (uint32_t i = lane; i < g.parts; i += 64) {
                    const Stat v = g.stat[(uint64_t)row * g.parts + i];
                    s += v.top == -kInf ? v.sum : v.sum * exp(((double)v.top - (double)top) * g.scale);
                }
                s = wave_sum(s);
                bad = !(s < (double)kInf) || top == kInf;    // a NaN or +inf among the logits: no distribution
                k = !bad && top > -kInf ? 1 : 0;
                from = (double)sc - log(s);
            }
        }
        if (lane == 0) {
            kind[b] = k;
            base[b] = from;
            tops[b] = (double)top;
            weight[b] = (double)w;
            if (bad) report(g.err, ZX_E_CORRUPT);
        }
    }
    __syncthreads();
    // entries: the parts' candidates of all rows, then one for each finished beam
    const uint32_t each = g.parts * g.n_out, all = g.beams * each;
    const Cand *cand = g.cand + (uint64_t)row0 * each;
    auto entry = [&](uint32_t e, Best &o) {
        const bool part = e < all;
        const uint32_t b = part ? e / each : e - all;
        if (kind[b] != (part ? 1u : 2u)) return false;
        if (part) {
            const Cand v = cand[e];
            if (v.x == -kInf) return false;
            o.total = base[b] + ((double)v.x - tops[b]) * g.scale;       // (score - ln sum) + s (x - top): no large logit swallows the rest
            o.place = (uint64_t)b << 32 | v.token;
        } else {
            o.total = base[b];
            o.place = (uint64_t)b << 32 | (uint32_t)g.end;
        }
        o.key = ordered(o.total * weight[b] + 0.0);
        return true;
    };
    uint64_t mine = 0;
    for (uint32_t e = tid; e < all + g.beams; e += NT) {
        Best v;
        if (entry(e, v) && v.key > mine) mine = v.key;
    }
    // n_out keys of one wave at least reach the edge (or it is zero), so n_out of the group do
    const uint32_t hi = nth_largest((uint32_t)(mine >> 32), g.n_out);
    if (lane == 0) edge_hi[wave] = hi;
    if (tid == 0) count = 0;
    __syncthreads();
    uint32_t h = 0;
    for (int i = 0; i < NT / 64; ++i) h = edge_hi[i] > h ? edge_hi[i] : h;
    uint64_t ek = (uint64_t)h << 32, ep = ~0ull;
    uint32_t n;
    for (uint32_t round = 0;; ++round) {
        for (uint32_t e = tid; e < all + g.beams; e += NT) {
            Best v;
            if (!entry(e, v) || better(ek, ep, v.key, v.place)) continue;
            const uint32_t to = atomicAdd(&count, 1u);
            if (to < kList) list[to] = v;
        }
        __syncthreads();
        n = count;
        const uint32_t some = n < kList ? n : kList;
        for (uint32_t i = tid; i < some; i += NT) {
            const Best v = list[i];
            uint32_t r = 0;
            for (uint32_t j = 0; j < some; ++j) r += better(list[j].key, list[j].place, v.key, v.place);
            if (n > kList) {
                if (r == g.n_out - 1) {          // more than fit: another round from the n_out-th of those that did on
                    edge_key = v.key;
                    edge_place = v.place;
                }
            } else if (r < g.n_out) {
                const uint64_t to = (uint64_t)blockIdx.x * g.n_out + r;
                const uint32_t b = (uint32_t)(v.place >> 32), t = (uint32_t)v.place;
                g.out_scores[to] = (float)v.total;
                g.parents[to] = (int32_t)b;
                g.tokens[to] = (int32_t)t;
                g.out_finished[to] = kind[b] == 2 || (g.end >= 0 && t == (uint32_t)g.end);
            }
        }
        __syncthreads();
        if (n <= kList || round > all / 512) break;          // (each round leaves out kList - n_out at least)
        ek = edge_key;
        ep = edge_place;
        if (tid == 0) count = 0;
        __syncthreads();
    }
    for (uint32_t i = n + tid; i < g.n_out; i += NT) {
        const uint64_t to = (uint64_t)blockIdx.x * g.n_out + i;
        g.out_scores[to] = -kInf;
        g.parents[to] = -1;
        g.tokens[to] = -1;
        g.out_finished[to] = 0;
    }
}

// Logits a lane holds: as many as leave the card about 1024 waves, up to 64 (32 in 32 bits: the same bytes).
inline uint32_t lane_logits(int type, uint64_t rows, uint32_t vocab)
{
    uint32_t e = type == F32 ? 32 : 64;
    while (e > 8 && rows * ((vocab + 64ull * e - 1) / (64ull * e)) < 1024) e >>= 1;
    return e;
}

template <int TY>
void launch_parts(const BeamArgs &g, uint32_t e, uint32_t wgs, hipStream_t stream)
{
    if (e == 8) hipLaunchKernelGGL((k_beam_parts<TY, 8>), dim3(wgs), dim3(256), 0, stream, g);
    else if (e == 16) hipLaunchKernelGGL((k_beam_parts<TY, 16>), dim3(wgs), dim3(256), 0, stream, g);
    else if (e == 32) hipLaunchKernelGGL((k_beam_parts<TY, 32>), dim3(wgs), dim3(256), 0, stream, g);
    else if constexpr (TY != F32) hipLaunchKernelGGL((k_beam_parts<TY, 64>), dim3(wgs), dim3(256), 0, stream, g);
}

// ZX_OK, and how the rows are split, where the sizes can be served.
inline zx_status plan(int type, uint32_t groups, uint32_t beams, uint32_t vocab, uint32_t n_out, uint32_t &e, uint32_t &parts)
{
    if (type != ZX_LOGITS_BF16 && type != ZX_LOGITS_F16 && type != ZX_LOGITS_F32) return ZX_E_UNSUPPORTED;
    if (beams == 0 || beams > kMostBeams || n_out == 0 || n_out > kMostOut || vocab == 0) return ZX_E_INVAL;
    if (vocab > kMostVocab) return ZX_E_LIMIT;
    const uint64_t rows = (uint64_t)groups * beams;
    e = lane_logits(type, rows, vocab);
    parts = (uint32_t)((vocab + 64ull * e - 1) / (64ull * e));
    // a launch counts its threads in 32 bits
    if (rows > 0x7FFFFFFFull || rows * parts > (1ull << 26) - 4) return ZX_E_LIMIT;
    return ZX_OK;
}

}  // namespace zxb

static_assert(zxb::BF16 == ZX_LOGITS_BF16 && zxb::F16 == ZX_LOGITS_F16 && zxb::F32 == ZX_LOGITS_F32, "logit types");

extern "C" size_t zx_beam_select_workspace_bytes(int32_t type, uint32_t n_groups, uint32_t beams, uint32_t vocab, uint32_t n_out)
{
    uint32_t e, parts;
    if (zxb::plan(type, n_groups, beams, vocab, n_out, e, parts) != ZX_OK) return 0;
    return (size_t)n_groups * beams * parts * (sizeof(zxb::Stat) + n_out * sizeof(zxb::Cand));
}

extern "C" zx_status zx_beam_select(const zx_beam_logits *in, const float *scores, const float *weights, const uint8_t *finished,
                                    int32_t end, const uint32_t *allowed, double scale, uint32_t n_out, float *out_scores,
                                    int32_t *parents, int32_t *tokens, uint8_t *out_finished, void *workspace, size_t ws_bytes,
                                    uint32_t *err, hipStream_t stream)
{
    using namespace zxb;
    if (!in) return ZX_E_INVAL;
    uint32_t e, parts;
    const zx_status st = plan(in->type, in->n_groups, in->beams, in->vocab, n_out, e, parts);
    if (st != ZX_OK) return st;
    if (in->n_groups == 0) return ZX_OK;
    const uintptr_t width = in->type == ZX_LOGITS_F32 ? 4 : 2;
    if (!in->logits || (uintptr_t)in->logits % width || !scores || !out_scores || !parents || !tokens || !out_finished) return ZX_E_INVAL;
    if (!(scale > 0.0) || !(scale <= 1e30) || end < -1 || (end >= 0 && (uint32_t)end >= in->vocab) || (finished && end < 0)) return ZX_E_INVAL;
    if (in->group_stride > (1ull << 40) || in->beam_stride > (1ull << 40)) return ZX_E_INVAL;
    const uint64_t rows = (uint64_t)in->n_groups * in->beams;
    if (!workspace || ((uintptr_t)workspace & 15u) || ws_bytes < zx_beam_select_workspace_bytes(in->type, in->n_groups, in->beams, in->vocab, n_out))
        return ZX_E_INVAL;
    BeamArgs g{};
    g.logits = in->logits;
    g.group_stride = (int64_t)in->group_stride;
    g.beam_stride = (int64_t)in->beam_stride;
    g.scores = scores;
    g.weights = weights;
    g.finished = finished;
    g.allowed = allowed;
    g.stat = static_cast<Stat *>(workspace);
    g.cand = reinterpret_cast<Cand *>(g.stat + rows * parts);
    g.out_scores = out_scores;
    g.parents = parents;
    g.tokens = tokens;
    g.out_finished = out_finished;
    g.err = err;
    g.scale = scale;
    g.groups = in->n_groups;
    g.beams = in->beams;
    g.vocab = in->vocab;
    g.n_out = n_out;
    g.parts = parts;
    g.words = (in->vocab + 31) / 32;
    g.end = end;
    const uint32_t wgs = (uint32_t)((rows * parts + 3) / 4);
    if (in->type == ZX_LOGITS_BF16) launch_parts<BF16>(g, e, wgs, stream);
    else if (in->type == ZX_LOGITS_F16) launch_parts<F16>(g, e, wgs, stream);
    else launch_parts<F32>(g, e, wgs, stream);
    if ((uint64_t)in->beams * parts * n_out > 4096) hipLaunchKernelGGL((k_beam_pick<1024>), dim3(in->n_groups), dim3(1024), 0, stream, g);
    else hipLaunchKernelGGL((k_beam_pick<256>), dim3(in->n_groups), dim3(256), 0, stream, g);
    return hipGetLastError() == hipSuccess ? ZX_OK : ZX_E_HIP;
}
