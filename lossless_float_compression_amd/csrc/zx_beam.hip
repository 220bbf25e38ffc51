// zx_beam.hip -- the choice of the next beams from the logits.
//
// With lse_b = ln sum_t exp(s x_bt) over the tokens that beam b may take, candidate (b, t) has the total
// score_b + s x_bt - lse_b, and the n_out candidates of a group with the largest weight_b * total are taken.
//
// Bound by reading the logits once.  k_beam_parts streams a part of a row: each thread keeps its running maximum and its sum of
// exponentials relative to that, and the maxima of its shares of the part's tiles.  The n_out largest logits of the part are found
// without sorting it: the n_out-th largest of the threads' maxima is no larger than the n_out-th largest logit,
// so only logits from there on can be among them, and hardly more than n_out are; the few tiles' shares that hold them are read again
// (from L2) and the logits ranked by counting.  k_beam_pick: one workgroup a group joins the parts' sums, turns the parts' candidates into totals and
// finds the n_out best of them the same way.
//
// 64 x 8 of 128256, BF16, 16 out, a seventh of the beams finished: 28 + 6 us, 3.9 TB/s of the 111 MB that it needs (119 MB are read: the first
// tile of a part is under way before its row's score and flag can leave it out; without what follows the last tile 27, with no exponentials 27); 256 x 8: 98 us, 5.4 TB/s; in 32 bits 179 us, 5.9 TB/s.  1 x 4 of 32000: 5.3 + 4.6.
// Tried, in us of k_beam_parts for 64 x 8: a part of 4096 logits held in registers by each wave, which ranks its own 75, then 34 with the maxima of
// pieces kept and cheaper ranking, 33 with parts of a workgroup (every part pays for its edge and ranking); the next two tiles under way
// 30.9, tiles of half the size 30.0.
//
// Many equal logits at the edge do not fit the list of 256 that are ranked; then the part is read again from a sharper edge on (all logits
// equal, whole calls: 64 x 8 of 128256 330 us, 1 x 4 of 32000 42).
//
// Rounding: exponentials are taken and summed in 32 bits by a thread (up to 256 logits, 128 in 32 bits, in four sums) and summed in 64 bits from there
// on; totals are formed and compared in 64 bits, which adds nothing to the sums' error.  That error (below 1e-5 of a score, 3e-8 measured) is one for all of
// a beam's candidates: their order is exact, and only beams closer than it may change places.
#include "zx_common.h"

namespace zxb {

using zxk::report;

typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef u4 u4_anywhere __attribute__((aligned(2)));  // 16 bytes that begin at any logit

constexpr float kInf = __builtin_huge_valf();
constexpr float kLowest = -3.4028234663852886e38f;
constexpr uint32_t kMostOut = 64, kMostBeams = 64;
constexpr uint32_t kMostVocab = 1u << 24;
// The scale times log2 e has to be a normal number in 32 bits (zero times -inf is NaN), and where a difference of two logits passes 32 bits
// (3.4e38; it is -inf then) its exponential has to be nothing: e^-340 here.
constexpr double kLeastScale = 1e-36;

enum { BF16, F16, F32 };

struct Stat {
    float top;                       // a wave's largest logit (-inf: none may be taken)
    uint32_t unused;
    double sum;                      // of exp(s (x - top)) over its logits
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
    Stat *stat;                                  // [row][part][wave]
    Cand *cand;                                  // [row][part][n_out], the largest first
    float *out_scores;
    int32_t *parents, *tokens;
    uint8_t *out_finished;
    uint32_t *err;
    double scale;
    uint32_t groups, beams, vocab, n_out, parts, words;
    uint32_t tiles;                              // of a part
    uint32_t depth;                              // candidates of a part that the join looks at first
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

template <class F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t x, F f)
{
    // within rows of 16 lanes by rotations, then across them
#define ROTATE(n) x = f(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x120 + n, 0xF, 0xF, true))
    ROTATE(8);
    ROTATE(4);
    ROTATE(2);
    ROTATE(1);
#undef ROTATE
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    const uint32_t y = f((uint32_t)r[0], (uint32_t)r[1]);
    const auto s = __builtin_amdgcn_permlane32_swap(y, y, false, false);
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)f((uint32_t)s[0], (uint32_t)s[1]));
}

constexpr int kLevels = 4;
template <int NT>
struct EdgeRoom {
    uint32_t low[NT / 64], high[NT / 64], keys[NT / 64], bins[kLevels][256];
};

// A value that n at least of the workgroup's keys reach (0 is no key), and few more: 1 where there are fewer than n keys.  From the
// first bit in which any two keys differ on, eight bits at a time are counted, and what follows the bin that
// the n-th largest key lies in is looked at only if that bin holds many.
template <int NT>
__device__ __forceinline__ uint32_t block_edge(uint32_t key, uint32_t n, EdgeRoom<NT> &m)
{
    const uint32_t tid = threadIdx.x, lane = tid & 63u;
    const uint32_t wl = wave_reduce(key ? key : 0xFFFFFFFFu, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
    const uint32_t wh = wave_reduce(key, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
    const uint64_t some_keys = __ballot(key != 0);
    if (lane == 0) {
        m.keys[tid >> 6] = (uint32_t)__popcll(some_keys);
        m.low[tid >> 6] = wl;
        m.high[tid >> 6] = wh;
    }
    for (uint32_t i = tid; i < kLevels * 256; i += NT) (&m.bins[0][0])[i] = 0;
    __syncthreads();
    uint32_t low = m.low[0], high = m.high[0], keys = m.keys[0];
#pragma unroll
    for (int i = 1; i < NT / 64; ++i) {
        keys += m.keys[i];
        low = m.low[i] < low ? m.low[i] : low;
        high = m.high[i] > high ? m.high[i] : high;
    }
    if (keys < n) return 1u;
    if (low == high) return high;
    uint32_t width = 32u - (uint32_t)__builtin_clz(low ^ high);      // bits below what all keys share
    uint32_t base = low & ~(uint32_t)((1ull << width) - 1ull);
    for (int level = 0;; ++level) {
        const uint32_t shift = width > 8 ? width - 8 : 0;
        const bool in = key >= base && (uint64_t)(key - base) >> width == 0 && key;
        const uint32_t bin = (key - base) >> shift;
        if (in && bin) atomicAdd(&m.bins[level][bin], 1u);   // (bin 0 is what is left)
        __syncthreads();
        uint32_t c[4], all;
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = m.bins[level][4 * lane + i];
        const uint32_t ahead = zxk::wave_excl_scan(c[0] + c[1] + c[2] + c[3], all);
        uint32_t from = all - ahead;             // keys in the lane's bins and higher ones
        int mine = -1;
        uint32_t reach = 0, above = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (from >= n) {
                mine = i;
                reach = from;
                above = from - c[i];
            }
            from -= c[i];
        }
        const uint64_t some = __ballot(mine >= 0);
        if (some) {
            const int l = 63 - __builtin_clzll(some);
            const uint32_t nth = 4u * (uint32_t)l + (uint32_t)__builtin_amdgcn_readlane(mine, l);
            reach = (uint32_t)__builtin_amdgcn_readlane((int)reach, l);
            above = (uint32_t)__builtin_amdgcn_readlane((int)above, l);
            base += nth << shift;
            // (bin 0 has not been counted)
            if (nth && reach <= n + n / 2 + 4) return base;
        } else {
            above = all;
        }
        if (shift == 0 || level + 1 == kLevels) return base ? base : 1u;
        n -= above < n ? above : n - 1;
        width = shift;
    }
}

template <int TY>
struct Type {
    static constexpr int N = TY == F32 ? 4 : 8;  // logits of 16 bytes
    static constexpr int W = TY == F32 ? 4 : 2;  // bytes of one
    static constexpr uint32_t LOW = TY == F32 ? 0xFF800000u : TY == BF16 ? 0xFF80u : 0xFC00u;    // -inf
};

template <int TY>
__device__ __forceinline__ void unpack(u4 w, float (&x)[Type<TY>::N])
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

// Which of a row's tokens t .. t + N - 1 are there (bit i for t + i).
__device__ __forceinline__ uint32_t there(uint32_t t, uint32_t n, uint32_t vocab)
{
    return t >= vocab ? 0u : t + n <= vocab ? 0xFFFFFFFFu : (1u << (vocab - t)) - 1u;
}
// The logits of these tokens: at the row's end the row's last 16 bytes, which `settle` moves to their places (a row shorter than that
// is read there, one by one); it makes those that are not in `bits` -inf.
template <int TY>
__device__ __forceinline__ u4 fetch(const uint8_t *row, uint32_t t, uint32_t vocab)
{
    constexpr uint32_t N = Type<TY>::N, W = Type<TY>::W;
    u4 r{0, 0, 0, 0};
    // (a row is read once: past the caches 256 x 8 of 128256 98 us, through them 105)
    if (vocab >= N) r = __builtin_nontemporal_load(reinterpret_cast<const u4_anywhere *>(row + (uint64_t)(t + N <= vocab ? t : vocab - N) * W));
    return r;
}
template <int TY>
__device__ __forceinline__ u4 settle(u4 r, const uint8_t *row, uint32_t t, uint32_t vocab, uint32_t bits)
{
    constexpr uint32_t N = Type<TY>::N, W = Type<TY>::W;
    if (t + N > vocab && t < vocab) {
        unsigned __int128 x = __builtin_bit_cast(unsigned __int128, r);
        if (vocab >= N) {
            x >>= (t + N - vocab) * W * 8;
        } else {
#pragma unroll 1
            for (uint32_t i = 0; i < vocab - t; ++i) {
                uint32_t one = 0;
                __builtin_memcpy(&one, row + (uint64_t)(t + i) * W, W);
                x |= (unsigned __int128)one << (i * W * 8);
            }
        }
        r = __builtin_bit_cast(u4, x);
    }
    if (bits != 0xFFFFFFFFu) {
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            if constexpr (W == 4) {
                if (!(bits >> i & 1u)) r[i] = Type<TY>::LOW;
            } else {
                if (!(bits >> (2 * i) & 1u)) r[i] = (r[i] & 0xFFFF0000u) | Type<TY>::LOW;
                if (!(bits >> (2 * i + 1) & 1u)) r[i] = (r[i] & 0xFFFFu) | Type<TY>::LOW << 16;
            }
        }
    }
    return r;
}

__device__ __forceinline__ float wave_max(float x)
{
    return __builtin_bit_cast(float, wave_reduce(__builtin_bit_cast(uint32_t, x), [](uint32_t a, uint32_t b) {
        return __builtin_bit_cast(uint32_t, fmaxf(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)));
    }));
}
__device__ __forceinline__ double wave_sum(double x)
{
    auto with = [](double a, uint32_t lo, uint32_t hi) { return a + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo); };
#define HALVES const uint64_t q = __builtin_bit_cast(uint64_t, x); const uint32_t lo = (uint32_t)q, hi = (uint32_t)(q >> 32)
#define ROTATE(n) \
    do { \
        HALVES; \
        x = with(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)lo, 0x120 + n, 0xF, 0xF, true), \
                 (uint32_t)__builtin_amdgcn_update_dpp(0, (int)hi, 0x120 + n, 0xF, 0xF, true)); \
    } while (0)
    ROTATE(8);
    ROTATE(4);
    ROTATE(2);
    ROTATE(1);
#undef ROTATE
    {
        HALVES;
        const auto a = __builtin_amdgcn_permlane16_swap(lo, lo, false, false), b = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
        x = with(__builtin_bit_cast(double, (uint64_t)(uint32_t)b[0] << 32 | (uint32_t)a[0]), (uint32_t)a[1], (uint32_t)b[1]);
    }
    {
        HALVES;
        const auto a = __builtin_amdgcn_permlane32_swap(lo, lo, false, false), b = __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
        x = with(__builtin_bit_cast(double, (uint64_t)(uint32_t)b[0] << 32 | (uint32_t)a[0]), (uint32_t)a[1], (uint32_t)b[1]);
    }
#undef HALVES
    return x;
}

constexpr uint32_t kThreads = 256, kWaves = kThreads / 64;
constexpr uint32_t kMostTiles = 8;               // of a part
constexpr uint32_t kRoom = 256;                  // logits of a part that are ranked at a time
constexpr uint32_t kHits = 256;                  // threads' shares of tiles with a logit that may be among the largest

// Keys that order by logit, then by place within the part, the earlier first; minus zero is no smaller than zero.
template <int TY>
struct Key {                                     // of 16-bit logits: the logit's bits in order, and 16 bits of place
    typedef uint32_t T;
    static __device__ __forceinline__ T of(float x, uint32_t place)
    {
        uint32_t h;
        if constexpr (TY == BF16) h = __builtin_bit_cast(uint32_t, x + 0.0f) >> 16;
        else h = __builtin_bit_cast(uint16_t, (_Float16)(x + 0.0f));
        return (h ^ (h & 0x8000u ? 0xFFFFu : 0x8000u)) << 16 | (0xFFFFu - place);
    }
    static __device__ __forceinline__ Cand cand(T k, uint32_t token0)
    {
        const uint32_t o = k >> 16, h = o ^ (o & 0x8000u ? 0x8000u : 0xFFFFu);
        if constexpr (TY == BF16) return Cand{__builtin_bit_cast(float, h << 16), token0 + (0xFFFFu - (k & 0xFFFFu))};
        else return Cand{(float)__builtin_bit_cast(_Float16, (uint16_t)h), token0 + (0xFFFFu - (k & 0xFFFFu))};
    }
};
template <>
struct Key<F32> {
    typedef uint64_t T;
    static __device__ __forceinline__ T of(float x, uint32_t place) { return (uint64_t)ordered(x + 0.0f) << 32 | (0xFFFFFFFFu - place); }
    static __device__ __forceinline__ Cand cand(T k, uint32_t token0) { return Cand{unordered((uint32_t)(k >> 32)), token0 + (0xFFFFFFFFu - (uint32_t)k)}; }
};

// One workgroup a part of up to eight tiles; of a tile a thread has TP pieces of 16 bytes, read while the tile before is worked on.
template <int TY, int TP, bool MASK>
__global__ __launch_bounds__(kThreads) void k_beam_parts(BeamArgs g)
{
    constexpr uint32_t N = Type<TY>::N, W = Type<TY>::W, kPiece = kThreads * N, kTile = TP * kPiece;
    static_assert(kMostTiles * kTile <= 65536, "places fit 16 bits");
    typedef typename Key<TY>::T K;
    __shared__ float tile_top[kMostTiles][kThreads];
    __shared__ K room[kRoom];
    __shared__ uint32_t hits[kHits], n_hits, n_room;
    __shared__ EdgeRoom<kThreads> edges;
    __shared__ K edge_key;
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
    const uint32_t row = blockIdx.x / g.parts, part = blockIdx.x - row * g.parts;
    const uint8_t *p = static_cast<const uint8_t *>(g.logits) +
                       ((int64_t)(row / g.beams) * g.group_stride + (int64_t)(row % g.beams) * g.beam_stride) * W;
    const uint32_t *allowed = MASK ? g.allowed + (uint64_t)row * g.words : nullptr;
    const uint32_t token0 = part * g.tiles * kTile, left = g.vocab - token0;
    const uint32_t n_tiles = left > g.tiles * kTile ? g.tiles : (left + kTile - 1) / kTile;
    if (tid == 0) n_hits = n_room = 0;

    // a thread's maximum so far and its sum of exponentials relative to that
    float top = -kInf, sum = 0.0f;
    const float c = (float)(g.scale * 1.4426950408889634);
    struct Buffer {
        u4 raw[TP];
        uint32_t bits[TP];
    };
    auto load = [&](uint32_t tile, Buffer &f) {
#pragma unroll
        for (int u = 0; u < TP; ++u) {
            const uint32_t t = token0 + tile * kTile + u * kPiece + tid * N;
            f.raw[u] = fetch<TY>(p, t, g.vocab);
            if (MASK) f.bits[u] = t < g.vocab ? allowed[t >> 5] >> (t & 31u) | ~((1u << N) - 1u) : 0;
        }
    };
    auto work = [&](uint32_t tile, Buffer &f) {
        if (MASK || left < (tile + 1) * kTile) {
#pragma unroll
            for (int u = 0; u < TP; ++u) {
                const uint32_t t = token0 + tile * kTile + u * kPiece + tid * N;
                f.raw[u] = settle<TY>(f.raw[u], p, t, g.vocab, there(t, N, g.vocab) & (MASK ? f.bits[u] : 0xFFFFFFFFu));
            }
        }
        float x[TP][N], best = -kInf;            // (NaN is left out of the maximum; it shows in the sum)
#pragma unroll
        for (int u = 0; u < TP; ++u) {
            unpack<TY>(f.raw[u], x[u]);
#pragma unroll
            for (uint32_t i = 0; i < N; ++i) best = fmaxf(best, x[u][i]);
        }
        tile_top[tile][tid] = best;
        const float now = fmaxf(top, best), from = now == -kInf ? 0.0f : now;
        float s[4] = {sum * __builtin_amdgcn_exp2f((top - from) * c), 0, 0, 0};
        top = now;
#pragma unroll
        for (int u = 0; u < TP; ++u)
#pragma unroll
            for (uint32_t i = 0; i < N; ++i) s[i & 3] += __builtin_amdgcn_exp2f((x[u][i] - from) * c);
        sum = (s[0] + s[1]) + (s[2] + s[3]);
    };
    Buffer a, b;
    load(0, a);                                  // beside the score and the flag that say whether the row is needed
    if (!row_runs(g, row)) return;
    for (uint32_t tile = 0; tile < n_tiles; tile += 2) {
        if (tile + 1 < n_tiles) load(tile + 1, b);
        work(tile, a);
        if (tile + 1 >= n_tiles) break;
        if (tile + 2 < n_tiles) load(tile + 2, a);
        work(tile + 1, b);
    }
    const float all = wave_max(top), from = all == -kInf ? 0.0f : all;
    const double total = wave_sum((double)(sum * __builtin_amdgcn_exp2f((top - from) * c)));
    if (lane == 0) {
        Stat &o = g.stat[(uint64_t)blockIdx.x * kWaves + wave];
        o.top = all;
        o.sum = total;
    }
    // n_out threads' maxima at least reach the edge, or all that there are; hardly more logits do
    const float edge = fmaxf(unordered(block_edge(top > -kInf ? ordered(top) : 0u, g.n_out, edges)), kLowest);
    auto take = [&](const float (&y)[N], uint32_t place, K ek) {     // a piece's logits from the edge on, with keys from ek on
        uint32_t yes = 0;
#pragma unroll
        for (uint32_t i = 0; i < N; ++i) yes |= (uint32_t)(y[i] >= edge && (ek == 0 || Key<TY>::of(y[i], place + i) >= ek)) << i;
        if (!yes) return;
        uint32_t to = atomicAdd(&n_room, (uint32_t)__builtin_popcount(yes));
#pragma unroll
        for (uint32_t i = 0; i < N; ++i)
            if (yes >> i & 1u) {
                if (to < kRoom) room[to] = Key<TY>::of(y[i], place + i);
                ++to;
            }
    };
    if (g.tiles == 1) {                          // all logits are at hand
        if (top >= edge) {
#pragma unroll
            for (int u = 0; u < TP; ++u) {
                float y[N];
                unpack<TY>(a.raw[u], y);
                take(y, u * kPiece + tid * N, 0);
            }
        }
    } else if (top >= edge) {
        // the threads and tiles that reach it, then their logits that do, read once more
        for (uint32_t i = 0; i < n_tiles; ++i) {
            if (tile_top[i][tid] < edge) continue;
            const uint32_t to = atomicAdd(&n_hits, 1u);
            if (to < kHits) hits[to] = i << 8 | tid;
        }
    }
    __syncthreads();
    const uint32_t v = n_hits;
    auto sift = [&](uint32_t place, K ek) {
        const uint32_t t = token0 + place;
        float y[N];
        uint32_t bits = there(t, N, g.vocab);
        if (MASK && t < g.vocab) bits &= allowed[t >> 5] >> (t & 31u) | ~((1u << N) - 1u);
        unpack<TY>(settle<TY>(fetch<TY>(p, t, g.vocab), p, t, g.vocab, bits), y);
        take(y, place, ek);
    };
    if (g.tiles > 1 && v <= kHits) {
        for (uint32_t i = tid; i < v * TP; i += kThreads) {
            const uint32_t h = hits[i / TP];
            sift((h >> 8) * kTile + (i % TP) * kPiece + (h & 255u) * N, 0);
        }
        __syncthreads();
    }
    uint32_t n = n_room;
    auto rank = [&](uint32_t some) {
        const K k = room[tid < some ? tid : 0];
        uint32_t r = 0;
#pragma unroll 8
        for (uint32_t j = 0; j < some; ++j) r += room[j] > k;
        return r;
    };
    if (v > kHits || n > kRoom) {
        // more than there is room for, as many equal logits are: the n_out-th of those that fit is a sharper edge, which
        // leaves out kRoom - n_out of them at least, so the rounds end
        K ek = 0;
        for (;;) {
            __syncthreads();
            if (tid == 0) n_room = 0;
            __syncthreads();
            for (uint32_t i = 0; i < n_tiles * TP; ++i) sift(i * kPiece + tid * N, ek);
            __syncthreads();
            n = n_room;
            if (n <= kRoom) break;
            if (rank(kRoom) == g.n_out - 1) edge_key = room[tid];
            __syncthreads();
            ek = edge_key;
        }
    }
    Cand *o = g.cand + (uint64_t)blockIdx.x * g.n_out;
    if (tid < n) {
        const uint32_t r = rank(n);
        if (r < g.n_out) o[r] = Key<TY>::cand(room[tid], token0);
    } else if (tid < g.n_out) {
        o[tid] = Cand{-kInf, 0};
    }
}

struct Best {
    uint64_t key;                                // orders like weight * total
    uint64_t place;                              // place_of
    double total;
};
constexpr uint32_t kList = 1024;

// The order among equal totals: the earlier beam, then the larger logit (in 64 bits the totals of unlike ones may be equal), then the earlier token.
// So a part's candidates, which are sorted by logit and token, are in this order too: whatever reaches an edge, all ahead of it do.
constexpr uint32_t kTokenBits = 24, kBeamShift = 32 + kTokenBits;
static_assert(kMostVocab <= 1u << kTokenBits && kMostBeams <= 1u << (64 - kBeamShift), "places fit 64 bits");
__device__ __forceinline__ uint64_t place_of(uint32_t beam, float x, uint32_t token)
{
    return (uint64_t)beam << kBeamShift | (uint64_t)(0xFFFFFFFFu - ordered(x)) << kTokenBits | token;
}

__device__ __forceinline__ bool better(uint64_t ka, uint64_t pa, uint64_t kb, uint64_t pb) { return ka > kb || (ka == kb && pa < pb); }

template <int NT>
__global__ __launch_bounds__(NT) void k_beam_pick(BeamArgs g)
{
    __shared__ Best list[kList];
    __shared__ double base[kMostBeams], tops[kMostBeams], weight[kMostBeams];
    __shared__ uint32_t kind[kMostBeams];        // 0: no candidates, 1: the parts', 2: finished
    __shared__ uint32_t count, few, survivors[kList];
    __shared__ EdgeRoom<NT> edges;
    __shared__ uint64_t edge_key, edge_place;
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
    const uint32_t row0 = blockIdx.x * g.beams;
    // the parts' candidates are sorted: an edge is found among the first `depth` of each, and a part's further ones are
    // looked at only while they reach it
    const uint32_t lists = g.beams * g.parts, entries = lists * g.depth;
    const Cand *cand = g.cand + (uint64_t)row0 * g.parts * g.n_out;
    Cand mine{-kInf, 0};                         // under way while the sums are joined (rows that are not needed hold anything)
    if (tid < entries) mine = cand[(uint64_t)(tid / g.depth) * g.n_out + tid % g.depth];
    for (uint32_t b = wave; b < g.beams; b += NT / 64) {
        const uint32_t row = row0 + b, stats = g.parts * kWaves;
        const Stat *stat = g.stat + (uint64_t)row * stats;
        Stat v{-kInf, 0, 0.0};
        if (lane < stats) v = stat[lane];
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
                top = v.top;
                for (uint32_t i = lane + 64; i < stats; i += 64) top = fmaxf(top, stat[i].top);
                top = wave_max(top);
                double s = 0.0;
                for (uint32_t i = lane; i < stats; i += 64) {
                    if (i >= 64) v = stat[i];
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
    if (tid == 0) count = 0;
    __syncthreads();
    auto value = [&](uint32_t list, Cand v, Best &o) {
        const uint32_t b = list / g.parts;
        if (kind[b] != 1 || v.x == -kInf) return false;
        o.total = base[b] + ((double)v.x - tops[b]) * g.scale;       // (score - ln sum) + s (x - top): no large logit swallows the rest
        o.place = place_of(b, v.x, v.token);
        o.key = ordered(o.total * weight[b] + 0.0);
        return true;
    };
    auto entry = [&](uint32_t list, uint32_t nth, Best &o) { return value(list, cand[(uint64_t)list * g.n_out + nth], o); };
    Best own;
    const bool have = tid < entries && value(tid / g.depth, mine, own);
    uint64_t key = have ? own.key : 0;
    for (uint32_t e = tid + NT; e < entries; e += NT) {
        Best v;
        if (entry(e / g.depth, e % g.depth, v) && v.key > key) key = v.key;
    }
    // n_out threads' keys at least reach the edge, or all that there are
    uint64_t ek = (uint64_t)block_edge((uint32_t)(key >> 32), g.n_out, edges) << 32, ep = ~0ull;
    uint32_t n;
    for (uint32_t round = 0;; ++round) {
        auto enter = [&](const Best &v) {
            if (better(ek, ep, v.key, v.place)) return false;
            const uint32_t to = atomicAdd(&count, 1u);
            if (to < kList) list[to] = v;
            return true;
        };
        for (uint32_t e = tid; e < entries; e += NT) {
            const uint32_t l = e / g.depth, nth = e % g.depth;
            Best v = own;
            if (!(e == tid ? have : entry(l, nth, v)) || !enter(v) || nth + 1 < g.depth) continue;
            // eight further ones under way at once
            for (uint32_t i = g.depth; i < g.n_out; i += 8) {
                Cand more[8];
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) more[j] = cand[(uint64_t)l * g.n_out + (i + j < g.n_out ? i + j : g.n_out - 1)];
                bool on = true;
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) on = on && i + j < g.n_out && value(l, more[j], v) && enter(v);
                if (!on) break;
            }
        }
        if (tid < g.beams && kind[tid] == 2) {   // finished: one candidate
            Best v;
            v.total = base[tid];
            v.place = place_of(tid, 0.0f, (uint32_t)g.end);
            v.key = ordered(v.total * weight[tid] + 0.0);
            enter(v);
        }
        __syncthreads();
        n = count;
        const uint32_t some = n < kList ? n : kList;
        auto rank_of = [&](const Best &v, uint32_t of, auto at) {
            uint32_t r = 0;
#pragma unroll 8
            for (uint32_t j = 0; j < of; ++j) {
                const Best &o = list[at(j)];
                r += better(o.key, o.place, v.key, v.place);
            }
            return r;
        };
        auto put = [&](const Best &v, uint32_t r) {
            if (r >= g.n_out) return;
            const uint64_t to = (uint64_t)blockIdx.x * g.n_out + r;
            const uint32_t b = (uint32_t)(v.place >> kBeamShift), t = (uint32_t)v.place & ((1u << kTokenBits) - 1u);
            g.out_scores[to] = (float)v.total;
            g.parents[to] = (int32_t)b;
            g.tokens[to] = (int32_t)t;
            g.out_finished[to] = kind[b] == 2 || (g.end >= 0 && t == (uint32_t)g.end);
        };
        if (n > kList) {
            // more than fit: another round from the n_out-th of those that did on
            for (uint32_t i = tid; i < some; i += NT)
                if (rank_of(list[i], some, [](uint32_t j) { return j; }) == g.n_out - 1) {
                    edge_key = list[i].key;
                    edge_place = list[i].place;
                }
        } else if (n <= 2 * g.n_out + 64) {
            for (uint32_t i = tid; i < n; i += NT) put(list[i], rank_of(list[i], n, [](uint32_t j) { return j; }));
        } else {
            // many: an edge among them first
            uint32_t top = 0;
            for (uint32_t i = tid; i < n; i += NT) {
                const uint32_t k = (uint32_t)(list[i].key >> 32);
                top = k > top ? k : top;
            }
            if (tid == 0) few = 0;
            const uint32_t e = block_edge(top, g.n_out, edges);
            for (uint32_t i = tid; i < n; i += NT)
                if ((uint32_t)(list[i].key >> 32) >= e) survivors[atomicAdd(&few, 1u)] = i;
            __syncthreads();
            const uint32_t left = few;
            for (uint32_t i = tid; i < left; i += NT) {
                const Best &v = list[survivors[i]];
                put(v, rank_of(v, left, [&](uint32_t j) { return survivors[j]; }));
            }
        }
        __syncthreads();
        if (n <= kList || round > lists) break;          // (each round leaves out kList - n_out at least)
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

template <int TY, bool MASK>
void launch_parts(const BeamArgs &g, uint32_t pieces, uint32_t wgs, hipStream_t stream)
{
    if (pieces == 1) hipLaunchKernelGGL((k_beam_parts<TY, 1, MASK>), dim3(wgs), dim3(kThreads), 0, stream, g);
    else hipLaunchKernelGGL((k_beam_parts<TY, 4, MASK>), dim3(wgs), dim3(kThreads), 0, stream, g);
}
template <int TY>
void launch_parts(const BeamArgs &g, uint32_t pieces, uint32_t wgs, hipStream_t stream)
{
    if (g.allowed) launch_parts<TY, true>(g, pieces, wgs, stream);
    else launch_parts<TY, false>(g, pieces, wgs, stream);
}

// How rows are split.
struct Split {
    uint32_t pieces, tiles, parts;               // pieces of a tile a thread, tiles of a part, parts of a row
};

// ZX_OK and the split, where the sizes can be served.
inline zx_status plan(int type, uint32_t groups, uint32_t beams, uint32_t vocab, uint32_t n_out, Split &o)
{
    if (type != ZX_LOGITS_BF16 && type != ZX_LOGITS_F16 && type != ZX_LOGITS_F32) return ZX_E_UNSUPPORTED;
    if (beams == 0 || beams > kMostBeams || n_out == 0 || n_out > kMostOut || vocab == 0) return ZX_E_INVAL;
    if (vocab > kMostVocab) return ZX_E_LIMIT;
    const uint64_t rows = (uint64_t)groups * beams;
    const uint32_t piece = kThreads * (type == F32 ? 4 : 8);
    auto up = [](uint64_t a, uint64_t b) { return (a + b - 1) / b; };
    // tiles of four pieces where that makes a workgroup a CU (parts of one such tile each: 7 x 5 of 50001 in 32 bits 7.2 us, of one piece 8.1);
    // parts as long as leave 1024 workgroups, four a CU (64 x 8 of 128256: 29.6 us; 1280 30.4, 2048 31.0, 4096 34.4, parts of a tile 49.7)
    o.pieces = rows * up(vocab, 4 * piece) < 256 ? 1 : 4;
    const uint64_t row_tiles = up(vocab, o.pieces * piece);
    uint64_t tiles = up(rows * row_tiles, 1024);
    if (tiles > kMostTiles) tiles = kMostTiles;
    if (tiles == 0) tiles = 1;
    o.parts = (uint32_t)up(row_tiles, tiles);
    o.tiles = (uint32_t)up(row_tiles, o.parts);
    // a launch counts its threads in 32 bits
    if (rows > 0x7FFFFFFFull || rows * o.parts >= 1ull << 24) return ZX_E_LIMIT;
    return ZX_OK;
}

}  // namespace zxb

static_assert(zxb::BF16 == ZX_LOGITS_BF16 && zxb::F16 == ZX_LOGITS_F16 && zxb::F32 == ZX_LOGITS_F32, "logit types");

extern "C" size_t zx_beam_select_workspace_bytes(int32_t type, uint32_t n_groups, uint32_t beams, uint32_t vocab, uint32_t n_out)
{
    zxb::Split sp;
    if (zxb::plan(type, n_groups, beams, vocab, n_out, sp) != ZX_OK) return 0;
    return (size_t)n_groups * beams * sp.parts * (zxb::kWaves * sizeof(zxb::Stat) + n_out * sizeof(zxb::Cand));
}

extern "C" zx_status zx_beam_select(const zx_beam_logits *in, const float *scores, const float *weights, const uint8_t *finished,
                                    int32_t end, const uint32_t *allowed, double scale, uint32_t n_out, float *out_scores,
                                    int32_t *parents, int32_t *tokens, uint8_t *out_finished, void *workspace, size_t ws_bytes,
                                    uint32_t *err, hipStream_t stream)
{
    using namespace zxb;
    if (!in) return ZX_E_INVAL;
    Split sp;
    const zx_status st = plan(in->type, in->n_groups, in->beams, in->vocab, n_out, sp);
    if (st != ZX_OK) return st;
    if (in->n_groups == 0) return ZX_OK;
    const uintptr_t width = in->type == ZX_LOGITS_F32 ? 4 : 2;
    if (!in->logits || (uintptr_t)in->logits % width || !scores || !out_scores || !parents || !tokens || !out_finished) return ZX_E_INVAL;
    if (((uintptr_t)scores | (uintptr_t)weights | (uintptr_t)allowed | (uintptr_t)out_scores | (uintptr_t)parents | (uintptr_t)tokens | (uintptr_t)err) & 3u)
        return ZX_E_INVAL;
    if (!(scale >= kLeastScale) || !(scale <= 1e30) || end < -1 || (end >= 0 && (uint32_t)end >= in->vocab) || (finished && end < 0)) return ZX_E_INVAL;
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
    g.cand = reinterpret_cast<Cand *>(g.stat + rows * sp.parts * kWaves);
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
    g.parts = sp.parts;
    g.tiles = sp.tiles;
    g.words = (in->vocab + 31) / 32;
    g.end = end;
    const uint32_t wgs = (uint32_t)(rows * sp.parts);
    if (in->type == ZX_LOGITS_BF16) launch_parts<BF16>(g, sp.pieces, wgs, stream);
    else if (in->type == ZX_LOGITS_F16) launch_parts<F16>(g, sp.pieces, wgs, stream);
    else launch_parts<F32>(g, sp.pieces, wgs, stream);
    // (more threads where there are more rows' sums to join or more candidates to look at: 64 x 8 6.1 us, with 256 threads 9.4)
    const uint32_t lists = in->beams * sp.parts, threads = lists > 512 || in->beams > 4 ? 1024 : 256;
    g.depth = lists >= threads ? 1 : threads / lists < n_out ? threads / lists : n_out;
    if (threads == 1024) hipLaunchKernelGGL((k_beam_pick<1024>), dim3(in->n_groups), dim3(1024), 0, stream, g);
    else hipLaunchKernelGGL((k_beam_pick<256>), dim3(in->n_groups), dim3(256), 0, stream, g);
    return hipGetLastError() == hipSuccess ? ZX_OK : ZX_E_HIP;
}
