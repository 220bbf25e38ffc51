// zx_paged_append.hip -- new keys and values into a paged K/V cache, with the position
// rotation on the way, and the checks that all entry points of the paged cache share.
//
// A pair (a, b) of channels of a row at place p becomes (a cos - b sin, b cos + a sin) of the angle
// p * inv_freq, times a magnitude.  Bound by the bytes: every row is read once and written once.
//
// A workgroup takes one segment of a sequence's new tokens (the tokens of one bounded
// block, or of 32 places where the cache has no bounds) and a group of eight heads: of the
// keys, of the values or of the queries.  It computes the cosines and sines of the
// segment's positions once, in LDS, and turns the rows of all its heads with them (with one
// head a workgroup the sines would cost more than the rows).  A thread holds 16 channels, eight
// rotated pairs, of two rows of keys or four of values and queries at a time, all read before
// the sines are worked out: 71 us for five prompts of up to 2900 tokens (BF16, 8 K/V and 32 query
// heads of 128 channels, 233 MB) with one role after the other, 55 us with the roles in workgroups of their own, 4.2 TB/s
// of the 5.15 TB/s of a large copy.  (More waves a SIMD spill: 63 us at five, 82 at six; 16 heads a
// workgroup 62.)  One token: 4.5 us, a launch; 256 tokens with bounds, E4M3: 10 us.
// One workgroup owns a block's bounds for its heads, so they are reduced in registers and
// LDS with no atomics and do not depend on any order.
//
// Rounding: keys and queries are turned in 32 bits and rounded once, to what is stored.  The angle is taken in
// 64 bits and its whole turns dropped there: in 32 bits a place of a million would be off by a sixteenth of a radian.
#include "zx_paged.h"

namespace zxp {

zx_status make_cache(const zx_paged_cache *c, Cache &o)
{
    if (!c) return ZX_E_INVAL;
    if (c->dtype != ZX_BF16 && c->dtype != ZX_FP8_E4M3FN) return ZX_E_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return ZX_E_INVAL;
    const uint64_t e = c->dtype == ZX_BF16 ? 2 : 1, per16 = 16 / e;
    if (!c->k || !c->v || !al16(c->k) || !al16(c->v) || c->n_pages == 0 || c->n_pages > 0x7FFFFFFFu || c->kv_heads == 0 ||
        c->kv_heads > 4096 || !pow2_in(c->page_tokens, 16, 4096))
        return ZX_E_INVAL;
    const uint64_t st[6] = {c->k_page_stride, c->k_head_stride, c->k_token_stride, c->v_page_stride, c->v_head_stride, c->v_token_stride};
    for (uint64_t s : st)
        if (s % per16 || s > (1ull << 40)) return ZX_E_INVAL;
    if (c->k_token_stride < c->head_dim || c->v_token_stride < c->head_dim || c->k_token_stride * e > (1u << 24) ||
        c->v_token_stride * e > (1u << 24))
        return ZX_E_INVAL;
    if (c->dtype == ZX_BF16 && (c->k_scale || c->v_scale)) return ZX_E_INVAL;
    if ((c->bounds == nullptr) != (c->block_tokens == 0)) return ZX_E_INVAL;
    if (c->block_tokens && (!pow2_in(c->block_tokens, 16, 256) || c->block_tokens > c->page_tokens || !al16(c->bounds)))
        return ZX_E_INVAL;
    o.k = static_cast<uint8_t *>(c->k);
    o.v = static_cast<uint8_t *>(c->v);
    o.k_page = (int64_t)(c->k_page_stride * e);
    o.k_head = (int64_t)(c->k_head_stride * e);
    o.k_token = (uint32_t)(c->k_token_stride * e);
    o.v_page = (int64_t)(c->v_page_stride * e);
    o.v_head = (int64_t)(c->v_head_stride * e);
    o.v_token = (uint32_t)(c->v_token_stride * e);
    o.k_scale = c->k_scale;
    o.v_scale = c->v_scale;
    o.bounds = reinterpret_cast<__bf16 *>(c->bounds);
    o.n_pages = c->n_pages;
    o.heads = c->kv_heads;
    o.log_page = log2_of(c->page_tokens);
    o.log_block = c->block_tokens ? log2_of(c->block_tokens) : 0;
    return ZX_OK;
}

zx_status make_batch(const zx_paged_batch *b, const zx_paged_cache *c, uint32_t n_tokens, uint32_t *err, Batch &o)
{
    if (!b || !c || n_tokens > 0x7FFFFFu || b->n_seqs > 65536) return ZX_E_INVAL;
    if (b->n_seqs && (!b->q_start || !b->kv_len || (b->table_width && !b->page_table))) return ZX_E_INVAL;
    const uint64_t room = (uint64_t)b->table_width * c->page_tokens, cap = b->max_kv < room ? b->max_kv : room;
    if (cap > 0x3FFFFFFFu) return ZX_E_INVAL;
    o.q_start = b->q_start;
    o.kv_len = b->kv_len;
    o.table = b->page_table;
    o.n_seqs = b->n_seqs;
    o.width = b->table_width;
    o.n_tokens = n_tokens;
    o.max_q = b->max_q;
    o.cap = (int32_t)cap;
    o.err = err;
    return ZX_OK;
}

zx_status make_rows(const zx_rows *r, Rows &o)
{
    if (!r || !r->p || !al16(r->p) || r->token_stride % 8 || r->head_stride % 8 || r->token_stride > (1ull << 40) ||
        r->head_stride > (1ull << 40))
        return ZX_E_INVAL;
    o.p = static_cast<__bf16 *>(r->p);
    o.token = (int64_t)r->token_stride;
    o.head = (int64_t)r->head_stride;
    return ZX_OK;
}

namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kSeg = 32;          // places of a segment where there are no bounds
constexpr uint32_t kTab = 32;          // tokens whose cosines and sines are held at a time
constexpr uint32_t kLogGroup = 3, kGroup = 1u << kLogGroup;   // heads of a workgroup

typedef int16_t i16x2 __attribute__((ext_vector_type(2)));

struct Turn {
    const double *inv_freq;
    const int32_t *positions;
    uint32_t half;                     // rotated pairs; 0: no rotation
    int32_t interleaved;
    float magnitude;
};

struct AppendArgs {
    Cache c;
    Batch b;
    Rows k, v, q, qo;
    Turn turn;
    uint32_t kv_groups, kv_log;        // K/V head groups; log2 of the heads of one (up to kLogGroup)
    uint32_t q_heads, log_seg;
};

__device__ __forceinline__ bf8 to_bf8(const float (&x)[8])
{
    bf8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (__bf16)x[i];
    return o;
}

// BF16 pairs as pairs of 16-bit integers that order like them (-0 below +0), and back.
__device__ __forceinline__ i16x2 ordered(uint32_t w)
{
    const i16x2 b = __builtin_bit_cast(i16x2, w);
    return b ^ ((b >> 15) & (int16_t)0x7FFF);
}
__device__ __forceinline__ uint16_t unordered(int16_t x) { return (uint16_t)(x ^ ((x >> 15) & 0x7FFF)); }
constexpr int16_t kTopBf16 = 0x7F80, kLowBf16 = (int16_t)~0x7F80;   // +inf and -inf in that order

// x / scale as E4M3, to the nearest, saturating at 448; NaN stays NaN.
__device__ __forceinline__ float fp8_in(float x, float scale)
{
    const float y = x / scale;
    return y != y ? y : fminf(fmaxf(y, -448.0f), 448.0f);
}

__device__ __forceinline__ u2 to_fp8(const float (&x)[8])
{
    u2 o;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        int r = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * w], x[4 * w + 1], 0, false);
        o[w] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[4 * w + 2], x[4 * w + 3], r, true);
    }
    return o;
}

__device__ __forceinline__ uint32_t bf16_pair_of_fp8(uint32_t w, bool high)
{
    const f2 x = high ? __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true) : __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const bf2 r = {(__bf16)x[0], (__bf16)x[1]};
    return __builtin_bit_cast(uint32_t, r);
}

// Store eight channels as the cache holds them; the stored values as BF16 pairs (exact).
template <int DT>
__device__ __forceinline__ u4 store8(uint8_t *row, uint32_t ch, float (&x)[8], float scale, bool yes)
{
    u4 r;
    if constexpr (DT == ZX_BF16) {
        const bf8 y = to_bf8(x);
        if (yes) *reinterpret_cast<bf8 *>(row + 2 * ch) = y;
        r = __builtin_bit_cast(u4, y);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fp8_in(x[i], scale);
        const u2 y = to_fp8(x);
        if (yes) *reinterpret_cast<u2 *>(row + ch) = y;
        r = u4{bf16_pair_of_fp8(y[0], false), bf16_pair_of_fp8(y[0], true), bf16_pair_of_fp8(y[1], false), bf16_pair_of_fp8(y[1], true)};
    }
    return r;
}

enum { KEYS, VALUES, QUERIES };

// The new tokens of one segment: places p0 .. p1 - 1 of a sequence, whose packed row of
// place p is row0 + p.
struct Segment {
    int32_t p0, p1, row0, start;     // start: first place of the segment's block
    const int32_t *table;
    bool older;                      // the block has tokens ahead of p0
};

template <int DT, int D, int ROLE>
__device__ __forceinline__ void append_rows(const AppendArgs &g, const Segment &sg, uint32_t group, float *lds)
{
    constexpr uint32_t TPR = D / 16;                    // threads of a row
    constexpr uint32_t ROWS = kThreads / TPR;           // rows at a time
    constexpr int kBatch = ROLE == KEYS ? 2 : 4;        // rows of a thread that are read together
    const uint32_t tid = threadIdx.x;
    const uint32_t log_lanes = ROLE == QUERIES ? kLogGroup : g.kv_log, lanes = 1u << log_lanes;      // lanes: heads side by side
    const uint32_t heads = ROLE == QUERIES ? g.q_heads : g.c.heads;
    const uint32_t h0 = group << log_lanes;
    const uint32_t slot = tid / TPR, c = tid % TPR;
    const uint32_t tslot = slot >> log_lanes, tstep = ROWS >> log_lanes;
    const bool live = h0 + (slot & (lanes - 1u)) < heads;
    const uint32_t head = live ? h0 + (slot & (lanes - 1u)) : heads - 1;
    const uint32_t half = ROLE == VALUES ? 0 : g.turn.half;
    const bool turned = 8 * c < half;
    // a thread's two pieces: the two sides of eight pairs, or 16 channels that are not turned or hold whole pairs
    const bool split = turned && !g.turn.interleaved;
    const uint32_t ca = split ? 8 * c : 16 * c, cb = split ? half + 8 * c : 16 * c + 8;
    const Rows &in = ROLE == QUERIES ? g.q : ROLE == KEYS ? g.k : g.v;
    const __bf16 *src = in.p + (int64_t)sg.row0 * in.token + (int64_t)head * in.head;
    float scale = 1.0f;
    if (DT != ZX_BF16 && ROLE != QUERIES) {
        const float *sc = ROLE == KEYS ? g.c.k_scale : g.c.v_scale;
        if (sc) scale = sc[head];
    }
    const bool bounds = ROLE == KEYS && g.c.bounds;
    i16x2 lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo[i] = i16x2{kTopBf16, kTopBf16};
        hi[i] = i16x2{kLowBf16, kLowBf16};
    }

    for (int32_t t0 = sg.p0; t0 < sg.p1; t0 += (int32_t)kTab) {
        const uint32_t nt = (uint32_t)(sg.p1 - t0) < kTab ? (uint32_t)(sg.p1 - t0) : kTab;
        bf8 ra[kBatch], rb[kBatch];
        uint32_t page[kBatch];
        auto fetch = [&](uint32_t t) {                  // rows past the last one repeat it
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const uint32_t tu = t + u * tstep < nt ? t + u * tstep : nt - 1;
                const int32_t p = t0 + (int32_t)tu;
                const __bf16 *r = src + (int64_t)p * in.token;
                ra[u] = *reinterpret_cast<const bf8 *>(r + ca);
                rb[u] = *reinterpret_cast<const bf8 *>(r + cb);
                if (ROLE != QUERIES) page[u] = (uint32_t)sg.table[p >> g.c.log_page];
            }
        };
        fetch(tslot);                                   // under way while the cosines and sines are worked out
        if (half) {
            if (t0 > sg.p0) __syncthreads();
            for (uint32_t i = tid; i < nt * half; i += kThreads) {
                const uint32_t t = i / half, j = i - t * half;
                const int32_t p = g.turn.positions ? g.turn.positions[sg.row0 + t0 + (int32_t)t] : t0 + (int32_t)t;
                // whole turns are dropped in 64 bits: what is left keeps its 24 bits at any position
                const double rev = (double)p * g.turn.inv_freq[j] * 0.15915494309189533577;
                const float r = (float)(rev - __builtin_rint(rev));
                float sn, cs;
                sincospif(2.0f * r, &sn, &cs);
                reinterpret_cast<f2 *>(lds)[t * half + j] = f2{cs * g.turn.magnitude, sn * g.turn.magnitude};
            }
            __syncthreads();
        }
        for (uint32_t tb = tslot; tb < nt; tb += kBatch * tstep) {
            if (tb != tslot) fetch(tb);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const uint32_t tu = tb + u * tstep;
                const bool yes = live && tu < nt;
                const uint32_t t = tu < nt ? tu : nt - 1;
                const int32_t p = t0 + (int32_t)t;
                float x[8], y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] = (float)ra[u][i];
                    y[i] = (float)rb[u][i];
                }
                if (turned) {
                    const f4 *tab = reinterpret_cast<const f4 *>(reinterpret_cast<const f2 *>(lds) + t * half + 8 * c);
                    auto turn = [](float &a, float &b, float cs, float sn) {
                        const float u = a * cs - b * sn;
                        b = b * cs + a * sn;
                        a = u;
                    };
                    if (split) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const f4 w = tab[i];        // of two pairs
                            turn(x[2 * i], y[2 * i], w[0], w[1]);
                            turn(x[2 * i + 1], y[2 * i + 1], w[2], w[3]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const f4 w = tab[i], v = tab[2 + i];
                            turn(x[4 * i], x[4 * i + 1], w[0], w[1]);
                            turn(x[4 * i + 2], x[4 * i + 3], w[2], w[3]);
                            turn(y[4 * i], y[4 * i + 1], v[0], v[1]);
                            turn(y[4 * i + 2], y[4 * i + 3], v[2], v[3]);
                        }
                    }
                }
                if constexpr (ROLE == QUERIES) {
                    __bf16 *dst = g.qo.p + (int64_t)(sg.row0 + p) * g.qo.token + (int64_t)head * g.qo.head;
                    if (yes) {
                        *reinterpret_cast<bf8 *>(dst + ca) = to_bf8(x);
                        *reinterpret_cast<bf8 *>(dst + cb) = to_bf8(y);
                    }
                } else {
                    const bool there = page[u] < g.c.n_pages;
                    if (!there) report(g.b.err, ZX_E_CORRUPT);
                    const uint32_t at = (uint32_t)p & ((1u << g.c.log_page) - 1u), pg = there ? page[u] : 0;
                    uint8_t *dst = ROLE == KEYS ? g.c.k + (int64_t)head * g.c.k_head + (int64_t)pg * g.c.k_page + (uint64_t)at * g.c.k_token
                                                : g.c.v + (int64_t)head * g.c.v_head + (int64_t)pg * g.c.v_page + (uint64_t)at * g.c.v_token;
                    if constexpr (DT == ZX_BF16 && ROLE == VALUES) {
                        if (yes && there) {             // bits as they are
                            *reinterpret_cast<bf8 *>(dst + 2 * ca) = ra[u];
                            *reinterpret_cast<bf8 *>(dst + 2 * cb) = rb[u];
                        }
                    } else {
                        const u4 wa = store8<DT>(dst, ca, x, scale, yes && there), wb = store8<DT>(dst, cb, y, scale, yes && there);
                        if (bounds) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const i16x2 a = ordered(wa[i]), b = ordered(wb[i]);
                                lo[i] = __builtin_elementwise_min(lo[i], a);
                                hi[i] = __builtin_elementwise_max(hi[i], a);
                                lo[4 + i] = __builtin_elementwise_min(lo[4 + i], b);
                                hi[4 + i] = __builtin_elementwise_max(hi[4 + i], b);
                            }
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);      // one row's values at a time
            }
        }
    }

    if constexpr (ROLE == KEYS) {
        if (!bounds) return;
        const uint32_t page = (uint32_t)sg.table[sg.start >> g.c.log_page];
        if (page >= g.c.n_pages) return;                // reported above; the whole workgroup leaves
        // [rows][smallest, largest][D] as ordered 16-bit integers
        int16_t *const sh = reinterpret_cast<int16_t *>(lds);
        __syncthreads();
        i16x2 *mine = reinterpret_cast<i16x2 *>(sh + slot * (2 * D));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mine[ca / 2 + i] = lo[i];
            mine[cb / 2 + i] = lo[4 + i];
            mine[(D + ca) / 2 + i] = hi[i];
            mine[(D + cb) / 2 + i] = hi[4 + i];
        }
        __syncthreads();
        const uint32_t nb = 1u << (g.c.log_page - g.c.log_block);
        const uint32_t blk = (uint32_t)(sg.start >> g.c.log_block) & (nb - 1u);
        const uint32_t nh = heads - h0 < lanes ? heads - h0 : lanes;
        const uint32_t used = (uint32_t)(sg.p1 - sg.p0) < tstep ? (uint32_t)(sg.p1 - sg.p0) : tstep;    // rows of a head that took part
        for (uint32_t i = tid; i < nh * 2 * D; i += kThreads) {
            const uint32_t h = i / (2 * D), w = i % (2 * D);
            const bool low = w < (uint32_t)D;
            int16_t x = sh[h * (2 * D) + w];
            for (uint32_t r = 1; r < used; ++r) {
                const int16_t y = sh[(r * lanes + h) * (2 * D) + w];
                x = low ? (y < x ? y : x) : (y > x ? y : x);
            }
            if (low ? x < kLowBf16 : x > kTopBf16) {
                // a NaN got in: the values once more, without it
                x = low ? kTopBf16 : kLowBf16;
                for (int32_t p = sg.p0; p < sg.p1; ++p) {
                    const uint64_t at = (uint32_t)p & ((1u << g.c.log_page) - 1u);
                    const uint8_t *row = g.c.k + (int64_t)page * g.c.k_page + (int64_t)(h0 + h) * g.c.k_head + at * g.c.k_token;
                    const uint32_t ch = w % D;
                    const uint32_t bits = DT == ZX_BF16 ? reinterpret_cast<const uint16_t *>(row)[ch] : bf16_pair_of_fp8(row[ch], false) & 0xFFFFu;
                    if ((bits & 0x7FFFu) > 0x7F80u) continue;
                    const int16_t y = ordered(bits)[0];
                    x = low ? (y < x ? y : x) : (y > x ? y : x);
                }
            }
            uint16_t *o = reinterpret_cast<uint16_t *>(g.c.bounds) + (((uint64_t)page * g.c.heads + h0 + h) * nb + blk) * (2 * D) + w;
            if (sg.older) {
                const uint32_t old = *o;
                if ((old & 0x7FFFu) <= 0x7F80u) {
                    const int16_t y = ordered(old)[0];
                    x = low ? (y < x ? y : x) : (y > x ? y : x);
                }
            }
            *o = unordered(x);
        }
    }
}

template <int DT, int D>
__global__ __launch_bounds__(kThreads, 4) void k_paged_append(AppendArgs g)
{
    // the cosines and sines of kTab tokens; then the bounds of every thread's 16 channels
    __shared__ __align__(16) float lds[kTab * D > kThreads * 16 ? kTab * D : kThreads * 16];
    uint32_t seq, seg, unused;
    Seq sv;
    const uint32_t ls = g.log_seg;
    const bool found = find_item(
        g.b, blockIdx.x,
        [ls](const Seq &v) {
            if (v.nq == 0 || v.kv == 0) return 0u;
            const int32_t p0 = v.kv > v.nq ? v.kv - v.nq : 0;
            return (uint32_t)((v.kv - 1) >> ls) - (uint32_t)(p0 >> ls) + 1u;
        },
        [](const Seq &) { return 0u; }, seq, sv, seg, unused);
    if (!found) return;
    const int32_t first = sv.kv > sv.nq ? sv.kv - sv.nq : 0;       // first new token that has a place
    Segment sg;
    sg.start = ((first >> ls) + (int32_t)seg) << ls;
    sg.p0 = sg.start > first ? sg.start : first;
    sg.p1 = sg.start + (1 << ls) < sv.kv ? sg.start + (1 << ls) : sv.kv;
    sg.row0 = sv.q0 + sv.nq - sv.kv;
    sg.table = g.b.table + (uint64_t)seq * g.b.width;
    sg.older = first > sg.start;
    // groups of heads: of the keys, of the values, of the queries
    if (blockIdx.y < g.kv_groups) append_rows<DT, D, KEYS>(g, sg, blockIdx.y, lds);
    else if (blockIdx.y < 2 * g.kv_groups) append_rows<DT, D, VALUES>(g, sg, blockIdx.y - g.kv_groups, lds);
    else append_rows<DT, D, QUERIES>(g, sg, blockIdx.y - 2 * g.kv_groups, lds);
}

template <int DT>
void launch(const AppendArgs &g, uint32_t D, dim3 grid, hipStream_t stream)
{
    if (D == 64) hipLaunchKernelGGL((k_paged_append<DT, 64>), grid, dim3(kThreads), 0, stream, g);
    else if (D == 128) hipLaunchKernelGGL((k_paged_append<DT, 128>), grid, dim3(kThreads), 0, stream, g);
    else hipLaunchKernelGGL((k_paged_append<DT, 256>), grid, dim3(kThreads), 0, stream, g);
}

}  // namespace
}  // namespace zxp

extern "C" zx_status zx_paged_append(const zx_paged_cache *cache, const zx_paged_batch *batch, uint32_t n_tokens,
                                     const zx_rows *k, const zx_rows *v, const zx_rotary *rot, const int32_t *positions,
                                     const zx_rows *q, uint32_t q_heads, const zx_rows *q_out, uint32_t *err,
                                     hipStream_t stream)
{
    using namespace zxp;
    AppendArgs g{};
    zx_status st = make_cache(cache, g.c);
    if (st == ZX_OK) st = make_batch(batch, cache, n_tokens, err, g.b);
    if (st != ZX_OK) return st;
    if (n_tokens == 0 || batch->n_seqs == 0) return ZX_OK;
    if ((st = make_rows(k, g.k)) != ZX_OK || (st = make_rows(v, g.v)) != ZX_OK) return st;
    if (q) {
        if (q_heads == 0 || q_heads > 65536) return ZX_E_INVAL;
        if ((st = make_rows(q, g.q)) != ZX_OK || (st = make_rows(q_out, g.qo)) != ZX_OK) return st;
        g.q_heads = q_heads;
    }
    if (rot) {
        if (!rot->inv_freq || ((uintptr_t)rot->inv_freq & 7u) || rot->dims == 0 || rot->dims % 16 || rot->dims > cache->head_dim)
            return ZX_E_INVAL;
        g.turn = Turn{rot->inv_freq, positions, rot->dims / 2, rot->interleaved, rot->magnitude};
    }
    g.log_seg = g.c.bounds ? g.c.log_block : log2_of(kSeg);
    while (g.kv_log < kLogGroup && (1u << g.kv_log) < g.c.heads) ++g.kv_log;
    g.kv_groups = ceil_div(g.c.heads, 1u << g.kv_log);
    const uint64_t by_len = ((uint64_t)n_tokens >> g.log_seg) + 2ull * batch->n_seqs;
    const uint32_t segs = (uint32_t)(by_len < n_tokens ? by_len : n_tokens);
    const dim3 grid(segs, 2 * g.kv_groups + ceil_div(g.q_heads, kGroup));
    if (cache->dtype == ZX_BF16) launch<ZX_BF16>(g, cache->head_dim, grid, stream);
    else launch<ZX_FP8_E4M3FN>(g, cache->head_dim, grid, stream);
    return hipGetLastError() == hipSuccess ? ZX_OK : ZX_E_HIP;
}
