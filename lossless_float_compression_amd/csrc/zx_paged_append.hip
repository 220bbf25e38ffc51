// zx_paged_append.hip -- new keys and values into a paged K/V cache, with the position
// rotation on the way, and the checks that all entry points of the paged cache share.
//
// A workgroup takes one segment of a sequence's new tokens (the tokens of one bounded
// block, or of 32 places where the cache has no bounds) and a group of heads: of the
// keys and values, or of the queries.  It computes the cosines and sines of the
// segment's positions once, in LDS, and turns the rows of all its heads with them.  A
// thread holds 16 channels, eight rotated pairs.  One workgroup owns a block's bounds
// for its heads, so they are reduced in registers and LDS with no atomics and do not
// depend on any order.
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
constexpr uint32_t kGroup = 8;         // heads of a workgroup

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
    uint32_t kv_groups, kv_lanes;      // K/V head groups and heads of one (a power of two up to kGroup)
    uint32_t q_heads, log_seg;
};

// Two 8-channel pieces of a row: channels a .. a + 7 and b .. b + 7.
struct Piece {
    float a[8], b[8];
};

__device__ __forceinline__ void load8(const __bf16 *p, float (&o)[8])
{
    const bf8 x = *reinterpret_cast<const bf8 *>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (float)x[i];
}

__device__ __forceinline__ bf8 to_bf8(const float (&x)[8])
{
    bf8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (__bf16)x[i];
    return o;
}

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

__device__ __forceinline__ void from_fp8(u2 v, float (&o)[8])
{
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const f2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[w], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[w], true);
        o[4 * w] = lo[0];
        o[4 * w + 1] = lo[1];
        o[4 * w + 2] = hi[0];
        o[4 * w + 3] = hi[1];
    }
}

// Store a piece of eight channels as the cache holds it; x becomes the stored values.
template <int DT>
__device__ __forceinline__ void store8(uint8_t *row, uint32_t ch, float (&x)[8], float scale)
{
    if constexpr (DT == ZX_BF16) {
        const bf8 y = to_bf8(x);
        *reinterpret_cast<bf8 *>(row + 2 * ch) = y;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)y[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fp8_in(x[i], scale);
        const u2 y = to_fp8(x);
        *reinterpret_cast<u2 *>(row + ch) = y;
        from_fp8(y, x);
    }
}

template <int DT, int D>
__global__ __launch_bounds__(kThreads) void k_paged_append(AppendArgs g)
{
    constexpr uint32_t TPR = D / 16;            // threads of a row
    constexpr uint32_t ROWS = kThreads / TPR;   // rows at a time
    // the cosines and sines of kTab tokens; then, for the bounds, every thread's 16 smallest and 16 largest
    __shared__ __align__(16) float lds[kTab * D > kThreads * 32 ? kTab * D : kThreads * 32];

    const uint32_t tid = threadIdx.x;
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
    const int32_t s0 = ((first >> ls) + (int32_t)seg) << ls;
    const int32_t p0 = s0 > first ? s0 : first;
    const int32_t p1 = s0 + (1 << ls) < sv.kv ? s0 + (1 << ls) : sv.kv;
    const int32_t row0 = sv.q0 + sv.nq - sv.kv;                     // packed row of position p: row0 + p

    const bool is_q = blockIdx.y >= g.kv_groups;
    const uint32_t lanes = is_q ? kGroup : g.kv_lanes;              // heads side by side
    const uint32_t h0 = is_q ? (blockIdx.y - g.kv_groups) * kGroup : blockIdx.y * g.kv_lanes;
    const uint32_t slot = tid / TPR, c = tid % TPR;
    const uint32_t head = h0 + slot % lanes, tslot = slot / lanes, tstep = ROWS / lanes;
    const bool live = head < (is_q ? g.q_heads : g.c.heads);
    const uint32_t half = g.turn.half;
    const bool turned = 8 * c < half;
    // a thread's two pieces: the two sides of eight pairs, or 16 channels that are not turned or hold whole pairs
    const bool split = turned && !g.turn.interleaved;
    const uint32_t ca = split ? 8 * c : 16 * c, cb = split ? half + 8 * c : 16 * c + 8;
    const int32_t *table = g.b.table + (uint64_t)seq * g.b.width;
    float ks = 1.0f, vs = 1.0f;
    if (DT != ZX_BF16 && !is_q && live) {
        ks = g.c.k_scale ? g.c.k_scale[head] : 1.0f;
        vs = g.c.v_scale ? g.c.v_scale[head] : 1.0f;
    }
    const bool bounds = !is_q && g.c.bounds;
    Piece lo, hi;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo.a[i] = lo.b[i] = __builtin_huge_valf();
        hi.a[i] = hi.b[i] = -__builtin_huge_valf();
    }

    for (int32_t t0 = p0; t0 < p1; t0 += (int32_t)kTab) {
        const uint32_t nt = (uint32_t)(p1 - t0) < kTab ? (uint32_t)(p1 - t0) : kTab;
        if (half) {
            __syncthreads();
            for (uint32_t i = tid; i < nt * half; i += kThreads) {
                const uint32_t t = i / half, j = i - t * half;
                const int32_t p = g.turn.positions ? g.turn.positions[row0 + t0 + (int32_t)t] : t0 + (int32_t)t;
                // whole turns are dropped in 64 bits: what is left keeps its 24 bits at any position
                const double rev = (double)p * g.turn.inv_freq[j] * 0.15915494309189533577;
                const float r = (float)(rev - __builtin_rint(rev));
                float sn, cs;
                sincospif(2.0f * r, &sn, &cs);
                reinterpret_cast<f2 *>(lds)[t * half + j] = f2{cs * g.turn.magnitude, sn * g.turn.magnitude};
            }
            __syncthreads();
        }
        if (!live) continue;
        for (uint32_t t = tslot; t < nt; t += tstep) {
            const int32_t p = t0 + (int32_t)t;
            const int64_t row = row0 + p;
            Piece x;
            const __bf16 *src = is_q ? g.q.p + row * g.q.token + (int64_t)head * g.q.head : g.k.p + row * g.k.token + (int64_t)head * g.k.head;
            load8(src + ca, x.a);
            load8(src + cb, x.b);
            if (turned) {
                const f4 *tab = reinterpret_cast<const f4 *>(reinterpret_cast<const f2 *>(lds) + t * half + 8 * c);
                float cs[8], sn[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f4 w = tab[i];
                    cs[2 * i] = w[0];
                    sn[2 * i] = w[1];
                    cs[2 * i + 1] = w[2];
                    sn[2 * i + 1] = w[3];
                }
                if (split) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float a = x.a[i], b = x.b[i];
                        x.a[i] = a * cs[i] - b * sn[i];
                        x.b[i] = b * cs[i] + a * sn[i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float a = x.a[2 * i], b = x.a[2 * i + 1], d = x.b[2 * i], e = x.b[2 * i + 1];
                        x.a[2 * i] = a * cs[i] - b * sn[i];
                        x.a[2 * i + 1] = b * cs[i] + a * sn[i];
                        x.b[2 * i] = d * cs[4 + i] - e * sn[4 + i];
                        x.b[2 * i + 1] = e * cs[4 + i] + d * sn[4 + i];
                    }
                }
            }
            if (is_q) {
                __bf16 *dst = g.qo.p + row * g.qo.token + (int64_t)head * g.qo.head;
                *reinterpret_cast<bf8 *>(dst + ca) = to_bf8(x.a);
                *reinterpret_cast<bf8 *>(dst + cb) = to_bf8(x.b);
                continue;
            }
            const uint32_t page = (uint32_t)table[p >> g.c.log_page];
            if (page >= g.c.n_pages) {
                report(g.b.err, ZX_E_CORRUPT);
                continue;
            }
            const uint32_t at = (uint32_t)p & ((1u << g.c.log_page) - 1u);
            uint8_t *kr = g.c.k + (int64_t)page * g.c.k_page + (int64_t)head * g.c.k_head + (uint64_t)at * g.c.k_token;
            store8<DT>(kr, ca, x.a, ks);
            store8<DT>(kr, cb, x.b, ks);
            if (bounds) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    lo.a[i] = fminf(lo.a[i], x.a[i]);
                    hi.a[i] = fmaxf(hi.a[i], x.a[i]);
                    lo.b[i] = fminf(lo.b[i], x.b[i]);
                    hi.b[i] = fmaxf(hi.b[i], x.b[i]);
                }
            }
            const __bf16 *vr = g.v.p + row * g.v.token + (int64_t)head * g.v.head + 16 * c;
            uint8_t *vd = g.c.v + (int64_t)page * g.c.v_page + (int64_t)head * g.c.v_head + (uint64_t)at * g.c.v_token;
            if constexpr (DT == ZX_BF16) {
                const u4 w0 = reinterpret_cast<const u4 *>(vr)[0], w1 = reinterpret_cast<const u4 *>(vr)[1];
                reinterpret_cast<u4 *>(vd + 32 * c)[0] = w0;
                reinterpret_cast<u4 *>(vd + 32 * c)[1] = w1;
            } else {
                load8(vr, x.a);
                load8(vr + 8, x.b);
                store8<DT>(vd, 16 * c, x.a, vs);
                store8<DT>(vd, 16 * c + 8, x.b, vs);
            }
        }
    }

    if (!bounds) return;
    const uint32_t page = (uint32_t)table[s0 >> g.c.log_page];
    if (page >= g.c.n_pages) return;            // reported above; the whole workgroup leaves
    __syncthreads();
    float *mine = lds + slot * (2 * D);         // [rows][smallest, largest][D]
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        mine[ca + i] = lo.a[i];
        mine[cb + i] = lo.b[i];
        mine[D + ca + i] = hi.a[i];
        mine[D + cb + i] = hi.b[i];
    }
    __syncthreads();
    const uint32_t nb = 1u << (g.c.log_page - g.c.log_block);
    const uint32_t blk = (uint32_t)(s0 >> g.c.log_block) & (nb - 1u);
    const uint32_t nh = g.c.heads - h0 < lanes ? g.c.heads - h0 : lanes;
    for (uint32_t i = tid; i < nh * 2 * D; i += kThreads) {
        const uint32_t h = i / (2 * D), w = i % (2 * D);
        float x = lds[h * (2 * D) + w];
        for (uint32_t r = 1; r < tstep; ++r) {
            const float y = lds[(r * lanes + h) * (2 * D) + w];
            x = w < (uint32_t)D ? fminf(x, y) : fmaxf(x, y);
        }
        __bf16 *o = g.c.bounds + (((uint64_t)page * g.c.heads + h0 + h) * nb + blk) * (2 * D) + w;
        if (first > s0) {                       // the block has older tokens
            const float y = (float)*o;
            x = w < (uint32_t)D ? fminf(x, y) : fmaxf(x, y);
        }
        *o = (__bf16)x;                         // a stored value: exact
    }
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
    g.kv_lanes = 1;
    while (g.kv_lanes < kGroup && g.kv_lanes < g.c.heads) g.kv_lanes *= 2;
    g.kv_groups = ceil_div(g.c.heads, g.kv_lanes);
    const uint64_t by_len = ((uint64_t)n_tokens >> g.log_seg) + 2ull * batch->n_seqs;
    const uint32_t segs = (uint32_t)(by_len < n_tokens ? by_len : n_tokens);
    const dim3 grid(segs, g.kv_groups + ceil_div(g.q_heads, kGroup));
    if (cache->dtype == ZX_BF16) launch<ZX_BF16>(g, cache->head_dim, grid, stream);
    else launch<ZX_FP8_E4M3FN>(g, cache->head_dim, grid, stream);
    return hipGetLastError() == hipSuccess ? ZX_OK : ZX_E_HIP;
}
