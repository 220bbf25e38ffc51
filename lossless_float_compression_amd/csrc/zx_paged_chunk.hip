// zx_paged_chunk.hip -- attention of many new tokens over a paged K/V cache: the tiled
// kernel.
//
// A workgroup takes 32 rows a wave (rows: the group's query heads for each new token)
// and goes over its tokens in tiles of 64.  K and V tiles are read from their pages into
// registers two steps ahead, written to LDS as BF16 one step ahead, and shared by all
// waves (read straight into LDS by the load instruction they are no faster for BF16, 10% slower for 64
// channels or E4M3).  With 32x32x16 products a lane has one query row; K is the left operand as it lies, V is
// read transposed (ds_read_b64_tr_b16), four tokens of 16 channels for 16 lanes at a
// time, in the order of tokens that the scores come out in, so weights go from one
// product to the next without leaving their lane.  LDS rows are padded so that the 16
// lanes of a read meet all 64 banks: keys by 16 bytes (a row of 16-byte pieces moves four
// banks on), values by 64 bytes (four rows of 32 bytes, 16 banks apart).
//
// A step of a wave is a matrix phase (the second product of tile i, the first of tile i + 1)
// and a vector phase (the softmax of tile i + 1), about 1000 cycles each.  Two waves share a
// SIMD; in step with each other they would both want the matrix unit and then both the
// vector unit, so the second half of the workgroup's waves runs one phase behind the
// first, held there by a barrier after every phase: 165 us against 185 in step, for 4096 new
// tokens at 32 query heads of 128 channels, 137 GFLOP over the tokens they see (151 us, 910 TFLOP/s, in short
// runs, where clocks are higher).  The products with their LDS reads alone take 125 us, without reads and barriers 115.
#include <type_traits>

#include "zx_paged_attend.h"

namespace zxp {
namespace {

constexpr int kTile = 64;

template <int DT, int D, int NW>
__global__ __launch_bounds__(NW * 64, D == 256 ? 1 : 2) void k_chunk(AttendArgs g)
{
    constexpr int ROWS = 32 * NW, NT = 64 * NW;
    constexpr int ES = DT == ZX_BF16 ? 2 : 1;
    constexpr int CPR = D * ES / 16;                       // 16-byte pieces of a row
    constexpr int NL = (kTile * CPR + NT - 1) / NT;        // pieces a thread moves
    constexpr int KS = D * 2 + 16, VS = D * 2 + 64;        // LDS row strides in bytes
    constexpr int NS = D / 16, ND = D / 32;
    __shared__ __align__(16) uint8_t kl[2][kTile * KS];
    __shared__ __align__(16) uint8_t vl[2][kTile * VS];
    __shared__ uint32_t any_odd;                           // whether store_v left infinities or NaN out

    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t lr = lane & 31u, lh = lane >> 5;
    const uint32_t G = g.group;
    const uint32_t h = blockIdx.x % g.c.heads, rest = blockIdx.x / g.c.heads;
    uint32_t seq, rt, part, nch, slot;
    Seq sv;
    if (!find_piece<ROWS, kTile>(g, rest, chunk_steps<ROWS, kTile>(g), seq, sv, rt, part, nch, slot)) return;
    const uint32_t all = (uint32_t)sv.nq * G;
    if (nch == 1) {
        // The last row tiles see the most tokens: they go first.  Of two workgroups on a CU
        // the second has the tiles from the other end, shortest first, while there are no more.
        const uint32_t tiles = div_up(all, ROWS), room = div_up(256, g.c.heads);
        rt = NW == 4 && rt >= room && tiles <= 2 * room ? rt - room : tiles - 1 - rt;
    }
    const uint32_t row0 = rt * ROWS, row9 = row0 + ROWS < all ? row0 + ROWS : all;
    const int32_t pos0 = sv.kv - sv.nq;
    const int32_t pa = pos0 + (int32_t)(row0 / G), pb = pos0 + (int32_t)((row9 - 1) / G);
    const int32_t lo_min = first_seen(g, pa), lo_max = first_seen(g, pb), hi_min = end_seen(g, pa, sv.kv), hi_max = end_seen(g, pb, sv.kv);

    // this wave's rows (one lane's row past the last repeats it)
    const uint32_t wr = row0 + wave * 32;
    const bool live = wr < row9;
    const uint32_t w9 = wr + 32 < row9 ? wr + 32 : row9;
    const uint32_t row = live ? (wr + lr < w9 ? wr + lr : w9 - 1) : row9 - 1;
    const int32_t wa = pos0 + (int32_t)((live ? wr : row9 - 1) / G), wb = pos0 + (int32_t)((live ? w9 - 1 : row9 - 1) / G);
    const int32_t wlo_max = first_seen(g, wb), whi_min = end_seen(g, wa, sv.kv);
    const int32_t mypos = pos0 + (int32_t)(row / G), lo = first_seen(g, mypos), hi = end_seen(g, mypos, sv.kv);
    const int64_t at = sv.q0 + (int32_t)(row / G);
    const uint32_t qh = h * G + row % G;
    u4 q[NS];
    {
        const __bf16 *qp = g.q.p + at * g.q.token + (int64_t)qh * g.q.head + 8 * lh;
#pragma unroll
        for (int s = 0; s < NS; ++s) q[s] = *reinterpret_cast<const u4 *>(qp + 16 * s);
    }

    uint32_t t0 = (uint32_t)lo_min / kTile, t1 = div_up((uint32_t)hi_max, kTile);
    if (t1 < t0) t1 = t0;
    const uint32_t per = div_up(t1 - t0, nch);
    t0 += part * per;
    if (t0 > t1) t0 = t1;
    if (t1 > t0 + per) t1 = t0 + per;

    const int32_t *table = g.b.table + (uint64_t)seq * g.b.width;
    const uint32_t pmask = (1u << g.c.log_page) - 1u;
    const uint8_t *const kmem = g.c.k + (int64_t)h * g.c.k_head, *const vmem = g.c.v + (int64_t)h * g.c.v_head;
    // Where the tiles' 16-token pieces lie: lane i has the addresses of piece i of the 16
    // tiles from `base` on (page 0, and a bit in `gone`, where there is no page), and the page
    // ids of the 16 tiles behind them are read ahead.  A tile's addresses are then lane
    // reads, not a trip to memory and 64-bit products.
    uint64_t kat, vat, gone;
    uint32_t base = t0, ahead;
    auto look = [&](uint32_t tile) {
        const uint32_t t = tile * kTile + 16 * lane;
        return t < (uint32_t)sv.kv ? (uint32_t)table[t >> g.c.log_page] : 0xFFFFFFFFu;
    };
    auto settle = [&](uint32_t id) {
        const uint32_t t = base * kTile + 16 * lane;
        const bool none = id >= g.c.n_pages;
        // (tiles begin at multiples of 64: pages of 16 or 32 tokens that no row sees may have been given away)
        if (none && t < (uint32_t)hi_max && t + 16 > (uint32_t)lo_min) report(g.b.err, ZX_E_CORRUPT);
        if (none) id = 0;
        kat = (uint64_t)kmem + (uint64_t)((int64_t)id * g.c.k_page) + (uint64_t)(t & pmask) * g.c.k_token;
        vat = (uint64_t)vmem + (uint64_t)((int64_t)id * g.c.v_page) + (uint64_t)(t & pmask) * g.c.v_token;
        gone = __ballot(none);
        ahead = look(base + 16);
    };
    settle(look(t0));
    // A thread's NL pieces of a tile lie in rows whose 16-token piece is the same for the whole wave.
    struct Spot {
        uint64_t at[NL];
    };
    struct Where {
        Spot k, v;
        uint32_t gone;               // pieces of the tile that have no page: four bits
    };
    auto lane64 = [](uint64_t x, uint32_t l) {
        return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, (int)l) |
               (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(x >> 32), (int)l) << 32;
    };
    auto where = [&](uint32_t tile) {
        if (tile - base >= 16) {
            base += 16;
            settle(ahead);
        }
        Where r;
        const uint32_t l = 4 * (tile - base);
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            uint32_t sub = (i * NT + wave * 64) / CPR / 16;
            if (kTile * CPR % NT) sub &= 3u;            // waves that have no piece
            r.k.at[i] = lane64(kat, l + sub);
            r.v.at[i] = lane64(vat, l + sub);
        }
        r.gone = (uint32_t)(gone >> l) & 15u;
        return r;
    };
    u4 kr[NL], vr[NL];
    // piece i of this thread's part of a tile, keys or values, into a register
    auto load = [&](u4 &r, const Spot &at, uint32_t token_stride, int i) {
        const uint32_t w = i * NT + wave * 64;
        if (kTile * CPR % NT && w >= (uint32_t)(kTile * CPR)) return;
        const uint32_t row = (threadIdx.x + i * NT) / CPR % 16u, ch = (threadIdx.x + i * NT) % CPR * 16u;
        r = *(const global_u4 *)((const global_u1 *)at.at[i] + (row * token_stride + ch));
    };
    auto load_k = [&](const Where &at, int i) { load(kr[i], at.k, g.c.k_token, i); };
    auto load_v = [&](const Where &at, int i) { load(vr[i], at.v, g.c.v_token, i); };
    // 16 bytes of the cache as BF16
    auto widen = [](u4 x, u4 (&y)[2 / ES == 1 ? 1 : 2]) {
        if constexpr (DT == ZX_BF16) {
            y[0] = x;
        } else {
            y[0] = u4{fp8_pair<false>(x[0]), fp8_pair<true>(x[0]), fp8_pair<false>(x[1]), fp8_pair<true>(x[1])};
            y[1] = u4{fp8_pair<false>(x[2]), fp8_pair<true>(x[2]), fp8_pair<false>(x[3]), fp8_pair<true>(x[3])};
        }
    };
    constexpr int NY = ES == 2 ? 1 : 2;
    auto store_k = [&](uint32_t tile, int i) {
        const uint32_t w = i * NT + wave * 64;
        if (kTile * CPR % NT && w >= (uint32_t)(kTile * CPR)) return;
        u4 y[NY];
        widen(kr[i], y);
        uint8_t *dst = kl[tile & 1u] + (w + lane) / CPR * KS + ((w + lane) % CPR) * (32 / ES);
#pragma unroll
        for (int j = 0; j < NY; ++j) reinterpret_cast<u4 *>(dst)[j] = y[j];
    };
    auto store_v = [&](uint32_t tile, uint32_t gone, int i) {
        const uint32_t w = i * NT + wave * 64;
        if (kTile * CPR % NT && w >= (uint32_t)(kTile * CPR)) return;
        const int32_t a = (int32_t)(tile * kTile);
        const bool edge = gone != 0 || a < lo_min || a + kTile > hi_max;      // some token that no row sees
        const bool mixed = a < lo_max || a + kTile > hi_min;                  // some token that some rows do not see
        u4 y[NY];
        widen(vr[i], y);
        if (edge) {
            const int32_t t = a + (int32_t)((w + lane) / CPR);
            const bool none = (gone >> (w / CPR / 16) & 1u) || t < lo_min || t >= hi_max;
#pragma unroll
            for (int j = 0; j < NY; ++j) y[j] = none ? u4{0, 0, 0, 0} : y[j];
        }
        if (mixed) {
            // An infinity or NaN that only some rows see: zero times it would reach the
            // others.  It is left out here and added at the end to the rows that see it.
            bool odd = false;
#pragma unroll
            for (int j = 0; j < NY; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    odd = odd || odd_pair(y[j][e]);
                    y[j][e] = tame_pair(y[j][e]);
                }
            if (odd) any_odd = 1;
        }
        uint8_t *dst = vl[tile & 1u] + (w + lane) / CPR * VS + ((w + lane) % CPR) * (32 / ES);
#pragma unroll
        for (int j = 0; j < NY; ++j) reinterpret_cast<u4 *>(dst)[j] = y[j];
    };

    float m = -kInf, l = 0.0f;
    f16v o[ND], s[2];
    u4 p[4];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
    // (not zero where a tiny scale meets a tiny k_scale: a masked score is -inf until it is multiplied)
    const float c0 = g.scale * (g.c.k_scale ? g.c.k_scale[h] : 1.0f), c = c0 == 0.0f ? 0x1p-149f : c0;

    typedef __attribute__((address_space(3))) const uint8_t *lds_ptr;
    const lds_ptr kp = (lds_ptr)&kl[0][0] + lr * KS + 16 * lh;
    const lds_ptr vp = (lds_ptr)&vl[0][0] + (4 * lh + (lane & 15u) / 4) * VS + ((lane >> 4) & 1u) * 32 + (lane & 3u) * 8;
    auto key = [](lds_ptr kp, int t, int j) { return *(__attribute__((address_space(3))) const u4 *)(kp + 32 * t * KS + 32 * j); };
    auto value = [](lds_ptr vp, int k, int d) {
        typedef short s4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s4 *lp;
        const s4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(vp + (16 * k) * VS + 64 * d));
        const s4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(vp + (16 * k + 8) * VS + 64 * d));
        const u2 xu = __builtin_bit_cast(u2, x), yu = __builtin_bit_cast(u2, y);
        return u4{xu[0], xu[1], yu[0], yu[1]};
    };
    // The products of a matrix phase: the second one of a tile (FIRST: none), then the first one
    // of the tile behind it, whose register i of s[t] is token 32 t + 8 (i / 4) + 4 lh + i % 4.
    // Reads and products stand in the order they are to run in, held there by scheduling
    // barriers: values are read ND products ahead, keys kAhead products ahead.
    constexpr int kAhead = D == 256 ? 4 : 8;
    // `between(n)` is called after product n of the first one, to run beside the products.
    auto products = [&](uint32_t tile, auto first, auto between) {
        const lds_ptr vq = vp + (tile & 1u) * (kTile * VS), kq = kp + ((tile + 1) & 1u) * (kTile * KS);
        u4 kf[kAhead];
        auto next_key = [&](int n) { kf[n % kAhead] = key(kq, n % 2, n / 2); };
        if constexpr (decltype(first)::value) {
#pragma unroll
            for (int n = 0; n < kAhead; ++n) next_key(n);
        } else {
            u4 vf[2][ND];
#pragma unroll
            for (int d = 0; d < ND; ++d) vf[0][d] = value(vq, 0, d);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8, vf[k % 2][d]), __builtin_bit_cast(bf8, p[k]), o[d], 0, 0, 0);
                    if (k < 3) {
                        vf[(k + 1) % 2][d] = value(vq, k + 1, d);
                    } else {
#pragma unroll
                        for (int n = d * kAhead / ND; n < (d + 1) * kAhead / ND; ++n) next_key(n);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
        }
        f16v zero;
#pragma unroll
        for (int i = 0; i < 16; ++i) zero[i] = 0.0f;
#pragma unroll
        for (int n = 0; n < 2 * NS; ++n) {
            s[n % 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8, kf[n % kAhead]), __builtin_bit_cast(bf8, q[n / 2]),
                                                               n < 2 ? zero : s[n % 2], 0, 0, 0);
            if (n + kAhead < 2 * NS) next_key(n + kAhead);
            between(n);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // The weights of a tile whose scores are in s, and what they change in m, l and o.
    auto soften = [&](uint32_t tile, uint32_t gone) {
        const int32_t a = (int32_t)(tile * kTile);
        if (gone || a < wlo_max || a + kTile > whi_min) {
            // in terms of the tokens' constants, so that only two values are kept
            const int32_t rl = lo - a - 4 * (int32_t)lh, rn = hi - lo;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    s[t][i] = (uint32_t)(32 * t + 8 * (i / 4) + i % 4 - rl) < (uint32_t)rn ? s[t][i] : -kInf;
            if (gone) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[t][i] = gone >> (2 * t + i / 8) & 1u ? -kInf : s[t][i];
            }
        }
        float mx = -kInf;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[t][i]);
        mx = max_halves(mx) * c;
        if (__any(mx > m + kSlack)) {
            const float nm = fmaxf(m, mx), base = nm == -kInf ? 0.0f : nm;
            const float f = __builtin_amdgcn_exp2f(m - base);
            m = nm;
            l *= f;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[d][i] *= f;
        }
        const float base = m == -kInf ? 0.0f : m;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[t][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][i], c, -base));
                l += s[t][i];
            }
        asm volatile("" : "+v"(l));      // here, not behind the matrix phase: s is to be free by then
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) p[k][i] = pack2(s[k / 2][8 * (k % 2) + 2 * i], s[k / 2][8 * (k % 2) + 2 * i + 1]);
    };
    if (threadIdx.x == 0) any_odd = 0;
    if (t0 < t1) {
        __syncthreads();
        // w1, w2: tiles i + 1, i + 2 (their loads are under way); the pieces of tile i without a page
        const Where w0 = where(t0);
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            load_k(w0, i);
            load_v(w0, i);
        }
        Where w1 = where(t0 + 1), w2 = where(t0 + 2);
        uint32_t gone0 = w0.gone;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            store_k(t0, i);
            store_v(t0, w0.gone, i);
            load_k(w1, i);
        }
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            store_k(t0 + 1, i);
            load_v(w1, i);
            load_k(w2, i);
        }
        __syncthreads();
        const bool behind = NW == 8 && wave >= NW / 2;
        if (behind) __syncthreads();
        products(t0 - 1, std::true_type{}, [](int) {});
        __syncthreads();
        for (uint32_t tile = t0; tile < t1; ++tile) {
            __builtin_amdgcn_sched_barrier(0);
            soften(tile, gone0);
            __builtin_amdgcn_sched_barrier(0);
            __syncthreads();
            // Every wave works on every tile: one that its rows do not see has weights of zero.
            // Behind the last tile, the scores are of whatever LDS holds and are not used.
            __builtin_amdgcn_s_setprio(1);
            // The tiles ahead, beside the products: what was read a step ago goes to LDS, where tile
            // i - 1's values and tile i's keys were last read before the barrier above; then the
            // next pieces are read.
            products(tile, std::false_type{}, [&](int n) {
                if (n < NL) {
                    store_v(tile + 1, w1.gone, n);
                    store_k(tile + 2, n);
                }
                if (n == NL) {
                    gone0 = w1.gone;
                    w1 = w2;
                    w2 = where(tile + 3);
                }
                if (n > NL && n <= 2 * NL) {
                    load_v(w1, n - NL - 1);
                    load_k(w2, n - NL - 1);
                }
            });
            __builtin_amdgcn_s_setprio(0);
            __syncthreads();
        }
        if (NW == 8 && !behind) __syncthreads();
        if (any_odd) {
            // the infinities and NaN that store_v left out, for the rows that see them
#pragma unroll 1
            for (int32_t tk = (int32_t)(t0 * kTile); tk < (int32_t)(t1 * kTile); ++tk) {
                const int32_t a = tk & ~(kTile - 1);
                if (!(a < lo_max || a + kTile > hi_min) || tk < lo_min || tk >= hi_max) continue;
                const uint32_t page = (uint32_t)table[tk >> g.c.log_page];
                if (page >= g.c.n_pages) continue;
                const bool see = tk >= lo && tk < hi;
                const uint8_t *row = vmem + (int64_t)page * g.c.v_page + (uint64_t)((uint32_t)tk & pmask) * g.c.v_token + 4 * lh * ES;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        u2 w;
                        if constexpr (DT == ZX_BF16) {
                            w = *reinterpret_cast<const u2 *>(row + 64 * d + 16 * i);
                        } else {
                            const uint32_t b = *reinterpret_cast<const uint32_t *>(row + 32 * d + 8 * i);
                            w = u2{fp8_pair<false>(b), fp8_pair<true>(b)};
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float x = __builtin_bit_cast(float, j % 2 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
                            o[d][4 * i + j] += see && !(__builtin_fabsf(x) < kInf) ? x : 0.0f;
                        }
                    }
            }
        }
    }

    if (!live) return;
    const bool mine = wr + lr < w9;              // (both lanes of a row are, or neither)
    l = sum_halves(l);
    if (nch == 1) {
        const float inv = l == 0.0f ? 0.0f : (g.c.v_scale ? g.c.v_scale[h] : 1.0f) / l;
        // A lane has channels 8 i + 4 lh .. + 3 of each 32; with the lane of the row's other half it trades four for
        // four, so that both write 16 bytes, next to each other.
        __bf16 *op = g.out.p + at * g.out.token + (int64_t)qh * g.out.head + 8 * lh;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                u4 y;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const auto r = __builtin_amdgcn_permlane32_swap(pack2(o[d][4 * i + 2 * j] * inv, o[d][4 * i + 2 * j + 1] * inv),
                                                                    pack2(o[d][4 * i + 4 + 2 * j] * inv, o[d][4 * i + 5 + 2 * j] * inv), false, false);
                    y[j] = (uint32_t)r[0];
                    y[2 + j] = (uint32_t)r[1];
                }
                if (mine) *reinterpret_cast<u4 *>(op + 32 * d + 8 * i) = y;
            }
        if (g.lse && mine && lh == 0) g.lse[at * g.q_heads + qh] = l == 0.0f ? -kInf : (m + log2f(l)) * kLn2;
    } else if (mine) {
        const uint64_t r = ((uint64_t)slot * g.c.heads + h) * ROWS + (row - row0);
        float *dst = g.part + r * D + 4 * lh;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<f4 *>(dst + 32 * d + 8 * i) = f4{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
        if (lh == 0) {
            g.stat[r * 2] = m;
            g.stat[r * 2 + 1] = l;
        }
    }
}

template <int DT, int D, int NW>
void launch(const ChunkPlan &p, const AttendArgs &g, hipStream_t stream)
{
    hipLaunchKernelGGL((k_chunk<DT, D, NW>), dim3(split_items(p.tiles, g) * g.c.heads), dim3(64 * NW), 0, stream, g);
    if (const uint32_t t = split_tiles(p.tiles, g)) hipLaunchKernelGGL((k_join<D, 32 * NW, kTile>), dim3(t * g.c.heads, 1, join_depth(t * g.c.heads, 32 * NW)), dim3(256), 0, stream, g);
}

template <int DT>
void by_size(uint32_t D, const ChunkPlan &p, const AttendArgs &g, hipStream_t stream)
{
    if (D == 256) launch<DT, 256, 4>(p, g, stream);
    else if (D == 128 && p.waves == 8) launch<DT, 128, 8>(p, g, stream);
    else if (D == 128) launch<DT, 128, 4>(p, g, stream);
    else if (p.waves == 8) launch<DT, 64, 8>(p, g, stream);
    else launch<DT, 64, 4>(p, g, stream);
}

}  // namespace

constexpr uint32_t kChunkRounds = 3;

ChunkPlan plan_chunk(uint64_t rows, uint32_t head_dim, uint32_t heads, uint64_t tokens, uint64_t seqs, uint64_t group, uint64_t cap, AttendArgs &g)
{
    ChunkPlan p{};
    const uint32_t wide = bound_tiles(tokens, seqs, group, 256);
    // Eight waves of 32 rows read a tile of keys half as often as four, four leave fewer CUs idle.  With 8 K/V heads of 128
    // channels and 4 heads on each, us at four / eight waves: 512 new tokens 23 / 26, 1024 37 / 40, 2048 68 / 71, 3 x 200 over
    // 3000 72 / 83, but 4096 181 / 169, 2 x 300 over 8000 127 / 117.  (Eight waves of 256 channels do not fit the registers.)
    p.waves = head_dim == 256 || rows <= 128 || ((uint64_t)wide * heads <= 256 && cap <= 4096) ? 4 : 8;
    p.tiles = p.waves == 8 ? wide : bound_tiles(tokens, seqs, group, 128);
    plan_split(p.tiles, ceil_div(p.waves == 8 || head_dim == 256 ? 256 : 512, heads), kChunkRounds, 8, 64, cap, kTile, g);
    return p;
}

void run_chunk(int dtype, uint32_t head_dim, const ChunkPlan &p, const AttendArgs &g, hipStream_t stream)
{
    if (dtype == ZX_BF16) by_size<ZX_BF16>(head_dim, p, g, stream);
    else by_size<ZX_FP8_E4M3FN>(head_dim, p, g, stream);
}

}  // namespace zxp
