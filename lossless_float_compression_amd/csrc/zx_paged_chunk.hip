// zx_paged_chunk.hip -- attention of many new tokens over a paged K/V cache: the tiled
// kernel.
//
// A workgroup takes 32 rows a wave (rows: the group's query heads for each new token)
// and goes over its tokens in tiles of 64.  K and V tiles are read from their pages into
// registers while the tile before is worked on, written to the other half of LDS as BF16,
// and shared by all waves: one barrier a tile.  With 32x32x16 products a lane has one query row;
// K is the left operand as it lies, V is read transposed (ds_read_b64_tr_b16), four
// tokens of 16 channels for 16 lanes at a time, in the order of tokens that the scores
// come out in, so weights go from one product to the next without leaving their lane.
// LDS rows are padded so that the 16 lanes of a read meet all 64 banks: keys by 16 bytes
// (a row of 16-byte pieces moves four banks on), values by 64 bytes (four rows of 32
// bytes, 16 banks apart).
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
    __shared__ uint32_t flag[2];                           // tile + 1 whose values hold an infinity or NaN

    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t lr = lane & 31u, lh = lane >> 5;
    const uint32_t G = g.group;
    const uint32_t h = blockIdx.x % g.c.heads, rest = blockIdx.x / g.c.heads;
    const uint32_t part = rest % g.target, item = rest / g.target;
    uint32_t seq, local, unused;
    Seq sv;
    if (!find_item(g.b, item, [&](const Seq &v) { return takes(g, v) ? div_up((uint32_t)v.nq * G, ROWS) : 0u; }, [](const Seq &) { return 0u; }, seq, sv,
                   local, unused))
        return;
    // the last row tiles see the most tokens: they go first
    const uint32_t all = (uint32_t)sv.nq * G, rt = div_up(all, ROWS) - 1 - local;
    const uint64_t slot = (uint64_t)(item - local + rt) * g.target + part;
    if (g.target > 1 && slot >= g.slots) return;       // overlapping sequences: more row tiles than there is room for
    const uint32_t row0 = rt * ROWS, row9 = row0 + ROWS < all ? row0 + ROWS : all;
    const int32_t pos0 = sv.kv - sv.nq;
    const int32_t pa = pos0 + (int32_t)(row0 / G), pb = pos0 + (int32_t)((row9 - 1) / G);
    const int32_t lo_min = first_seen(g, pa), lo_max = first_seen(g, pb), hi_min = end_seen(g, pa, sv.kv), hi_max = end_seen(g, pb, sv.kv);

    // this wave's rows (one lane's row past the last repeats it)
    const uint32_t w0 = row0 + wave * 32;
    const bool live = w0 < row9;
    const uint32_t w9 = w0 + 32 < row9 ? w0 + 32 : row9;
    const uint32_t row = live ? (w0 + lr < w9 ? w0 + lr : w9 - 1) : row9 - 1;
    const int32_t wa = pos0 + (int32_t)((live ? w0 : row9 - 1) / G), wb = pos0 + (int32_t)((live ? w9 - 1 : row9 - 1) / G);
    const int32_t wlo_min = first_seen(g, wa), wlo_max = first_seen(g, wb), whi_min = end_seen(g, wa, sv.kv), whi_max = end_seen(g, wb, sv.kv);
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
    const uint32_t per = div_up(t1 - t0, g.target);
    t0 += part * per;
    if (t0 > t1) t0 = t1;
    if (t1 > t0 + per) t1 = t0 + per;

    const int32_t *table = g.b.table + (uint64_t)seq * g.b.width;
    const uint32_t pmask = (1u << g.c.log_page) - 1u;
    // Pages of the tiles' 16-token pieces, 0xFFFFFFFF where there is none: lane i has the
    // piece i of the 16 tiles from `base` on (and, read ahead, of the 16 behind them), so a
    // tile's pages are a lane read and not a trip to memory.
    auto look = [&](uint32_t tile) {
        const uint32_t t = tile * kTile + 16 * lane;
        uint32_t id = 0xFFFFFFFFu;
        if (t < (uint32_t)sv.kv) id = (uint32_t)table[t >> g.c.log_page];
        return id;
    };
    auto vet = [&](uint32_t id, uint32_t tile) {
        if (id >= g.c.n_pages) {
            if (tile * kTile + 16 * lane < (uint32_t)sv.kv) report(g.b.err, ZX_E_CORRUPT);
            id = 0xFFFFFFFFu;
        }
        return id;
    };
    uint32_t base = t0, ids = vet(look(t0), t0), ahead = look(t0 + 16);
    auto pages = [&](uint32_t tile) {
        if (tile - base >= 16) {
            base += 16;
            ids = vet(ahead, base);
            ahead = look(base + 16);
        }
        u4 id;
#pragma unroll
        for (int i = 0; i < 4; ++i) id[i] = (uint32_t)__builtin_amdgcn_readlane((int)ids, (int)(4 * (tile - base)) + i);
        return id;
    };
    u4 kr[NL], vr[NL];
    auto load = [&](uint32_t tile, u4 id) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const uint32_t w = i * NT + wave * 64;          // first piece of the wave: its rows lie in one 16-token piece
            if (kTile * CPR % NT && w >= (uint32_t)(kTile * CPR)) continue;
            const uint32_t sub = w / CPR / 16;
            uint32_t p = id[0];
#pragma unroll
            for (int j = 1; j < 4; ++j) p = sub == (uint32_t)j ? id[j] : p;
            if (p == 0xFFFFFFFFu) p = 0;                    // any page: its tokens are not used
            const uint32_t tok = (tile * kTile + 16 * sub) & pmask;
            const uint32_t r = (w + lane) / CPR - 16 * sub, ch = ((w + lane) % CPR) * 16;
            const uint8_t *kb = g.c.k + (int64_t)p * g.c.k_page + (int64_t)h * g.c.k_head + (uint64_t)tok * g.c.k_token;
            const uint8_t *vb = g.c.v + (int64_t)p * g.c.v_page + (int64_t)h * g.c.v_head + (uint64_t)tok * g.c.v_token;
            kr[i] = *reinterpret_cast<const u4 *>(kb + (r * g.c.k_token + ch));
            vr[i] = *reinterpret_cast<const u4 *>(vb + (r * g.c.v_token + ch));
        }
    };
    auto put = [](uint8_t *dst, u4 x) {                     // 16 bytes of the cache as BF16
        if constexpr (DT == ZX_BF16) {
            *reinterpret_cast<u4 *>(dst) = x;
        } else {
            reinterpret_cast<u4 *>(dst)[0] = u4{fp8_pair<false>(x[0]), fp8_pair<true>(x[0]), fp8_pair<false>(x[1]), fp8_pair<true>(x[1])};
            reinterpret_cast<u4 *>(dst)[1] = u4{fp8_pair<false>(x[2]), fp8_pair<true>(x[2]), fp8_pair<false>(x[3]), fp8_pair<true>(x[3])};
        }
    };
    auto store = [&](uint32_t tile, uint32_t buf, u4 id) {
        const int32_t a = (int32_t)(tile * kTile);
        const bool gone = id[0] == 0xFFFFFFFFu || id[1] == 0xFFFFFFFFu || id[2] == 0xFFFFFFFFu || id[3] == 0xFFFFFFFFu;
        const bool edge = gone || a < lo_min || a + kTile > hi_max;      // some token that no row sees
        const bool mixed = a < lo_max || a + kTile > hi_min;             // some token that some rows do not see
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const uint32_t w = i * NT + wave * 64;
            if (kTile * CPR % NT && w >= (uint32_t)(kTile * CPR)) continue;
            const uint32_t r = (w + lane) / CPR, ch = ((w + lane) % CPR) * (32 / ES);
            if (edge) {
                const uint32_t sub = w / CPR / 16;
                uint32_t p = id[0];
#pragma unroll
                for (int j = 1; j < 4; ++j) p = sub == (uint32_t)j ? id[j] : p;
                const int32_t t = a + (int32_t)r;
                if (p == 0xFFFFFFFFu || t < lo_min || t >= hi_max) vr[i] = u4{0, 0, 0, 0};
            }
            put(kl[buf] + r * KS + ch, kr[i]);
            put(vl[buf] + r * VS + ch, vr[i]);
            if (mixed) {
                bool odd = false;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (DT == ZX_BF16) odd = odd || odd_pair(vr[i][j]);
                    else odd = odd || odd_pair(fp8_pair<false>(vr[i][j])) || odd_pair(fp8_pair<true>(vr[i][j]));
                }
                if (odd) flag[buf] = tile + 1;
            }
        }
    };

    float m = -kInf, l = 0.0f;
    f16v o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
    const float c = g.scale * (g.c.k_scale ? g.c.k_scale[h] : 1.0f);

    if (threadIdx.x < 2) flag[threadIdx.x] = 0;
    __syncthreads();
    u4 here = {0, 0, 0, 0}, next = here;
    if (t0 < t1) {
        here = pages(t0);
        load(t0, here);
        next = pages(t0 + 1);
        store(t0, 0, here);
    }
    for (uint32_t tile = t0; tile < t1; ++tile) {
        const uint32_t buf = (tile - t0) & 1u;
        const bool more = tile + 1 < t1;
        __syncthreads();
        if (more) load(tile + 1, next);
        __builtin_amdgcn_sched_barrier(0);
        // An infinity or NaN in the values of a tile that only some rows see in full: zero
        // times it would reach the others.  It is taken out of the tile, kept in the other half
        // (free until this tile is done), and added afterwards to the rows that see it.
        const bool odd = flag[buf] == tile + 1;
        if (odd) {
            for (uint32_t i = threadIdx.x; i < kTile * D / 8; i += NT) {
                const uint32_t at8 = (i / (D / 8)) * VS + (i % (D / 8)) * 16;
                u4 x = *reinterpret_cast<const u4 *>(vl[buf] + at8);
                *reinterpret_cast<u4 *>(vl[buf ^ 1u] + at8) = x;
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = tame_pair(x[j]);
                *reinterpret_cast<u4 *>(vl[buf] + at8) = x;
            }
            __syncthreads();
        }
        const int32_t a = (int32_t)(tile * kTile);
        if (live && a < whi_max && a + kTile > wlo_min) {
            f16v s[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int i = 0; i < 16; ++i) s[t][i] = 0.0f;
                const uint8_t *kp = kl[buf] + (32 * t + lr) * KS + 16 * lh;
#pragma unroll
                for (int j = 0; j < NS; ++j)
                    s[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8, *reinterpret_cast<const u4 *>(kp + 32 * j)),
                                                                   __builtin_bit_cast(bf8, q[j]), s[t], 0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            // register i of tile t: token 32 t + 8 (i / 4) + 4 lh + i % 4
            const bool gone = here[0] == 0xFFFFFFFFu || here[1] == 0xFFFFFFFFu || here[2] == 0xFFFFFFFFu || here[3] == 0xFFFFFFFFu;
            const bool mixed = gone || a < wlo_max || a + kTile > whi_min;
            float mx = -kInf;
            if (mixed) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int32_t tk = a + 32 * t + 8 * (i / 4) + 4 * (int32_t)lh + i % 4;
                        const bool in = tk >= lo && tk < hi && here[2 * t + i / 8] != 0xFFFFFFFFu;
                        s[t][i] = in ? s[t][i] : -kInf;
                    }
            }
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
            u4 p[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) p[k][i] = pack2(s[k / 2][8 * (k % 2) + 2 * i], s[k / 2][8 * (k % 2) + 2 * i + 1]);

            __builtin_amdgcn_sched_barrier(0);
            typedef __attribute__((address_space(3))) const uint8_t *lds_ptr;
            const lds_ptr vp = (lds_ptr)vl[buf] + (4 * lh + (lane & 15u) / 4) * VS + ((lane >> 4) & 1u) * 32 + (lane & 3u) * 8;
            auto value = [](lds_ptr vp, int k, int d) {
                typedef short s4 __attribute__((ext_vector_type(4)));
                typedef __attribute__((address_space(3))) s4 *lp;
                const s4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(vp + (16 * k) * VS + 64 * d));
                const s4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(vp + (16 * k + 8) * VS + 64 * d));
                const u2 xu = __builtin_bit_cast(u2, x), yu = __builtin_bit_cast(u2, y);
                return u4{xu[0], xu[1], yu[0], yu[1]};
            };
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int d = 0; d < ND; ++d)
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8, value(vp, k, d)), __builtin_bit_cast(bf8, p[k]), o[d], 0, 0, 0);
            if (odd) {
                // the infinities and NaN that were taken out, for the rows that see them
#pragma unroll 1
                for (int t = 0; t < kTile; ++t) {
                    const bool see = a + t >= lo && a + t < hi;
                    const uint8_t *vo = vl[buf ^ 1u] + t * VS + 8 * lh;
#pragma unroll
                    for (int d = 0; d < ND; ++d)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const u2 w = *reinterpret_cast<const u2 *>(vo + 64 * d + 16 * i);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float x = __builtin_bit_cast(float, j % 2 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
                                o[d][4 * i + j] += see && !(__builtin_fabsf(x) < kInf) ? x : 0.0f;
                            }
                        }
                }
            }
        }
        if (odd) __syncthreads();
        if (more) {
            store(tile + 1, buf ^ 1u, next);
            here = next;
            next = pages(tile + 2);
        }
    }

    if (!live || w0 + lr >= w9) return;
    l = sum_halves(l);
    if (g.target == 1) {
        const float inv = l == 0.0f ? 0.0f : (g.c.v_scale ? g.c.v_scale[h] : 1.0f) / l;
        __bf16 *op = g.out.p + at * g.out.token + (int64_t)qh * g.out.head + 4 * lh;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<u2 *>(op + 32 * d + 8 * i) =
                    u2{pack2(o[d][4 * i] * inv, o[d][4 * i + 1] * inv), pack2(o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv)};
        if (g.lse && lh == 0) g.lse[at * g.q_heads + qh] = l == 0.0f ? -kInf : (m + log2f(l)) * kLn2;
    } else {
        const uint64_t r = (slot * g.c.heads + h) * ROWS + (row - row0);
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
void launch(uint32_t items, uint32_t split, const AttendArgs &g, hipStream_t stream)
{
    hipLaunchKernelGGL((k_chunk<DT, D, NW>), dim3(items * split * g.c.heads), dim3(64 * NW), 0, stream, g);
    if (split > 1) hipLaunchKernelGGL((k_join<D, 32 * NW, JOIN_CHUNK>), dim3(items * g.c.heads, 1, 16), dim3(256), 0, stream, g);
}

template <int DT>
void by_size(uint32_t D, uint32_t waves, uint32_t items, uint32_t split, const AttendArgs &g, hipStream_t stream)
{
    if (D == 256) launch<DT, 256, 4>(items, split, g, stream);
    else if (D == 128 && waves == 8) launch<DT, 128, 8>(items, split, g, stream);
    else if (D == 128) launch<DT, 128, 4>(items, split, g, stream);
    else if (waves == 8) launch<DT, 64, 8>(items, split, g, stream);
    else launch<DT, 64, 4>(items, split, g, stream);
}

}  // namespace

uint32_t chunk_waves(uint64_t rows, uint32_t head_dim) { return head_dim == 256 || rows <= 128 ? 4 : 8; }

void run_chunk(int dtype, uint32_t head_dim, uint32_t waves, uint32_t items, uint32_t split, const AttendArgs &g, hipStream_t stream)
{
    if (dtype == ZX_BF16) by_size<ZX_BF16>(head_dim, waves, items, split, g, stream);
    else by_size<ZX_FP8_E4M3FN>(head_dim, waves, items, split, g, stream);
}

}  // namespace zxp
