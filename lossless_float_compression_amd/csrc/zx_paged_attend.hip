// zx_paged_attend.hip -- attention of new tokens over a paged K/V cache.
//
// For query row r and the tokens t it sees: s_t = scale q.k_t, o = sum e^(s_t - m) v_t /
// sum e^(s_t - m).  Both kernels go over the tokens once, with the running maximum m and
// sum l of a softmax, in powers of two (s_t log2 e).  The rows of one K/V head are its
// group's query heads for each new token, r = token * group + head, so a token's keys and
// values are read once for the whole group.
//
// Scores are computed transposed, S^T = K Q^T, and the output too, O^T = V^T P^T: in the
// matrix instruction's result layout a lane then holds one query row, so the row's
// statistics are lane-local values, and a lane's scores are, in their order, the operand
// that the second product wants (any order of tokens will do there, if the values' order
// is the same).
//
//   k_rows   few rows (single tokens, groups of a few), or little to read: bound by the bytes of K and V.
//            Every wave reads its own tokens straight into the operand registers, with no
//            LDS in the loop; the waves and the workgroups that share a row are joined at the end.
//            64 single tokens over 5 .. 16384 tokens, BF16: 262 us, 5.4 TB/s; 4 over 131072, E4M3: 188 us, 5.7 TB/s
//            (a large copy: 5.15); one over 1000: 7.6 us and 4 for the join, bound by the launches and one
//            trip to memory after the other (lengths, page ids, keys).
//   k_chunk  many rows: bound by the matrix units and the softmax beside them.  Tiles of K and V in LDS serve 32 rows a wave.
//            4096 new tokens 151 us, 910 TFLOP/s; 2 x 777 over 32768 620 us, 870 TFLOP/s (a large matrix product: 1140 to 1370).
//   k_join   adds up what the workgroups of one row left.
//
// Roundings: weights go into the second product as BF16, the matrix unit's type: up to 2^-8 of each, either way, so
// an output is off by at most 2^-8 of sum w |v| for it beside the 2^-8 of its own rounding to BF16 (rms against 64 bits over the
// cases timed here: 0.0023 of the output, 0.0016 with weights of 32 bits).  Weights of 32 bits would take two products
// and halve the rate.  Scores, maxima, the sums of the weights (of the unrounded ones) and products are 32-bit.
#include "zx_paged_attend.h"

namespace zxp {
namespace {

// ---------------------------------------------------------------- few rows

// An infinity or NaN in a dword of values becomes zero; whether there was one.
template <int DT>
__device__ __forceinline__ bool tame(uint32_t &w)
{
    if constexpr (DT == ZX_BF16) {
        const bool odd = odd_pair(w);
        w = tame_pair(w);
        return odd;
    } else {                                     // E4M3 has no infinity; NaN is 0x7F in the low seven bits
        const uint32_t m = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
        w &= ~((m >> 7) * 0xFFu);
        return m != 0;
    }
}

// Waves of one SIMD that k_rows leaves registers for.
constexpr int rows_waves(int d, int mt) { return d == 256 ? 1 : mt == 3 ? 2 : mt == 2 ? (d == 64 ? 3 : 2) : d == 64 ? 4 : 3; }

template <int DT, int D, int MT, bool LIST, int NW>
__global__ __launch_bounds__(64 * NW, rows_waves(D, MT) * 4 >= NW ? rows_waves(D, MT) : NW / 4) void k_rows(AttendArgs g)
{
    constexpr int ROWS = 16 * MT;
    constexpr uint32_t kPieces = 2 * NW;             // 16-token pieces of a step
    constexpr int ES = DT == ZX_BF16 ? 2 : 1;
    constexpr int NK = D / 32;                       // matrix steps over the channels
    constexpr int VW = D < 128 ? D / 16 : 8;         // value channels a lane reads of one token
    constexpr int NP = D / (16 * VW);                // such pieces of a row
    constexpr int VD = VW * ES / 4;                  // dwords of one
    constexpr int KL = D * 16 * ES / 64 / 16;        // 16-byte loads a lane makes of 16 keys
    constexpr int OS = D + 4;                        // LDS row of the join, in floats
    __shared__ __align__(16) float ods[NW * 16 * OS];
    __shared__ float mls[2][MT][NW][16];

    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t lr = lane & 15u, lq = lane >> 4;
    const uint32_t h = blockIdx.x % g.c.heads, item = blockIdx.x / g.c.heads;
    const uint32_t G = g.group;

    // which rows, which tokens
    uint32_t seq, rt, part, nch, chunk = 1, piece_slot;
    Seq sv;
    if constexpr (LIST) {
        const uint32_t tiles = div_up(G, ROWS);
        uint32_t local, unused;
        nch = g.pieces;
        if (!find_item(g.b, item, [&](const Seq &v) { return (uint32_t)v.nq * tiles * nch; }, [](const Seq &) { return 0u; }, seq, sv, local, unused)) return;
        rt = local / nch;
        part = local % nch;
        piece_slot = item;
    } else {
        chunk = chunk_steps<ROWS, 32 * NW>(g);
        if (!find_piece<ROWS, 32 * NW>(g, item, chunk, seq, sv, rt, part, nch, piece_slot)) return;
    }
    uint32_t row0, nrows, tok0;                      // rows row0 .. of the token list starting at tok0
    if constexpr (LIST) {
        const uint32_t tiles = div_up(G, ROWS);
        tok0 = rt / tiles;
        row0 = (rt % tiles) * ROWS;
        nrows = G - row0 < (uint32_t)ROWS ? G - row0 : (uint32_t)ROWS;
    } else {
        tok0 = 0;
        row0 = rt * ROWS;
        const uint32_t all = (uint32_t)sv.nq * G;
        nrows = all - row0 < (uint32_t)ROWS ? all - row0 : (uint32_t)ROWS;
    }

    // each lane's rows: what they see, and their queries in the operand's layout.  Rows
    // past the last one repeat it.
    int32_t lo[MT], hi[MT];
    u4 q[MT][NK];
    const int32_t pos0 = sv.kv - sv.nq;
    int32_t lo_min = 0x7FFFFFFF, lo_max = 0, hi_min = 0x7FFFFFFF, hi_max = 0;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        uint32_t r = t * 16 + lr;
        r = row0 + (r < nrows ? r : nrows - 1);
        const uint32_t tok = tok0 + r / G, gh = r % G;
        const int32_t p = pos0 + (int32_t)tok;
        lo[t] = first_seen(g, p);
        hi[t] = end_seen(g, p, sv.kv);
        const __bf16 *qp = g.q.p + (int64_t)(sv.q0 + (int32_t)tok) * g.q.token + (int64_t)(h * G + gh) * g.q.head;
#pragma unroll
        for (int s = 0; s < NK; ++s) {
            // BF16 keys: step s, lane quarter lq holds channels 32 s + 8 lq ..; E4M3 keys come 16
            // channels a load: 64 (s / 2) + 16 lq + 8 (s % 2) ..
            const int ch = DT == ZX_BF16 ? 32 * s + 8 * (int)lq : 64 * (s / 2) + 16 * (int)lq + 8 * (s % 2);
            q[t][s] = *reinterpret_cast<const u4 *>(qp + ch);
        }
    }
    {
        const uint32_t ta = tok0 + row0 / G, tb = tok0 + (row0 + nrows - 1) / G;   // first and last token of the rows
        const int32_t pa = pos0 + (int32_t)ta, pb = pos0 + (int32_t)tb;
        lo_min = first_seen(g, pa);
        lo_max = first_seen(g, pb);
        hi_min = end_seen(g, pa, sv.kv);
        hi_max = end_seen(g, pb, sv.kv);
    }

    // the pieces of 16 tokens this workgroup reads: u0 .. u1 - 1
    const int32_t *table = g.b.table + (uint64_t)seq * g.b.width;
    const int32_t *list = nullptr;
    uint32_t u0, u1;
    const uint32_t lb = g.c.log_block;
    if constexpr (LIST) {
        list = g.blocks + ((uint64_t)(sv.q0 + (int32_t)tok0) * g.c.heads + h) * g.n_blocks;
        uint32_t n = 0;
        while (n < g.n_blocks) {
            const uint64_t neg = __ballot(n + lane >= g.n_blocks || list[n + lane < g.n_blocks ? n + lane : 0] < 0);
            if (neg) {
                n += (uint32_t)__builtin_ctzll(neg);
                break;
            }
            n += 64;
        }
        const uint32_t steps = div_up(n << (lb - 4), kPieces), per = div_up(steps, nch);
        u0 = part * per * kPieces;
        u1 = u0 + per * kPieces;
        if (u1 > n << (lb - 4)) u1 = n << (lb - 4);
    } else {
        const uint32_t base = (uint32_t)(first_seen(g, pos0) >> 4);
        u0 = base;
        u1 = 0x7FFFFFFFu;
        if (nch > 1) {
            u0 += part * chunk * kPieces;
            u1 = u0 + chunk * kPieces;
        }
        if (u0 < (uint32_t)(lo_min >> 4)) u0 = (uint32_t)(lo_min >> 4);
        if (u1 > (uint32_t)((hi_max + 15) >> 4)) u1 = (uint32_t)((hi_max + 15) >> 4);
    }

    // Where the wave's pieces lie: lane 2 i + a has piece a of the wave's step i, 32 steps at a
    // time, as addresses (page 0, and no bit in `held`, where there is no page).  A step's
    // addresses are then lane reads, not trips to memory and 64-bit products.
    const uint32_t pmask = (1u << g.c.log_page) - 1u;
    uint64_t kat, vat, held;
    int32_t first_token;
    auto settle = [&](uint32_t u) {
        u += kPieces * (lane >> 1) + (lane & 1u);
        bool there = u < u1;
        uint32_t t = u << 4;
        if constexpr (LIST) {
            const uint32_t e = there ? (uint32_t)list[u >> (lb - 4)] : 0u;
            there = there && e <= (uint32_t)sv.kv >> lb;        // entries past the sequence see nothing
            t = (e << lb) + ((u & ((1u << (lb - 4)) - 1u)) << 4);
            there = there && t < (uint32_t)sv.kv;
        }
        uint32_t page = 0;
        if (there) {
            page = (uint32_t)table[t >> g.c.log_page];
            if (page >= g.c.n_pages) {
                report(g.b.err, ZX_E_CORRUPT);
                page = 0;
                there = false;
            }
        }
        const uint64_t at = t & pmask;
        kat = (uint64_t)g.c.k + (uint64_t)((int64_t)page * g.c.k_page + (int64_t)h * g.c.k_head) + at * g.c.k_token;
        vat = (uint64_t)g.c.v + (uint64_t)((int64_t)page * g.c.v_page + (int64_t)h * g.c.v_head) + at * g.c.v_token;
        first_token = (int32_t)t;
        held = __ballot(there);
    };
    auto lane64 = [](uint64_t x, uint32_t l) {
        return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, (int)l) |
               (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(x >> 32), (int)l) << 32;
    };
    const uint32_t koff = lr * g.c.k_token + lq * 16u;
    const uint32_t voff = lq * 4u * g.c.v_token + lr * (VW * ES);

    u4 kreg[2][KL];
    uint32_t vreg[8][NP][VD];
    auto load_k = [&](uint32_t i) {              // step i of the 32
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const global_u1 *b = (const global_u1 *)lane64(kat, 2 * i + a) + koff;
#pragma unroll
            for (int e = 0; e < KL; ++e) kreg[a][e] = *(const global_u4 *)(b + 64 * e);
        }
    };
    auto load_v = [&](uint32_t i) {
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const global_u1 *b = (const global_u1 *)lane64(vat, 2 * i + a);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int n = 0; n < NP; ++n) {
                    const global_u1 *s = b + (voff + (uint32_t)e * g.c.v_token) + n * (16 * VW * ES);
                    if constexpr (VD == 4) {
                        const u4 x = *(const global_u4 *)s;
#pragma unroll
                        for (int w = 0; w < 4; ++w) vreg[4 * a + e][n][w] = x[w];
                    } else if constexpr (VD == 2) {
                        const u2 x = *(const global_u2 *)s;
                        vreg[4 * a + e][n][0] = x[0];
                        vreg[4 * a + e][n][1] = x[1];
                    } else {
                        vreg[4 * a + e][n][0] = *(const global_u32 *)s;
                    }
                }
        }
    };

    float m[MT], l[MT];
    f4 o[MT][NP][VW];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        m[t] = -kInf;
        l[t] = 0.0f;
#pragma unroll
        for (int n = 0; n < NP; ++n)
#pragma unroll
            for (int j = 0; j < VW; ++j) o[t][n][j] = f4{0, 0, 0, 0};
    }
    const float c = g.scale * (g.c.k_scale ? g.c.k_scale[h] : 1.0f);

    uint32_t u = u0 + 2 * wave, step = 0;
    bool any_odd = false;                        // values with infinities or NaN were left out
    if (u < u1) {
        settle(u);
        load_k(0);
        load_v(0);
    }
    for (; u < u1; u += kPieces) {
        const int32_t token[2] = {__builtin_amdgcn_readlane(first_token, (int)(2 * step)), __builtin_amdgcn_readlane(first_token, (int)(2 * step + 1))};
        const bool there[2] = {(held >> (2 * step) & 1u) != 0, (held >> (2 * step + 1) & 1u) != 0};
        // scores: 16 tokens x 16 rows a tile; a lane has row lr, tokens 4 lq .. 4 lq + 3 of each piece
        f4 s[MT][2];
#pragma unroll
        for (int a = 0; a < 2; ++a) {
#pragma unroll
            for (int t = 0; t < MT; ++t) s[t][a] = f4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                u4 kk;
                if constexpr (DT == ZX_BF16) {
                    kk = kreg[a][i];
                } else {
                    const uint32_t w0 = kreg[a][i / 2][2 * (i % 2)], w1 = kreg[a][i / 2][2 * (i % 2) + 1];
                    kk = u4{fp8_pair<false>(w0), fp8_pair<true>(w0), fp8_pair<false>(w1), fp8_pair<true>(w1)};
                }
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    s[t][a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, kk), __builtin_bit_cast(bf8, q[t][i]), s[t][a], 0, 0, 0);
            }
        }
        const bool more = u + kPieces < u1;
        if (more) {
            step = (step + 1) & 31u;
            if (step == 0) settle(u + kPieces);
            load_k(step);
        }

        // does any row not see any of these tokens?
        bool part_seen = false;
#pragma unroll
        for (int a = 0; a < 2; ++a)
            part_seen = part_seen || !there[a] || token[a] < lo_max || token[a] + 16 > hi_min;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            float mx = -kInf;
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x = s[t][a][i] * c;
                    if (part_seen) {
                        const int32_t tk = token[a] + 4 * (int32_t)lq + i;
                        x = there[a] && tk >= lo[t] && tk < hi[t] ? x : -kInf;
                    }
                    s[t][a][i] = x;
                    mx = fmaxf(mx, x);
                }
            mx = max_quarters(mx);
            if (__any(mx > m[t] + kSlack)) {
                const float nm = fmaxf(m[t], mx), base = nm == -kInf ? 0.0f : nm;
                const float f = __builtin_amdgcn_exp2f(m[t] - base);
                m[t] = nm;
                l[t] *= f;
#pragma unroll
                for (int n = 0; n < NP; ++n)
#pragma unroll
                    for (int j = 0; j < VW; ++j) o[t][n][j] *= f;
            }
            const float base = m[t] == -kInf ? 0.0f : m[t];
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[t][a][i] = __builtin_amdgcn_exp2f(s[t][a][i] - base);
                    l[t] += s[t][a][i];
                }
        }
        // weights as the second product's operand: tokens 4 lq .. + 3 of both pieces, as the values have them
        u4 p[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t)
            p[t] = u4{pack2(s[t][0][0], s[t][0][1]), pack2(s[t][0][2], s[t][0][3]), pack2(s[t][1][0], s[t][1][1]), pack2(s[t][1][2], s[t][1][3])};

        // values that no row sees are not there (pages hold anything behind a sequence's end)
        if (part_seen) {
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int32_t tk = token[a] + 4 * (int32_t)lq + i;
                    const bool seen = there[a] && tk >= lo_min && tk < hi_max;
#pragma unroll
                    for (int n = 0; n < NP; ++n)
#pragma unroll
                        for (int w = 0; w < VD; ++w) vreg[4 * a + i][n][w] = seen ? vreg[4 * a + i][n][w] : 0u;
                }
            if (lo_min != lo_max || hi_min != hi_max) {
                // An infinity or NaN that only some rows see: zero times it would reach the
                // others.  It is left out here and added at the end to the rows that see it.
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int n = 0; n < NP; ++n)
#pragma unroll
                        for (int w = 0; w < VD; ++w) any_odd = tame<DT>(vreg[i][n][w]) || any_odd;
            }
        }
#pragma unroll
        for (int n = 0; n < NP; ++n) {
#pragma unroll
            for (int w = 0; w < VW / 2; ++w) {
                // channel pair w of eight tokens, as BF16 pairs of channels ...
                uint32_t x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if constexpr (DT == ZX_BF16) x[i] = vreg[i][n][w];
                    else x[i] = w % 2 ? fp8_pair<true>(vreg[i][n][w / 2]) : fp8_pair<false>(vreg[i][n][w / 2]);
                }
                // ... and turned into pairs of tokens
                u4 v0, v1;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v0[i] = __builtin_amdgcn_perm(x[2 * i + 1], x[2 * i], 0x05040100u);
                    v1[i] = __builtin_amdgcn_perm(x[2 * i + 1], x[2 * i], 0x07060302u);
                }
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    o[t][n][2 * w] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, v0), __builtin_bit_cast(bf8, p[t]), o[t][n][2 * w], 0, 0, 0);
                    o[t][n][2 * w + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, v1), __builtin_bit_cast(bf8, p[t]), o[t][n][2 * w + 1], 0, 0, 0);
                }
            }
        }
        if (more) load_v(step);
    }
    if (__any(any_odd)) {
        // the infinities and NaN that were left out, for the rows that see them
#pragma unroll 1
        for (u = u0 + 2 * wave, step = 0; u < u1; u += kPieces, step = (step + 1) & 31u) {
            if (step == 0) settle(u);
#pragma unroll 1
            for (uint32_t e = 0; e < 32; ++e) {
                const uint32_t at = 2 * step + (e >> 4);
                const int32_t tk = __builtin_amdgcn_readlane(first_token, (int)at) + (int32_t)(e & 15u);
                if (!(held >> at & 1u) || tk < lo_min || tk >= hi_max) continue;
                const uint8_t *b = (const uint8_t *)lane64(vat, at) + (uint64_t)(e & 15u) * g.c.v_token;
#pragma unroll
                for (int n = 0; n < NP; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < VW; ++j) {
                            const uint32_t ch = n * 16 * VW + (4 * lq + i) * VW + j;
                            float x;
                            if constexpr (DT == ZX_BF16) x = (float)reinterpret_cast<const __bf16 *>(b)[ch];
                            else x = __builtin_bit_cast(float, fp8_pair<false>(b[ch]) << 16);
                            if (__builtin_fabsf(x) < kInf) x = 0.0f;
#pragma unroll
                            for (int t = 0; t < MT; ++t) o[t][n][j][i] += tk >= lo[t] && tk < hi[t] ? x : 0.0f;
                        }
            }
        }
    }

    // join the waves, 16 rows at a time
    const float vs = g.c.v_scale ? g.c.v_scale[h] : 1.0f;
    const uint64_t slot = ((uint64_t)piece_slot * g.c.heads + h) * ROWS;
    // (all statistics first: what stays in registers across the loops below is then the sums alone, which lie
    // in accumulation registers and are not moved about)
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        l[t] = sum_quarters(l[t]);
        if (lq == 0) {
            mls[0][t][wave][lr] = m[t];
            mls[1][t][wave][lr] = l[t];
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        if (t) __syncthreads();
        // a lane has, of row lr, channels n * 16 VW + (4 lq + i) VW + j
        float *dst = ods + (wave * 16 + lr) * OS;
#pragma unroll
        for (int n = 0; n < NP; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < VW; j += 4)
                    *reinterpret_cast<f4 *>(dst + n * 16 * VW + (4 * lq + i) * VW + j) = f4{o[t][n][j][i], o[t][n][j + 1][i], o[t][n][j + 2][i], o[t][n][j + 3][i]};
        __syncthreads();
        for (uint32_t e = threadIdx.x; e < 16 * (D / 8); e += 64 * NW) {
            const uint32_t r = e / (D / 8), ch = (e % (D / 8)) * 8;
            const uint32_t row = t * 16 + r;
            if (row >= nrows) continue;
            float mm = -kInf;
#pragma unroll
            for (int w = 0; w < NW; ++w) mm = fmaxf(mm, mls[0][t][w][r]);
            const float base = mm == -kInf ? 0.0f : mm;
            float ll = 0.0f, x[8] = {};
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float f = __builtin_amdgcn_exp2f(mls[0][t][w][r] - base);
                ll += mls[1][t][w][r] * f;
                const float *src = ods + (w * 16 + r) * OS + ch;
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] += src[i] * f;
            }
            if (nch == 1) {
                const uint32_t tok = tok0 + (row0 + row) / G, gh = (row0 + row) % G;
                const int64_t at = sv.q0 + (int32_t)tok;
                const float inv = ll == 0.0f ? 0.0f : vs / ll;
                bf8 y;
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = (__bf16)(x[i] * inv);
                *reinterpret_cast<bf8 *>(g.out.p + at * g.out.token + (int64_t)(h * G + gh) * g.out.head + ch) = y;
                if (g.lse && ch == 0) g.lse[at * g.q_heads + h * G + gh] = ll == 0.0f ? -kInf : (mm + log2f(ll)) * kLn2;
            } else {
                float *dst2 = g.part + (slot + row) * D + ch;
                reinterpret_cast<f4 *>(dst2)[0] = f4{x[0], x[1], x[2], x[3]};
                reinterpret_cast<f4 *>(dst2)[1] = f4{x[4], x[5], x[6], x[7]};
                if (ch == 0) {
                    g.stat[(slot + row) * 2] = mm;
                    g.stat[(slot + row) * 2 + 1] = ll;
                }
            }
        }
    }
}

// ---------------------------------------------------------------- host

struct Plan {
    bool rows, chunk;                // which kernels run
    AttendArgs r, c;                 // their arguments: how sequences are split
    uint32_t mt, rows_items, rows_join, rows_max;   // rows_join: row tiles that may be split (0: none)
    bool wide;                       // k_rows with eight waves, and nothing split
    ChunkPlan cp;
    uint64_t rows_part, rows_stat, chunk_part, chunk_stat, bytes;   // offsets into the workspace
};

constexpr uint32_t kFewRows = 64;    // rows of a sequence that k_rows takes in any case
// With a row tile of its own for every CU at most (every second with 256 channels, whose workgroups fill a CU), and so many
// tokens met by all of them together, k_rows takes sequences of any number of rows: without tiles in LDS to fill it is done
// sooner, until the keys and values that its row tiles read again outweigh that.  Us with k_rows / k_chunk (row tiles, tokens
// met), 128 channels: 20 new tokens of 32 heads over 2000 (24, 48,000) 15 / 25, 100 of 10 heads over 6000 (32, 192,000) 25 / 32, 4 x 50 of 32
// heads over 1000 (224, 224,000) 18 / 28, but 4 x 64 (256, 256,000) 32 / 29, 100 of 32 heads over 6000 (104, 624,000) 44 / 34, a prompt
// of 256 (256, 66,000) 18 / 15; 64 channels, 28 heads: 4 x 60 over 1000 (144, 144,000) 19 / 21, 6 x 50 (192, 192,000) 23 / 22, 8 x 30 over 3000 (160,
// 480,000) 28 / 25; 256 channels, 8 heads: 400 over 1500 (100, 150,000) 37 / 48, 8 x 30 over 3000 (64, 192,000) 39 / 45, 3 x 169 over 1283
// (132, 169,000) 60 / 43, 8 x 64 over 3000 (128, 384,000) 66 / 51.
constexpr uint64_t most_row_tiles(uint32_t d) { return d == 256 ? 128 : 255; }
constexpr uint64_t most_tile_tokens(uint32_t d) { return d == 64 ? 160000 : 250000; }
// Up to so many bytes of keys and values a row tile, one workgroup of eight waves reads them all, and there is no
// second launch to join pieces (about 4 us).  A CU draws about 57 bytes a nanosecond, so with few row tiles
// pieces on several CUs are sooner read from twice 128 KB on; with a workgroup for half the CUs or more, later.
// Us a call in one launch / in pieces, 8 K/V heads of 128 channels, BF16: one token over 250 8.0 / 11.9, over 500
// 9.8 / 11.9, over 1000 14.4 / 11.9; 16 tokens, each over its 700, 13.4 / 16.6, over 16 blocks of 64 16.2 / 19.7,
// but of lengths from 62 to 1000 15.6 / 14.3; 123 tokens, 2 heads, over 40 blocks of 32, E4M3, 13.9 / 21.3.
constexpr uint64_t wide_bytes(uint64_t tiles) { return tiles < 128 ? 256 << 10 : 512 << 10; }
// Workgroups of k_rows that the card holds at a time.
constexpr uint32_t rows_groups(uint32_t d, uint32_t mt) { return 256u * (uint32_t)rows_waves((int)d, (int)mt); }

Plan make_plan(const zx_paged_cache *c, const zx_paged_batch *b, uint32_t n, uint32_t q_heads, uint32_t n_blocks, const AttendArgs &g)
{
    Plan p{};
    p.r = p.c = g;
    const uint32_t G = q_heads / c->kv_heads, H = c->kv_heads, D = c->head_dim, es = c->dtype == ZX_BF16 ? 2 : 1;
    const uint64_t room = (uint64_t)b->table_width * c->page_tokens, all = b->max_kv < room ? b->max_kv : room;
    const uint32_t max_q = b->max_q < n ? b->max_q : n;
    // tokens that the rows of one sequence can see
    const uint64_t near = (uint64_t)g.window + max_q + 15, cap = g.window && near < all ? near : all;
    const uint32_t seqs = b->n_seqs < n ? b->n_seqs : n;      // sequences with new tokens
    const uint64_t most = (uint64_t)max_q * G < 1 ? 1 : (uint64_t)max_q * G;
    auto area = [&](uint64_t bytes) {
        const uint64_t at = p.bytes;
        p.bytes += (bytes + 255) & ~255ull;
        return at;
    };
    uint64_t rows_slots = 0;
    if (n_blocks) {
        p.rows = true;
        p.mt = 1;
        const uint32_t tiles = n * ceil_div(G, 16), steps = ceil_div((uint64_t)n_blocks * c->block_tokens, kStep);
        const uint32_t s = ceil_div(rows_groups(D, 1), (uint64_t)tiles * H);
        p.wide = D <= 128 && s > 1 && 2 * (uint64_t)n_blocks * c->block_tokens * D * es <= wide_bytes((uint64_t)tiles * H);
        p.r.pieces = p.wide ? 1 : s > steps ? steps : s;
        p.rows_items = tiles * p.r.pieces;
        p.rows_max = G < 16 ? G : 16;
        if (p.r.pieces > 1) {
            p.rows_join = tiles;
            rows_slots = p.rows_items;
        }
    } else {
        // 16, 32 or 48 rows a tile, so that keys and values are read once for a few rows (48 only where the registers
        // hold them): 90 sequences of 7 x 4 rows, 256 channels, E4M3, 54 us in tiles of 32, 65 of 16; 16 of 5 x 8 rows, 64 channels,
        // 23 us in tiles of 48, 30 of 32.
        p.mt = D == 64 && most > 32 ? 3 : most > 16 ? 2 : 1;
        const uint64_t row_tiles = ceil_div(most, 16 * p.mt) * (uint64_t)seqs * H;
        p.chunk = most > kFewRows && (row_tiles > most_row_tiles(D) || row_tiles * cap > most_tile_tokens(D));
        // A batch may mix single tokens with long chunks.  k_chunk can serve both; k_rows and its join read the
        // single tokens' caches faster but cost two launches.  Us without / with them, 8 heads of 128 channels: 4 sequences
        // of up to 100 new tokens over 1000 29 / 32, over 4000 39 / 46; 512 new beside 16 single tokens over 2000 60 / 91,
        // but beside 64 of them 193 / 174, and beside 16 over 16000 449 / 352.
        p.rows = !p.chunk || (seqs > 1 && (cap > 4096 || (uint64_t)seqs * H > 256));
        if (p.rows) {
            const uint32_t R = 16 * p.mt, tiles = p.chunk ? seqs * ceil_div(kFewRows, R) : bound_tiles(n, seqs, G, R);
            plan_split(tiles, ceil_div(rows_groups(D, p.mt), H), 2, 1, 1, cap, kStep, p.r);
            p.wide = D <= 128 && p.mt <= 2 && p.r.one_round && p.r.slots && 2 * cap * D * es <= wide_bytes((uint64_t)tiles * H);
            if (p.wide) p.r.slots = 0;
            rows_slots = p.r.slots;
            p.rows_items = split_items(tiles, p.r);
            p.rows_join = split_tiles(tiles, p.r);
            p.rows_max = (uint32_t)(most < R ? most : R);
        }
        if (p.chunk) {
            p.cp = plan_chunk(most, D, H, n, seqs, G, cap, p.c);
            if (p.c.slots) {
                const uint64_t r = (uint64_t)p.c.slots * H * 32 * p.cp.waves;
                p.chunk_part = area(r * D * 4);
                p.chunk_stat = area(r * 8);
            }
        }
    }
    if (rows_slots) {
        const uint64_t r = rows_slots * H * 16 * p.mt;
        p.rows_part = area(r * D * 4);
        p.rows_stat = area(r * 8);
    }
    p.r.lo_rows = 0;
    p.r.hi_rows = p.chunk ? kFewRows : 0xFFFFFFFFu;
    p.c.lo_rows = p.rows ? kFewRows : 0;
    p.c.hi_rows = 0xFFFFFFFFu;
    return p;
}

template <int DT, int D, int MT, bool LIST, int UNIT>
void launch_rows(const Plan &p, const AttendArgs &a, dim3 grid, dim3 jgrid, hipStream_t stream)
{
    if constexpr (D <= 128 && MT <= 2) {
        if (p.wide) {
            hipLaunchKernelGGL((k_rows<DT, D, MT, LIST, 8>), grid, dim3(512), 0, stream, a);
            return;
        }
    }
    hipLaunchKernelGGL((k_rows<DT, D, MT, LIST, 4>), grid, dim3(256), 0, stream, a);
    if (p.rows_join) hipLaunchKernelGGL((k_join<D, 16 * MT, UNIT>), jgrid, dim3(256), 0, stream, a);
}

template <int DT, int D>
void run_plan(Plan &p, uint32_t n_blocks, uint8_t *ws, hipStream_t stream)
{
    if (p.rows) {
        AttendArgs &a = p.r;
        a.part = reinterpret_cast<float *>(ws + p.rows_part);
        a.stat = reinterpret_cast<float *>(ws + p.rows_stat);
        const dim3 grid(p.rows_items * a.c.heads), jgrid(p.rows_join * a.c.heads, 1, join_depth(p.rows_join * a.c.heads, p.rows_max));
        if (n_blocks) {
            launch_rows<DT, D, 1, true, 0>(p, a, grid, jgrid, stream);
        } else if (p.mt == 1) {
            launch_rows<DT, D, 1, false, (int)kStep>(p, a, grid, jgrid, stream);
        } else if (p.mt == 2) {
            launch_rows<DT, D, 2, false, (int)kStep>(p, a, grid, jgrid, stream);
        } else if constexpr (D == 64) {
            launch_rows<DT, D, 3, false, (int)kStep>(p, a, grid, jgrid, stream);
        }
    }
    if (p.chunk) {
        AttendArgs &a = p.c;
        a.part = reinterpret_cast<float *>(ws + p.chunk_part);
        a.stat = reinterpret_cast<float *>(ws + p.chunk_stat);
        run_chunk(DT, D, p.cp, a, stream);
    }
}

zx_status checks(const zx_paged_cache *cache, const zx_paged_batch *batch, uint32_t n_tokens, uint32_t q_heads, uint32_t n_blocks, uint32_t window,
                 uint32_t *err, AttendArgs &g)
{
    zx_status st = make_cache(cache, g.c);
    if (st == ZX_OK) st = make_batch(batch, cache, n_tokens, err, g.b);
    if (st != ZX_OK) return st;
    if (q_heads == 0 || q_heads % cache->kv_heads || q_heads > 65536 || n_blocks > 65536) return ZX_E_INVAL;
    if (n_blocks && !cache->block_tokens) return ZX_E_INVAL;
    g.window = (int32_t)window;
    const uint64_t work = (uint64_t)n_tokens * q_heads;
    if (work > 0x3FFFFFFFull) return ZX_E_LIMIT;
    // the kernels count steps and pieces in 32 bits
    const uint64_t tiles = (uint64_t)n_tokens * ceil_div(q_heads / cache->kv_heads, 16);
    if (tiles * ((uint64_t)g.b.cap / kStep + 1) > 0x7FFFFFFFull || tiles * cache->kv_heads * (n_blocks ? 64 : 1) > 0x7FFFFFFFull) return ZX_E_LIMIT;
    return ZX_OK;
}

}  // namespace
}  // namespace zxp

extern "C" size_t zx_paged_attend_workspace_bytes(const zx_paged_cache *cache, const zx_paged_batch *batch, uint32_t n_tokens,
                                                  uint32_t q_heads, uint32_t window, uint32_t n_blocks)
{
    zxp::AttendArgs g{};
    if (window > 0x3FFFFFFFu || zxp::checks(cache, batch, n_tokens, q_heads, n_blocks, window, nullptr, g) != ZX_OK || n_tokens == 0 || batch->n_seqs == 0) return 0;
    return (size_t)zxp::make_plan(cache, batch, n_tokens, q_heads, n_blocks, g).bytes;
}

extern "C" zx_status zx_paged_attend(const zx_paged_cache *cache, const zx_paged_batch *batch, uint32_t n_tokens, const zx_rows *q,
                                     uint32_t q_heads, const zx_rows *out, float *lse, float scale, int causal, uint32_t window,
                                     const int32_t *blocks, uint32_t n_blocks, void *workspace, size_t ws_bytes, uint32_t *err,
                                     hipStream_t stream)
{
    using namespace zxp;
    AttendArgs g{};
    if ((blocks == nullptr) != (n_blocks == 0)) return ZX_E_INVAL;
    if (window > 0x3FFFFFFFu) return ZX_E_INVAL;
    zx_status st = checks(cache, batch, n_tokens, q_heads, n_blocks, window, err, g);
    if (st != ZX_OK) return st;
    if (!(scale > 0.0f) || scale > 1e30f || (blocks && (!causal || window))) return ZX_E_INVAL;
    if (n_tokens == 0 || batch->n_seqs == 0) return ZX_OK;
    if ((st = make_rows(q, g.q)) != ZX_OK || (st = make_rows(out, g.out)) != ZX_OK) return st;
    g.lse = lse;
    g.blocks = blocks;
    g.n_blocks = n_blocks;
    g.scale = scale * kLog2e;
    g.causal = causal;
    g.group = q_heads / cache->kv_heads;
    g.q_heads = q_heads;
    Plan p = make_plan(cache, batch, n_tokens, q_heads, n_blocks, g);
    const uint64_t H = cache->kv_heads;
    if ((p.rows && !launchable(p.rows_items * H, 512)) || (p.chunk && !launchable(split_items(p.cp.tiles, p.c) * H, 64 * p.cp.waves)))
        return ZX_E_LIMIT;
    if (p.bytes && (!workspace || ws_bytes < p.bytes || !al16(workspace))) return ZX_E_INVAL;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const uint32_t D = cache->head_dim;
    if (cache->dtype == ZX_BF16) {
        if (D == 64) run_plan<ZX_BF16, 64>(p, n_blocks, ws, stream);
        else if (D == 128) run_plan<ZX_BF16, 128>(p, n_blocks, ws, stream);
        else run_plan<ZX_BF16, 256>(p, n_blocks, ws, stream);
    } else {
        if (D == 64) run_plan<ZX_FP8_E4M3FN, 64>(p, n_blocks, ws, stream);
        else if (D == 128) run_plan<ZX_FP8_E4M3FN, 128>(p, n_blocks, ws, stream);
        else run_plan<ZX_FP8_E4M3FN, 256>(p, n_blocks, ws, stream);
    }
    return hipGetLastError() == hipSuccess ? ZX_OK : ZX_E_HIP;
}
