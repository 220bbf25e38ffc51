// zx_paged.h -- what the kernels of the paged K/V cache share: the device form of a
// cache and a batch, the checks of lengths and page ids, and the search for the piece
// of work a workgroup does.
#pragma once

#include "zx_common.h"

namespace zxp {

using zxk::report;
using zxk::wave_excl_scan;

typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

struct Cache {
    uint8_t *k, *v;
    int64_t k_page, k_head, v_page, v_head;   // byte strides
    uint32_t k_token, v_token;                // byte strides (at most 2^24: a 16-token offset fits 32 bits)
    const float *k_scale, *v_scale;
    __bf16 *bounds;
    uint32_t n_pages, heads, log_page, log_block;
};

struct Batch {
    const int32_t *q_start, *kv_len, *table;
    uint32_t n_seqs, width, n_tokens, max_q;
    int32_t cap;                              // largest length: min(max_kv, width * page_tokens)
    uint32_t *err;
};

struct Rows {
    __bf16 *p;
    int64_t token, head;                      // element strides
};

// Lengths of one sequence; nq = 0 where it is left out.
struct Seq {
    int32_t q0, nq, kv;
};

__device__ __forceinline__ Seq load_seq(const Batch &b, uint32_t s)
{
    const int32_t q0 = b.q_start[s], q1 = b.q_start[s + 1], kv = b.kv_len[s];
    Seq r{q0, q1 - q0, kv};
    if (q0 < 0 || q1 < q0 || (uint32_t)q1 > b.n_tokens || (uint32_t)(q1 - q0) > b.max_q || kv < 0 || kv > b.cap) {
        report(b.err, ZX_E_CORRUPT);
        r = Seq{0, 0, 0};
    }
    return r;
}

// The sequence that holds item `idx` when sequence s has count(seq) items, by one wave:
// 64 sequences a step, counted, scanned across the lanes, and searched by ballot.  All
// lanes get the same answer.  `local` is the item's index within the sequence; `before`
// the sum of weight(seq) over the sequences ahead of it.  False past the last item.
template <class Count, class Weight>
__device__ __forceinline__ bool find_item(const Batch &b, uint32_t idx, Count count, Weight weight, uint32_t &seq, Seq &sv,
                                          uint32_t &local, uint32_t &before)
{
    constexpr int kAtOnce = 4;                   // steps whose lengths are read together
    const uint32_t lane = threadIdx.x & 63u;
    uint32_t acc = 0, wacc = 0;
    for (uint32_t s0 = 0; s0 < b.n_seqs; s0 += 64 * kAtOnce) {
        Seq v[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            v[i] = Seq{0, 0, 0};
            if (s0 + 64 * i + lane < b.n_seqs) v[i] = load_seq(b, s0 + 64 * i + lane);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            if (s0 + 64 * i >= b.n_seqs) break;
            const bool in = s0 + 64 * i + lane < b.n_seqs;
            const uint32_t c = in ? count(v[i]) : 0, w = in ? weight(v[i]) : 0;
            uint32_t total, wtotal;
            const uint32_t ex = wave_excl_scan(c, total);
            const uint32_t wex = wave_excl_scan(w, wtotal);
            if (idx < acc + total) {
                const uint64_t m = __ballot(idx >= acc + ex && idx < acc + ex + c);
                const int l = __builtin_ctzll(m);
                seq = s0 + 64 * i + (uint32_t)l;
                sv.q0 = __builtin_amdgcn_readlane(v[i].q0, l);
                sv.nq = __builtin_amdgcn_readlane(v[i].nq, l);
                sv.kv = __builtin_amdgcn_readlane(v[i].kv, l);
                local = idx - acc - (uint32_t)__builtin_amdgcn_readlane((int)ex, l);
                before = wacc + (uint32_t)__builtin_amdgcn_readlane((int)wex, l);
                return true;
            }
            acc += total;
            wacc += wtotal;
        }
    }
    return false;
}

__device__ __forceinline__ uint32_t div_up(uint32_t a, uint32_t b) { return (a + b - 1) / b; }

// ---- host side: checks shared by the entry points
inline bool pow2_in(uint32_t x, uint32_t lo, uint32_t hi) { return x >= lo && x <= hi && (x & (x - 1)) == 0; }
inline bool al16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline uint32_t log2_of(uint32_t x) { return 31u - (uint32_t)__builtin_clz(x); }
inline uint32_t ceil_div(uint64_t a, uint64_t b) { return (uint32_t)((a + b - 1) / b); }

// ZX_OK and the device form, or the first thing wrong with the cache.
zx_status make_cache(const zx_paged_cache *c, Cache &o);
zx_status make_batch(const zx_paged_batch *b, const zx_paged_cache *c, uint32_t n_tokens, uint32_t *err, Batch &o);
zx_status make_rows(const zx_rows *r, Rows &o);

}  // namespace zxp
