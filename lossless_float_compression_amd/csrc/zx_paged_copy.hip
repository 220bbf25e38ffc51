// zx_paged_copy.hip -- tokens of pages copied to other pages, in the caches of all layers at once; and attention
// over parts of a context joined.
//
// Both are bound by the bytes: every byte is read once and written once.  Copies: 512 pages of 8 heads x 64 tokens x 128 channels, BF16,
// in 32 layers 5.2 TB/s read and written (a large copy 4.9 to 5.4); of 31 of the 64 tokens 4.2 (every other 8 KB: the card's
// channels are not all met).  Joins: 4096 x 32 heads, five parts 36 us, 5.7 TB/s.
#include <type_traits>

#include "zx_paged.h"

namespace zxp {
namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kMostCaches = 40;             // of one launch: its arguments fit 4 KB
constexpr uint32_t kVecs = 4;                    // 16-byte pieces a thread reads before it writes any

struct One {
    uint8_t *k, *v, *bounds;
    int64_t k_page, k_head, v_page, v_head;      // byte strides
    uint32_t k_token, v_token;
};

struct CopyArgs {
    One c[kMostCaches];
    const int32_t *pairs, *count;
    uint32_t *err;
    uint32_t cap, n_pages, heads, log_page, log_block, n_caches;
    uint32_t log_row, log_bound;                 // 16-byte pieces of a token's channels, and of a block's bounds
    uint32_t kv_items, bound_items;              // workgroups' shares of a page's keys (or values) and of its bounds
};

// Whether a list of so many shares of 16 KB goes past the caches: 256 MB of whole pages, which is what the last of them holds.  Shares are counted
// by the list's length and the size of a page, whatever part of the pages is copied (the tokens stand on the device), so lists of partly filled pages go past
// earlier.  512 pages in 32 layers (4.3 GB) 1736 us through them, 1645 past them; 8 pages in 32 layers, 31 tokens (33 MB), 17.5 and 19.6;
// between these it has not been measured.
constexpr uint64_t kManyShares = 16384;

// `n` rows of 2^log_vecs pieces of each head, from piece `first` of them on.
template <bool PAST>
__device__ __forceinline__ void copy_rows(const uint8_t *src, uint8_t *dst, int64_t head, uint32_t token, uint32_t n, uint32_t heads,
                                          uint32_t log_vecs, uint32_t first)
{
    const uint32_t all = (n * heads) << log_vecs;
    if (first >= all) return;                    // fewer tokens than a page has
    u4 x[kVecs];
    int64_t at[kVecs];
#pragma unroll
    for (uint32_t i = 0; i < kVecs; ++i) {
        const uint32_t v = first + i * kThreads + threadIdx.x, row = v >> log_vecs, h = row / n, t = row - h * n;
        at[i] = v < all ? (int64_t)h * head + (int64_t)((uint64_t)t * token + ((v & ((1u << log_vecs) - 1)) << 4)) : -1;
        if (at[i] < 0) continue;
        const u4 *from = reinterpret_cast<const u4 *>(src + at[i]);
        x[i] = PAST ? __builtin_nontemporal_load(from) : *from;
    }
#pragma unroll
    for (uint32_t i = 0; i < kVecs; ++i)
        if (at[i] >= 0) {
            u4 *to = reinterpret_cast<u4 *>(dst + at[i]);
            if (PAST) __builtin_nontemporal_store(x[i], to);
            else *to = x[i];
        }
}

// Items: for each pair and cache, shares of its keys, of its values and of its bounds.  A share is kThreads * kVecs
// pieces (16 KB) of the tokens that are copied, one head's after the other's: no workgroup is left with the
// short end of every head.
__global__ __launch_bounds__(kThreads) void k_paged_copy(CopyArgs g)
{
    const int32_t said = *g.count;
    const uint32_t n_pairs = said < 0 ? 0 : (uint32_t)said < g.cap ? (uint32_t)said : g.cap;
    const uint32_t each = 2 * g.kv_items + g.bound_items, per_pair = each * g.n_caches;
    if (blockIdx.x == 0 && threadIdx.x == 0 && (uint32_t)said != n_pairs) report(g.err, ZX_E_CORRUPT);
    const uint64_t all = (uint64_t)n_pairs * per_pair;
    for (uint64_t item = blockIdx.x; item < all; item += gridDim.x) {
        const uint32_t pair = (uint32_t)(item / per_pair), in_pair = (uint32_t)(item - (uint64_t)pair * per_pair);
        const uint32_t layer = in_pair / each, share = in_pair - layer * each;
        const uint32_t from = (uint32_t)g.pairs[3 * (uint64_t)pair], to = (uint32_t)g.pairs[3 * (uint64_t)pair + 1],
                       n = (uint32_t)g.pairs[3 * (uint64_t)pair + 2];
        if (from >= g.n_pages || to >= g.n_pages || n > (1u << g.log_page)) {
            if (threadIdx.x == 0) report(g.err, ZX_E_CORRUPT);
            continue;
        }
        if (from == to || n == 0) continue;
        const One &c = g.c[layer];
        constexpr uint32_t kShare = kThreads * kVecs;
        const uint8_t *src;
        uint8_t *dst;
        int64_t head;
        uint32_t token, rows = n, log_vecs = g.log_row, at = share;
        if (share < g.kv_items) {
            src = c.k + (int64_t)from * c.k_page;
            dst = c.k + (int64_t)to * c.k_page;
            head = c.k_head;
            token = c.k_token;
        } else if (share < 2 * g.kv_items) {
            src = c.v + (int64_t)from * c.v_page;
            dst = c.v + (int64_t)to * c.v_page;
            head = c.v_head;
            token = c.v_token;
            at -= g.kv_items;
        } else {
            rows = ((n - 1) >> g.log_block) + 1;
            log_vecs = g.log_bound;
            token = 16u << g.log_bound;
            head = (int64_t)token << (g.log_page - g.log_block);
            src = c.bounds + from * (head * g.heads);
            dst = c.bounds + to * (head * g.heads);
            at -= 2 * g.kv_items;
        }
        if (all > kManyShares) copy_rows<true>(src, dst, head, token, rows, g.heads, log_vecs, at * kShare);
        else copy_rows<false>(src, dst, head, token, rows, g.heads, log_vecs, at * kShare);
    }
}

// ---------------------------------------------------------------- attention over parts

constexpr uint32_t kMostParts = 16;

struct MergeArgs {
    Rows part[kMostParts], out;
    const float *lse[kMostParts];
    float *out_lse;
    uint32_t heads;
    uint64_t n_rows;                             // tokens * heads
};

// With l_i the ln of a part's sum of exponentials: l = m + ln sum_i e^(l_i - m), out = sum_i e^(l_i - l) out_i.  A part of
// -inf has seen nothing and its output is not looked at.  A thread has eight channels of a row.
template <int D, int P, bool PAST>
__global__ __launch_bounds__(kThreads) void k_attention_merge(MergeArgs g)
{
    constexpr uint32_t TPR = D / 8;
    const uint64_t i = ((uint64_t)blockIdx.x * kThreads + threadIdx.x) / TPR;
    const uint32_t ch = threadIdx.x % TPR * 8;
    if (i >= g.n_rows) return;
    const uint32_t token = (uint32_t)(i / g.heads), h = (uint32_t)(i - (uint64_t)token * g.heads);
    float l[P], m = -__builtin_huge_valf();
    bf8 x[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        l[p] = g.lse[p][i];
        const bf8 *from = reinterpret_cast<const bf8 *>(g.part[p].p + (int64_t)token * g.part[p].token + (int64_t)h * g.part[p].head + ch);
        x[p] = PAST ? __builtin_nontemporal_load(from) : *from;
    }
#pragma unroll
    for (int p = 0; p < P; ++p) m = fmaxf(m, l[p]);
    const float base = m == -__builtin_huge_valf() ? 0.0f : m;
    float sum = 0.0f, y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const float w = __expf(l[p] - base);
        sum += w;
        if (w == 0.0f) continue;                 // (NaN is no zero)
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] += w * (float)x[p][j];
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    bf8 o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = (__bf16)(y[j] * inv);
    *reinterpret_cast<bf8 *>(g.out.p + (int64_t)token * g.out.token + (int64_t)h * g.out.head + ch) = o;
    if (g.out_lse && ch == 0) g.out_lse[i] = sum == 0.0f ? -__builtin_huge_valf() : m + logf(sum);
}

template <int D, bool PAST>
void launch_merge(const MergeArgs &g, uint32_t parts, hipStream_t stream)
{
    const dim3 grid((uint32_t)((g.n_rows * (D / 8) + kThreads - 1) / kThreads)), block(kThreads);
#define MERGE(P) \
    case P: hipLaunchKernelGGL((k_attention_merge<D, P, PAST>), grid, block, 0, stream, g); break
    switch (parts) {
        MERGE(1); MERGE(2); MERGE(3); MERGE(4); MERGE(5); MERGE(6); MERGE(7); MERGE(8);
        MERGE(9); MERGE(10); MERGE(11); MERGE(12); MERGE(13); MERGE(14); MERGE(15); MERGE(16);
    }
#undef MERGE
}

}  // namespace
}  // namespace zxp

extern "C" zx_status zx_paged_copy(const zx_paged_cache *caches, uint32_t n_caches, const zx_page_copies *copies, uint32_t *err,
                                   hipStream_t stream)
{
    using namespace zxp;
    if (n_caches == 0) return ZX_OK;
    if (!caches || !copies || !copies->count || (copies->cap && !copies->pairs)) return ZX_E_INVAL;
    if (((uintptr_t)copies->count | (uintptr_t)copies->pairs | (uintptr_t)err) & 3u) return ZX_E_INVAL;
    if (n_caches > 65536) return ZX_E_LIMIT;
    const zx_paged_cache &f = caches[0];
    for (uint32_t i = 0; i < n_caches; ++i) {
        const zx_paged_cache &c = caches[i];
        Cache o;
        const zx_status st = make_cache(&c, o);
        if (st != ZX_OK) return st;
        if (c.dtype != f.dtype || c.n_pages != f.n_pages || c.kv_heads != f.kv_heads || c.head_dim != f.head_dim ||
            c.page_tokens != f.page_tokens || c.block_tokens != f.block_tokens)
            return ZX_E_INVAL;
    }
    if (copies->cap == 0) return ZX_OK;
    CopyArgs g{};
    g.pairs = copies->pairs;
    g.count = copies->count;
    g.err = err;
    g.cap = copies->cap;
    for (uint32_t i0 = 0; i0 < n_caches; i0 += kMostCaches) {
        const uint32_t n = n_caches - i0 < kMostCaches ? n_caches - i0 : kMostCaches;
        Cache o;
        for (uint32_t i = 0; i < n; ++i) {
            (void)make_cache(&caches[i0 + i], o);
            g.c[i] = One{o.k, o.v, reinterpret_cast<uint8_t *>(o.bounds), o.k_page, o.k_head, o.v_page, o.v_head, o.k_token, o.v_token};
        }
        g.n_pages = o.n_pages;
        g.heads = o.heads;
        g.log_page = o.log_page;
        g.log_block = o.log_block;
        g.n_caches = n;
        g.log_row = log2_of(f.head_dim * (f.dtype == ZX_BF16 ? 2 : 1) / 16);
        g.log_bound = log2_of(f.head_dim / 4);
        const uint32_t share = kThreads * kVecs;
        g.kv_items = ceil_div((uint64_t)o.heads << (o.log_page + g.log_row), share);
        g.bound_items = f.block_tokens ? ceil_div((uint64_t)o.heads << (o.log_page - o.log_block + g.log_bound), share) : 0;
        const uint64_t items = (uint64_t)copies->cap * n * (2ull * g.kv_items + g.bound_items);
        // (the list's length is known on the device only: workgroups take shares in turn until it ends)
        hipLaunchKernelGGL(k_paged_copy, dim3((uint32_t)(items < 8192 ? items : 8192)), dim3(kThreads), 0, stream, g);
    }
    return hipGetLastError() == hipSuccess ? ZX_OK : ZX_E_HIP;
}

extern "C" zx_status zx_attention_merge(const zx_rows *parts, const float *const *lses, uint32_t n_parts, uint32_t n_tokens, uint32_t heads,
                                        uint32_t head_dim, const zx_rows *out, float *out_lse, hipStream_t stream)
{
    using namespace zxp;
    if (!parts || !lses || n_parts == 0 || n_parts > kMostParts || heads == 0 || heads > 65536) return ZX_E_INVAL;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return ZX_E_INVAL;
    MergeArgs g{};
    zx_status st = make_rows(out, g.out);
    for (uint32_t i = 0; i < n_parts && st == ZX_OK; ++i) {
        st = make_rows(&parts[i], g.part[i]);
        if (!lses[i] || ((uintptr_t)lses[i] & 3u)) st = ZX_E_INVAL;
        g.lse[i] = lses[i];
    }
    if (st == ZX_OK && ((uintptr_t)out_lse & 3u)) st = ZX_E_INVAL;
    if (st != ZX_OK) return st;
    if (n_tokens == 0) return ZX_OK;
    g.out_lse = out_lse;
    g.heads = heads;
    g.n_rows = (uint64_t)n_tokens * heads;
    if (g.n_rows * (head_dim / 8) > 0xFFFFFF00ull) return ZX_E_LIMIT;      // a launch counts its threads in 32 bits
    // what the last cache does not hold beside the result (256 MB) is not there from when it was written: 16384 x 32 of two parts 66 us past the
    // caches, 72 through them, 8192 x 64 of eight 202 and 233
    const bool past = g.n_rows * head_dim * 2 * (n_parts + 1) > 256ull << 20;
    auto launch = [&](auto p) {
        constexpr bool PAST = decltype(p)::value;
        if (head_dim == 64) launch_merge<64, PAST>(g, n_parts, stream);
        else if (head_dim == 128) launch_merge<128, PAST>(g, n_parts, stream);
        else launch_merge<256, PAST>(g, n_parts, stream);
    };
    if (past) launch(std::true_type{});
    else launch(std::false_type{});
    return hipGetLastError() == hipSuccess ? ZX_OK : ZX_E_HIP;
}
