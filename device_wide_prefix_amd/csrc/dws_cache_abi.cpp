// C entry points of the cached keys and values: argument checks, workspace
// layout and dispatch. The contract is in include/dws_scan.h.
#include "dws_scan.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cfloat>
#include <cmath>
#include <new>

#include "dws_abi_arrays.h"
#include "dws_cache.h"

namespace {

using namespace dws;

constexpr int64_t kMaxCount = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxPages = (int64_t)1 << 24;
constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int kMaxHeads = 65535;
constexpr int kMaxDim = 256;

dws_status status_of(hipError_t e)
{
    if (e == hipSuccess) return DWS_OK;
    return e == hipErrorOutOfMemory ? DWS_ERR_OOM : DWS_ERR_HIP;
}
size_t size_of(int dtype)
{
    return dtype == DWS_FLOAT32 ? 4 : (dtype == DWS_FLOAT16 || dtype == DWS_BFLOAT16 ? 2 : 0);
}

// Sizes of a cache and a call's tokens; no pointers.
dws_status check_sizes(const dws_kv_cache& c, const dws_page_seqs& s, int heads_q)
{
    if (size_of(c.dtype) == 0 || c.n_pages < 1 || c.n_rows < 0 || c.max_pages < 0 || c.page_tokens < 1 || c.heads < 1 ||
        c.dim_k < 1 || c.dim_v < 1 || heads_q < 0 || s.tokens < 0 || s.n < 0)
        return DWS_ERR_INVALID_ARG;
    if (s.n == 0 && s.tokens > 0 && s.d_offsets == nullptr) return DWS_ERR_INVALID_ARG;
    if (s.n > 0 && s.d_offsets == nullptr && s.tokens % s.n != 0) return DWS_ERR_INVALID_ARG;
    if (c.n_pages > kMaxPages || c.n_rows > kMaxCount || c.max_pages > kMaxCount || c.page_tokens > kMaxCount ||
        c.heads > kMaxHeads || heads_q > kMaxHeads || c.dim_k > kMaxDim || c.dim_v > kMaxDim || s.tokens > kMaxCount ||
        s.n > kMaxCount || c.n_rows * c.max_pages > kMaxArrayBytes / 4)
        return DWS_ERR_UNSUPPORTED;
    return DWS_OK;
}

dws_status add_pool(Arrays* arrays, const dws_page_pool& a, const dws_kv_cache& c, int dim, bool written, PagePool* out)
{
    *out = {a.data, a.page_stride, a.token_stride, a.head_stride};
    for (int64_t s : {a.page_stride, a.token_stride, a.head_stride})
        if (s < 0 || s > kMaxStride) return DWS_ERR_INVALID_ARG;
    const int64_t e = (int64_t)size_of(c.dtype);
    const Strided shape{{a.page_stride * e, a.token_stride * e, a.head_stride * e}, {c.n_pages, c.page_tokens, c.heads}, dim * e};
    return arrays->add(a.data, shape, written, (size_t)e);
}
dws_status add_rows(Arrays* arrays, const dws_rows& a, int64_t tokens, int heads, int dim, int dtype, bool written, HeadRows* out)
{
    *out = {a.data, a.token_stride, a.head_stride};
    if (tokens == 0 || heads == 0) return DWS_OK;
    for (int64_t s : {a.token_stride, a.head_stride})
        if (s < 0 || s > kMaxStride) return DWS_ERR_INVALID_ARG;
    const int64_t e = (int64_t)size_of(dtype);
    const Strided shape{{a.token_stride * e, a.head_stride * e, 0}, {tokens, heads, 1}, dim * e};
    return arrays->add(a.data, shape, written, (size_t)e);
}
// Whether each run of `dim` elements is whole, aligned units of `bytes` bytes.
bool whole(const void* data, int64_t e, int64_t bytes, int64_t dim, int64_t s0, int64_t s1, int64_t s2 = 0)
{
    return reinterpret_cast<uintptr_t>(data) % bytes == 0 && dim * e % bytes == 0 && s0 * e % bytes == 0 &&
           s1 * e % bytes == 0 && s2 * e % bytes == 0;
}

// The cache's and the tokens' arrays.
dws_status check_view(Arrays* arrays, const dws_kv_cache& c, const dws_page_seqs& s, bool written, KvView* v)
{
    dws_status st = add_pool(arrays, c.keys, c, c.dim_k, written, &v->keys);
    if (st == DWS_OK) st = add_pool(arrays, c.values, c, c.dim_v, written, &v->values);
    if (st == DWS_OK) st = arrays->add(c.d_table, c.n_rows * c.max_pages * 4, false, 4);
    if (st == DWS_OK) st = arrays->add(c.d_lengths, c.n_rows * 4, false, 4);
    if (st == DWS_OK && s.d_offsets != nullptr) st = arrays->add(s.d_offsets, (s.n + 1) * 8, false, 8);
    if (st == DWS_OK && s.d_rows != nullptr) st = arrays->add(s.d_rows, s.n * 4, false, 4);
    v->table = c.d_table;
    v->lengths = c.d_lengths;
    v->n_rows = c.n_rows;
    v->max_pages = c.max_pages;
    v->n_pages = (int)c.n_pages;
    v->page_tokens = (int)c.page_tokens;
    // 31-bit numbers divided by page_tokens: with 2^l the power of two at or above it,
    // ceil(2^(31 + l) / page_tokens) is exact enough and below 2^32
    int l = 0;
    while (((int64_t)1 << l) < c.page_tokens) ++l;
    v->page_magic = l == 0 ? 0 : (uint32_t)((((unsigned __int128)1 << (31 + l)) + c.page_tokens - 1) / c.page_tokens);
    v->page_shift = l == 0 ? 0 : (uint32_t)(l - 1);
    v->heads = c.heads;
    v->dim_k = c.dim_k;
    v->dim_v = c.dim_v;
    v->tokens = s.tokens;
    v->n = s.n;
    v->offsets = reinterpret_cast<const int64_t*>(s.d_offsets);
    v->each = s.n > 0 ? s.tokens / s.n : 0;
    v->rows = s.d_rows;
    return st;
}

dws_status append_entry(const dws_pages_append_args* a, hipStream_t stream)
{
    if (a == nullptr) return DWS_ERR_INVALID_ARG;
    const dws_kv_cache& c = a->cache;
    dws_status st = check_sizes(c, a->seqs, a->heads_q);
    if (st != DWS_OK) return st;
    if (a->seqs.tokens > kMaxAppendTokens) return DWS_ERR_UNSUPPORTED;
    if (a->pairs < 0 || a->pairs > c.dim_k / 2) return DWS_ERR_INVALID_ARG;
    AppendParams p{};
    Arrays arrays;
    const int64_t tokens = a->seqs.tokens;
    st = check_view(&arrays, c, a->seqs, true, &p.c);
    if (st == DWS_OK && a->d_granted != nullptr) st = arrays.add(a->d_granted, a->seqs.n * 4, false, 4);
    if (st == DWS_OK && a->d_positions != nullptr) st = arrays.add(a->d_positions, tokens * 4, false, 4);
    if (st == DWS_OK) st = arrays.add(a->d_freqs, (int64_t)a->pairs * 4, false, 4);
    if (st == DWS_OK) st = add_rows(&arrays, a->k, tokens, c.heads, c.dim_k, c.dtype, false, &p.k);
    if (st == DWS_OK) st = add_rows(&arrays, a->v, tokens, c.heads, c.dim_v, c.dtype, false, &p.v);
    const bool in_place = a->q.data == a->q_out.data && a->q.token_stride == a->q_out.token_stride &&
                          a->q.head_stride == a->q_out.head_stride;
    if (st == DWS_OK && !in_place) st = add_rows(&arrays, a->q, tokens, a->heads_q, c.dim_k, c.dtype, false, &p.q);
    if (st == DWS_OK) st = add_rows(&arrays, a->q_out, tokens, a->heads_q, c.dim_k, c.dtype, true, &p.q_out);
    if (st != DWS_OK) return st;
    if (in_place) p.q = p.q_out;
    if (arrays.overlap()) return DWS_ERR_OVERLAP;
    if (tokens == 0) return DWS_OK;
    p.granted = a->d_granted;
    p.positions = a->d_positions;
    p.freqs = a->d_freqs;
    p.pairs = a->pairs;
    p.adjacent = a->adjacent != 0;
    p.heads_q = a->heads_q;
    p.zero_rest = a->zero_rest != 0;
    const int64_t e = (int64_t)size_of(c.dtype);
    p.whole = whole(c.keys.data, e, 16, c.dim_k, c.keys.page_stride, c.keys.token_stride, c.keys.head_stride) &&
              whole(c.values.data, e, 16, c.dim_v, c.values.page_stride, c.values.token_stride, c.values.head_stride) &&
              whole(a->k.data, e, 16, c.dim_k, a->k.token_stride, a->k.head_stride) &&
              whole(a->v.data, e, 16, c.dim_v, a->v.token_stride, a->v.head_stride) &&
              (a->heads_q == 0 || (whole(a->q.data, e, 16, c.dim_k, a->q.token_stride, a->q.head_stride) &&
                                   whole(a->q_out.data, e, 16, c.dim_k, a->q_out.token_stride, a->q_out.head_stride))) &&
              a->pairs * e * (a->adjacent ? 2 : 1) % 16 == 0;
    return status_of(launch_pages_append(p, c.dtype, stream));
}

// ---- attention ---------------------------------------------------------------

struct Plan {
    int padded, waves, tile_rows, workgroups, cost_shift;
    int64_t tiles, apart;
    size_t segs, done, tiles_at, apart_sum, apart_stat, part_sum, part_stat, bytes;
};
// Sizes of the workspace's arrays; the caller's sizes have passed
// check_attention_sizes. Each workgroup has an equal share of the work, so at most its
// first and its last tile are parts. Results that are always joined are those of
// groups and their sequences, which are apart only while a group's rows fill less than
// half a tile a sequence.
dws_status plan_of(const dws_pages_attention_args* a, Plan* z)
{
    const dws_kv_cache& c = a->cache;
    const int64_t share = a->heads_q / c.heads, n = a->seqs.n, groups = a->n_groups;
    z->padded = attn_padded_dim(c.dim_k, c.dim_v);
    z->waves = attn_waves(c.dtype, z->padded);
    const int64_t full = kAttnRows * z->waves;
    const __int128 rows = (__int128)a->seqs.tokens * share;
    __int128 tiles = rows / full + n;
    if (groups > 0) tiles += rows / full + groups;
    if (tiles * c.heads > kMaxCount / 2 || n + groups > kMaxCount / 2) return DWS_ERR_UNSUPPORTED;
    z->tiles = (int64_t)tiles;
    __int128 apart = 0;
    if (groups > 0) apart = 2 * (rows < (__int128)n * (full / 2) ? rows : (__int128)n * (full / 2));
    if (apart > kMaxCount || apart * c.heads * (z->padded + 2) * 4 > kMaxArrayBytes) return DWS_ERR_UNSUPPORTED;
    z->apart = (int64_t)apart;
    z->tile_rows = (int)(rows < full ? (rows < 1 ? 1 : rows) : full);
    // no row is longer than its pages
    const __int128 most = (__int128)c.max_pages * c.page_tokens, step = kKvTokens * z->waves;
    const int64_t tile_cost = kCostTile + (int64_t)kCostWide * (int64_t)((most < kMaxCount ? most : kMaxCount) / step + 1);
    const __int128 cost = tiles * c.heads * tile_cost;
    const int groups_at_once = attn_groups(c.dtype, z->padded);
    z->workgroups = cost < (__int128)groups_at_once * kCostLeast ? (int)(cost / kCostLeast) + 1 : groups_at_once;
    z->cost_shift = 0;
    while (tiles * c.heads * (1 + (tile_cost >> z->cost_shift)) > kMaxCount) ++z->cost_shift;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t was = at;
        at += (bytes + 255) / 256 * 256;
        return was;
    };
    const size_t part = (size_t)z->workgroups * 2 * (size_t)z->tile_rows, always = (size_t)z->apart * c.heads;
    z->segs = take((size_t)(groups + n + 1) * sizeof(AttnSeg));
    z->done = take((size_t)z->tiles * c.heads * sizeof(AttnDone));
    z->tiles_at = take(4);
    z->apart_sum = take(always * z->padded * 4);
    z->apart_stat = take(always * 8);
    z->part_sum = take(part * z->padded * 4);
    z->part_stat = take(part * 8);
    z->bytes = at;
    return DWS_OK;
}

dws_status check_attention_sizes(const dws_pages_attention_args* a)
{
    if (a == nullptr) return DWS_ERR_INVALID_ARG;
    const dws_status st = check_sizes(a->cache, a->seqs, a->heads_q);
    if (st != DWS_OK) return st;
    if (a->heads_q < 1 || a->heads_q % a->cache.heads != 0 || a->n_groups < 0) return DWS_ERR_INVALID_ARG;
    return a->n_groups > kMaxCount ? DWS_ERR_UNSUPPORTED : DWS_OK;
}

template <class P>
P* part(void* workspace, size_t at)
{
    return reinterpret_cast<P*>(static_cast<char*>(workspace) + at);
}

dws_status attention_entry(const dws_pages_attention_args* a, hipStream_t stream)
{
    dws_status st = check_attention_sizes(a);
    if (st != DWS_OK) return st;
    const dws_kv_cache& c = a->cache;
    // 0 leaves the queries out, so that any factor will do
    const double by = a->scale == 0.f ? 1.0 : std::fabs((double)a->scale) * 1.4426950408889634;
    if (!(by <= (double)FLT_MAX) || (a->options & ~DWS_ATTENTION_ONE_PART) != 0) return DWS_ERR_INVALID_ARG;
    const int64_t tokens = a->seqs.tokens;
    AttentionParams p{};
    Arrays arrays;
    st = check_view(&arrays, c, a->seqs, false, &p.c);
    if (st == DWS_OK && a->n_groups > 0) st = arrays.add(a->d_groups, (a->n_groups + 1) * 8, false, 8);
    if (st == DWS_OK && a->n_groups > 0) st = arrays.add(a->d_shared, a->n_groups * 4, false, 4);
    if (st == DWS_OK) st = add_rows(&arrays, a->q, tokens, a->heads_q, c.dim_k, c.dtype, false, &p.q);
    if (st == DWS_OK) st = add_rows(&arrays, a->out, tokens, a->heads_q, c.dim_v, c.dtype, true, &p.out);
    if (st == DWS_OK && a->d_lse != nullptr) st = arrays.add(a->d_lse, tokens * a->heads_q * 4, true, 4);
    if (st != DWS_OK) return st;
    Plan z{};
    if ((st = plan_of(a, &z)) != DWS_OK) return st;
    if (a->d_workspace == nullptr || a->workspace_bytes < z.bytes) return DWS_ERR_INVALID_ARG;
    if ((st = arrays.add(a->d_workspace, (int64_t)z.bytes, true, 256)) != DWS_OK) return st;
    if (arrays.overlap()) return DWS_ERR_OVERLAP;
    if (tokens == 0) return DWS_OK;
    p.heads_q = a->heads_q;
    p.share = a->heads_q / c.heads;
    p.scale = a->scale;
    p.n_groups = a->n_groups;
    p.groups = reinterpret_cast<const int64_t*>(a->d_groups);
    p.shared = a->d_shared;
    p.zero_rest = a->zero_rest != 0;
    p.one_part = (a->options & DWS_ATTENTION_ONE_PART) != 0;
    const int64_t e = (int64_t)size_of(c.dtype);
    p.whole_q = whole(a->q.data, e, 16, c.dim_k, a->q.token_stride, a->q.head_stride);
    const bool whole_kv = whole(c.keys.data, e, 16, c.dim_k, c.keys.page_stride, c.keys.token_stride, c.keys.head_stride) &&
                          whole(c.values.data, e, 16, c.dim_v, c.values.page_stride, c.values.token_stride, c.values.head_stride);
    // (arrays.r[0] and [1] are the keys and the values)
    const bool near = arrays.r[0].end - arrays.r[0].begin <= (uintptr_t)1 << 36 && arrays.r[1].end - arrays.r[1].begin <= (uintptr_t)1 << 36;
    p.kv_access = !whole_kv ? kElements : (near ? kNear : kFar);
    if (p.kv_access == kNear) {
        // a stride that nothing is apart by may be any
        auto units = [&](int64_t stride, int64_t count) { return count > 1 ? (uint32_t)(stride * e / 16) : 0u; };
        p.key_ps = units(c.keys.page_stride, c.n_pages);
        p.key_ts = units(c.keys.token_stride, c.page_tokens);
        p.value_ps = units(c.values.page_stride, c.n_pages);
        p.value_ts = units(c.values.token_stride, c.page_tokens);
    }
    p.whole_out = whole(a->out.data, e, 4 * e, c.dim_v, a->out.token_stride, a->out.head_stride);
    p.lse = a->d_lse;
    p.dtype = c.dtype;
    p.padded = z.padded;
    p.shift = z.waves == 4 ? 7 : 6;
    p.workgroups = z.workgroups;
    p.cost_shift = z.cost_shift;
    p.log2_scale = (float)by;
    p.log2_rest = (float)(by - (double)p.log2_scale);
    p.sign = a->scale > 0.f ? 1.f : (a->scale < 0.f ? -1.f : 0.f);
    p.tile_rows = z.tile_rows;
    p.own_plan = a->seqs.n + a->n_groups <= kAttnSegs;
    p.max_tiles = z.tiles;
    p.max_apart = z.apart;
    p.segs = part<AttnSeg>(a->d_workspace, z.segs);
    p.done = part<AttnDone>(a->d_workspace, z.done);
    p.tiles = part<int>(a->d_workspace, z.tiles_at);
    p.apart = part<float>(a->d_workspace, z.apart_sum);
    p.apart_stat = part<float2>(a->d_workspace, z.apart_stat);
    p.part = part<float>(a->d_workspace, z.part_sum);
    p.part_stat = part<float2>(a->d_workspace, z.part_stat);
    return status_of(launch_attention(p, stream));
}

template <class F>
dws_status guarded(F f)
{
    try {
        return f();
    } catch (const std::bad_alloc&) {
        return DWS_ERR_OOM;
    } catch (...) {
        return DWS_ERR_HIP;
    }
}

}  // namespace

extern "C" {

dws_status dws_pages_append(const dws_pages_append_args* args, hipStream_t stream)
{
    return guarded([&] { return append_entry(args, stream); });
}

dws_status dws_pages_attention_workspace(const dws_pages_attention_args* args, size_t* bytes)
{
    return guarded([&] {
        if (bytes == nullptr) return DWS_ERR_INVALID_ARG;
        dws_status st = check_attention_sizes(args);
        Plan z{};
        if (st == DWS_OK) st = plan_of(args, &z);
        if (st == DWS_OK) *bytes = z.bytes;
        return st;
    });
}

dws_status dws_pages_attention(const dws_pages_attention_args* args, hipStream_t stream)
{
    return guarded([&] { return attention_entry(args, stream); });
}

}  // extern "C"
