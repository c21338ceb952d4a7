// Attention over cached keys and values: who computes what, and the joining of
// partial results.
//
// Lengths are known on the device alone, so one workgroup lays out the work before
// the attention kernel: tiles of queries (AttnTile), and their keys shared out in
// parts (AttnItem) of about equal time, kAttnTarget in all, whatever the lengths are.
#include "dws_cache_device.hpp"

namespace dws {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kSegInLds = 4096;
// A part has at least this many pieces (of 128 tokens): below, joining the parts
// costs more than it saves.
constexpr int kLeastSteps = 2;
// Time of a piece for a tile of more than 32 rows, whose waves each go through the
// whole piece, to one for a smaller tile.
constexpr int kWideCost = 2;

// Exclusive sum over the workgroup's threads; *total gets the sum of all.
__device__ int64_t block_scan(int64_t x, int64_t* total, int64_t* lds)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t sum = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t y = __shfl_up(sum, d, 64);
        if (lane >= d) sum += y;
    }
    __syncthreads();
    if (lane == 63) lds[wave] = sum;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
        const int64_t y = lds[w];
        before += w < wave ? y : 0;
        all += y;
    }
    *total = all;
    return before + sum - x;
}

__device__ __forceinline__ int64_t clamped(int64_t x, int64_t most) { return x < 0 ? 0 : (x > most ? most : x); }

// A sequence's tokens and its cache row; length 0 where it has none.
struct Seq {
    int64_t begin, end, row;
    int length;
};
__device__ Seq sequence(const AttentionParams& p, int64_t i)
{
    Seq s;
    s.begin = clamped(seq_begin(p.c, i), p.c.tokens);
    s.end = clamped(seq_begin(p.c, i + 1), p.c.tokens);
    if (s.end < s.begin) s.end = s.begin;
    s.row = p.c.rows != nullptr ? p.c.rows[i] : i;
    int64_t length = s.row >= 0 && s.row < p.c.n_rows ? p.c.lengths[s.row] : 0;
    if (length > p.c.max_pages * p.c.page_tokens || length < s.end - s.begin) length = 0;
    s.length = (int)length;
    return s;
}
__device__ __forceinline__ int tiles_of(int64_t rows, int tile_rows)
{
    return (int)((rows + tile_rows - 1) / tile_rows);
}

__global__ __launch_bounds__(kPlanThreads) void k_attention_plan(AttentionParams p)
{
    __shared__ int64_t sums[kPlanWaves];
    __shared__ int seg_lds[kSegInLds];
    const int tid = threadIdx.x;
    const int64_t n = p.c.n, groups = p.n_groups, segs = groups + n;
    const int tile_rows = kAttnRows * p.waves, step_tokens = kKvTokens * p.waves;
    const bool in_lds = segs < kSegInLds;
    int64_t total = 0, base = 0;

    // groups: what they share, and whether it pays
    for (int64_t g0 = 0; g0 < groups; g0 += kPlanThreads) {
        const int64_t g = g0 + tid;
        int tiles = 0;
        if (g < groups) {
            const int64_t s0 = clamped(p.groups[g], n), s1 = clamped(p.groups[g + 1], n);
            int from = 0;
            if (s1 - s0 > 1) {
                const Seq lead = sequence(p, s0);
                const int64_t end = clamped(seq_begin(p.c, s1), p.c.tokens);
                const int64_t rows = (end - lead.begin) * p.share;
                const int shared = p.shared[g] < lead.length ? p.shared[g] : lead.length;
                // larger tiles are full with the rows of one sequence
                if (rows > 0 && shared > 0 && rows < (s1 - s0) * (tile_rows / 2)) {
                    from = shared;
                    tiles = tiles_of(rows, tile_rows);
                }
            }
            p.from[g] = from;
        }
        const int64_t first = base + block_scan(tiles, &total, sums);
        if (g < groups) {
            const int at = (int)(first < p.max_tiles ? first : p.max_tiles);
            p.seg[g] = at;
            if (in_lds) seg_lds[g] = at;
        }
        base += total;
    }
    __syncthreads();
    // sequences
    for (int64_t i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int64_t i = i0 + tid;
        int tiles = 0;
        if (i < n) {
            const Seq s = sequence(p, i);
            tiles = tiles_of((s.end - s.begin) * p.share, tile_rows);
        }
        const int64_t first = base + block_scan(tiles, &total, sums);
        if (i < n) {
            const int at = (int)(first < p.max_tiles ? first : p.max_tiles);
            p.seg[groups + i] = at;
            if (in_lds) seg_lds[groups + i] = at;
        }
        base += total;
    }
    const int tiles = (int)(base < p.max_tiles ? base : p.max_tiles);
    if (tid == 0) {
        p.seg[segs] = tiles;
        if (in_lds) seg_lds[segs] = tiles;
    }
    __syncthreads();

    // tiles: the last segment that begins at or before the tile has it
    int64_t cost = 0;
    for (int t = tid; t < tiles; t += kPlanThreads) {
        int64_t lo = 0, hi = segs - 1;
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) / 2;
            if ((in_lds ? seg_lds[mid] : p.seg[mid]) <= t)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int j = t - (in_lds ? seg_lds[lo] : p.seg[lo]);
        AttnTile a;
        a.row = (int64_t)j * tile_rows;
        a.other = -1;
        a.other_row = 0;
        a.slot = -1;
        a.begin = 0;
        int64_t rows;
        if (lo < groups) {
            const Seq lead = sequence(p, clamped(p.groups[lo], n));
            rows = (clamped(seq_begin(p.c, clamped(p.groups[lo + 1], n)), p.c.tokens) - lead.begin) * p.share;
            a.token = lead.begin;
            a.table = lead.row * p.c.max_pages;
            a.end = p.from[lo];
            a.position = 0;
            a.group = 1;
        } else {
            const int64_t i = lo - groups;
            const Seq s = sequence(p, i);
            rows = (s.end - s.begin) * p.share;
            a.token = s.begin;
            a.table = s.length > 0 ? s.row * p.c.max_pages : 0;
            a.position = s.length - (int)(s.end - s.begin);
            a.group = 0;
            if (groups > 0) {
                int64_t g = 0, last = groups - 1;
                while (g < last) {
                    const int64_t mid = (g + last + 1) / 2;
                    if (p.groups[mid] <= i)
                        g = mid;
                    else
                        last = mid - 1;
                }
                const int64_t s0 = clamped(p.groups[g], n);
                if (p.from[g] > 0 && s0 <= i && i < p.groups[g + 1]) {
                    a.begin = p.from[g] < s.length ? p.from[g] : s.length;
                    a.other = in_lds ? seg_lds[g] : p.seg[g];
                    a.other_row = (s.begin - clamped(seq_begin(p.c, s0), p.c.tokens)) * p.share + a.row;
                    if (j == 0)
                        for (int64_t x = s.begin; x < s.end; ++x)
                            p.positions[x] = s.length > 0 ? a.position + (int)(x - s.begin) : -1;
                }
            }
            a.end = s.length;
        }
        a.rows = (int)(rows - a.row < tile_rows ? rows - a.row : tile_rows);
        if (a.group == 0 && a.end > 0) {
            // the last row's own token is the last one that any of them sees
            const int64_t last = a.position + (a.row + a.rows - 1) / p.share + 1;
            a.end = (int)(last < a.end ? last : a.end);
        }
        if (a.end < a.begin) a.end = a.begin;
        a.steps = (a.end - a.begin + step_tokens - 1) / step_tokens;
        a.parts = a.rows > kAttnRows ? kWideCost : 1;
        cost += (int64_t)a.steps * a.parts;
        p.tile[t] = a;
        p.wild[t] = 0;
    }
    int64_t all = 0;
    block_scan(cost, &all, sums);
    int64_t piece = (all * p.c.heads + kAttnTarget - 1) / kAttnTarget;
    if (piece < kLeastSteps) piece = kLeastSteps;

    int64_t items = 0, rows = 0;
    for (int t0 = 0; t0 < tiles; t0 += kPlanThreads) {
        const int t = t0 + tid;
        AttnTile a;
        int parts = 0;
        int64_t partial = 0;
        if (t < tiles) {
            a = p.tile[t];
            parts = (int)((a.steps * (int64_t)a.parts + piece - 1) / piece);
            parts = parts < 1 ? 1 : (parts > a.steps && a.steps > 0 ? a.steps : parts);
            partial = parts > 1 || a.group || a.other >= 0 ? (int64_t)parts * a.rows : 0;
        }
        int64_t all_items = 0, all_rows = 0;
        const int64_t item = items + block_scan(parts, &all_items, sums);
        const int64_t slot = rows + block_scan(partial, &all_rows, sums);
        if (t < tiles) {
            // offsets that decrease can ask for more than there is: that is left out
            const bool fits = item + parts <= p.max_items && slot + partial <= p.max_rows;
            p.tile[t].slot = fits && partial > 0 ? slot : -1;
            p.tile[t].parts = parts;
            for (int x = 0; x < parts && item + x < p.max_items; ++x) p.item[item + x] = {t, fits ? x : -1};
        }
        items += all_items;
        rows += all_rows;
    }
    if (tid == 0) {
        p.head->tiles = tiles;
        p.head->items = (int)(items < p.max_items ? items : p.max_items);
    }
}

__device__ __forceinline__ void store_out(const AttentionParams& p, int64_t at, float x)
{
    if (p.dtype == DWS_FLOAT32)
        static_cast<float*>(p.out.data)[at] = x;
    else if (p.dtype == DWS_BFLOAT16)
        static_cast<bf16_t*>(p.out.data)[at] = (bf16_t)x;
    else
        static_cast<f16_t*>(p.out.data)[at] = (f16_t)x;
}

constexpr int kJoinThreads = 256;

__device__ __forceinline__ float load_as_float(const void* from, int64_t at, int dtype)
{
    if (dtype == DWS_FLOAT32) return static_cast<const float*>(from)[at];
    if (dtype == DWS_BFLOAT16) return (float)static_cast<const bf16_t*>(from)[at];
    return (float)static_cast<const f16_t*>(from)[at];
}

// One row of queries by the whole workgroup, 256 tokens at a time, each token's score
// by a thread and each dimension's sum by a thread: only what the row sees is touched,
// so that values which are not finite stay with those that see them.
struct Again {
    float score[kJoinThreads], red[kJoinThreads / 64];
    int64_t value[kJoinThreads];
};
__device__ void row_again(const AttentionParams& p, const AttnTile& a, int h, int r, Again& s)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t behind = a.row + r, token = a.token + behind / p.share;
    const int head = h * p.share + (int)(behind % p.share);
    const int position = a.position + (int)(behind / p.share);
    const int64_t q = token * p.q.ts + head * p.q.hs;
    const float c = p.scale * 1.44269504088896f;
    float m = -__builtin_inff(), l = 0.f, sum = 0.f;
    for (int t0 = 0; t0 <= position; t0 += kJoinThreads) {
        const int t = t0 + tid;
        float x = -__builtin_inff();
        int64_t value = -1;
        if (t <= position) {
            const int page = p.c.table[a.table + t / p.c.page_tokens], place = t % p.c.page_tokens;
            if (page >= 0 && page < p.c.n_pages) {
                const int64_t key = page * p.c.keys.ps + place * p.c.keys.ts + h * p.c.keys.hs;
                value = page * p.c.values.ps + place * p.c.values.ts + h * p.c.values.hs;
                float dot = 0.f;
                for (int d = 0; d < p.c.dim_k; ++d)
                    dot = __builtin_fmaf(load_as_float(p.q.data, q + d, p.dtype), load_as_float(p.c.keys.data, key + d, p.dtype), dot);
                x = dot * c;
            }
        }
        float top = x;
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
        if (lane == 0) s.red[wave] = top;
        s.value[tid] = value;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kJoinThreads / 64; ++w) top = fmaxf(top, s.red[w]);
        const float now = fmaxf(m, top), base = now == -__builtin_inff() ? 0.f : now;
        const float by = now == m ? 1.f : __builtin_amdgcn_exp2f(m - now);
        s.score[tid] = value < 0 ? 0.f : __builtin_amdgcn_exp2f(x - base);
        __syncthreads();
        l *= by;
        sum *= by;
        m = now;
        const int some = position - t0 + 1 < kJoinThreads ? position - t0 + 1 : kJoinThreads;
        for (int i = 0; i < some; ++i) {
            if (s.value[i] < 0) continue;
            l += s.score[i];
            if (tid < p.c.dim_v) sum += s.score[i] * load_as_float(p.c.values.data, s.value[i] + tid, p.dtype);
        }
        __syncthreads();
    }
    if (tid < p.c.dim_v) store_out(p, token * p.out.ts + head * p.out.hs + tid, l == 0.f ? 0.f : sum / l);
    if (tid == 0 && p.lse != nullptr)
        p.lse[token * p.heads_q + head] = l == 0.f ? -__builtin_inff() : (m + __builtin_log2f(l)) * 0.693147180559945f;
}

// Joins the parts of each row of queries: with m and l the largest score and the
// sum of a part, out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i. Four
// dimensions a thread.
__global__ __launch_bounds__(kJoinThreads) void k_attention_join(AttentionParams p)
{
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    __shared__ Again again;
    const int tile_rows = kAttnRows * p.waves, quads = p.padded / 4;
    const int tiles = p.head->tiles;
    const int64_t all = (int64_t)tiles * p.c.heads;
    for (int64_t x = blockIdx.x; x < all; x += gridDim.x) {
        const int number = (int)(x / p.c.heads), h = (int)(x % p.c.heads);
        const AttnTile a = p.tile[number];
        if (a.group) continue;
        bool wild = p.wild[number] != 0;
        const int64_t shared0 = a.other + a.other_row / tile_rows, shared1 = a.other + (a.other_row + a.rows - 1) / tile_rows;
        if (a.other >= 0 && a.other_row >= 0)
            for (int64_t g = shared0; g <= shared1 && g < tiles; ++g) wild |= p.wild[g] != 0;
        if (wild) {
            for (int r = 0; r < a.rows; ++r) row_again(p, a, h, r, again);
            continue;
        }
        if (a.slot < 0) continue;
        for (int at = threadIdx.x; at < a.rows * quads; at += kJoinThreads) {
            const int r = at / quads, q = at - r * quads;
            f32x4 sum = {0.f, 0.f, 0.f, 0.f};
            float m = -__builtin_inff(), l = 0.f;
            auto add = [&](int64_t slot, int rows, int parts) {
                const int64_t first = (int64_t)h * p.max_rows + slot;
                for (int i = 0; i < parts; ++i) {
                    const float2 s = p.stat[first + (int64_t)i * rows];
                    const f32x4 o = *reinterpret_cast<const f32x4*>(p.partial + (first + (int64_t)i * rows) * p.padded + 4 * q);
                    if (s.y == 0.f) continue;       // saw nothing
                    const float top = fmaxf(m, s.x);
                    const float was = m == top ? 1.f : __builtin_amdgcn_exp2f(m - top);
                    const float is = s.x == top ? 1.f : __builtin_amdgcn_exp2f(s.x - top);
                    sum = sum * was + o * is;
                    l = l * was + s.y * is;
                    m = top;
                }
            };
            add(a.slot + r, a.rows, a.parts);
            if (a.other >= 0) {
                const int64_t row = a.other_row + r, tile = a.other + row / tile_rows;
                if (row >= 0 && tile < tiles) {
                    const AttnTile& g = p.tile[tile];
                    if (g.group && g.slot >= 0 && row % tile_rows < g.rows) add(g.slot + row % tile_rows, g.rows, g.parts);
                }
            }
            const int64_t behind = a.row + r, token = a.token + behind / p.share;
            const int head = h * p.share + (int)(behind % p.share);
            const float by = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (4 * q + j < p.c.dim_v)
                    store_out(p, token * p.out.ts + head * p.out.hs + 4 * q + j, l == 0.f ? 0.f : sum[j] * by);
            if (q == 0 && p.lse != nullptr)
                p.lse[token * p.heads_q + head] = l == 0.f ? -__builtin_inff() : (m + __builtin_log2f(l)) * 0.693147180559945f;
        }
    }
    if (!p.zero_rest) return;
    const int64_t first = clamped(seq_begin(p.c, 0), p.c.tokens), last = clamped(seq_begin(p.c, p.c.n), p.c.tokens);
    const int64_t rest = first + (p.c.tokens - last), per = (int64_t)p.heads_q * p.c.dim_v;
    if (last < first) return;
    for (int64_t r = blockIdx.x; r < rest; r += gridDim.x) {
        const int64_t token = r < first ? r : last + (r - first);
        for (int64_t x = threadIdx.x; x < per; x += kJoinThreads)
            store_out(p, token * p.out.ts + x / p.c.dim_v * p.out.hs + x % p.c.dim_v, 0.f);
        if (p.lse != nullptr)
            for (int64_t x = threadIdx.x; x < p.heads_q; x += kJoinThreads) p.lse[token * p.heads_q + x] = -__builtin_inff();
    }
}

}  // namespace

hipError_t launch_attention(const AttentionParams& p, hipStream_t stream)
{
    k_attention_plan<<<1, kPlanThreads, 0, stream>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    e = p.dtype == DWS_FLOAT32    ? launch_attention_f32(p, stream)
        : p.dtype == DWS_BFLOAT16 ? launch_attention_bf16(p, stream)
                                  : launch_attention_f16(p, stream);
    if (e != hipSuccess) return e;
    const int64_t most = p.max_tiles * p.c.heads + (p.zero_rest ? p.c.tokens : 0);
    k_attention_join<<<(unsigned)(most < 2048 ? most : 2048), kJoinThreads, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace dws
