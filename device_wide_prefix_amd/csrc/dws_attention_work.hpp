// Attention over cached keys and values: who computes what.
//
// Lengths are known on the device alone. The work is laid out in a line: for each key
// head all segments (AttnSeg), for each segment its tiles of queries, for each tile its
// pieces of keys, each with its cost. Every workgroup takes an equal stretch of that
// line, whatever the lengths are; a tile that lies in several stretches is joined from
// their partial results afterwards. Where the stretches end follows from the segments'
// costs by arithmetic, in whole numbers, for the workgroups and the joining alike.
#pragma once

#include "dws_cache_device.hpp"

namespace dws {
namespace {

// Tokens of a row: those of a piece behind them are still numbers.
constexpr int64_t kMaxLength = INT32_MAX - 4096;

__device__ __forceinline__ int64_t clamped(int64_t x, int64_t most) { return x < 0 ? 0 : (x > most ? most : x); }

__device__ __forceinline__ uint32_t sum_of(uint32_t x, uint32_t y)
{
    return x + y < x ? 0xffffffffu : x + y;
}
// Cost, tiles and rows joined always, of a segment or of those before it; at most 2^32 - 1.
struct AttnSums {
    uint32_t cost, tiles, apart;
    __device__ __forceinline__ void add(const AttnSums& y)
    {
        cost = sum_of(cost, y.cost);
        tiles = sum_of(tiles, y.tiles);
        apart = sum_of(apart, y.apart);
    }
};
// Exclusive sums over the workgroup's threads; *total gets those of all.
template <int WAVES>
__device__ AttnSums block_scan(AttnSums x, AttnSums* total, AttnSums* lds)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    AttnSums sum = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const AttnSums y{__shfl_up(sum.cost, d, 64), __shfl_up(sum.tiles, d, 64), __shfl_up(sum.apart, d, 64)};
        if (lane >= d) sum.add(y);
    }
    __syncthreads();
    if (lane == 63) lds[wave] = sum;
    const AttnSums up{__shfl_up(sum.cost, 1, 64), __shfl_up(sum.tiles, 1, 64), __shfl_up(sum.apart, 1, 64)};
    __syncthreads();
    AttnSums before = lane > 0 ? up : AttnSums{0, 0, 0}, all{0, 0, 0};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        if (w < wave) before.add(lds[w]);
        all.add(lds[w]);
    }
    *total = all;
    return before;
}

__device__ __forceinline__ int64_t divided(int64_t x, int by)
{
    return x >= 0 && x <= INT32_MAX ? (int64_t)((uint32_t)x / (uint32_t)by) : x / by;
}

// A segment's tiles: their number, and the pieces of the first and the last one.
struct AttnShape {
    int tiles, first, last;
    uint32_t last_cost;     // of a piece of the last tile
};
// Tile j of a segment.
struct AttnTile {
    int64_t row;            // its first row
    int rows;
    int begin, end;         // its keys
    int steps;              // pieces of them
};
struct AttnWork {
    const AttentionParams& p;
    __device__ __forceinline__ AttnWork(const AttentionParams& p) : p(p) {}

    __device__ __forceinline__ int tile_rows() const { return 1 << p.shift; }
    __device__ __forceinline__ static uint32_t step_cost(int rows) { return rows <= 32 ? kCostNarrow : (rows <= 64 ? kCostMiddle : kCostWide); }
    __device__ __forceinline__ int64_t rows(const AttnSeg& s) const { return (int64_t)s.count * p.share; }
    __device__ __forceinline__ int tiles(const AttnSeg& s) const { return (int)((rows(s) + tile_rows() - 1) >> p.shift); }
    __device__ __forceinline__ AttnTile tile(const AttnSeg& s, int j, bool group) const
    {
        AttnTile t;
        const int64_t all = rows(s);
        t.row = (int64_t)j << p.shift;
        t.rows = (int)(all - t.row < tile_rows() ? all - t.row : tile_rows());
        t.begin = s.from;
        t.end = s.length;
        if (!group && s.count > 1) {
            // the last row's own token is the last one that any of them sees
            const int64_t last = s.length - s.count + divided(t.row + t.rows - 1, p.share) + 1;
            t.end = (int)(last < t.end ? last : t.end);
        }
        if (t.end < t.begin) t.end = t.begin;
        t.steps = (int)(((uint32_t)t.end - (uint32_t)t.begin + tile_rows() - 1) >> p.shift);
        return t;
    }
    __device__ __forceinline__ AttnShape shape(const AttnSeg& s, bool group) const
    {
        AttnShape x{tiles(s), 0, 0, kCostWide};
        if (x.tiles > 0) {
            const AttnTile last = tile(s, x.tiles - 1, group);
            x.last = last.steps;
            x.last_cost = step_cost(last.rows);
            x.first = x.tiles > 1 ? tile(s, 0, group).steps : x.last;
        }
        return x;
    }
    // Cost of the first j tiles, at least 1 for each. Those of a sequence have more keys the
    // later they are: of several tiles a straight line from the first to the last one's.
    __device__ __forceinline__ uint32_t cost(const AttnShape& x, int j) const
    {
        if (x.tiles <= 1) return j > 0 && x.tiles > 0 ? 1 + ((kCostTile - 1 + x.last * x.last_cost) >> p.cost_shift) : 0;
        const double slope = (double)kCostWide * (x.last - x.first) / (2.0 * (x.tiles - 1));
        const double y = (double)j * (kCostTile - 1.0 + (double)kCostWide * x.first) + slope * ((double)j * (double)(j - 1));
        return (uint32_t)j + (uint32_t)(y * __builtin_ldexp(1.0, -p.cost_shift));
    }
    // The tile that has place x of its segment.
    __device__ __forceinline__ int tile_at(const AttnShape& s, uint32_t x) const
    {
        int j = 0, last = s.tiles - 1;
        while (j < last) {
            const int mid = j + (last - j + 1) / 2;
            if (cost(s, mid) <= x)
                j = mid;
            else
                last = mid - 1;
        }
        return j;
    }
    // How many of a tile's pieces lie before its place x of `cost`.
    __device__ __forceinline__ int step_at(const AttnShape& s, uint32_t x, uint32_t cost, int steps) const
    {
        if (x >= cost) return steps;
        if (s.tiles == 1 && p.cost_shift == 0) return x <= kCostTile ? 0 : (int)((x - kCostTile) / s.last_cost);
        return (int)((double)x * (double)steps / (double)cost);
    }
    // What a workgroup takes of a line of this length.
    __device__ __forceinline__ uint32_t stretch(uint32_t line) const
    {
        const uint32_t x = (line + p.workgroups - 1) / (uint32_t)p.workgroups;
        return x < kCostLeast ? kCostLeast : x;
    }
};

// A sequence's tokens and its cache row; length 0 where it has none.
__device__ __forceinline__ AttnSeg sequence(const AttentionParams& p, int64_t i)
{
    AttnSeg s;
    const int64_t b = clamped(seq_begin(p.c, i), p.c.tokens), e = clamped(seq_begin(p.c, i + 1), p.c.tokens);
    const int64_t row = p.c.rows != nullptr ? p.c.rows[i] : i;
    const bool in = row >= 0 && row < p.c.n_rows;
    int64_t length = in ? p.c.lengths[row] : 0;
    s.begin = (int)b;
    s.count = e > b ? (int)(e - b) : 0;
    if (length > p.c.max_pages * p.c.page_tokens || length > kMaxLength || length < s.count) length = 0;
    s.row = length > 0 ? (int)row : -1;
    s.length = (int)length;
    s.from = 0;
    s.group = -1;
    s.apart = -1;
    s.cost = 0;
    s.tile = 0;
    return s;
}

// Lays out the segments, n_groups + n and one that ends them, with all threads of a
// workgroup; `segs` in LDS or global memory. Ends with a barrier.
// (Inlined always: called, it would have the parameters in scratch memory, and every
// access by their pointers would be one that might be of the LDS.)
template <int THREADS>
__device__ __forceinline__ void lay_out(const AttentionParams& p, AttnSeg* segs, AttnSums* scratch)
{
    const AttnWork work(p);
    const int tid = threadIdx.x;
    const int64_t n = p.c.n, groups = p.n_groups, all = groups + n;
    // the sequences are looked up by the first waves, while the last ones look at the groups
    AttnSeg mine{};
    if (tid >= groups && tid < all) mine = sequence(p, tid - groups);
    for (int64_t g = THREADS - 1 - tid; g < groups; g += THREADS) {
        const int64_t s0 = clamped(p.groups[g], n), s1 = clamped(p.groups[g + 1], n);
        AttnSeg s{};
        s.row = s.apart = -1;
        s.group = (int)s0;
        if (s1 - s0 > 1) {
            // the first one that has a row (the last one of a group shares with none)
            AttnSeg lead = sequence(p, s0);
#pragma unroll 1
            for (int64_t i = s0 + 1; i < s1 - 1 && lead.length == 0; ++i) lead = sequence(p, i);
            const int64_t begin = clamped(seq_begin(p.c, s0), p.c.tokens), end = clamped(seq_begin(p.c, s1), p.c.tokens);
            const int64_t count = end - begin;
            const int shared = p.shared[g] < lead.length ? p.shared[g] : lead.length;
            // (from half a tile of rows a sequence on, all read the shared tokens for themselves: their
            // own tiles are half full at least)
            if (count > 0 && shared > 0 && count * p.share < (s1 - s0) * (work.tile_rows() / 2)) {
                s.begin = (int)begin;
                s.count = (int)count;
                s.row = lead.row;
                s.length = shared;
            }
        }
        segs[g] = s;
    }
    if (groups > 0) __syncthreads();
    AttnSums sums{0, 0, 0};
    for (int64_t i0 = 0; i0 < all; i0 += THREADS) {
        const int64_t i = i0 + tid;
        AttnSeg s{};
        AttnSums of_mine{0, 0, 0}, of_all;
        if (i < all) {
            const bool group = i < groups;
            s = group ? segs[i] : (i0 == 0 ? mine : sequence(p, i - groups));
            if (!group && groups > 0) {
                int64_t lo = 0, hi = groups - 1;
                while (lo < hi) {
                    const int64_t mid = (lo + hi + 1) / 2;
                    if (segs[mid].group <= i - groups)
                        lo = mid;
                    else
                        hi = mid - 1;
                }
                // (the group's end: the next one begins there, or what p.groups says)
                const AttnSeg g = segs[lo];
                if (g.count > 0 && g.group <= i - groups && i - groups < p.groups[lo + 1]) {
                    s.group = (int)lo;
                    s.from = g.length < s.length ? g.length : s.length;
                }
            }
            const AttnShape shape = work.shape(s, group);
            const int64_t rows = group || s.group >= 0 ? work.rows(s) : 0;
            of_mine = {work.cost(shape, shape.tiles), (uint32_t)shape.tiles, (uint32_t)(rows < UINT32_MAX ? rows : UINT32_MAX)};
        }
        AttnSums before = block_scan<THREADS / 64>(of_mine, &of_all, scratch);
        before.add(sums);
        sums.add(of_all);
        // Offsets that decrease can ask for more than there is room for: such a segment is left out.
        AttnSums after = before;
        after.add(of_mine);
        s.cost = before.cost;
        s.tile = (int)(before.tiles < p.max_tiles ? before.tiles : p.max_tiles);
        s.apart = of_mine.apart > 0 ? (int)before.apart : -1;
        if (after.tiles > p.max_tiles || after.apart > p.max_apart || after.cost > INT32_MAX) s.row = -2;
        if (i < all) segs[i] = s;
    }
    if (tid == 0) {
        AttnSeg s{};
        s.cost = sums.cost;
        s.tile = (int)(sums.tiles < p.max_tiles ? sums.tiles : p.max_tiles);
        segs[all] = s;
    }
    __syncthreads();
}

// The last segment whose cost is not behind x; segments without tiles lie before the one
// that has it. Every lane calls it with the same x; 64 segments a round.
__device__ __forceinline__ int seg_at_cost(const AttnSeg* segs, int n, uint32_t x, int lane)
{
    int lo = 0, hi = n - 1;
    while (hi > lo) {
        const int step = (hi - lo) / 64 + 1, at = lo + lane * step;
        const uint64_t found = __ballot(at <= hi && segs[at <= hi ? at : hi].cost <= x);
        lo += found == 0 ? 0 : (63 - __builtin_clzll(found)) * step;
        if (found == 0) hi = lo;
        if (lo + step - 1 < hi) hi = lo + step - 1;
    }
    return lo;
}

}  // namespace
}  // namespace dws
