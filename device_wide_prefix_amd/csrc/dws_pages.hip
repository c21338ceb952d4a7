// Pages of a cache: reference counts, page tables and the pages themselves.
//
// A page is free when its count is 0 (or less), so the counts are all the state
// there is: giving out pages is a selection of the free ones, lowest first, and
// compaction a partition by the counts. Both are two passes over the counts: one
// counts each tile's pages in use, the next adds up the tiles before its own
// (at most 4,096 numbers) and ranks its pages. A third launch applies the result,
// since every request may need pages of any tile. All sums are of integers, so
// no result depends on an order.
#include "dws_pages.h"

namespace dws {
namespace {

constexpr int kThreads = 256;
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int wave_sum(int x)
{
#pragma unroll
    for (int d = 32; d > 0; d /= 2) x += __shfl_xor(x, d, 64);
    return x;
}
template <class I>
__device__ __forceinline__ I wave_scan(I x, int lane)     // inclusive
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const I o = __shfl_up(x, d, 64);
        if (lane >= d) x += o;
    }
    return x;
}
// Sum over the workgroup, known to every thread. `part` holds a number a wave.
template <int THREADS>
__device__ __forceinline__ int block_sum(int x, int* part, int tid)
{
    x = wave_sum(x);
    __syncthreads();
    if ((tid & 63) == 0) part[tid >> 6] = x;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) s += part[w];
    return s;
}
// Sum of x over the threads before this one, and in *total over all.
template <int THREADS, class I>
__device__ __forceinline__ I block_exclusive(I x, I* part, int tid, I* total)
{
    const I incl = wave_scan(x, tid & 63);
    __syncthreads();
    if ((tid & 63) == 63) part[tid >> 6] = incl;
    __syncthreads();
    I before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) {
        before += w < (tid >> 6) ? part[w] : 0;
        all += part[w];
    }
    *total = all;
    return before + incl - x;
}
template <int THREADS>
__device__ __forceinline__ int sum_of(const int* x, int64_t n, int* part, int tid)
{
    int s = 0;
    for (int64_t i = tid; i < n; i += THREADS) s += x[i];
    return block_sum<THREADS>(s, part, tid);
}
__device__ __forceinline__ int64_t pages_of(int64_t tokens, int64_t page_tokens)
{
    return (tokens + page_tokens - 1) / page_tokens;
}
int64_t tiles_of(int64_t pages) { return (pages + kPageTile - 1) / kPageTile; }

// Pages in use in each tile; and every row's claim set to none.
__global__ __launch_bounds__(kThreads) void k_pages_count(PageCache c, int* live, int* claim)
{
    __shared__ int part[kThreads / 64];
    const int tid = threadIdx.x;
    const int64_t base = (int64_t)blockIdx.x * kPageTile;
    if (base < c.pages) {
        int n = 0;
        for (uint32_t i = tid; i < kPageTile; i += kThreads)
            if (base + i < c.pages) n += c.refs[base + i] > 0;
        n = block_sum<kThreads>(n, part, tid);
        if (tid == 0) live[blockIdx.x] = n;
    }
    if (claim != nullptr)
        for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < c.rows; i += (int64_t)gridDim.x * kThreads)
            claim[i] = INT32_MAX;
}

// What request i needs, if the row it names is its own: *length the tokens to
// start from (-1: refused), and the pages.
template <bool FORK>
__device__ __forceinline__ long long pages_needed(const PageCache& c, const PageRequests& r, int64_t i, int row, int64_t* length)
{
    *length = -1;
    if constexpr (FORK) {
        const int parent = r.a[i];
        if (parent < 0 || parent >= c.rows || c.lengths[row] != 0) return 0;
        const int64_t n = c.lengths[parent];
        if (n < 0 || n > c.max_pages * c.page_tokens) return 0;
        *length = n;
        return n % c.page_tokens != 0;
    } else {
        const int64_t old = c.lengths[row], now = r.b[i];
        if (old < 0 || now < old || pages_of(now, c.page_tokens) > c.max_pages) return 0;
        *length = old;
        return pages_of(now, c.page_tokens) - pages_of(old, c.page_tokens);
    }
}
// Entry k of the row of granted request i; `first`: its first new page in `fresh`.
template <bool FORK>
__device__ __forceinline__ void apply_entry(const PageCache& c, const PageRequests& r, int64_t i, int64_t k, int64_t length,
                                            int rank, const int* fresh)
{
    if constexpr (FORK) {
        const int* held = c.table + (int64_t)r.a[i] * c.max_pages;
        const int64_t whole = length / c.page_tokens;
        int page = -1;
        if (k < whole) {
            page = held[k];
            if (page >= 0 && page < c.pages) atomicAdd(&c.refs[page], 1);
        } else if (k == whole && rank >= 0) {
            page = fresh[rank];
            c.refs[page] = 1;
            r.src[rank] = held[k];
            r.dst[rank] = page;
        }
        c.table[(int64_t)r.b[i] * c.max_pages + k] = page;
    } else {
        const int64_t first = pages_of(length, c.page_tokens);
        if (k < first || k >= pages_of(r.b[i], c.page_tokens)) return;
        const int page = fresh[rank + (k - first)];
        c.table[(int64_t)r.a[i] * c.max_pages + k] = page;
        c.refs[page] = 1;
    }
}

// Workgroup 0: which requests are granted, in order. The others: the free pages
// of their tile, by rank, as far as `most` can be asked for.
template <bool FORK>
__global__ __launch_bounds__(kPlanThreads) void k_pages_plan(PageCache c, PageRequests r)
{
    __shared__ int part[kPlanThreads / 64];
    __shared__ long long wide[kPlanThreads / 64];
    const int tid = threadIdx.x;
    if (blockIdx.x > 0) {
        const int64_t tile = blockIdx.x - 1, base = tile * kPageTile;
        int64_t rank = base - sum_of<kPlanThreads>(r.live, tile, part, tid);
        if (rank >= r.most) return;
        constexpr int EACH = kPageTile / kPlanThreads;
        int free[EACH], n = 0, all;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int64_t p = base + tid * EACH + i;
            free[i] = p < c.pages && c.refs[p] <= 0;
            n += free[i];
        }
        rank += block_exclusive<kPlanThreads>(n, part, tid, &all);
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            if (free[i]) {
                if (rank < r.most) r.fresh[rank] = (int)(base + tid * EACH + i);
                ++rank;
            }
        return;
    }
    // a row that two requests name goes to the first
    for (int64_t i = tid; i < r.n; i += kPlanThreads) {
        const int row = FORK ? r.b[i] : r.a[i];
        if (row >= 0 && row < c.rows) atomicMin(&r.claim[row], (int)i);
    }
    __threadfence();
    const int64_t tiles = (c.pages + kPageTile - 1) / kPageTile;
    const int64_t n_free = c.pages - sum_of<kPlanThreads>(r.live, tiles, part, tid);
    int64_t taken = 0;       // pages that the requests so far need
    int64_t given = 0;       // pages they got
    for (int64_t base = 0; base < r.n; base += kPlanThreads) {
        const int64_t i = base + tid;
        long long need = 0, all;
        int64_t length = -1;
        if (i < r.n) {
            const int row = FORK ? r.b[i] : r.a[i];
            if (row >= 0 && row < c.rows &&
                __hip_atomic_load(&r.claim[row], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (int)i) {
                need = pages_needed<FORK>(c, r, i, row, &length);
            }
        }
        const int64_t first = taken + block_exclusive<kPlanThreads>(need, wide, tid, &all);
        const bool ok = length >= 0 && (need == 0 || first + need <= n_free);
        if (i < r.n) {
            r.length[i] = ok ? (int)length : -1;
            r.rank[i] = ok && need > 0 ? (int)first : -1;
            r.granted[i] = ok;
        }
        if constexpr (FORK) given += block_sum<kPlanThreads>(ok && need > 0, part, tid);
        taken += all;
    }
    if constexpr (FORK)
        if (tid == 0) *r.count = given;
}

constexpr int64_t kSplit = 2048;      // table entries of a row that one workgroup handles

// Workgroup (i, split): entries split * kSplit .. of request i's row.
template <bool FORK>
__global__ __launch_bounds__(kThreads) void k_pages_apply(PageCache c, PageRequests r, uint32_t splits)
{
    const int64_t i = blockIdx.x / splits, from = (int64_t)(blockIdx.x % splits) * kSplit;
    const bool one = from == 0 && threadIdx.x == 0;
    if constexpr (FORK)
        if (one && i >= *r.count) r.src[i] = r.dst[i] = -1;
    const int64_t length = r.length[i];
    if (length < 0) return;
    const int64_t end = c.max_pages < from + kSplit ? c.max_pages : from + kSplit;
    const int rank = r.rank[i];
    for (int64_t k = from + threadIdx.x; k < end; k += kThreads) apply_entry<FORK>(c, r, i, k, length, rank, r.fresh);
    if (one) c.lengths[FORK ? r.b[i] : r.a[i]] = FORK ? (int)length : r.b[i];
}

// All three steps in one workgroup, with LDS in the place of the workspace: a
// small cache's pass over the counts takes less than two more launches. Growing 4
// rows of 64 entries over 512 pages 5.5 us against 11.6 us, 128 of 32 over 8,192
// pages 9.4 against 13.5; but 32 of 1,024, which want more than one compute unit,
// 23.3 against 14.2. (Compaction of the three caches: 4.1 and 9.1, 11.6 and 12.1,
// 20.0 and 11.9 us.)
constexpr int kSmallPages = 8192, kSmallRows = 4096;
constexpr int64_t kSmallEntries = 8192;       // table entries
template <bool FORK>
__global__ __launch_bounds__(kPlanThreads) void k_pages_small(PageCache c, PageRequests r)
{
    __shared__ int part[kPlanThreads / 64];
    __shared__ long long wide[kPlanThreads / 64];
    __shared__ int claim[kSmallRows], fresh[kSmallPages], lengths[kPlanThreads], ranks[kPlanThreads];
    const int tid = threadIdx.x, n = (int)r.n;
    const int row = tid < n ? (FORK ? r.b[tid] : r.a[tid]) : -1;
    const bool named = row >= 0 && row < c.rows;
    if (named) claim[row] = INT32_MAX;
    int free[kSmallPages / kPlanThreads], mine = 0, n_free;
#pragma unroll
    for (int i = 0; i < kSmallPages / kPlanThreads; ++i) {
        const int64_t p = tid * (kSmallPages / kPlanThreads) + i;
        free[i] = p < c.pages && c.refs[p] <= 0;
        mine += free[i];
    }
    int at = block_exclusive<kPlanThreads>(mine, part, tid, &n_free);
#pragma unroll
    for (int i = 0; i < kSmallPages / kPlanThreads; ++i)
        if (free[i]) fresh[at++] = tid * (kSmallPages / kPlanThreads) + i;
    if (named) atomicMin(&claim[row], tid);
    __syncthreads();
    long long need = 0, all;
    int64_t length = -1;
    if (named && claim[row] == tid) need = pages_needed<FORK>(c, r, tid, row, &length);
    const long long first = block_exclusive<kPlanThreads>(need, wide, tid, &all);
    const bool ok = length >= 0 && (need == 0 || first + need <= n_free);
    const int given = block_sum<kPlanThreads>(ok && need > 0, part, tid);
    lengths[tid] = ok ? (int)length : -1;
    ranks[tid] = ok && need > 0 ? (int)first : -1;
    if (tid < n) {
        r.granted[tid] = ok;
        if constexpr (FORK)
            if (tid >= given) r.src[tid] = r.dst[tid] = -1;
    }
    if constexpr (FORK)
        if (tid == 0) *r.count = given;
    __syncthreads();
    const int most = (int)c.max_pages;
    for (int e = tid; e < n * most; e += kPlanThreads) {
        const int i = e / most;
        if (lengths[i] >= 0) apply_entry<FORK>(c, r, i, e - i * most, lengths[i], ranks[i], fresh);
    }
    if (ok) c.lengths[row] = FORK ? (int)length : r.b[tid];
}

// Takes the rows' lengths: of requests for the same row one gets it, the others 0.
__global__ __launch_bounds__(kThreads) void k_pages_take(PageCache c, PageFree f)
{
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i == 0) *f.freed = 0;
    if (i >= f.n) return;
    const int row = f.row[i];
    f.length[i] = row >= 0 && row < c.rows ? atomicExch(&c.lengths[row], 0) : 0;
}

__global__ __launch_bounds__(kThreads) void k_pages_free(PageCache c, PageFree f, uint32_t splits)
{
    __shared__ int part[kThreads / 64];
    const int64_t i = blockIdx.x / splits, from = (int64_t)(blockIdx.x % splits) * kSplit;
    const int64_t length = f.length[i];
    if (length <= 0) return;
    int64_t end = pages_of(length, c.page_tokens);
    if (end > c.max_pages) end = c.max_pages;
    if (end > from + kSplit) end = from + kSplit;
    if (end <= from) return;
    int* row = c.table + (int64_t)f.row[i] * c.max_pages;
    int n = 0;
    for (int64_t k = from + threadIdx.x; k < end; k += kThreads) {
        const int page = row[k];
        if (page >= 0 && page < c.pages) n += atomicSub(&c.refs[page], 1) == 1;
        row[k] = -1;
    }
    n = block_sum<kThreads>(n, part, threadIdx.x);
    if (threadIdx.x == 0 && n > 0) atomicAdd(reinterpret_cast<unsigned long long*>(f.freed), (unsigned long long)n);
}

// Both steps in one workgroup, for few entries (16 rows of 32: 2.1 us against
// 3.8 us with two launches; 32 rows of 128: 6.8 against 4.3).
constexpr int64_t kSmallFree = 1024;
__global__ __launch_bounds__(kPlanThreads) void k_pages_free_small(PageCache c, PageFree f)
{
    __shared__ int part[kPlanThreads / 64], lengths[kPlanThreads];
    const int tid = threadIdx.x, n = (int)f.n, most = (int)c.max_pages;
    if (tid < n) {
        const int row = f.row[tid];
        lengths[tid] = row >= 0 && row < c.rows ? atomicExch(&c.lengths[row], 0) : 0;
    }
    __syncthreads();
    int freed = 0;
    for (int e = tid; e < n * most; e += kPlanThreads) {
        const int i = e / most, k = e - i * most;
        if (lengths[i] <= 0 || k >= pages_of(lengths[i], c.page_tokens)) continue;
        int* entry = c.table + (int64_t)f.row[i] * c.max_pages + k;
        const int page = *entry;
        if (page >= 0 && page < c.pages) freed += atomicSub(&c.refs[page], 1) == 1;
        *entry = -1;
    }
    freed = block_sum<kPlanThreads>(freed, part, tid);
    if (tid == 0) *f.freed = freed;
}

// With `live` pages in use: the k-th free page before place `live` (a hole) takes
// the k-th page in use behind it. A page p's rank r(p) among those in use
// numbers both: hole p is the (p - r(p))-th, page p behind the front the
// (r(p) - r(live))-th. Pages that move are marked -2 - k in the remap until the
// next launch, which knows all holes.
__global__ __launch_bounds__(kPlanThreads) void k_pages_rank(PageCache c, PageCompact k)
{
    __shared__ int part[kPlanThreads / 64];
    const int tid = threadIdx.x;
    const int64_t tiles = (c.pages + kPageTile - 1) / kPageTile, tile = blockIdx.x, base = tile * kPageTile;
    const int64_t live = sum_of<kPlanThreads>(k.live, tiles, part, tid);
    const int64_t edge = live / kPageTile;            // tile of the first place behind the front
    int64_t before_front = sum_of<kPlanThreads>(k.live, edge, part, tid);
    int n = 0;
    for (int64_t p = edge * kPageTile + tid; p < live; p += kPlanThreads) n += c.refs[p] > 0;
    before_front += block_sum<kPlanThreads>(n, part, tid);
    int64_t rank = sum_of<kPlanThreads>(k.live, tile, part, tid);
    constexpr int EACH = kPageTile / kPlanThreads;
    int used[EACH], all;
    n = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int64_t p = base + tid * EACH + i;
        used[i] = p < c.pages && c.refs[p] > 0;
        n += used[i];
    }
    rank += block_exclusive<kPlanThreads>(n, part, tid, &all);
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int64_t p = base + tid * EACH + i;
        if (p < c.pages) {
            if (used[i]) {
                const int64_t t = rank - before_front;
                k.remap[p] = p < live ? (int)p : (int)(-2 - t);
                if (p >= live) k.src[t] = (int)p;
                ++rank;
            } else {
                k.remap[p] = -1;
                if (p < live) k.dst[p - rank] = (int)p;
            }
        }
    }
    if (tile == 0 && tid == 0) {
        *k.count = live;
        *k.moves = live - before_front;
    }
}

__global__ __launch_bounds__(kThreads) void k_pages_renumber(PageCache c, PageCompact k)
{
    const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x, step = (int64_t)gridDim.x * kThreads;
    const int64_t moves = *k.moves;
    for (int64_t t = at; t < k.list; t += step) {
        if (t < moves) {
            const int from = k.src[t], to = k.dst[t];
            c.refs[to] = c.refs[from];
            c.refs[from] = 0;
            // a table entry may be looked up at the same time: it finds the mark or this, which say the same
            __hip_atomic_store(&k.remap[from], to, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        } else {
            k.src[t] = k.dst[t] = -1;
        }
    }
    for (int64_t e = at; e < c.rows * c.max_pages; e += step) {
        const int page = c.table[e];
        if (page < 0 || page >= c.pages) continue;
        int to = __hip_atomic_load(&k.remap[page], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (to <= -2) to = k.dst[-2 - to];
        if (to >= 0 && to != page) c.table[e] = to;
    }
}

// All of it in one workgroup, with the remap in LDS.
__global__ __launch_bounds__(kPlanThreads) void k_pages_compact_small(PageCache c, PageCompact k)
{
    __shared__ int part[kPlanThreads / 64], remap[kSmallPages], hole[kSmallPages / 2], front;
    const int tid = threadIdx.x, pages = (int)c.pages;
    constexpr int EACH = kSmallPages / kPlanThreads;
    int used[EACH], refs[EACH], n = 0, live;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int p = tid * EACH + i;
        refs[i] = p < pages ? c.refs[p] : 0;
        used[i] = refs[i] > 0;
        n += used[i];
    }
    const int before = block_exclusive<kPlanThreads>(n, part, tid, &live);
    int rank = before;
    if (tid == 0) front = live;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int p = tid * EACH + i;
        if (p == live) front = rank;           // pages in use among the first `live` places
        if (p < live && p < pages && !used[i]) hole[p - rank] = p;
        rank += used[i];
    }
    __syncthreads();
    const int moves = live - front;
    rank = before;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int p = tid * EACH + i;
        if (p < pages) {
            int to = used[i] ? p : -1;
            if (used[i] && p >= live) {
                const int t = rank - front;
                to = hole[t];
                k.src[t] = p;
                k.dst[t] = to;
                c.refs[to] = refs[i];
                c.refs[p] = 0;
            }
            remap[p] = to;
            k.remap[p] = to;
        }
        rank += used[i];
    }
    for (int t = moves + tid; t < (int)k.list; t += kPlanThreads) k.src[t] = k.dst[t] = -1;
    if (tid == 0) {
        *k.count = live;
        *k.moves = moves;
    }
    __syncthreads();
    for (int64_t e = tid; e < c.rows * c.max_pages; e += kPlanThreads) {
        const int page = c.table[e];
        if (page >= 0 && page < pages && remap[page] >= 0 && remap[page] != page) c.table[e] = remap[page];
    }
}

// One workgroup copies kSlice bytes of one page in one layer at a time, past
// the caches: 6,000 pages of 32 KiB in two layers take 155 us (5.05 TB/s), and 4%
// more with accesses through the caches. 4,096 workgroups, a quarter as many, take
// 1% more (again and again on the same pages, 147 us against 138), since their
// last round leaves most compute units idle; far more than 16,384 cost where a
// list is longer than its count (8,350 of 30,000 pairs: 103 us, 109 with 60,000).
// 8 loads in flight a thread stay within 1%.
constexpr int64_t kSlice = 16384;
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

template <class V>
__global__ __launch_bounds__(kThreads) void k_pages_copy(PageCopy c)
{
    int64_t n = c.n;
    if (c.count != nullptr && *c.count < n) n = *c.count < 0 ? 0 : *c.count;
    const int64_t slices = (c.page_bytes + kSlice - 1) / kSlice;
    const int64_t each = c.layers * slices;
    for (int64_t w = blockIdx.x; w < n * each; w += gridDim.x) {
        const int64_t i = w / each, rest = w - i * each, layer = rest / slices, first = (rest - layer * slices) * kSlice;
        const int src = c.src[i], dst = c.dst[i];
        if (src < 0 || dst < 0 || src >= c.pages || dst >= c.pages || src == dst) continue;
        const int64_t bytes = c.page_bytes - first < kSlice ? c.page_bytes - first : kSlice;
        const V* from = reinterpret_cast<const V*>(c.pool + layer * c.layer_stride + src * c.page_bytes + first);
        V* to = reinterpret_cast<V*>(c.pool + layer * c.layer_stride + dst * c.page_bytes + first);
        const int units = (int)(bytes / (int64_t)sizeof(V));
        constexpr int EACH = 4;
        for (int u = threadIdx.x; u < units; u += EACH * kThreads) {
            V x[EACH];
#pragma unroll
            for (int j = 0; j < EACH; ++j)
                if (u + j * kThreads < units) x[j] = __builtin_nontemporal_load(from + u + j * kThreads);
#pragma unroll
            for (int j = 0; j < EACH; ++j)
                if (u + j * kThreads < units) __builtin_nontemporal_store(x[j], to + u + j * kThreads);
        }
    }
}

// Workgroups for the entries of one row.
uint32_t splits_of(const PageCache& c) { return c.max_pages <= kSplit ? 1u : (uint32_t)((c.max_pages + kSplit - 1) / kSplit); }
uint32_t clamp_grid(int64_t blocks, int64_t most) { return (uint32_t)(blocks < 1 ? 1 : (blocks < most ? blocks : most)); }

template <bool FORK>
hipError_t launch_requests(const PageCache& c, const PageRequests& r, hipStream_t stream)
{
    if (c.pages <= kSmallPages && c.rows <= kSmallRows && r.n <= kPlanThreads && r.n * c.max_pages <= kSmallEntries) {
        k_pages_small<FORK><<<dim3(1), dim3(kPlanThreads), 0, stream>>>(c, r);
        return hipGetLastError();
    }
    const int64_t tiles = tiles_of(c.pages);
    const uint32_t splits = splits_of(c);
    // workgroups for the claims of many rows, too, which may be far more than pages
    const int64_t clears = (c.rows + kPageTile - 1) / kPageTile;
    k_pages_count<<<dim3(clamp_grid(tiles > clears ? tiles : clears, 1 << 16)), dim3(kThreads), 0, stream>>>(c, r.live, r.claim);
    k_pages_plan<FORK><<<dim3((uint32_t)tiles + 1), dim3(kPlanThreads), 0, stream>>>(c, r);
    if (r.n == 0) return hipGetLastError();
    k_pages_apply<FORK><<<dim3((uint32_t)r.n * splits), dim3(kThreads), 0, stream>>>(c, r, splits);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_pages_grow(const PageCache& c, const PageRequests& r, hipStream_t stream)
{
    return launch_requests<false>(c, r, stream);
}

hipError_t launch_pages_fork(const PageCache& c, const PageRequests& r, hipStream_t stream)
{
    return launch_requests<true>(c, r, stream);
}

hipError_t launch_pages_free(const PageCache& c, const PageFree& f, hipStream_t stream)
{
    if (f.n <= kPlanThreads && f.n * c.max_pages <= kSmallFree) {
        k_pages_free_small<<<dim3(1), dim3(kPlanThreads), 0, stream>>>(c, f);
        return hipGetLastError();
    }
    const uint32_t splits = splits_of(c);
    k_pages_take<<<dim3((uint32_t)(f.n / kThreads + 1)), dim3(kThreads), 0, stream>>>(c, f);
    if (f.n == 0) return hipGetLastError();
    k_pages_free<<<dim3((uint32_t)f.n * splits), dim3(kThreads), 0, stream>>>(c, f, splits);
    return hipGetLastError();
}

hipError_t launch_pages_compact(const PageCache& c, const PageCompact& k, hipStream_t stream)
{
    if (c.pages <= kSmallPages && c.rows * c.max_pages <= kSmallEntries) {
        k_pages_compact_small<<<dim3(1), dim3(kPlanThreads), 0, stream>>>(c, k);
        return hipGetLastError();
    }
    const int64_t tiles = tiles_of(c.pages);
    k_pages_count<<<dim3((uint32_t)tiles), dim3(kThreads), 0, stream>>>(c, k.live, nullptr);
    k_pages_rank<<<dim3((uint32_t)tiles), dim3(kPlanThreads), 0, stream>>>(c, k);
    const int64_t work = c.rows * c.max_pages > k.list ? c.rows * c.max_pages : k.list;
    k_pages_renumber<<<dim3(clamp_grid((work + kThreads - 1) / kThreads, 2048)), dim3(kThreads), 0, stream>>>(c, k);
    return hipGetLastError();
}

hipError_t launch_pages_copy(const PageCopy& c, hipStream_t stream)
{
    const int64_t items = c.n * c.layers * ((c.page_bytes + kSlice - 1) / kSlice);
    const dim3 grid(clamp_grid(items, 16384)), threads(kThreads);
    if (c.unit == 16)
        k_pages_copy<u32x4_t><<<grid, threads, 0, stream>>>(c);
    else if (c.unit == 4)
        k_pages_copy<uint32_t><<<grid, threads, 0, stream>>>(c);
    else
        k_pages_copy<uint8_t><<<grid, threads, 0, stream>>>(c);
    return hipGetLastError();
}

}  // namespace dws
