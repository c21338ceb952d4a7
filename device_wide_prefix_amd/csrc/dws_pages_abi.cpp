// C entry points of the page operators: argument checks, workspace layout and
// dispatch. The contract is in include/dws_scan.h.
#include "dws_scan.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <new>

#include "dws_pages.h"

namespace {

using namespace dws;

constexpr int64_t kMaxCount = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxGrid = (((int64_t)1 << 32) - 1) / 256;      // workgroups of 256 threads in a launch
constexpr int64_t kMaxBytes = (int64_t)1 << 50;

dws_status status_of(hipError_t e) { return e == hipSuccess ? DWS_OK : DWS_ERR_HIP; }

// A call's arrays, to refuse written ones that overlap others.
struct Arrays {
    struct {
        uintptr_t begin, end;
        bool written;
    } r[16];
    int n = 0;

    dws_status add(const void* ptr, int64_t bytes, bool written, size_t align)
    {
        if (bytes == 0) return DWS_OK;
        if (ptr == nullptr) return DWS_ERR_INVALID_ARG;
        const uintptr_t b = reinterpret_cast<uintptr_t>(ptr);
        if (b % align) return DWS_ERR_MISALIGNED;
        if (bytes > kMaxBytes || b + (uintptr_t)bytes < b) return DWS_ERR_INVALID_ARG;
        r[n++] = {b, b + (uintptr_t)bytes, written};
        return DWS_OK;
    }
    bool overlap() const
    {
        for (int i = 0; i < n; ++i)
            for (int j = 0; j < i; ++j)
                if ((r[i].written || r[j].written) && r[i].begin < r[j].end && r[j].begin < r[i].end) return true;
        return false;
    }
};

// `lengths`: whether the call uses them.
dws_status check_cache(const dws_page_cache* a, bool lengths, Arrays* arrays, PageCache* c)
{
    if (a == nullptr || a->n_pages < 1 || a->n_rows < 0 || a->max_pages < 0) return DWS_ERR_INVALID_ARG;
    if (lengths && a->page_tokens < 1) return DWS_ERR_INVALID_ARG;
    if (a->n_pages > kMaxPages || a->n_rows > kMaxCount || a->max_pages > kMaxCount || a->page_tokens > kMaxCount ||
        a->n_rows * a->max_pages > kMaxBytes / 4)
        return DWS_ERR_UNSUPPORTED;
    *c = {a->d_refs, a->n_pages, a->d_table, a->n_rows, a->max_pages, a->d_lengths, a->page_tokens};
    dws_status st = arrays->add(a->d_refs, a->n_pages * 4, true, 4);
    if (st == DWS_OK) st = arrays->add(a->d_table, a->n_rows * a->max_pages * 4, true, 4);
    if (st == DWS_OK && lengths) st = arrays->add(a->d_lengths, a->n_rows * 4, true, 4);
    return st;
}

// Requests: at most kMaxGrid workgroups, 2,048 table entries each.
dws_status check_requests(const PageCache& c, long long n)
{
    if (n < 0) return DWS_ERR_INVALID_ARG;
    if (n > kMaxCount || n * (c.max_pages / 2048 + 1) > kMaxGrid) return DWS_ERR_UNSUPPORTED;
    return DWS_OK;
}

struct Sizes {
    size_t live, claim, length, rank, fresh, bytes;
};
Sizes workspace_of(int64_t pages, int64_t rows, int64_t n)
{
    Sizes z{};
    size_t at = 0;
    auto take = [&](int64_t count) {
        const size_t was = at;
        at += ((size_t)count * 4 + 255) / 256 * 256;
        return was;
    };
    z.live = take((pages + kPageTile - 1) / kPageTile);
    z.claim = take(rows);
    z.length = take(n);
    z.rank = take(n);
    z.fresh = take(pages);
    z.bytes = at;
    return z;
}
dws_status check_workspace(Arrays* arrays, const Sizes& z, void* workspace, size_t bytes)
{
    if (workspace == nullptr || bytes < z.bytes) return DWS_ERR_INVALID_ARG;
    return arrays->add(workspace, (int64_t)z.bytes, true, 256);
}
template <class P>
P* part(void* workspace, size_t at)
{
    return reinterpret_cast<P*>(static_cast<char*>(workspace) + at);
}

dws_status requests_entry(const dws_page_cache* cache, const int* a, const int* b, long long n, int* granted, int* src,
                          int* dst, long long* count, bool fork, void* workspace, size_t bytes, hipStream_t stream)
{
    Arrays arrays;
    PageCache c{};
    dws_status st = check_cache(cache, true, &arrays, &c);
    if (st == DWS_OK) st = check_requests(c, n);
    if (st == DWS_OK) st = arrays.add(a, n * 4, false, 4);
    if (st == DWS_OK) st = arrays.add(b, n * 4, false, 4);
    if (st == DWS_OK) st = arrays.add(granted, n * 4, true, 4);
    if (st == DWS_OK && fork) st = arrays.add(src, n * 4, true, 4);
    if (st == DWS_OK && fork) st = arrays.add(dst, n * 4, true, 4);
    if (st == DWS_OK && fork) st = arrays.add(count, 8, true, 8);
    if (st != DWS_OK) return st;
    const Sizes z = workspace_of(c.pages, c.rows, n);
    if ((st = check_workspace(&arrays, z, workspace, bytes)) != DWS_OK) return st;
    if (arrays.overlap()) return DWS_ERR_OVERLAP;
    PageRequests r{};
    r.a = a;
    r.b = b;
    r.n = n;
    r.granted = granted;
    r.src = src;
    r.dst = dst;
    r.count = count;
    r.live = part<int>(workspace, z.live);
    r.claim = part<int>(workspace, z.claim);
    r.length = part<int>(workspace, z.length);
    r.rank = part<int>(workspace, z.rank);
    r.fresh = part<int>(workspace, z.fresh);
    r.most = fork && n < c.pages ? n : c.pages;
    return status_of(fork ? launch_pages_fork(c, r, stream) : launch_pages_grow(c, r, stream));
}

dws_status free_entry(const dws_page_cache* cache, const int* rows, long long n, long long* freed, void* workspace,
                      size_t bytes, hipStream_t stream)
{
    Arrays arrays;
    PageCache c{};
    dws_status st = check_cache(cache, true, &arrays, &c);
    if (st == DWS_OK) st = check_requests(c, n);
    if (st == DWS_OK) st = arrays.add(rows, n * 4, false, 4);
    if (st == DWS_OK) st = arrays.add(freed, 8, true, 8);
    if (st != DWS_OK) return st;
    const Sizes z = workspace_of(c.pages, c.rows, n);
    if ((st = check_workspace(&arrays, z, workspace, bytes)) != DWS_OK) return st;
    if (arrays.overlap()) return DWS_ERR_OVERLAP;
    const PageFree f{rows, n, freed, part<int>(workspace, z.length)};
    return status_of(launch_pages_free(c, f, stream));
}

dws_status compact_entry(const dws_page_cache* cache, int* remap, int* src, int* dst, long long* moves, long long* count,
                         void* workspace, size_t bytes, hipStream_t stream)
{
    Arrays arrays;
    PageCache c{};
    dws_status st = check_cache(cache, false, &arrays, &c);
    if (st == DWS_OK) st = arrays.add(remap, c.pages * 4, true, 4);
    if (st == DWS_OK) st = arrays.add(src, c.pages / 2 * 4, true, 4);
    if (st == DWS_OK) st = arrays.add(dst, c.pages / 2 * 4, true, 4);
    if (st == DWS_OK) st = arrays.add(moves, 8, true, 8);
    if (st == DWS_OK) st = arrays.add(count, 8, true, 8);
    if (st != DWS_OK) return st;
    const Sizes z = workspace_of(c.pages, c.rows, 0);
    if ((st = check_workspace(&arrays, z, workspace, bytes)) != DWS_OK) return st;
    if (arrays.overlap()) return DWS_ERR_OVERLAP;
    const PageCompact k{remap, src, dst, c.pages / 2, moves, count, part<int>(workspace, z.live)};
    return status_of(launch_pages_compact(c, k, stream));
}

dws_status copy_entry(void* pool, long long pages, long long page_bytes, long long layers, long long layer_stride,
                      const int* src, const int* dst, long long n, const long long* count, hipStream_t stream)
{
    if (pages < 0 || page_bytes < 0 || layers < 0 || layer_stride < 0 || n < 0) return DWS_ERR_INVALID_ARG;
    if (pages > kMaxCount || n > kMaxCount || layers > kMaxCount || page_bytes > kMaxBytes || layer_stride > kMaxBytes)
        return DWS_ERR_UNSUPPORTED;
    if (n == 0 || pages == 0 || layers == 0 || page_bytes == 0) return DWS_OK;
    const __int128 layer_bytes = (__int128)pages * page_bytes, all = (__int128)(layers - 1) * layer_stride + layer_bytes;
    if (all > kMaxBytes) return DWS_ERR_UNSUPPORTED;
    if (layers > 1 && layer_stride < layer_bytes) return DWS_ERR_INVALID_ARG;
    if ((__int128)n * layers * (page_bytes / 16384 + 1) > ((__int128)1 << 62)) return DWS_ERR_UNSUPPORTED;
    Arrays arrays;
    dws_status st = arrays.add(pool, (int64_t)all, true, 1);
    if (st == DWS_OK) st = arrays.add(src, n * 4, false, 4);
    if (st == DWS_OK) st = arrays.add(dst, n * 4, false, 4);
    if (st == DWS_OK && count != nullptr) st = arrays.add(count, 8, false, 8);
    if (st != DWS_OK) return st;
    if (arrays.overlap()) return DWS_ERR_OVERLAP;
    PageCopy c{static_cast<char*>(pool), pages, page_bytes, layers, layers > 1 ? layer_stride : 0, src, dst, n, count, 1};
    const uintptr_t bits = reinterpret_cast<uintptr_t>(pool) | (uintptr_t)page_bytes | (uintptr_t)c.layer_stride;
    c.unit = bits % 16 == 0 ? 16 : (bits % 4 == 0 ? 4 : 1);
    return status_of(launch_pages_copy(c, stream));
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

dws_status dws_pages_workspace(const dws_page_cache* cache, long long n, size_t* bytes)
{
    if (bytes == nullptr || cache == nullptr || cache->n_pages < 1 || cache->n_rows < 0 || n < 0)
        return DWS_ERR_INVALID_ARG;
    if (cache->n_pages > kMaxPages || cache->n_rows > kMaxCount || n > kMaxCount) return DWS_ERR_UNSUPPORTED;
    *bytes = workspace_of(cache->n_pages, cache->n_rows, n).bytes;
    return DWS_OK;
}

dws_status dws_pages_grow(const dws_page_cache* cache, const int* d_rows, const int* d_new_lengths, long long n,
                          int* d_granted, void* d_workspace, size_t workspace_bytes, hipStream_t stream)
{
    return guarded([&] {
        return requests_entry(cache, d_rows, d_new_lengths, n, d_granted, nullptr, nullptr, nullptr, false, d_workspace,
                              workspace_bytes, stream);
    });
}

dws_status dws_pages_fork(const dws_page_cache* cache, const int* d_parents, const int* d_children, long long n,
                          int* d_granted, int* d_src, int* d_dst, long long* d_count, void* d_workspace,
                          size_t workspace_bytes, hipStream_t stream)
{
    return guarded([&] {
        return requests_entry(cache, d_parents, d_children, n, d_granted, d_src, d_dst, d_count, true, d_workspace,
                              workspace_bytes, stream);
    });
}

dws_status dws_pages_free(const dws_page_cache* cache, const int* d_rows, long long n, long long* d_freed,
                          void* d_workspace, size_t workspace_bytes, hipStream_t stream)
{
    return guarded([&] { return free_entry(cache, d_rows, n, d_freed, d_workspace, workspace_bytes, stream); });
}

dws_status dws_pages_compact(const dws_page_cache* cache, int* d_remap, int* d_src, int* d_dst, long long* d_moves,
                             long long* d_count, void* d_workspace, size_t workspace_bytes, hipStream_t stream)
{
    return guarded([&] {
        return compact_entry(cache, d_remap, d_src, d_dst, d_moves, d_count, d_workspace, workspace_bytes, stream);
    });
}

dws_status dws_pages_copy(void* d_pool, long long n_pages, long long page_bytes, long long n_layers,
                          long long layer_stride, const int* d_src, const int* d_dst, long long n,
                          const long long* d_count, hipStream_t stream)
{
    return guarded([&] {
        return copy_entry(d_pool, n_pages, page_bytes, n_layers, layer_stride, d_src, d_dst, n, d_count, stream);
    });
}

}  // extern "C"
