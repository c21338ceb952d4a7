// Host-side interface between the page operators' C entry points
// (dws_pages_abi.cpp) and their kernels. Not installed; not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dws {

constexpr uint32_t kPageTile = 4096;                   // reference counts a workgroup looks through
constexpr int64_t kMaxPages = (int64_t)1 << 24;        // 4,096 tiles: every workgroup can add up their counts

struct PageCache {
    int* refs;
    int64_t pages;
    int* table;
    int64_t rows;
    int64_t max_pages;
    int* lengths;
    int64_t page_tokens;
};

// Requests of a grow (rows, new lengths) or a fork (parents, children).
struct PageRequests {
    const int* a;
    const int* b;
    int64_t n;
    int* granted;
    int* src;              // fork
    int* dst;
    long long* count;
    // workspace
    int* live;             // [tiles] pages in use in each tile
    int* claim;            // [rows] first request that names the row
    int* length;           // [n] tokens before (grow), of the parent (fork); -1: refused
    int* rank;             // [n] rank of the request's first new page, -1: needs none
    int* fresh;            // [most] pages not in use, by rank
    int64_t most;
};
hipError_t launch_pages_grow(const PageCache& c, const PageRequests& r, hipStream_t stream);
hipError_t launch_pages_fork(const PageCache& c, const PageRequests& r, hipStream_t stream);

struct PageFree {
    const int* row;
    int64_t n;
    long long* freed;
    int* length;           // workspace: [n]
};
hipError_t launch_pages_free(const PageCache& c, const PageFree& f, hipStream_t stream);

struct PageCompact {
    int* remap;            // [pages]
    int* src;              // [list]
    int* dst;
    int64_t list;
    long long* moves;
    long long* count;
    int* live;             // workspace: [tiles]
};
hipError_t launch_pages_compact(const PageCache& c, const PageCompact& k, hipStream_t stream);

struct PageCopy {
    char* pool;
    int64_t pages, page_bytes, layers, layer_stride;
    const int* src;
    const int* dst;
    int64_t n;
    const long long* count;
    int unit;              // bytes of a load: 16, 4 or 1
};
hipError_t launch_pages_copy(const PageCopy& c, hipStream_t stream);

}  // namespace dws
