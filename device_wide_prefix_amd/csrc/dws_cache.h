// Host-side interface between the C entry points of the cached keys and values
// (dws_cache_abi.cpp) and their kernels. Not installed; not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dws_scan.h"

namespace dws {

// One (tokens, heads, dim) operand: strides in elements, dim contiguous.
struct HeadRows {
    void* data;
    int64_t ts, hs;
};
struct PagePool {
    void* data;
    int64_t ps, ts, hs;
};

// Keys, values and the tokens of a call, as every kernel is given them.
struct KvView {
    PagePool keys, values;
    const int* table;
    const int* lengths;
    int64_t n_rows, max_pages;
    int n_pages, page_tokens;
    int heads, dim_k, dim_v;
    int64_t tokens, n;
    const int64_t* offsets;     // n + 1, or null: tokens / n each
    const int* rows;            // n, or null: row i
};

struct AppendParams {
    KvView c;
    const int* granted;
    const int* positions;
    const float* freqs;
    int pairs, adjacent, heads_q, zero_rest;
    int whole;                  // every run is made of whole, aligned 16-byte units
    HeadRows k, v, q, q_out;
};
hipError_t launch_pages_append(const AppendParams& p, int dtype, hipStream_t stream);

// ---- attention ---------------------------------------------------------------

constexpr int kKvTokens = 32;       // tokens of a wave's tile of keys and values
constexpr int kAttnRows = 32;       // queries of a wave's tile
constexpr int attn_padded_dim(int dim_k, int dim_v)
{
    const int d = dim_k > dim_v ? dim_k : dim_v;
    return d <= 64 ? 64 : (d <= 128 ? 128 : 256);
}
// Waves of a workgroup: their tiles of keys and values share 160 KB of LDS, two
// workgroups of them up to 128 dimensions of 16 bits.
constexpr int attn_waves(int dtype, int padded) { return dtype == DWS_FLOAT32 && padded == 256 ? 2 : 4; }

// Workgroups that the keys are shared out to, two a compute unit.
constexpr int kAttnTarget = 512;

// A tile of queries that belong together: rows (token, head of the key head) of one
// sequence or of one group.
struct AttnTile {
    int64_t token;          // first token of the sequence (of the group)
    int64_t row;            // the tile's first row behind it
    int64_t table;          // first table entry of the cache row
    int64_t slot;           // first row of its partial results; -1: written as it is
    int64_t other_row;      // where a sequence's shared tokens are computed apart: the tile's first row in its group,
    int other;              // and the group's first tile; else -1
    int rows;
    int begin, end;         // its keys: tokens of the cache row
    int position;           // of `token`; a group's are in AttentionParams.positions
    int group;              // 1: the shared tokens of a group
    int steps, parts;       // pieces of kKvTokens tokens a wave, and the workgroups they are shared out to
};
struct AttnHead {
    int tiles, items;
};
struct AttnItem {
    int tile, part;
};

struct AttentionParams {
    KvView c;
    int heads_q, share;         // share: query heads of a key head
    float scale;
    int64_t n_groups;
    const int64_t* groups;
    const int* shared;
    int zero_rest, whole_q, whole_kv, whole_out;
    HeadRows q, out;
    float* lse;
    int dtype, padded, waves;
    // plan and partial results, in the workspace
    int64_t max_tiles, max_items, max_rows;
    AttnHead* head;
    int* seg;                   // [n_groups + n + 1] first tile of each group, then of each sequence
    int* from;                  // [n_groups] tokens that are computed once for the group
    int* positions;             // [tokens], with groups
    AttnTile* tile;             // [max_tiles]
    AttnItem* item;             // [max_items]
    int* wild;                  // [max_tiles] 1: rows to compute again one by one
    float* partial;             // [heads][max_rows][padded] sums
    float2* stat;               // [heads][max_rows] largest score (log2) and sum of the exponentials
};
hipError_t launch_attention(const AttentionParams& p, hipStream_t stream);
hipError_t launch_attention_bf16(const AttentionParams& p, hipStream_t stream);
hipError_t launch_attention_f16(const AttentionParams& p, hipStream_t stream);
hipError_t launch_attention_f32(const AttentionParams& p, hipStream_t stream);

}  // namespace dws
