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
    uint32_t page_magic, page_shift;    // t / page_tokens = (t * magic >> 32) >> shift for t < 2^31; magic 0: t
    int heads, dim_k, dim_v;
    int64_t tokens, n;
    const int64_t* offsets;     // n + 1, or null: `each` tokens a sequence
    int64_t each;
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
// Tokens of a call at most: workgroups of four waves, a token each, and fewer than 2^32
// threads in a launch.
constexpr int64_t kMaxAppendTokens = (((int64_t)1 << 32) - 1) / 256 * 4;
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

// Workgroups that the work is shared out to at most, as many as are there at a time: two
// a compute unit, one where its four waves have all registers (23 sequences of 64 heads of
// 256 dimensions: 73 us, with 512 of them 96).
constexpr int attn_groups(int dtype, int padded)
{
    return padded * (dtype == DWS_FLOAT32 ? 4 : 2) > 256 && attn_waves(dtype, padded) == 4 ? 256 : 512;
}
// The time of a piece of kKvTokens tokens a wave for tiles of up to 32, 64 and 128
// queries, of a tile beside its pieces, and the least for a workgroup of its own. (With
// weights in two parts the pieces of 64 and 128 take 6 and 10, but spread worse by that: 64
// sequences behind 32,773 shared tokens took 101 us instead of 99, 12 x 8 beams 49 instead of 47.)
constexpr uint32_t kCostNarrow = 4, kCostMiddle = 5, kCostWide = 8, kCostTile = 12, kCostLeast = 8;
// Segments that a workgroup lays out for itself.
constexpr int kAttnSegs = 256;

// A segment of the work: a group's shared tokens for the queries of all its
// sequences, or a sequence's other tokens (all without a group). Its queries, rows
// (token, head of the key head), are cut into tiles.
struct AttnSeg {
    uint32_t cost;          // of the segments before it
    int begin, count;       // tokens of the call
    int row;                // of the cache; -1: none
    int from, length;       // its keys: tokens of that row
    int group;              // a sequence: its group if that shares tokens, else -1; a group: its first sequence
    int tile;               // number of its first tile
    int apart;              // where its tiles are always joined with others: first row of their results; else -1
};

// How a tile was computed, for the joining.
struct AttnDone {
    int first, last;        // workgroups that have a part of it; first < 0: one has it all, -2: and its rows are to be computed again
    int kind;               // 0: as it is, 1: together with its group's tiles, 2: a group's own, or left out
    int rows;
    int64_t row;            // first row of the sequence
    int64_t slot;           // kind 1 and 2: first row of the results that one workgroup has
    int64_t group_row;      // kind 1: the tile's first row in the group,
    int group_tile;         // and the group's first tile
    int begin;              // first token of the sequence, its place in the row, and the cache row
    int position, table;
};

// Rows that are not made of whole, aligned 16 bytes; rows that are; and those in pools
// whose places, in 16 bytes, are 32-bit numbers.
enum AttnAccess { kElements, kFar, kNear };

struct AttentionParams {
    KvView c;
    int heads_q, share;         // share: query heads of a key head
    float scale;
    float log2_scale, log2_rest, sign;      // |scale| log2(e), what fp32 loses of it, and the sign
    int64_t n_groups;
    const int64_t* groups;
    const int* shared;
    int zero_rest, whole_q, whole_out;
    int one_part;               // 16-bit weights of tiles of more than 32 queries rounded once
    int kv_access;              // how keys and values are read (AttnAccess)
    uint32_t key_ps, key_ts, value_ps, value_ts;    // kNear: strides in 16 bytes
    HeadRows q, out;
    float* lse;
    int dtype, padded;
    int shift;                  // log2 of the queries of a whole tile, and of the tokens of a piece
    int cost_shift;             // of costs, so that all of them together stay below 2^31
    int workgroups, tile_rows;  // tile_rows: of a tile at most
    int own_plan;               // every workgroup lays the segments out for itself
    // plan and partial results, in the workspace
    int64_t max_tiles, max_apart;
    AttnSeg* segs;              // [n_groups + n + 1], where not every workgroup has them
    AttnDone* done;             // [max_tiles][heads]
    int* tiles;                 // their number
    float* apart;               // [heads][max_apart][padded] sums,
    float2* apart_stat;         // [heads][max_apart] largest score (log2) and sum of the exponentials
    float* part;                // [workgroups][2][tile_rows][padded]
    float2* part_stat;          // [workgroups][2][tile_rows]
};
hipError_t launch_attention(const AttentionParams& p, hipStream_t stream);
hipError_t launch_attention_bf16(const AttentionParams& p, hipStream_t stream);
hipError_t launch_attention_f16(const AttentionParams& p, hipStream_t stream);
hipError_t launch_attention_f32(const AttentionParams& p, hipStream_t stream);

}  // namespace dws
