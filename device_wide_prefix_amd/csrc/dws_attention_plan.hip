// Attention over cached keys and values: the layout of large batches' work, and the
// joining of partial results.
#include "dws_attention_work.hpp"

namespace dws {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kJoinThreads = 256;      // (at least one a dimension)
constexpr int kJoinRows = 64;          // of a tile, for a workgroup: 32 to 128 take as long
static_assert(kJoinThreads >= 256, "row_again has a thread for each dimension");

__global__ __launch_bounds__(kPlanThreads) void k_attention_plan(AttentionParams p)
{
    __shared__ AttnSums scratch[kPlanThreads / 64];
    lay_out<kPlanThreads>(p, p.segs, scratch);
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

__device__ __forceinline__ float load_as_float(const void* from, int64_t at, int dtype)
{
    if (dtype == DWS_FLOAT32) return static_cast<const float*>(from)[at];
    if (dtype == DWS_BFLOAT16) return (float)static_cast<const bf16_t*>(from)[at];
    return (float)static_cast<const f16_t*>(from)[at];
}

// Four dimensions from d on, which are whole units where whole_out says so.
template <class T, class V>
__device__ __forceinline__ void store_four_as(const AttentionParams& p, int64_t at, int d, V x)
{
    typedef T Four __attribute__((ext_vector_type(4)));
    T* to = static_cast<T*>(p.out.data) + at + d;
    if (p.whole_out) {
        if (d < p.c.dim_v) *reinterpret_cast<Four*>(to) = __builtin_convertvector(x, Four);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (d + k < p.c.dim_v) to[k] = (T)x[k];
    }
}
template <class V>
__device__ __forceinline__ void store_four(const AttentionParams& p, int64_t at, int d, V x)
{
    if (p.dtype == DWS_FLOAT32)
        store_four_as<float>(p, at, d, x);
    else if (p.dtype == DWS_BFLOAT16)
        store_four_as<bf16_t>(p, at, d, x);
    else
        store_four_as<f16_t>(p, at, d, x);
}

// One row of queries by the whole workgroup, 256 tokens at a time, each token's score
// by a thread and each dimension's sum by a thread: only what the row sees is touched,
// so that values which are not finite stay with those that see them.
struct Again {
    float score[kJoinThreads], red[kJoinThreads / 64];
    int64_t value[kJoinThreads];
};
__device__ void row_again(const AttentionParams& p, const AttnDone& a, int h, int64_t behind, Again& s)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t token = a.begin + behind / p.share;
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
            const int page = p.c.table[a.table * p.c.max_pages + t / p.c.page_tokens], place = t % p.c.page_tokens;
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
// dimensions a thread; with few rows the parts are shared out to threads, too. Bound
// by the bytes of the parts, (padded + 2) 4 for each of their rows, and with few of
// them by three trips to memory.
__global__ __launch_bounds__(kJoinThreads) void k_attention_join(AttentionParams p)
{
    typedef float f32x4 __attribute__((ext_vector_type(4)));
    __shared__ float sums[kJoinThreads][4];
    __shared__ float2 stats[kJoinThreads];
    __shared__ Again again;
    const int tid = threadIdx.x, quads = p.padded / 4, lines = kJoinThreads / quads;        // rows, or parts of rows, at a time
    const int q = tid & (quads - 1), line = tid / quads;
    const int row0 = blockIdx.y * kJoinRows;
    const uint32_t tiles = (uint32_t)*p.tiles * (uint32_t)p.c.heads;
    for (uint32_t number = blockIdx.x; number < p.max_tiles * p.c.heads; number += gridDim.x) {
        const AttnDone a = p.done[number];
        if (number >= tiles) break;
        const int h = (int)(number % (uint32_t)p.c.heads);
        const int end = a.rows < row0 + kJoinRows ? a.rows : row0 + kJoinRows;
        if (a.kind == 2 || row0 >= end || (a.kind == 0 && a.first == -1)) continue;
        int ways = 1;
        while (ways * 2 * (end - row0) <= lines) ways *= 2;
        const int way = line & (ways - 1);
        bool wild = a.first == -2;
        for (int r0 = row0; r0 < end; r0 += lines / ways) {
            const int r = r0 + line / ways;
            f32x4 sum = {0.f, 0.f, 0.f, 0.f};
            float m = -__builtin_inff(), l = 0.f;
            auto add = [&](f32x4 o, float2 y) {
                if (y.y == 0.f) return;         // saw nothing
                const float top = fmaxf(m, y.x);
                const float was = m == top ? 1.f : __builtin_amdgcn_exp2f(m - top);
                const float is = y.x == top ? 1.f : __builtin_amdgcn_exp2f(y.x - top);
                sum = sum * was + o * is;
                l = l * was + y.y * is;
                m = top;
            };
            // a tile's row: of the one workgroup that has all of it, or of all that have a part
            auto gather = [&](const AttnDone& t, int row) {
                if (t.first < 0) {
                    if (t.kind == 0 || way > 0) return;
                    const int64_t at = h * p.max_apart + t.slot + row;
                    const float2 y = p.apart_stat[at];
                    wild |= y.y < 0.f;
                    add(*reinterpret_cast<const f32x4*>(p.apart + at * p.padded + 4 * q), y);
                    return;
                }
                const int n = t.last - t.first + 1;
                for (int k0 = way; k0 < n; k0 += 8 * ways) {
                    f32x4 o[8];
                    float2 y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int k = k0 + i * ways;
                        if (k >= n) break;
                        const int64_t at = (2 * (int64_t)(t.first + k) + (k == 0 ? 1 : 0)) * p.tile_rows + row;
                        y[i] = p.part_stat[at];
                        o[i] = *reinterpret_cast<const f32x4*>(p.part + at * p.padded + 4 * q);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (k0 + i * ways >= n) break;
                        wild |= y[i].y < 0.f;
                        add(o[i], y[i]);
                    }
                }
            };
            if (r < end && a.table >= 0) {
                // the group's tile with the row is on its way while the own parts are added
                AttnDone g{};
                int in = 0;
                if (a.kind == 1) {
                    const int64_t row = a.group_row + r, tile = a.group_tile + (row >> p.shift);
                    in = (int)(row & ((1 << p.shift) - 1));
                    if (row >= 0 && tile < *p.tiles) g = p.done[tile * p.c.heads + h];
                }
                gather(a, r);
                if (in < g.rows) gather(g, in);
            }
            if (ways > 1) {
                *reinterpret_cast<f32x4*>(sums[tid]) = sum;
                stats[tid] = make_float2(m, l);
                __syncthreads();
                if (way == 0)
                    for (int k = 1; k < ways; ++k) add(*reinterpret_cast<const f32x4*>(sums[tid + k * quads]), stats[tid + k * quads]);
                __syncthreads();
            }
            if (r >= end || way > 0 || a.first == -2) continue;
            const int64_t behind = a.row + r, token = a.begin + behind / p.share;
            const int head = h * p.share + (int)(behind % p.share);
            const float by = l == 0.f ? 0.f : 1.f / l;
            store_four(p, token * p.out.ts + head * p.out.hs, 4 * q, l == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f} : sum * by);
            if (q == 0 && p.lse != nullptr)
                p.lse[token * p.heads_q + head] = l == 0.f ? -__builtin_inff() : (m + __builtin_log2f(l)) * 0.693147180559945f;
        }
        if (__syncthreads_or(wild))
            for (int r = row0; r < end; ++r) row_again(p, a, h, a.row + r, again);
    }
    if (!p.zero_rest || blockIdx.y > 0) return;
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
    if (!p.own_plan) {
        k_attention_plan<<<1, kPlanThreads, 0, stream>>>(p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const hipError_t e = p.dtype == DWS_FLOAT32    ? launch_attention_f32(p, stream)
                         : p.dtype == DWS_BFLOAT16 ? launch_attention_bf16(p, stream)
                                                   : launch_attention_f16(p, stream);
    if (e != hipSuccess) return e;
    const int64_t most = p.max_tiles * p.c.heads;
    const dim3 grid((unsigned)(most < 1 ? 1 : (most < 2048 ? most : 2048)), (unsigned)((p.tile_rows + kJoinRows - 1) / kJoinRows));
    k_attention_join<<<grid, kJoinThreads, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace dws
