// Attention over cached keys and values: the kernel.
//
//   out = sum_t p_t v_t / sum_t p_t,  p_t = 2^(c q . k_t - m),  c = scale log2(e)
//
// in one pass over the tokens t, with m a running maximum. A wave holds 32 queries
// (rows (token, head) that share a key head) in registers and takes 32 tokens at a
// time: S^T = K Q^T leaves a query's scores in one lane and the lane 32 beside it, so
// that the softmax needs one exchange between lanes, and P^T is, as it lies, the
// operand of O^T = V^T P^T, whose columns are again queries: rescaling is a product
// with the lane's own factor.
//
// Tiles of up to 32 queries are memory bound (2 operations a query for each byte of
// keys): their waves work on 32 tokens each and are joined at the end. Larger ones are
// bound by the matrix products and the softmax beside them: each wave brings 16 tokens,
// and goes with its own 32 queries (of 128 in all) through the 64 of all waves, or (of 64)
// through half of them. The next piece's keys and values are on their way meanwhile: to the
// other half of the LDS by themselves, or in registers where two pieces do not fit there or
// rows are not whole units of 16 bytes.
//
// Measured, with the joining, a call: 96 sequences of 1 to 16,000 tokens, 8 heads of 128, 4
// queries each, bf16: 156 us, 4.7 TB/s of keys and values. 3 prompts of 900 to 2,000 tokens
// behind 4,097: 731 us, 610 TFLOP/s without the weights' second part, where a large matrix
// product reaches 1,274 in the same session. Each SIMD's vector instructions take 52% of the
// time (scores to weights: 5 of 32 bits for each, 4 times one for the exponential) and its
// matrix products 48%: two waves hide what one waits for, and hardly overlap the two. Tiles
// of 256 queries would halve the reads of the LDS (23% of the time), but leave one wave a
// SIMD. With weights in one part, where a caller asks for that, 583 us.
//
// Fragments (32 x 32 tiles, h = lane / 32):
//   operand  lane holds row (or column) lane % 32, contraction indices 8 h .. 8 h + 7 of
//            16 (16 bits), or h of 2 (fp32, where a chunk of four takes four products)
//   result   lane holds column lane % 32, rows 8 (i / 4) + 4 h + i % 4, i = 0 .. 15
// A contraction may run in any order that both operands share: P's eight elements of a
// step are the rows above, and the transposing LDS reads bring V's in the same order.
#pragma once

#include <stddef.h>

#include <type_traits>

#include "dws_attention_work.hpp"

namespace dws {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char* LdsBytes;      // 32-bit addresses, so that offsets fold into the accesses
template <class X>
using InLds = __attribute__((address_space(3))) X*;
template <class T>
using Chunk = T __attribute__((ext_vector_type(16 / sizeof(T))));

__device__ __forceinline__ f32x16_t mma(Chunk<bf16_t> a, Chunk<bf16_t> b, f32x16_t c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16_t mma(Chunk<f16_t> a, Chunk<f16_t> b, f32x16_t c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16_t mma(Chunk<float> a, Chunk<float> b, f32x16_t c)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
    return c;
}

// The larger (the sum) of a lane's value and that of the lane 32 beside it.
__device__ __forceinline__ float max_halves(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float sum_halves(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

// PARTS: of the weights in tiles of more than 32 queries.
template <class T, int D, int NW, int ACCESS, int PARTS>
struct Attention {
    static constexpr bool WHOLE = ACCESS != kElements;
    static constexpr int CH = 16 / sizeof(T);           // elements of a chunk
    static constexpr int NCH = D / CH;                  // chunks of a row
    static constexpr int ROW = D * (int)sizeof(T);      // bytes of a row
    static constexpr int TILE = kKvTokens * ROW;        // bytes of 32 rows
    static constexpr int RESULT = kAttnRows * D * 4;    // of a wave's results
    static constexpr int N = kKvTokens * NCH / 64;      // chunks of a tile in a lane
    static constexpr int STEP = 64 / NCH;               // rows that 64 lanes hold at a time
    static constexpr int BLOCKS = D / 32;
    static constexpr int THREADS = 64 * NW;
    // Whether a piece waits in registers: not where 4 N of them do not fit.
    static constexpr bool kAhead = N <= 16 && (WHOLE || ROW <= 256);
    static constexpr int kBatch = N > 16 ? 16 : 8;      // loads at a time where it does not
    // Whether a small tile's keys and values both do.
    static constexpr bool kBoth = kAhead && D * sizeof(T) <= 256;
    static constexpr int SUB = NW / 2;                  // tiles of 32 tokens that all waves go through at a time
    // Whether the pieces of larger tiles go from memory to the LDS by themselves: two fit there.
    static constexpr bool kStream = ACCESS == kNear && sizeof(T) == 2 && D <= 128;
    static_assert(!kStream || 4 * SUB * TILE <= NW * RESULT, "two pieces of keys and values");

    struct Lds {
        // a wave's keys, then its values; or all waves' keys, and their values; then results
        alignas(16) char kv[NW * (TILE > RESULT ? TILE : RESULT)];
        AttnSeg segs[kAttnSegs + 1];
        // where a token's keys and values are: elements, or 16 bytes of 32-bit numbers
        std::conditional_t<ACCESS == kNear, uint32_t, int64_t> at[NW][2][kKvTokens];
        uint32_t there[2][NW];          // which of a wave's tokens are there, of a piece and the next
        int wild[2];                    // rows to compute again, of this tile and the next
        float m[kAttnRows * NW], l[kAttnRows * NW];
    };

    // (m0 has 16 bits for the place in the LDS, where this is the kernel's only variable)
    static_assert(!kStream || (offsetof(Lds, kv) == 0 && sizeof(Lds::kv) <= 1 << 16), "streamed within the first 64 KB");

    // Chunks of a row are permuted so that reads of one column by 16 rows (keys), and
    // of four rows by 16 columns (values), go to different banks.
    static constexpr int SPAN = NCH < 16 ? 16 / NCH : 1;        // rows of 256 bytes
    static constexpr int MASK = (NCH < 16 ? NCH : 16) - 1;
    static __device__ __forceinline__ int key_swizzle(int row) { return (row / SPAN) & MASK; }
    static __device__ __forceinline__ int value_swizzle(int row)
    {
        if constexpr (sizeof(T) == 4) return ((row >> 2) & 1) << 3;
        return ((row / SPAN) << 2) & MASK & 12;
    }

    const AttentionParams& p;
    Lds& s;
    int lane, half, col;
    const int wave;
    int kv_head, sets;                  // sets: of 32 queries, 1, 2 or 4
    AttnSeg seg;
    AttnTile a;
    bool group;
    int turn;                           // which of Lds.wild
    int64_t table;
    const T *keys_of_head, *values_of_head;
    int stop;                           // tokens of the stretch end here
    Chunk<T> q[NCH / 2];
    int position;                       // of the lane's query
    int least;                          // smallest of the wave's queries
    float c, c_rest;                    // scale log2(e), and what fp32 loses of it
    f32x16_t o[BLOCKS];
    float m, l;

    uint32_t there;                     // which of the wave's tokens are

    __device__ __forceinline__ Attention(const AttentionParams& p, Lds& s)
        : p(p), s(s), lane(threadIdx.x & 63), half(lane >> 5), col(lane & 31), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6))
    {
    }

    __device__ __forceinline__ void row_place(int64_t r, int64_t* token, int* head) const
    {
        const int64_t at = a.row + r;
        if (at < (int64_t)1 << 31) {
            const uint32_t t = (uint32_t)at / (uint32_t)p.share;
            *token = seg.begin + t;
            *head = kv_head * p.share + (int)((uint32_t)at - t * (uint32_t)p.share);
        } else {
            *token = seg.begin + at / p.share;
            *head = kv_head * p.share + (int)(at % p.share);
        }
    }

    // Where a query of a group's tile stands in its own row. Of a sequence without a row: behind
    // everything, so that no piece has places that it alone must not see; the joining leaves it out.
    __device__ __forceinline__ int position_in_group(const AttnSeg* segs, int64_t token) const
    {
        int64_t lo = 0, hi = p.c.n - 1;
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) / 2;
            if (segs[p.n_groups + mid].begin <= token)
                lo = mid;
            else
                hi = mid - 1;
        }
        const AttnSeg& x = segs[p.n_groups + lo];
        return x.length > 0 ? x.length - x.count + (int)(token - x.begin) : INT32_MAX;
    }
    __device__ __forceinline__ void load_queries(const AttnSeg* segs)
    {
        const int r = (wave & (sets - 1)) * kAttnRows + col;
        const bool in = r < a.rows;
        int64_t token = 0;
        int head = 0;
        if (in) row_place(r, &token, &head);
        position = INT32_MAX;
        if (in) position = group ? position_in_group(segs, token) : seg.length - seg.count + (int)(token - seg.begin);
        least = position;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            const int y = __shfl_xor(least, d, 64);
            least = y < least ? y : least;
        }
        least = __builtin_amdgcn_readfirstlane(least);
        // the scale's sign goes to the queries, so that the largest product has the largest score
        const float sign = p.sign;
        c = p.log2_scale;
        c_rest = p.log2_rest;
        const T* from = static_cast<const T*>(p.q.data) + token * p.q.ts + head * p.q.hs;
#pragma unroll
        for (int i = 0; i < NCH / 2; ++i) {
            const int d = (2 * i + half) * CH;
            Chunk<T> x;
            if (p.whole_q) {
                x = in && d < p.c.dim_k ? *reinterpret_cast<const Chunk<T>*>(from + d) : Chunk<T>{};
            } else {
#pragma unroll
                for (int j = 0; j < CH; ++j) x[j] = in && d + j < p.c.dim_k ? from[d + j] : (T)0.f;
            }
            if (sign != 1.f) {
#pragma unroll
                for (int j = 0; j < CH; ++j) x[j] = sign == 0.f ? (T)0.f : -x[j];
            }
            q[i] = x;
        }
    }

    __device__ __forceinline__ uint32_t page_number(uint32_t t) const
    {
        return p.c.page_magic == 0 ? t : __umulhi(t, p.c.page_magic) >> p.c.page_shift;
    }
    // The page of the token that the lane looks up, of `tokens`.
    __device__ __forceinline__ int page_of(int first, int tokens) const
    {
        const int t = first + lane;
        if (lane >= tokens || (uint32_t)t >= (uint32_t)stop) return -1;
        return (p.c.table + table)[page_number((uint32_t)t)];
    }
    // Finds the tokens of a tile, and returns which are there. (The others are read from
    // the pool's beginning, and become 0 before they are used.)
    __device__ __forceinline__ uint32_t places(int first, int page)
    {
        const uint32_t t = (uint32_t)(first + lane), place = t - page_number(t) * (uint32_t)p.c.page_tokens;
        const bool there = (uint32_t)page < (uint32_t)p.c.n_pages;
        if (lane < kKvTokens) {
            if constexpr (ACCESS == kNear) {
                s.at[wave][0][lane] = there ? (uint32_t)page * p.key_ps + place * p.key_ts : 0;
                s.at[wave][1][lane] = there ? (uint32_t)page * p.value_ps + place * p.value_ts : 0;
            } else {
                s.at[wave][0][lane] = there ? page * p.c.keys.ps + place * p.c.keys.ts : 0;
                s.at[wave][1][lane] = there ? page * p.c.values.ps + place * p.c.values.ts : 0;
            }
        }
        wave_sync();
        return (uint32_t)__ballot(there);
    }
    using Place = std::conditional_t<ACCESS == kNear, uint32_t, int64_t>;
    template <bool VALUES>
    __device__ __forceinline__ Place place_of(int i) const
    {
        return s.at[wave][VALUES][i * STEP + lane / NCH];
    }
    // 128 bits moved down by 0 to 127.
    static __device__ __forceinline__ u32x4_t shifted(u32x4_t x, int by)
    {
        const uint64_t lo = (uint64_t)x[1] << 32 | x[0], hi = (uint64_t)x[3] << 32 | x[2];
        const uint64_t up = hi >> (by & 63);
        const uint64_t a = by < 64 ? lo >> (by & 63) | hi << 1 << (63 - (by & 63)) : up, b = by < 64 ? up : 0;
        return u32x4_t{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)};
    }
    template <bool VALUES>
    __device__ __forceinline__ u32x4_t load(Place at) const
    {
        const int dim = VALUES ? p.c.dim_v : p.c.dim_k, d = (lane % NCH) * CH;
        const T* from = VALUES ? values_of_head : keys_of_head;
        if constexpr (ACCESS == kNear) {
            // (chunks behind the last dimension are read from the first one)
            return *reinterpret_cast<const u32x4_t*>(reinterpret_cast<const char*>(from + (d < dim ? d : 0)) + ((uint64_t)at << 4));
        } else if constexpr (WHOLE) {
            return *reinterpret_cast<const u32x4_t*>(from + at + (d < dim ? d : 0));
        } else {
            // rows at any address, 16 bytes at a time too; the last ones end with the row (`only_there`
            // moves them to the front)
            if (dim >= CH) {
                // (as memory that is global: loads that might be of the LDS too may not be at any address)
                typedef u32x4_t Loose __attribute__((aligned(2)));
                return *(const __attribute__((address_space(1))) Loose*)(from + at + (d + CH <= dim ? d : dim - CH));
            }
            Chunk<T> x;
#pragma unroll
            for (int j = 0; j < CH; ++j) x[j] = from[at + (d + j < dim ? d + j : 0)];
            return __builtin_bit_cast(u32x4_t, x);
        }
    }
    // The chunk with 0 where the row or the dimension is not there.
    __device__ __forceinline__ u32x4_t only_there(int i, u32x4_t x, uint32_t there, int dim) const
    {
        const int d = (lane % NCH) * CH;
        const bool row = (there >> (i * STEP + lane / NCH)) & 1;
        if constexpr (WHOLE) return row && d < dim ? x : u32x4_t{};
        const int behind = d + CH - dim;        // elements of the chunk
        Chunk<T> y = __builtin_bit_cast(Chunk<T>, dim >= CH && behind > 0 && behind < CH ? shifted(x, 8 * (int)sizeof(T) * behind) : x);
#pragma unroll
        for (int j = 0; j < CH; ++j) y[j] = row && d + j < dim ? y[j] : (T)0.f;
        return __builtin_bit_cast(u32x4_t, y);
    }
    // Row i * STEP + lane / NCH; what depends on the lane alone stands apart.
    template <bool VALUES>
    __device__ __forceinline__ void put_chunk(LdsBytes to, int i, u32x4_t x)
    {
        static_assert(STEP * SPAN == 1 || (16 % STEP == 0 && (STEP % SPAN == 0 || SPAN == 1)), "rows' bits stand apart");
        const int r = lane / NCH;
        const int c = (lane % NCH) ^ (VALUES ? value_swizzle(r) : key_swizzle(r));
        *(InLds<u32x4_t>)(to + r * ROW + ((c ^ (VALUES ? value_swizzle(i * STEP) : key_swizzle(i * STEP))) << 4) + i * STEP * ROW) = x;
    }
    // Keys (values) of the wave's tokens, whose places are known, to registers and then to
    // the LDS; 0 for what is not there.
    template <bool VALUES, int COUNT>
    __device__ __forceinline__ void fetch(u32x4_t (&next)[kAhead ? N : 1]) const
    {
        if constexpr (kAhead) {
            Place at[COUNT];
#pragma unroll
            for (int i = 0; i < COUNT; ++i) at[i] = place_of<VALUES>(i);
            __builtin_amdgcn_sched_barrier(0);          // all places before the first load
#pragma unroll
            for (int i = 0; i < COUNT; ++i) next[i] = load<VALUES>(at[i]);
        }
    }
    template <bool VALUES, int COUNT>
    __device__ __forceinline__ void put(LdsBytes to, u32x4_t (&next)[kAhead ? N : 1])
    {
        const int dim = VALUES ? p.c.dim_v : p.c.dim_k;
        if constexpr (kAhead) {
            if (there != (uint32_t)((1ull << (COUNT * STEP)) - 1) || dim != D) {
#pragma unroll
                for (int i = 0; i < COUNT; ++i) next[i] = only_there(i, next[i], there, dim);
            }
#pragma unroll
            for (int i = 0; i < COUNT; ++i) put_chunk<VALUES>(to, i, next[i]);
        } else {
#pragma unroll kBatch
            for (int i = 0; i < COUNT; ++i) put_chunk<VALUES>(to, i, only_there(i, load<VALUES>(place_of<VALUES>(i)), there, dim));
        }
    }

    // Eight (four) values of V's column (dimension) 32 block + col, of the tokens that
    // step u's eight (four) elements of P belong to.
    __device__ __forceinline__ Chunk<T> value_fragment(LdsBytes values, int block, int u) const
    {
        if constexpr (sizeof(T) == 2) {
            const int r = (lane >> 2) & 3;      // the row that the lane points at, of four
            const int low = 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
            const LdsBytes at = values + (4 * half + r) * ROW + 8 * (lane & 1) + (((4 * block) ^ (low ^ value_swizzle(r))) << 4) + 16 * u * ROW;
            const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((InLds<s16x4_t>)at);
            const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((InLds<s16x4_t>)(at + 8 * ROW));
            return __builtin_bit_cast(Chunk<T>, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            Chunk<T> x;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = value_at(values, 8 * u + 4 * half + j, 32 * block + col);
            return x;
        }
    }
    static __device__ __forceinline__ T value_at(LdsBytes values, int row, int d)
    {
        return *(InLds<T>)(values + row * ROW + (((d / CH) ^ value_swizzle(row)) << 4) + (d % CH) * sizeof(T));
    }
    static __device__ __forceinline__ bool finite(T x) { return __builtin_fabsf((float)x) < __builtin_inff(); }

    // Operands are read from the LDS before their products begin, and those of a second
    // tile among the products of the first: left to itself, the compiler waits for each
    // before its product.
    static constexpr bool kAmong = D * sizeof(T) <= 256;       // registers for two tiles
    struct Operands {
        Chunk<T> x[NCH / 2];
    };
    static __device__ __forceinline__ void reads_before_products()
    {
        if constexpr (kAmong) __builtin_amdgcn_sched_barrier(0);
    }
    template <int COUNT, int READS, int PRODUCTS = 1>
    static __device__ __forceinline__ void reads_among_products()
    {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);                              // LDS reads
            __builtin_amdgcn_sched_group_barrier(0x008, PRODUCTS * (sizeof(T) == 2 ? 1 : CH), 0);            // matrix products
        }
    }
    __device__ __forceinline__ Chunk<T> key_fragment(LdsBytes keys, int i) const
    {
        return *(InLds<Chunk<T>>)(keys + col * ROW + (((2 * i) ^ (half ^ key_swizzle(col))) << 4));
    }
    // Products of a tile's 32 keys and the wave's queries; of two.
    __device__ __forceinline__ f32x16_t scores(LdsBytes keys) const
    {
        Operands k;
#pragma unroll
        for (int i = 0; i < NCH / 2; ++i) k.x[i] = key_fragment(keys, i);
        reads_before_products();
        f32x16_t x = {};
#pragma unroll
        for (int i = 0; i < NCH / 2; ++i) x = mma(k.x[i], q[i], x);
        return x;
    }
    __device__ __forceinline__ void scores(LdsBytes keys, f32x16_t (&x)[1]) const { x[0] = scores(keys); }
    __device__ __forceinline__ void scores(LdsBytes keys, f32x16_t (&x)[2]) const
    {
        if constexpr (!kAmong) {
            x[0] = scores(keys);
            x[1] = scores(keys + TILE);
            return;
        }
        Operands k[2];
#pragma unroll
        for (int i = 0; i < NCH / 2; ++i) k[0].x[i] = key_fragment(keys, i);
        reads_before_products();
        x[0] = x[1] = f32x16_t{};
#pragma unroll
        for (int i = 0; i < NCH / 2; ++i) {
            k[1].x[i] = key_fragment(keys + TILE, i);
            x[0] = mma(k[0].x[i], q[i], x[0]);
        }
        reads_among_products<NCH / 2, 1>();
        reads_before_products();
#pragma unroll
        for (int i = 0; i < NCH / 2; ++i) x[1] = mma(k[1].x[i], q[i], x[1]);
    }
    // Whether there are tokens among the 32 from `first` on that not every query sees.
    __device__ __forceinline__ bool masked(uint32_t there, int first) const
    {
        return there != 0xffffffffu || (int64_t)first + kKvTokens - 1 > least;
    }
    // A value that is not finite, of a token that not every query sees: 0 times it is not
    // 0. Such a tile's rows are computed again, one by one, where the parts are joined.
    __device__ __forceinline__ void note_wild(LdsBytes values)
    {
        bool bad = false;
#pragma unroll 1
        for (int i = 0; i < NCH / 2; ++i) {
            const Chunk<T> v = *(InLds<Chunk<T>>)(values + col * ROW + ((2 * i + half) << 4));
#pragma unroll
            for (int j = 0; j < CH; ++j) bad |= !finite(v[j]);
        }
        if (__ballot(bad)) s.wild[turn] = 1;
    }

    // Scores of 32 tokens, of which the bits in `here` are there: -infinity for those that
    // the lane's query does not see; returns the largest.
    __device__ __forceinline__ float only_seen(f32x16_t& x, uint32_t here, int first) const
    {
        if (masked(here, first)) {
            const int past = position - first;      // the last token that the query sees
            const uint32_t sees = (here & (past < 0 ? 0u : 0xffffffffu >> (past > 31 ? 0 : 31 - past))) >> (4 * half);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = sees >> (8 * (e / 4) + e % 4) & 1 ? x[e] : -__builtin_inff();
        }
        float top = x[0];
#pragma unroll
        for (int e = 1; e < 16; ++e) top = fmaxf(top, x[e]);
        return top;
    }
    // The maximum follows once a score is 2^kLag times above it: until then sums grow by
    // that, and the results need no rescaling. fp16 holds numbers from 2^-24 to 2^16, so its
    // weights go by 2^11 times less than the maximum: what is up to 2^36 below it still counts.
    // (With the maximum itself, what is 2^25 below it was lost from the products and not from the
    // sum: 3% of the results of 100,001 tokens of which one outweighs each other by e^17.7 and has a
    // 16th of their values.)
    static constexpr bool kNarrow = std::is_same_v<T, f16_t>;
    static constexpr float kLag = kNarrow ? 4.f : 8.f, kHeadroom = kNarrow ? 11.f : 0.f;
    __device__ __forceinline__ void follow(float top)
    {
        top = max_halves(top) * c;
        if (__ballot(top > m + kLag)) {
            const float now = fmaxf(m, top);
            const float by = now == m ? 1.f : __builtin_amdgcn_exp2f(m - now);
            l *= by;
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) o[b] *= by;
            m = now;
        }
    }
    static constexpr int STEPS = 16 / CH;       // steps of the second product
    static constexpr int kSmallParts = sizeof(T) == 2 ? 2 : 1;
    struct Weights {
        Chunk<T> p[STEPS];
    };
    // Two weights in 16 bits, less than they are, and what that leaves of them in `rest`. Both
    // parts are above 0 where the weight is, so that a value that is infinite stays so: rounded to the
    // nearest, the second part is 0 or below it for every other weight, and the sum of the products NaN.
    static __device__ __forceinline__ uint32_t parted(float x, float y, float (&rest)[2])
    {
        if constexpr (kNarrow) {
            typedef uint16_t Pair __attribute__((ext_vector_type(2)));
            typedef f16_t Halves __attribute__((ext_vector_type(2)));
            const Pair down = __builtin_elementwise_sub_sat(__builtin_bit_cast(Pair, __builtin_amdgcn_cvt_pkrtz(x, y)), Pair{1, 1});
            const Halves w = __builtin_bit_cast(Halves, down);
            rest[0] = x - (float)w[0];
            rest[1] = y - (float)w[1];
            return __builtin_bit_cast(uint32_t, down);
        } else {
            // (the 2^-20 added are a 2^11th of the result's rounding)
            const uint32_t a = __builtin_bit_cast(uint32_t, x), b = __builtin_bit_cast(uint32_t, y);
            rest[0] = __builtin_fmaf(x, 1.f + 0x1p-20f, -__builtin_bit_cast(float, a & 0xffff0000u));
            rest[1] = __builtin_fmaf(y, 1.f + 0x1p-20f, -__builtin_bit_cast(float, b & 0xffff0000u));
            return __builtin_amdgcn_perm(b, a, 0x07060302);         // the upper halves
        }
    }
    // `rest`: the second part, if they are wanted in two.
    template <int COUNT>
    __device__ __forceinline__ Weights weights(const f32x16_t& x, Weights& rest)
    {
        Weights w;
        const float base = m == -__builtin_inff() ? 0.f : m - kHeadroom;
        float y[16], sum = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            y[e] = __builtin_fmaf(x[e], c, -base);
            if constexpr (sizeof(T) == 4)
                if (x[e] != -__builtin_inff()) y[e] = __builtin_fmaf(x[e], c_rest, y[e]);
            y[e] = __builtin_amdgcn_exp2f(y[e]);
            sum += y[e];
            if constexpr (COUNT == 1) {
                w.p[e / CH][e % CH] = (T)y[e];
            } else if (e % 2) {
                typedef T Pair __attribute__((ext_vector_type(2)));
                float left[2];
                const Pair both = __builtin_bit_cast(Pair, parted(y[e - 1], y[e], left));
                w.p[e / CH][e % CH - 1] = both[0];
                w.p[e / CH][e % CH] = both[1];
                rest.p[e / CH][e % CH - 1] = (T)left[0];
                rest.p[e / CH][e % CH] = (T)left[1];
            }
        }
        l += sum;
        return w;
    }
    // Products of a tile's 32 values and the weights, added to the results; of two tiles.
    static constexpr int FRAGMENTS = BLOCKS * STEPS;
    struct Values {
        Chunk<T> x[FRAGMENTS];
    };
    template <int COUNT>
    __device__ __forceinline__ void add_product(int i, const Values& v, const Weights& w, const Weights& rest)
    {
        o[i / STEPS] = mma(v.x[i], w.p[i % STEPS], o[i / STEPS]);
        if constexpr (COUNT == 2) o[i / STEPS] = mma(v.x[i], rest.p[i % STEPS], o[i / STEPS]);
    }
    template <int COUNT>
    __device__ __forceinline__ void accumulate(LdsBytes values, const Weights& w, const Weights& rest)
    {
        Values v;
#pragma unroll
        for (int i = 0; i < FRAGMENTS; ++i) v.x[i] = value_fragment(values, i / STEPS, i % STEPS);
        reads_before_products();
#pragma unroll
        for (int i = 0; i < FRAGMENTS; ++i) add_product<COUNT>(i, v, w, rest);
    }
    template <int COUNT>
    __device__ __forceinline__ void accumulate(LdsBytes values, const Weights (&w)[1], const Weights (&rest)[1])
    {
        accumulate<COUNT>(values, w[0], rest[0]);
    }
    template <int COUNT>
    __device__ __forceinline__ void accumulate(LdsBytes values, const Weights (&w)[2], const Weights (&rest)[2])
    {
        if constexpr (!kAmong) {
            accumulate<COUNT>(values, w[0], rest[0]);
            accumulate<COUNT>(values + TILE, w[1], rest[1]);
            return;
        }
        Values v[2];
#pragma unroll
        for (int i = 0; i < FRAGMENTS; ++i) v[0].x[i] = value_fragment(values, i / STEPS, i % STEPS);
        reads_before_products();
#pragma unroll
        for (int i = 0; i < FRAGMENTS; ++i) {
            v[1].x[i] = value_fragment(values + TILE, i / STEPS, i % STEPS);
            add_product<COUNT>(i, v[0], w[0], rest[0]);
        }
        reads_among_products<FRAGMENTS, sizeof(T) == 2 ? 2 : CH, COUNT>();
        reads_before_products();
#pragma unroll
        for (int i = 0; i < FRAGMENTS; ++i) add_product<COUNT>(i, v[1], w[1], rest[1]);
    }
    // Addresses are worked out anew for each piece: kept, they push results out of the registers.
    __device__ __forceinline__ void forget_addresses()
    {
        asm volatile("" : "+v"(lane));
        lane &= 63;         // (not negative, for divisions)
        half = lane >> 5;
        col = lane & 31;
    }

    // Tokens t .. end - 1 for up to 32 queries: 32 a wave.
    __device__ __forceinline__ void pieces_apart(int t, int end, int page)
    {
        constexpr int TOKENS = kKvTokens * NW;
        const LdsBytes mine = (LdsBytes)&s.kv[0] + wave * TILE;
        t += wave * kKvTokens;
        if (t >= end) return;
        // (without kBoth one set of registers serves both in turn)
        u32x4_t next[kAhead ? N : 1], also[kBoth ? N : 1];
        u32x4_t(&v)[kAhead ? N : 1] = value_registers(next, also);
        uint32_t after = places(t, page);
        fetch<false, N>(next);
        if (kBoth) fetch<true, N>(v);
        page = page_of(t + TOKENS, kKvTokens);
        for (; t < end; t += TOKENS) {
            forget_addresses();
            there = after;
            wave_sync();
            put<false, N>(mine, next);
            wave_sync();
            const bool more = t + TOKENS < end;
            if (!kBoth) fetch<true, N>(v);
            if (kBoth && more) {
                after = places(t + TOKENS, page);
                fetch<false, N>(next);
            }
            f32x16_t x = scores(mine);
            follow(only_seen(x, there, t));
            // In two parts 16-bit weights leave no error beside the result's own rounding (0.0017 of bf16
            // results instead of 0.0020), here for half a percent of 96 sequences of 1 to 16,000 tokens. In
            // larger tiles (0.0017 instead of 0.0023) for a quarter of prompts' time: PARTS.
            Weights w, rest;
            w = weights<kSmallParts>(x, rest);
            wave_sync();
            put<true, N>(mine, v);
            wave_sync();
            if (more) {
                if (kBoth) {
                    fetch<true, N>(v);
                } else {
                    after = places(t + TOKENS, page);
                    fetch<false, N>(next);
                }
                page = page_of(t + 2 * TOKENS, kKvTokens);
            }
            if (masked(there, t)) note_wild(mine);
            accumulate<kSmallParts>(mine, w, rest);
        }
    }
    static __device__ __forceinline__ auto value_registers(u32x4_t (&next)[kAhead ? N : 1], u32x4_t (&also)[kBoth ? N : 1])
        -> u32x4_t (&)[kAhead ? N : 1]
    {
        if constexpr (kBoth)
            return also;
        else
            return next;
    }
    // The same for more queries: the waves go through each other's tokens, SUBS tiles of them each.
    template <int SUBS>
    __device__ __forceinline__ void pieces_together(int t, int end, int page)
    {
        constexpr int TOKENS = 16 * NW, HALF = N / 2;
        const LdsBytes keys = (LdsBytes)&s.kv[0], values = keys + SUB * TILE;
        const int mine = wave * 16 * ROW;
        const int first_sub = SUBS == SUB ? 0 : wave / 2;
        uint32_t after = places(t + wave * 16, page);
        u32x4_t next[kAhead ? N : 1];
        fetch<false, HALF>(next);
        page = page_of(t + wave * 16 + TOKENS, 16);
        for (; t < end; t += TOKENS) {
            // Of the two workgroups on a compute unit the older one goes first, and would be done
            // long before the other: they take turns.
            if (((t / TOKENS) ^ (blockIdx.x / 256)) & 1)
                __builtin_amdgcn_s_setprio(1);
            else
                __builtin_amdgcn_s_setprio(0);
            forget_addresses();
            there = after;
            put<false, HALF>(keys + mine, next);
            if (lane == 0) s.there[0][wave] = there;
            fetch<true, HALF>(next);
            __syncthreads();
            // tiles of which a token is not there, in 32 bits
            f32x16_t x[SUBS];
            Weights w[SUBS], rest[SUBS];
            scores(keys + first_sub * TILE, x);
            uint32_t here[SUBS];
#pragma unroll
            for (int r = 0; r < SUBS; ++r)
                here[r] = __builtin_amdgcn_readfirstlane(s.there[0][2 * (first_sub + r)] | s.there[0][2 * (first_sub + r) + 1] << 16);
            float top = -__builtin_inff();
#pragma unroll
            for (int r = 0; r < SUBS; ++r) top = fmaxf(top, only_seen(x[r], here[r], t + (first_sub + r) * kKvTokens));
            follow(top);
#pragma unroll
            for (int r = 0; r < SUBS; ++r) w[r] = weights<PARTS>(x[r], rest[r]);
            put<true, HALF>(values + mine, next);
            if (t + TOKENS < end) {
                after = places(t + wave * 16 + TOKENS, page);
                fetch<false, HALF>(next);
                page = page_of(t + wave * 16 + 2 * TOKENS, 16);
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < SUBS; ++r)
                if (masked(here[r], t + (first_sub + r) * kKvTokens)) note_wild(values + (first_sub + r) * TILE);
            accumulate<PARTS>(values + first_sub * TILE, w, rest);
        }
        __builtin_amdgcn_s_setprio(0);
    }
    // Keys (values) of the wave's 16 tokens, whose places are known, from memory to the LDS, 64
    // lanes' chunks one behind the other, without a register between; each lane brings the chunk
    // that belongs into its place. In assembly, since of the compiler's own such loads every
    // read of the LDS would wait for all; `landed` does.
    template <bool VALUES>
    __device__ __forceinline__ uint32_t chunk_of(int i) const
    {
        const int r = lane / NCH;
        return (uint32_t)(lane % NCH) ^ (uint32_t)(VALUES ? value_swizzle(r) ^ value_swizzle(i * STEP) : key_swizzle(r) ^ key_swizzle(i * STEP));
    }
    template <bool VALUES>
    __device__ __forceinline__ void stream(LdsBytes to) const
    {
        const uint32_t chunks = (uint32_t)(VALUES ? p.c.dim_v : p.c.dim_k) / CH;
        const char* head = reinterpret_cast<const char*>(VALUES ? values_of_head : keys_of_head);
        Place at[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) at[i] = place_of<VALUES>(i);
        __builtin_amdgcn_sched_barrier(0);          // all places before the first load
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const uint32_t c = chunk_of<VALUES>(i);
            asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                         :
                         : "v"(head + ((uint64_t)(at[i] + (c < chunks ? c : 0)) << 4)), "s"((uint32_t)(uintptr_t)(to + i * STEP * ROW))
                         : "m0", "memory");
        }
    }
    __device__ __forceinline__ void stream_piece(LdsBytes keys) const
    {
        stream<false>(keys);
        stream<true>(keys + SUB * TILE);
    }
    // What has been streamed is there, and 0 where a token's values or a dimension are not.
    __device__ __forceinline__ void landed(LdsBytes keys) const
    {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        if (there == 0xffffu && p.c.dim_k == D && p.c.dim_v == D) return;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const InLds<u32x4_t> at = (InLds<u32x4_t>)(keys + i * STEP * ROW + lane * 16);
            if ((int)chunk_of<false>(i) * CH >= p.c.dim_k) *at = u32x4_t{};
            if (!(there >> (i * STEP + lane / NCH) & 1) || (int)chunk_of<true>(i) * CH >= p.c.dim_v) at[SUB * TILE / 16] = u32x4_t{};
        }
    }
    // pieces_together with the next piece's keys and values on their way to the other half of the LDS.
    template <int SUBS>
    __device__ __forceinline__ void pieces_streamed(int t, int end, int page)
    {
        constexpr int TOKENS = 16 * NW, PIECE = 2 * SUB * TILE;
        const LdsBytes kv = (LdsBytes)&s.kv[0];
        const int mine = wave * 16 * ROW, first_sub = SUBS == SUB ? 0 : wave / 2;
        uint32_t after = places(t + wave * 16, page);
        stream_piece(kv + mine);
        page = page_of(t + wave * 16 + TOKENS, 16);
        for (int turn = 0; t < end; t += TOKENS, turn ^= 1) {
            // Of the two workgroups on a compute unit the older one goes first, and would be done
            // long before the other: they take turns (2% of the prompts above).
            if ((turn ^ (blockIdx.x / 256)) & 1)
                __builtin_amdgcn_s_setprio(1);
            else
                __builtin_amdgcn_s_setprio(0);
            there = after;
            const LdsBytes keys = kv + turn * PIECE, values = keys + SUB * TILE;
            landed(keys + mine);
            if (lane == 0) s.there[turn][wave] = there;
            __syncthreads();            // and the other half has been read
            // tiles of which a token is not there, in 32 bits
            f32x16_t x[SUBS];
            Weights w[SUBS], rest[SUBS];
            scores(keys + first_sub * TILE, x);
            if (t + TOKENS < end) {
                after = places(t + wave * 16 + TOKENS, page);
                stream_piece(kv + (turn ^ 1) * PIECE + mine);
                page = page_of(t + wave * 16 + 2 * TOKENS, 16);
            }
            uint32_t here[SUBS];
#pragma unroll
            for (int r = 0; r < SUBS; ++r)
                here[r] = __builtin_amdgcn_readfirstlane(s.there[turn][2 * (first_sub + r)] | s.there[turn][2 * (first_sub + r) + 1] << 16);
            float top = -__builtin_inff();
#pragma unroll
            for (int r = 0; r < SUBS; ++r) top = fmaxf(top, only_seen(x[r], here[r], t + (first_sub + r) * kKvTokens));
            follow(top);
#pragma unroll
            for (int r = 0; r < SUBS; ++r) w[r] = weights<PARTS>(x[r], rest[r]);
#pragma unroll
            for (int r = 0; r < SUBS; ++r)
                if (masked(here[r], t + (first_sub + r) * kKvTokens)) note_wild(values + (first_sub + r) * TILE);
            accumulate<PARTS>(values + first_sub * TILE, w, rest);
        }
        __builtin_amdgcn_s_setprio(0);
    }
    template <int SUBS>
    __device__ __forceinline__ void pieces(int t, int end, int page)
    {
        if constexpr (kStream)
            pieces_streamed<SUBS>(t, end, page);
        else
            pieces_together<SUBS>(t, end, page);
    }

    __device__ __forceinline__ void store(int64_t at, f32x4_t x, int d)
    {
        T* to = static_cast<T*>(p.out.data) + at + d;
        if (p.whole_out) {
            typedef T Four __attribute__((ext_vector_type(4)));
            Four y;
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = (T)x[j];
            if (d < p.c.dim_v) *reinterpret_cast<Four*>(to) = y;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (d + j < p.c.dim_v) to[j] = (T)x[j];
        }
    }

    // Pieces first_step .. last_step - 1 of the tile's keys. `part`: where partial results go.
    __device__ __forceinline__ void run(const AttnSeg* segs, int first_step, int last_step, bool whole, int64_t part)
    {
        if (!whole && first_step >= last_step) {
            // a stretch that ends before the tile's first piece
            for (int r = threadIdx.x; r < a.rows; r += THREADS) p.part_stat[part * p.tile_rows + r] = make_float2(-__builtin_inff(), 0.f);
            if (threadIdx.x == 0) s.wild[turn ^ 1] = 0;
            return;
        }
        sets = a.rows <= kAttnRows ? 1 : (a.rows <= 2 * kAttnRows || NW == 2 ? 2 : NW);
        stop = a.end;
        table = seg.row * p.c.max_pages;
        keys_of_head = static_cast<const T*>(p.c.keys.data) + kv_head * p.c.keys.hs;
        values_of_head = static_cast<const T*>(p.c.values.data) + kv_head * p.c.values.hs;
        constexpr int PIECE = kKvTokens * NW;
        const int t = a.begin + first_step * PIECE;
        // (64 bits: the last piece may reach beyond 2^31)
        const int64_t behind = (int64_t)a.begin + (int64_t)last_step * PIECE;
        stop = behind < stop ? (int)behind : stop;
        // the first pages are looked up while the queries come
        const int mine = sets == 1 ? kKvTokens : 16, page = page_of(t + wave * mine, mine);
        load_queries(segs);
        m = -__builtin_inff();
        l = 0.f;
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) o[b] = f32x16_t{};
        if (t < stop) {
            if (sets == 1)
                pieces_apart(t, stop, page);
            else if (sets == NW)
                pieces<SUB>(t, stop, page);
            else if constexpr (NW > 2)
                pieces<1>(t, stop, page);
        }
        l = sum_halves(l);
        if (half == 0) {
            s.m[wave * kAttnRows + col] = m - kHeadroom;       // what the sums go by
            s.l[wave * kAttnRows + col] = l;
        }

        float* to = nullptr;
        float2* to_stat = nullptr;
        if (!whole) {
            to = p.part + part * p.tile_rows * D;
            to_stat = p.part_stat + part * p.tile_rows;
        } else if (seg.apart >= 0) {
            const int64_t row = kv_head * p.max_apart + seg.apart + a.row;
            to = p.apart + row * D;
            to_stat = p.apart_stat + row;
        }
        // Results by way of the LDS (a wave's own part of it), so that rows are written whole.
        constexpr int QUADS = D / 4;
        __syncthreads();            // the other waves are done with keys and values
        const InLds<float> mine_out = (InLds<float>)((LdsBytes)&s.kv[0] + wave * RESULT);
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *(InLds<f32x4_t>)(mine_out + col * D + (((8 * b + 2 * j + half) ^ (col & 15)) << 2)) =
                    f32x4_t{o[b][4 * j], o[b][4 * j + 1], o[b][4 * j + 2], o[b][4 * j + 3]};
        if (threadIdx.x == 0) s.wild[turn ^ 1] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < a.rows * QUADS; i += THREADS) {
            const int r = i / QUADS, quad = i % QUADS, in = r % kAttnRows;
            const int place = in * D + ((quad ^ (in & 15)) << 2);
            f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
            float most = -__builtin_inff(), total = 0.f;
            // the waves that have the row's queries
            for (int w = r / kAttnRows; w < NW; w += sets)
                if (s.l[w * kAttnRows + in] != 0.f) most = fmaxf(most, s.m[w * kAttnRows + in]);
            for (int w = r / kAttnRows; w < NW; w += sets) {
                const float lw = s.l[w * kAttnRows + in], mw = s.m[w * kAttnRows + in];
                if (lw == 0.f) continue;
                const float by = mw == most ? 1.f : __builtin_amdgcn_exp2f(mw - most);
                sum += *(InLds<f32x4_t>)((InLds<float>)((LdsBytes)&s.kv[0] + w * RESULT) + place) * by;
                total += lw * by;
            }
            if (to != nullptr) {
                *reinterpret_cast<f32x4_t*>(to + (int64_t)r * D + 4 * quad) = sum;
                // (a sum below 0: rows to compute again)
                if (quad == 0) to_stat[r] = make_float2(most, s.wild[turn] ? -1.f : total);
            } else {
                int64_t token;
                int head;
                row_place(r, &token, &head);
                const float by = total == 0.f ? 0.f : 1.f / total;
                store(token * p.out.ts + head * p.out.hs, total == 0.f ? f32x4_t{0.f, 0.f, 0.f, 0.f} : sum * by, 4 * quad);
                if (quad == 0 && p.lse != nullptr)
                    p.lse[token * p.heads_q + head] =
                        total == 0.f ? -__builtin_inff() : (most + __builtin_log2f(total)) * 0.693147180559945f;
            }
        }
    }
};

template <class X>
__device__ __forceinline__ X uniform(X x)
{
    static_assert(sizeof(X) % 4 == 0, "whole words");
    uint32_t w[sizeof(X) / 4];
    __builtin_memcpy(w, &x, sizeof(X));
#pragma unroll
    for (size_t i = 0; i < sizeof(X) / 4; ++i) w[i] = __builtin_amdgcn_readfirstlane(w[i]);
    __builtin_memcpy(&x, w, sizeof(X));
    return x;
}

// Waves a SIMD: queries, results, scores and the next keys take D sizeof(T) / 4 times 1/2
// and 1 registers, 16 to 32, and as many as the queries.
constexpr int attn_occupancy(int dim, int size) { return dim * size <= 128 ? 3 : (dim * size <= 256 ? 2 : 1); }

template <class T, int D, int NW, int ACCESS, int PARTS>
__global__ __launch_bounds__(64 * NW, attn_occupancy(D, sizeof(T))) void k_attention(
    AttentionParams given)
{
    __shared__ typename Attention<T, D, NW, ACCESS, PARTS>::Lds lds;
    if (threadIdx.x < 2) lds.wild[threadIdx.x] = 0;
    if (given.own_plan) lay_out<64 * NW>(given, lds.segs, reinterpret_cast<AttnSums*>(lds.kv));
    // The arguments once more, from where they are (the only ones, so at the beginning): held in scalar
    // registers across the layout, up to 190 of them are written to lanes of vector registers and
    // read back a thousand times. One sequence of 700 tokens 16.5 us instead of 18.1, 96 of 1 to
    // 16,000 148 instead of 154, the prompts above 696 instead of 715, one graph after another.
    auto args = (const __attribute__((address_space(4))) AttentionParams*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(args));
    const AttentionParams& p = *(const AttentionParams*)args;
    Attention<T, D, NW, ACCESS, PARTS> w(p, lds);
    const AttnWork work(p);
    const int all = (int)(p.n_groups + p.c.n);
    const AttnSeg* segs = p.own_plan ? lds.segs : p.segs;
    __syncthreads();
    const AttnSeg last = p.own_plan ? lds.segs[all] : p.segs[all];
    const uint32_t line = __builtin_amdgcn_readfirstlane(last.cost), whole_line = line * (uint32_t)p.c.heads;
    // (costs that sum up beyond 2^31 are of offsets that make no sense)
    const bool sane = line <= INT32_MAX / (uint32_t)p.c.heads;
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.tiles = sane ? last.tile : 0;
    const uint32_t stretch = __builtin_amdgcn_readfirstlane(work.stretch(whole_line));
    // neighbours in the line, which may read the same keys, on the same XCD (every eighth workgroup)
    const uint32_t x = p.workgroups % 8 == 0 ? blockIdx.x % 8 * (p.workgroups / 8) + blockIdx.x / 8 : blockIdx.x;
    if (!sane || (uint64_t)x * stretch >= whole_line) return;
    uint32_t at = x * stretch;
    const uint32_t end = whole_line - at < stretch ? whole_line : at + stretch;
    w.turn = 0;
    while (at < end) {
        const uint32_t head = __builtin_amdgcn_readfirstlane(at / line), off = at - head * line;
        const int i = __builtin_amdgcn_readfirstlane(p.own_plan ? seg_at_cost(lds.segs, all, off, threadIdx.x & 63)
                                                                : seg_at_cost(p.segs, all, off, threadIdx.x & 63));
        w.group = i < p.n_groups;
        w.seg = uniform(p.own_plan ? lds.segs[i] : p.segs[i]);
        w.kv_head = (int)head;
        const AttnShape shape = work.shape(w.seg, w.group);
        const int j = __builtin_amdgcn_readfirstlane(work.tile_at(shape, off - w.seg.cost));
        w.a = uniform(work.tile(w.seg, j, w.group));
        const uint32_t before = __builtin_amdgcn_readfirstlane(work.cost(shape, j));
        const uint32_t cost = __builtin_amdgcn_readfirstlane(work.cost(shape, j + 1)) - before;
        const uint32_t x0 = off - w.seg.cost - before, x1 = x0 + (end - at < cost - x0 ? end - at : cost - x0);
        const int s0 = __builtin_amdgcn_readfirstlane(work.step_at(shape, x0, cost, w.a.steps));
        const int s1 = __builtin_amdgcn_readfirstlane(work.step_at(shape, x1, cost, w.a.steps));
        const bool whole = x0 == 0 && x1 == cost, left_out = w.seg.row == -2;
        const int number = w.seg.tile + j;
        AttnDone* done = p.done + ((int64_t)number * p.c.heads + w.kv_head);
        const bool notes = threadIdx.x == 64 * NW - 1 && x0 == 0 && number < p.max_tiles;
        if (notes) {
            AttnDone d{};
            d.first = whole ? -1 : (int)x;
            d.last = (int)((at + (cost - 1)) / stretch);
            d.kind = w.group || left_out ? 2 : (w.seg.apart >= 0 ? 1 : 0);
            d.rows = left_out ? 0 : w.a.rows;
            d.row = w.a.row;
            d.slot = w.seg.apart + w.a.row;
            d.begin = w.seg.begin;
            d.position = w.seg.length - w.seg.count;
            d.table = w.seg.row;
            if (d.kind == 1) {
                const AttnSeg& g = segs[w.seg.group];
                d.group_row = (int64_t)(w.seg.begin - g.begin) * p.share + w.a.row;
                d.group_tile = g.tile;
            }
            *done = d;
        }
        if (!left_out) {
            w.run(segs, s0, s1, whole, 2 * (int64_t)x + (x0 > 0 ? 0 : 1));
            if (notes && whole && lds.wild[w.turn]) done->first = -2;
            w.turn ^= 1;
            __syncthreads();
        }
        at += cost - x0;
    }
}

template <class T, int D, int PARTS>
hipError_t launch_parts(const AttentionParams& p, hipStream_t stream)
{
    constexpr int NW = attn_waves(sizeof(T) == 4 ? DWS_FLOAT32 : DWS_BFLOAT16, D);
    const unsigned grid = (unsigned)p.workgroups;
    if (p.kv_access == kNear)
        k_attention<T, D, NW, kNear, PARTS><<<grid, 64 * NW, 0, stream>>>(p);
    else if (p.kv_access == kFar)
        k_attention<T, D, NW, kFar, PARTS><<<grid, 64 * NW, 0, stream>>>(p);
    else
        k_attention<T, D, NW, kElements, PARTS><<<grid, 64 * NW, 0, stream>>>(p);
    return hipGetLastError();
}
template <class T, int D>
hipError_t launch_dim(const AttentionParams& p, hipStream_t stream)
{
    if constexpr (sizeof(T) == 2)
        if (!p.one_part) return launch_parts<T, D, 2>(p, stream);
    return launch_parts<T, D, 1>(p, stream);
}
template <class T>
hipError_t launch_type(const AttentionParams& p, hipStream_t stream)
{
    if (p.padded == 64) return launch_dim<T, 64>(p, stream);
    if (p.padded == 128) return launch_dim<T, 128>(p, stream);
    return launch_dim<T, 256>(p, stream);
}

}  // namespace
}  // namespace dws
