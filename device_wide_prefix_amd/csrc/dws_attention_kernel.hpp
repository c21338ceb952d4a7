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
// Each wave brings 32 tokens of keys and values into its part of the LDS, the next
// ones on their way meanwhile in registers. Tiles of up to 32 queries are memory bound
// (2 queries' products for each byte): there the waves work on their own tokens and
// are joined at the end of the part. Larger ones are bound by the matrix products and
// the softmax beside them: there each wave has 32 queries of its own and goes through
// the tokens of all waves.
//
// Fragments (32 x 32 tiles, h = lane / 32):
//   operand  lane holds row (or column) lane % 32, contraction indices 8 h .. 8 h + 7 of
//            16 (16 bits), or h of 2 (fp32, where a chunk of four takes four products)
//   result   lane holds column lane % 32, rows 8 (i / 4) + 4 h + i % 4, i = 0 .. 15
// A contraction may run in any order that both operands share: P's eight elements of a
// step are the rows above, and the transposing LDS reads bring V's in the same order.
#pragma once

#include "dws_cache_device.hpp"

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

template <class T, int D, int NW, bool WHOLE>
struct Attention {
    static constexpr int CH = 16 / sizeof(T);           // elements of a chunk
    static constexpr int NCH = D / CH;                  // chunks of a row
    static constexpr int ROW = D * (int)sizeof(T);      // bytes of a row
    static constexpr int TILE = kKvTokens * ROW;        // bytes of 32 rows
    static constexpr int N = kKvTokens * NCH / 64;      // chunks of a tile in a lane
    static constexpr int STEP = 64 / NCH;               // rows that 64 lanes hold at a time
    static constexpr int BLOCKS = D / 32;
    static constexpr int THREADS = 64 * NW;
    // Whether the next tiles wait in registers (8 N): not where they do not fit beside the
    // queries' and the results', nor where rows are read element by element.
    static constexpr bool kAhead = WHOLE && N <= 16;
    static constexpr int kBatch = WHOLE ? 8 : 1;

    struct Lds {
        char kv[NW][2 * TILE];          // keys, values; then results
        int64_t at[NW][2][kKvTokens];   // where a token's keys and values are, -1: nowhere
        uint32_t there[NW];             // which tokens of a tile are
        float m[kAttnRows * NW], l[kAttnRows * NW];
    };

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
    const int lane, wave, half, col;
    int kv_head, tile_number;
    AttnTile a;
    int stop;                           // tokens of the part end here
    Chunk<T> q[NCH / 2];
    int position;                       // of the lane's query
    int least;                          // smallest of the wave's queries
    float c, c_rest;                    // scale log2(e), and what fp32 loses of it
    f32x16_t o[BLOCKS];
    float m, l;

    struct Ahead {
        u32x4_t k[kAhead ? N : 1], v[kAhead ? N : 1];
        uint32_t there;
    };

    __device__ __forceinline__ Attention(const AttentionParams& p, Lds& s)
        : p(p), s(s), lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), half(lane >> 5), col(lane & 31)
    {
    }

    __device__ __forceinline__ void row_place(int64_t r, int64_t* token, int* head) const
    {
        const int64_t at = a.row + r;
        if (at < (int64_t)1 << 31) {
            const uint32_t t = (uint32_t)at / (uint32_t)p.share;
            *token = a.token + t;
            *head = kv_head * p.share + (int)((uint32_t)at - t * (uint32_t)p.share);
        } else {
            *token = a.token + at / p.share;
            *head = kv_head * p.share + (int)(at % p.share);
        }
    }

    __device__ __forceinline__ void load_queries(bool wide)
    {
        const int r = (wide ? wave * kAttnRows : 0) + col;
        const bool in = r < a.rows;
        int64_t token = 0;
        int head = 0;
        if (in) row_place(r, &token, &head);
        position = !in ? INT32_MAX : (a.group ? p.positions[token] : a.position + (int)(token - a.token));
        least = position;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            const int y = __shfl_xor(least, d, 64);
            least = y < least ? y : least;
        }
        least = __builtin_amdgcn_readfirstlane(least);
        // the scale's sign goes to the queries, so that the largest product has the largest score
        const float sign = p.scale > 0.f ? 1.f : (p.scale < 0.f ? -1.f : 0.f);
        const double wide_c = p.scale == 0.f ? 1.0 : fabs((double)p.scale) * 1.4426950408889634;
        c = (float)wide_c;
        c_rest = (float)(wide_c - (double)c);
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

    // The page of the token that the lane looks up (lanes 32 and on look up nothing).
    __device__ __forceinline__ int page_of(int first) const
    {
        const int t = first + lane;
        if (lane >= kKvTokens || (uint32_t)t >= (uint32_t)stop) return -1;
        return p.c.table[a.table + (uint32_t)t / (uint32_t)p.c.page_tokens];
    }
    // Finds the tokens of a tile, and returns which are there. (The others are read from
    // the pool's beginning, and become 0 before they are used.)
    __device__ __forceinline__ uint32_t places(int first, int page)
    {
        const uint32_t t = (uint32_t)(first + lane), place = t % (uint32_t)p.c.page_tokens;
        const bool there = page >= 0 && page < p.c.n_pages;
        if (lane < kKvTokens) {
            s.at[wave][0][lane] = there ? page * p.c.keys.ps + place * p.c.keys.ts + kv_head * p.c.keys.hs : 0;
            s.at[wave][1][lane] = there ? page * p.c.values.ps + place * p.c.values.ts + kv_head * p.c.values.hs : 0;
        }
        wave_sync();
        return (uint32_t)__ballot(there);
    }
    __device__ __forceinline__ u32x4_t load_chunk(const void* data, int64_t at, int dim) const
    {
        const int d = (lane % NCH) * CH;
        const T* from = static_cast<const T*>(data) + at;
        if constexpr (WHOLE) {
            return *reinterpret_cast<const u32x4_t*>(from + (d < dim ? d : 0));
        } else {
            Chunk<T> x;
#pragma unroll
            for (int j = 0; j < CH; ++j) x[j] = from[d + j < dim ? d + j : 0];
            return __builtin_bit_cast(u32x4_t, x);
        }
    }
    // The chunk with 0 where the row or the dimension is not there.
    __device__ __forceinline__ u32x4_t only_there(int i, u32x4_t x, uint32_t there, int dim) const
    {
        const int d = (lane % NCH) * CH;
        const bool row = (there >> (i * STEP + lane / NCH)) & 1;
        if constexpr (WHOLE) return row && d < dim ? x : u32x4_t{};
        Chunk<T> y = __builtin_bit_cast(Chunk<T>, x);
#pragma unroll
        for (int j = 0; j < CH; ++j) y[j] = row && d + j < dim ? y[j] : (T)0.f;
        return __builtin_bit_cast(u32x4_t, y);
    }
    __device__ __forceinline__ u32x4_t load_key(int i) const
    {
        return load_chunk(p.c.keys.data, s.at[wave][0][i * STEP + lane / NCH], p.c.dim_k);
    }
    __device__ __forceinline__ u32x4_t load_value(int i) const
    {
        return load_chunk(p.c.values.data, s.at[wave][1][i * STEP + lane / NCH], p.c.dim_v);
    }
    // Row i * STEP + lane / NCH; what depends on the lane alone stands apart.
    __device__ __forceinline__ void put_key(int i, u32x4_t x)
    {
        const int r = lane / NCH, c = (lane % NCH) ^ key_swizzle(r);
        static_assert(STEP * SPAN == 1 || (16 % STEP == 0 && (STEP % SPAN == 0 || SPAN == 1)), "rows' bits stand apart");
        *(InLds<u32x4_t>)(tile(wave) + r * ROW + ((c ^ key_swizzle(i * STEP)) << 4) + i * STEP * ROW) = x;
    }
    __device__ __forceinline__ void put_value(int i, u32x4_t x)
    {
        const int r = lane / NCH, c = (lane % NCH) ^ value_swizzle(r);
        *(InLds<u32x4_t>)(tile(wave) + r * ROW + ((c ^ value_swizzle(i * STEP)) << 4) + TILE + i * STEP * ROW) = x;
    }
    __device__ __forceinline__ LdsBytes tile(int w) const { return (LdsBytes)&s.kv[0][0] + w * (2 * TILE); }
    __device__ __forceinline__ void fetch(Ahead* x, int first, int page)
    {
        x->there = places(first, page);
        if constexpr (kAhead) {
#pragma unroll
            for (int i = 0; i < N; ++i) x->k[i] = load_key(i);
#pragma unroll
            for (int i = 0; i < N; ++i) x->v[i] = load_value(i);
        }
    }
    __device__ __forceinline__ void put(Ahead& x)
    {
        const bool rest = x.there != 0xffffffffu || p.c.dim_k != D || p.c.dim_v != D;
        if constexpr (kAhead) {
            if (rest) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    x.k[i] = only_there(i, x.k[i], x.there, p.c.dim_k);
                    x.v[i] = only_there(i, x.v[i], x.there, p.c.dim_v);
                }
            }
#pragma unroll
            for (int i = 0; i < N; ++i) put_key(i, x.k[i]);
#pragma unroll
            for (int i = 0; i < N; ++i) put_value(i, x.v[i]);
        } else {
#pragma unroll kBatch
            for (int i = 0; i < N; ++i) {
                const u32x4_t k = load_key(i), v = load_value(i);
                put_key(i, only_there(i, k, x.there, p.c.dim_k));
                put_value(i, only_there(i, v, x.there, p.c.dim_v));
            }
        }
        if (lane == 0) s.there[wave] = x.there;
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

    // The wave's queries and the 32 tokens from `first` on, which wave w brought.
    __device__ __forceinline__ void step(int w, int first)
    {
        const LdsBytes keys = tile(w), values = keys + TILE;
        const uint32_t there = s.there[w];
        f32x16_t x = {};
        const int swizzle = half ^ key_swizzle(col);
#pragma unroll
        for (int i = 0; i < NCH / 2; ++i)
            x = mma(*(InLds<Chunk<T>>)(keys + col * ROW + (((2 * i) ^ swizzle) << 4)), q[i], x);
        const bool masked = there != 0xffffffffu || (int64_t)first + kKvTokens - 1 > least;
        if (masked) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int t = 8 * (i / 4) + 4 * half + i % 4;
                const bool sees = (there >> t & 1) && first + t <= position;
                x[i] = sees ? x[i] : -__builtin_inff();
            }
        }
        float top = x[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, x[i]);
        top = max_halves(top) * c;
        // The maximum follows once a score is 2^8 times above it: until then sums grow
        // by that, which fp32 and fp16 hold, and the results need no rescaling.
        if (__ballot(top > m + 8.f)) {
            const float now = fmaxf(m, top);
            const float by = now == m ? 1.f : __builtin_amdgcn_exp2f(m - now);
            l *= by;
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) o[b] *= by;
            m = now;
        }
        const float base = m == -__builtin_inff() ? 0.f : m;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float y = __builtin_fmaf(x[i], c, -base);
            if constexpr (sizeof(T) == 4)
                if (c_rest != 0.f && x[i] != -__builtin_inff()) y = __builtin_fmaf(x[i], c_rest, y);
            x[i] = __builtin_amdgcn_exp2f(y);
        }
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) sum += x[i];
        l += sum;

        constexpr int STEPS = 16 / CH;          // steps of the second product
        Chunk<T> pr[STEPS];
#pragma unroll
        for (int u = 0; u < STEPS; ++u)
#pragma unroll
            for (int j = 0; j < CH; ++j) pr[u][j] = (T)x[u * CH + j];
        if (masked) {
            // A value that is not finite, of a token that not every query sees: 0 times it is
            // not 0. Such a tile's rows are computed again, one by one, where the parts are joined.
            bool bad = false;
#pragma unroll 1
            for (int i = 0; i < NCH / 2; ++i) {
                const Chunk<T> v = *(InLds<Chunk<T>>)(values + col * ROW + ((2 * i + half) << 4));
#pragma unroll
                for (int j = 0; j < CH; ++j) bad |= !finite(v[j]);
            }
            if (__ballot(bad)) p.wild[tile_number] = 1;
        }
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
            for (int u = 0; u < STEPS; ++u) o[b] = mma(value_fragment(values, b, u), pr[u], o[b]);
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

    __device__ __forceinline__ void run(int part)
    {
        const bool wide = a.rows > kAttnRows;
        const int per = (a.steps + a.parts - 1) / a.parts;
        constexpr int TOKENS = kKvTokens * NW;
        const int first_step = part * per, last_step = first_step + per < a.steps ? first_step + per : a.steps;
        stop = a.end;
        int t = a.begin + first_step * TOKENS + wave * kKvTokens;
        load_queries(wide);
        m = -__builtin_inff();
        l = 0.f;
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) o[b] = f32x16_t{};
        Ahead x;
        int page = -1;
        if (first_step < last_step) {
            fetch(&x, t, page_of(t));
            page = page_of(t + TOKENS);
        }
        for (int i = first_step; i < last_step; ++i, t += TOKENS) {
            put(x);
            if (i + 1 < last_step) {
                fetch(&x, t + TOKENS, page);
                page = page_of(t + 2 * TOKENS);
            }
            if (wide) __syncthreads();
            wave_sync();
            const int last = wide ? NW : wave + 1;
#pragma unroll 1
            for (int w = wide ? 0 : wave; w < last; ++w) step(w, t + (w - wave) * kKvTokens);
            if (wide) __syncthreads();
            wave_sync();
        }
        l = sum_halves(l);

        // Results by way of the LDS (a wave's own part of it), so that rows are written whole.
        float* mine = reinterpret_cast<float*>(s.kv[wave]);
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int quad = 8 * b + 2 * j + half;
                *reinterpret_cast<f32x4_t*>(mine + col * D + ((quad ^ (col & 15)) << 2)) =
                    f32x4_t{o[b][4 * j], o[b][4 * j + 1], o[b][4 * j + 2], o[b][4 * j + 3]};
            }
        if (half == 0) {
            s.m[wave * kAttnRows + col] = m;
            s.l[wave * kAttnRows + col] = l;
        }
        __syncthreads();
        constexpr int QUADS = D / 4;
        for (int i = threadIdx.x; i < a.rows * QUADS; i += THREADS) {
            const int r = i / QUADS, quad = i % QUADS;
            const int place = (r % kAttnRows) * D + ((quad ^ (r & 15)) << 2);
            f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
            float most = -__builtin_inff(), total = 0.f;
            if (wide) {
                most = s.m[r];
                total = s.l[r];
                sum = *reinterpret_cast<const f32x4_t*>(reinterpret_cast<const float*>(s.kv[r / kAttnRows]) + place);
            } else {
#pragma unroll
                for (int w = 0; w < NW; ++w) most = fmaxf(most, s.l[w * kAttnRows + r] == 0.f ? most : s.m[w * kAttnRows + r]);
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float lw = s.l[w * kAttnRows + r], mw = s.m[w * kAttnRows + r];
                    if (lw == 0.f) continue;
                    const float by = mw == most ? 1.f : __builtin_amdgcn_exp2f(mw - most);
                    sum += *reinterpret_cast<const f32x4_t*>(reinterpret_cast<const float*>(s.kv[w]) + place) * by;
                    total += lw * by;
                }
            }
            if (a.slot >= 0) {
                const int64_t row = (int64_t)kv_head * p.max_rows + a.slot + (int64_t)part * a.rows + r;
                *reinterpret_cast<f32x4_t*>(p.partial + row * D + 4 * quad) = sum;
                if (quad == 0) p.stat[row] = make_float2(most, total);
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

// An entry of the plan, the same for all lanes.
template <class X>
__device__ __forceinline__ X uniform_load(const X* from)
{
    static_assert(sizeof(X) % 4 == 0, "whole words");
    X x;
    uint32_t w[sizeof(X) / 4];
#pragma unroll
    for (size_t i = 0; i < sizeof(X) / 4; ++i)
        w[i] = __builtin_amdgcn_readfirstlane(reinterpret_cast<const uint32_t*>(from)[i]);
    __builtin_memcpy(&x, w, sizeof(X));
    return x;
}

// Waves a SIMD that the LDS allows.
constexpr int attn_occupancy(int bytes) { return bytes <= 80 * 1024 ? 2 : 1; }

template <class T, int D, int NW, bool WHOLE>
__global__ __launch_bounds__(64 * NW, attn_occupancy(sizeof(typename Attention<T, D, NW, WHOLE>::Lds))) void k_attention(
    AttentionParams p)
{
    __shared__ typename Attention<T, D, NW, WHOLE>::Lds lds;
    Attention<T, D, NW, WHOLE> w(p, lds);
    const int all = __builtin_amdgcn_readfirstlane(p.head->items) * p.c.heads;
    for (int x = blockIdx.x; x < all; x += gridDim.x) {
        const AttnItem item = uniform_load(p.item + x / p.c.heads);
        w.kv_head = x % p.c.heads;
        if (item.part < 0) continue;
        w.tile_number = item.tile;
        w.a = uniform_load(p.tile + item.tile);
        w.run(item.part);
        __syncthreads();
    }
}

template <class T, int D>
hipError_t launch_dim(const AttentionParams& p, hipStream_t stream)
{
    constexpr int NW = attn_waves(sizeof(T) == 4 ? DWS_FLOAT32 : DWS_BFLOAT16, D);
    const int64_t most = p.max_items * p.c.heads;
    const unsigned grid = (unsigned)(most < kAttnTarget ? most : kAttnTarget);
    if (p.whole_kv)
        k_attention<T, D, NW, true><<<grid, 64 * NW, 0, stream>>>(p);
    else
        k_attention<T, D, NW, false><<<grid, 64 * NW, 0, stream>>>(p);
    return hipGetLastError();
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
