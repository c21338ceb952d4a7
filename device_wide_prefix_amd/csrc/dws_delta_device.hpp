// Device pieces the delta-rule kernels share: matrix fragments, their products
// and loads, and the map from chunk slots to sequences.
//
// Fragment layouts (16 x 16 tiles, 64 lanes, gq = lane / 16, lr = lane % 16):
//   operand   lane holds 8 elements of row (or column) lr along the contraction
//   acc       lane holds column lr, rows 4 gq + r, r = 0..3
// A contraction may run over its 32 indices in any order that both operands
// share. In "natural" order element j of lane group gq is index 8 gq + j: one
// 16-byte read of a row. In "acc" order it is 4 gq + j for j < 4 and
// 16 + 4 gq + (j - 4) above: exactly the rows that two stacked acc tiles hold, so
// a product's result is the next product's operand without leaving its lane.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dws_delta.h"

namespace dws {

// Waves a SIMD: the kernels' LDS allows no more workgroups, so the compiler may
// as well use all 256 registers to have reads in flight.
#define DWS_TWO_WAVES __attribute__((amdgpu_waves_per_eu(2, 2)))

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16_t;
typedef _Float16 f16_t;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

template <class T>
using Vec8 = T __attribute__((ext_vector_type(8)));
template <class T>
using Vec4 = T __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mma(Vec8<bf16_t> a, Vec8<bf16_t> b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(Vec8<f16_t> a, Vec8<f16_t> b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
// fp32: eight products of depth 4. Step j contracts element j of every lane
// group, so the 32 indices are covered in whichever order the elements are in.
__device__ __forceinline__ f32x4 mma(Vec8<float> a, Vec8<float> b, f32x4 c)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
    return c;
}

// An operand computed in fp32 as NP parts of type T: the rounded value and the
// rounded rests. One bf16 part is off by at most 2^-8 of the value, two by
// 2^-16, three hold all of fp32 (fp16: 2^-11, then 2^-22); fp32 is one part.
template <class T, int NP>
struct Parts {
    Vec8<T> p[NP];
};
template <class T, int NP>
__device__ __forceinline__ Parts<T, NP> parts_of(f32x8 x)
{
    Parts<T, NP> r;
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        r.p[n] = __builtin_convertvector(x, Vec8<T>);
        if (n + 1 < NP) x -= __builtin_convertvector(r.p[n], f32x8);
    }
    return r;
}
template <class T, int NP>
__device__ __forceinline__ Parts<T, NP> parts_of(f32x4 lo, f32x4 hi)
{
    return parts_of<T, NP>(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}
// Product of two operands in parts, smallest terms first. Terms whose parts'
// numbers sum to more than the longer one's last part are below its rounding
// and are left out.
template <class T, int NA, int NB>
__device__ __forceinline__ f32x4 mma(const Parts<T, NA>& a, const Parts<T, NB>& b, f32x4 c)
{
    constexpr int LAST = (NA > NB ? NA : NB) - 1;
#pragma unroll
    for (int s = LAST; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB) c = mma(a.p[i], b.p[s - i], c);
    return c;
}

// c[m] += a[m] b for M independent results: consecutive products never wait
// for each other. LEFT: c[m] += b a[m], the transposed results.
template <bool LEFT = false, class T, int NA, int NB, int M>
__device__ __forceinline__ void mma_each(const Parts<T, NA> (&a)[M], const Parts<T, NB>& b, f32x4 (&c)[M], int from = 0,
                                         int to = M)
{
    constexpr int LAST = (NA > NB ? NA : NB) - 1;
#pragma unroll
    for (int s = LAST; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB)
#pragma unroll
                for (int m = 0; m < M; ++m)
                    if (m >= from && m < to)
                        c[m] = LEFT ? mma(b.p[s - i], a[m].p[i], c[m]) : mma(a[m].p[i], b.p[s - i], c[m]);
}

// ---- LDS tiles: rows of `stride` elements --------------------------------

// LDS row length: 16 bytes more than the row, so that the 16 rows a fragment
// read touches start in different banks.
template <class T>
constexpr int lds_stride(int cols) { return cols + 16 / (int)sizeof(T); }

// Operand rows r0..r0+15, contraction columns c0..c0+31, natural order.
template <class T>
__device__ __forceinline__ Vec8<T> frag_nat(const T* tile, int stride, int r0, int c0, int lane)
{
    const T* p = tile + (r0 + (lane & 15)) * stride + c0 + (lane >> 4) * 8;
    if constexpr (sizeof(T) == 2) {
        return *reinterpret_cast<const Vec8<T>*>(p);
    } else {
        const Vec4<T> a = *reinterpret_cast<const Vec4<T>*>(p), b = *reinterpret_cast<const Vec4<T>*>(p + 4);
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
}
// The same in acc order.
template <class T>
__device__ __forceinline__ Vec8<T> frag_acc(const T* tile, int stride, int r0, int c0, int lane)
{
    const T* p = tile + (r0 + (lane & 15)) * stride + c0 + (lane >> 4) * 4;
    const Vec4<T> a = *reinterpret_cast<const Vec4<T>*>(p), b = *reinterpret_cast<const Vec4<T>*>(p + 16);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
// The parts of an operand in as many tiles, one behind the other.
template <int NP, class T>
__device__ __forceinline__ Parts<T, NP> parts_acc(const T* tile, int tile_elems, int stride, int r0, int c0, int lane)
{
    Parts<T, NP> a;
#pragma unroll
    for (int n = 0; n < NP; ++n) a.p[n] = frag_acc(tile + n * tile_elems, stride, r0, c0, lane);
    return a;
}
// Four elements of column c0 + lr in rows r0 + 4 gq + (0..3): what an acc tile
// of these rows and columns holds. The 16-bit types use the transposing LDS
// read: within 16 lanes, lane i points at 4 elements of row i / 4 and receives
// column i of the 4 x 16 block.
template <class T>
__device__ __forceinline__ Vec4<T> quad_tr(const T* tile, int stride, int r0, int c0, int lane)
{
    if constexpr (sizeof(T) == 2) {
        const T* p = tile + (r0 + (lane >> 4) * 4 + ((lane >> 2) & 3)) * stride + c0 + (lane & 3) * 4;
        const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4*)(reinterpret_cast<uintptr_t>(p)));
        return __builtin_bit_cast(Vec4<T>, v);
    } else {
        const T* p = tile + (r0 + (lane >> 4) * 4) * stride + c0 + (lane & 15);
        return Vec4<T>{p[0], p[stride], p[2 * stride], p[3 * stride]};
    }
}
// Operand of the transposed tile: its rows are the tile's columns c0..c0+15,
// the contraction the tile's rows r0..r0+31 in acc order.
template <class T>
__device__ __forceinline__ Vec8<T> frag_tr(const T* tile, int stride, int r0, int c0, int lane)
{
    const Vec4<T> a = quad_tr(tile, stride, r0, c0, lane), b = quad_tr(tile, stride, r0 + 16, c0, lane);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

template <int NP, class T>
__device__ __forceinline__ Parts<T, NP> parts_tr(const T* tile, int tile_elems, int stride, int r0, int c0, int lane)
{
    Parts<T, NP> a;
#pragma unroll
    for (int n = 0; n < NP; ++n) a.p[n] = frag_tr(tile + n * tile_elems, stride, r0, c0, lane);
    return a;
}
// Four values as NP parts of four, `step` elements apart.
template <int NP, class T>
__device__ __forceinline__ void store_parts4(T* at, int64_t step, f32x4 x)
{
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        const Vec4<T> y = __builtin_convertvector(x, Vec4<T>);
        *reinterpret_cast<Vec4<T>*>(at + n * step) = y;
        if (n + 1 < NP) x -= __builtin_convertvector(y, f32x4);
    }
}

// ---- global memory --------------------------------------------------------

__device__ __forceinline__ float load_gate(const DeltaRows& r, int64_t token, int head, int dtype)
{
    const int64_t at = token * r.ts + head * r.hs;
    if (dtype == DWS_FLOAT32) return static_cast<const float*>(r.data)[at];
    if (dtype == DWS_BFLOAT16) return (float)static_cast<const bf16_t*>(r.data)[at];
    return (float)static_cast<const f16_t*>(r.data)[at];
}

// A log decay below -104 gives a factor that fp32 rounds to 0 (e^-104 is less
// than half its least number), so it is taken as -104: sums of a chunk's decays and
// their differences then stay finite for -infinity too. NaN stays NaN.
__device__ __forceinline__ float clamp_decay(float g) { return g < -104.f ? -104.f : g; }

// Buffer access: a resource over the rows of a chunk (32-bit offsets, and one
// compare in hardware instead of 64-bit addresses and branches): reads outside
// give 0, writes outside are dropped. kOutside is outside of every resource:
// rows of a chunk span less than 2^30 bytes, which the C entry points check.
constexpr int kOutside = (int)0x80000000u;
constexpr int kRsrcFlags = 0x00020000;      // untyped dwords, as the scan kernels' resources

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* first, int64_t row_bytes, int rows, int bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(first), (short)0,
                                             (int)((rows - 1) * row_bytes) + bytes, kRsrcFlags);
}
// Bytes of a row's elements in whole 16-byte units: the units are there (copied
// rows are padded), and a unit's last dwords are checked by themselves.
template <class T>
__device__ __forceinline__ int whole_bytes(int elems) { return (elems * (int)sizeof(T) + 15) & ~15; }

template <class T>
__device__ __forceinline__ T buffer_load(__amdgpu_buffer_rsrc_t r, int at)
{
    if constexpr (sizeof(T) == 16) return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
    if constexpr (sizeof(T) == 8) return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0));
    if constexpr (sizeof(T) == 4) return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0));
    if constexpr (sizeof(T) == 2) return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(r, at, 0, 0));
}
template <class T>
__device__ __forceinline__ void buffer_store(__amdgpu_buffer_rsrc_t r, int at, T x)
{
    if constexpr (sizeof(T) == 16) __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, x), r, at, 0, 0);
    if constexpr (sizeof(T) == 8) __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2_t, x), r, at, 0, 0);
    if constexpr (sizeof(T) == 4) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, x), r, at, 0, 0);
    if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, x), r, at, 0, 0);
}

// A tile of ROWS x COLS elements on its way from global memory to LDS through
// registers, 16 bytes at a time: load() for the next chunk is issued before a
// chunk's products and store() after them, so that the loads are in flight
// meanwhile. Rows from `rows` and columns from `cols` on become 0.
template <class T, int ROWS, int COLS, int THREADS>
struct TileRegs {
    static constexpr int V = 16 / (int)sizeof(T), UNITS = COLS / V, ALL = ROWS * UNITS;
    static constexpr int N = (ALL + THREADS - 1) / THREADS;
    typedef T VecT __attribute__((ext_vector_type(V)));
    VecT x[N];

    __device__ __forceinline__ void load(const T* src, int64_t ld, int rows, int cols, int tid)
    {
        const auto rsrc = rows_rsrc(src, ld * (int)sizeof(T), rows, whole_bytes<T>(cols));
        const int step = (int)ld * (int)sizeof(T);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int u = tid + i * THREADS, r = u / UNITS, c = u % UNITS * V;
            x[i] = buffer_load<VecT>(rsrc, r < rows && c < cols ? r * step + c * (int)sizeof(T) : kOutside);
        }
    }
    __device__ __forceinline__ void store(T* tile, int stride, int tid) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int u = tid + i * THREADS, r = u / UNITS, c = u % UNITS * V;
            if (ALL % THREADS == 0 || u < ALL) *reinterpret_cast<VecT*>(tile + r * stride + c) = x[i];
        }
    }
    // ROWS columns of COLS elements, 16 at a time as the lanes of a scan wave
    // hold them, to a row for each
    __device__ __forceinline__ void store_columns(T* tile, int stride, int tid) const
    {
        constexpr int EACH = COLS * 16 / (64 * V);       // units of a lane
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int u = tid + i * THREADS, lane = u % 64, t = u / 64 % EACH, group = u / 64 / EACH;
            if (ALL % THREADS != 0 && u >= ALL) break;
            T* to = tile + (group * 16 + lane % 16) * stride + t * (V * 4) + lane / 16 * 4;
            if constexpr (V == 8) {
                *reinterpret_cast<Vec4<T>*>(to) = __builtin_shufflevector(x[i], x[i], 0, 1, 2, 3);
                *reinterpret_cast<Vec4<T>*>(to + 16) = __builtin_shufflevector(x[i], x[i], 4, 5, 6, 7);
            } else {
                *reinterpret_cast<VecT*>(to) = x[i];
            }
        }
    }
};
// 8 elements as an operand, of a row that has `left` more from there on. Rows are
// whole 16-byte units, so an fp32 row may end between the two: what lies behind it,
// another head's elements or a gap, is not read. It would meet zeros, but
// infinity and NaN times 0 are NaN.
template <class T>
__device__ __forceinline__ Vec8<T> buffer_frag(__amdgpu_buffer_rsrc_t r, int at, int left)
{
    if constexpr (sizeof(T) == 2) {
        return buffer_load<Vec8<T>>(r, at);
    } else {
        const Vec4<T> a = buffer_load<Vec4<T>>(r, at), b = buffer_load<Vec4<T>>(r, at == kOutside || left <= 4 ? kOutside : at + 16);
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
}

// ---- sequences ------------------------------------------------------------

// First row and length of sequence i; whatever the offsets hold, the rows lie
// in [0, tokens).
__device__ __forceinline__ int64_t seq_begin(const int64_t* offsets, int64_t tokens, int64_t n_seqs, int64_t i)
{
    if (offsets == nullptr) return i * (tokens / n_seqs);
    const int64_t b = offsets[i];
    return b < 0 ? 0 : (b > tokens ? tokens : b);
}
__device__ __forceinline__ int64_t seq_length(const int64_t* offsets, int64_t tokens, int64_t n_seqs, int64_t i,
                                              int64_t begin)
{
    if (offsets == nullptr) return tokens / n_seqs;
    const int64_t e = offsets[i + 1];
    const int64_t end = e < begin ? begin : (e > tokens ? tokens : e);
    return end - begin;
}

// Chunk c of sequence i is chunk slot begin_i / C + i + c. Its ceil(len / C)
// chunks end before the next sequence's first slot, since
// ceil((b + C x - a) / C) <= x + 1 + floor(b / C) - floor(a / C), and the last
// one before tokens / C + n_seqs.
__device__ __forceinline__ int64_t first_slot(int64_t begin, int64_t i, int chunk) { return begin / chunk + i; }

// A value that all lanes have, for the compiler to know it: a buffer resource
// made of one that it takes for different in each lane costs a loop over the
// lanes at every access.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x)
{
    const uint32_t lo = (uint32_t)uniform((int)x), hi = (uint32_t)uniform((int)(x >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

struct SlotInfo {
    int64_t seq;
    int64_t row;       // first row of the chunk
    int rows;          // its tokens, 0 for a slot without any
    int64_t beyond;    // for a slot behind the last sequence's: how far, else -1
};
// Every lane of the wave calls it. The last sequence whose first slot is not
// behind `slot`, 64 candidates a round: a round is one trip to memory, and a
// binary search's six would be most of a small kernel's time.
template <int C>
__device__ __forceinline__ SlotInfo slot_info(const int64_t* offsets, int64_t tokens, int64_t n_seqs, int64_t slot, int lane)
{
    int64_t lo = 0, hi = n_seqs - 1;
    while (hi - lo >= 64) {
        const int64_t step = (hi - lo) / 64 + 1, at = lo + lane * step;
        const bool in = at <= hi && first_slot(seq_begin(offsets, tokens, n_seqs, at <= hi ? at : hi), at, C) <= slot;
        const uint64_t found = __ballot(in);
        lo += found == 0 ? 0 : (63 - __builtin_clzll(found)) * step;
        if (lo + step - 1 < hi) hi = lo + step - 1;
    }
    // the last round brings the sequence's rows along
    const int64_t at = lo + lane <= hi ? lo + lane : hi;
    const int64_t b = seq_begin(offsets, tokens, n_seqs, at), n = seq_length(offsets, tokens, n_seqs, at, b);
    const uint64_t found = __ballot(lo + lane <= hi && first_slot(b, at, C) <= slot);
    const int k = found == 0 ? 0 : 63 - __builtin_clzll(found);
    lo = uniform(lo + k);
    SlotInfo s;
    s.seq = lo;
    const int64_t begin = uniform(__shfl(b, k, 64)), len = uniform(__shfl(n, k, 64));
    const int64_t c = slot - first_slot(begin, lo, C);
    const int64_t left = len - c * C;
    s.row = begin + c * C;
    s.rows = c < 0 || left <= 0 ? 0 : (left < C ? (int)left : C);
    s.beyond = lo == n_seqs - 1 && c >= 0 && left <= 0 ? c - (len + C - 1) / C : -1;
    return s;
}

// Whether sequence i takes part: its slot is in the pool and no earlier
// sequence of the call names it. Every thread of the workgroup calls it.
template <int THREADS>
__device__ __forceinline__ bool slot_taken(const int* slots, int64_t n_states, int64_t i, int64_t* state, int tid)
{
    if (slots == nullptr) {
        *state = i;
        return true;
    }
    const int mine = slots[i];
    bool again = false;
    // Eight loads in flight a thread (behind slot i - 1 of slot i, not counted). All
    // workgroups together read the square of n_seqs: a step of 8 heads of 64 x 64 takes
    // 60 us without slots and 67 with for 1,024 sequences, 728 and 954 for 16,384
    // (1,183 with one load in flight), 2,174 and 3,808 for 49,152 (5,635).
    for (int64_t j = tid; j < i; j += 8 * THREADS) {
        int other[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) other[u] = slots[j + u * THREADS < i ? j + u * THREADS : i];
#pragma unroll
        for (int u = 0; u < 8; ++u) again |= j + u * THREADS < i && other[u] == mine;
    }
    *state = mine;
    const bool dup = __syncthreads_or(again);
    return mine >= 0 && mine < n_states && !dup;
}

// Workgroup index -> (group, part of `parts`) such that the parts of a group
// are dealt to one XCD (workgroups go to the 8 XCDs in turn): they read the same
// rows, which that XCD's L2 then holds once. `blocks` is a multiple of 8 parts.
__device__ __forceinline__ void xcd_split(uint32_t block, uint32_t parts, uint32_t* group, uint32_t* part)
{
    const uint32_t eight = block / (8 * parts), rest = block - eight * 8 * parts;
    *part = rest / 8;
    *group = eight * 8 + rest % 8;
}

}  // namespace dws
