// The chunked gated delta rule: kernels over chunks of C tokens.
//
// With G_i the sum of a chunk's first i log decays, D_ij = e^(G_i - G_j) for
// i >= j, S the state at the chunk's start and B = diag(beta):
//   L = tril(D o K K^T, -1)          X = V - diag(e^G) K S
//   U' = (I + L B)^-1 X              u = B U'       (what each token writes)
//   O = scale diag(e^G) Q S + P u    P = scale tril(D o Q K^T)
//   S <- e^(G_C) S + K^T diag(e^(G_C - G)) u
// k_delta_prep does for every chunk at once what does not depend on S (P and
// the inverse); k_delta_scan then goes through a sequence's chunks. The columns
// of S never meet: each wave owns 16 of them for the whole sequence, S in its
// registers, and passes products on as operands without a transfer.
#pragma once

#include "dws_delta_device.hpp"

#include <type_traits>

namespace dws {

// Tokens of a chunk: 64, and 32 where a chunk's tiles twice over (the next
// chunk's arrive while this one is worked on) would not fit 160 KB of LDS.
template <class T, int DK>
constexpr int kChunk = sizeof(T) == 4 || DK > 128 ? 32 : 64;

// Whether products with key columns behind dim_k, which are zeros, are left out:
// for fp32, whose products take most of the time (heads of 72 x 40: 103 us with
// them, 91 without). In 16 bits the branches cost more than they save (heads of
// 96 x 96: 134 us with all products, 153 with branches), as they do with the
// registers that fp32 heads above 128 take (160 x 128: 204 and 224 us).
template <class T, int DK>
constexpr bool kSkip = sizeof(T) == 4 && DK <= 128;

// Parts of the 16-bit operands that are computed in fp32. With one part for
// all, bf16 outputs and gradients are off by 3.3e-3 to 4.9e-3 (2-norm), twice
// what rounding the result itself gives (1.7e-3). The arrays of a chunk's size,
// P, X, U', Z, dU, e^G dX, scale e^G dO, W1 and W2, make up nearly all of that; in two
// parts they leave at most 1.4 times the result's own rounding. So does the
// inverse: where keys repeat, its rows subtract neighbouring tokens from each
// other, and what is left is far smaller than its entries' rounding. S in the
// outputs, which is larger and costs the most products, adds 0.35 times at most
// and keeps one part.
template <class T>
constexpr int kFine = sizeof(T) == 4 ? 1 : 2;
// Parts of the states (and of their gradients) in the backward pass. The decays'
// gradients sum terms with both that cancel: in one part each, d_g was off by 1.3
// times its own rounding at the median and 1.5 to 2.5 at the worst of 40 random
// calls; with the states in two, at 10% of a training step's time, by 1.1 and 1.3
// for heads up to 128. Chunks of wider heads are half as long, so that more comes
// through the states: with both in two parts 1.03 instead of 1.6. Both for all
// heads take 505 us a training step instead of 464, and leave each gradient's own
// rounding alone (0.01 of it before); a caller can ask for that.
template <class T>
constexpr int kStored = kFine<T>;
template <class T, int DK>
constexpr int kStoredGrad = DK > 128 ? kFine<T> : 1;
// Parts of everything that a final state depends on, for fp32 accuracy.
template <class T>
constexpr int kPrecise = __is_same(T, bf16_t) ? 3 : kFine<T>;

// ---- triangular chunk x chunk matrices as operands -------------------------

// Where four consecutive elements (row, col .. col + 3) of a lower (upper)
// triangular C x C matrix are when it is kept as operand fragments of 16 rows
// and 32 columns, 64 lanes x 8 elements each: only the fragments that are not
// all zero, each read with one 16-byte access a lane (two for fp32). `acc` and
// `nat`: the order of the contraction.
template <int C>
struct Triangle {
    static constexpr int frags = C == 64 ? 6 : 2, elems = frags * 512;
    // fragment (row tile mt, column block kb)
    static __device__ constexpr int lower(int mt, int kb) { return kb == 0 ? mt : 2 + mt; }
    static __device__ constexpr int upper(int mt, int kb) { return kb == 0 ? mt : 2 + mt; }
    static __device__ constexpr int acc(int row, int col) { return ((col % 16 / 4) * 16 + row % 16) * 8 + col % 32 / 16 * 4; }
    static __device__ constexpr int nat(int row, int col) { return ((col % 32 / 8) * 16 + row % 16) * 8 + col % 8; }
    static __device__ constexpr int lower_nat(int row, int col) { return lower(row / 16, col / 32) * 512 + nat(row, col); }
    static __device__ constexpr int upper_acc(int row, int col) { return upper(row / 16, col / 32) * 512 + acc(row, col); }
};
// The parts of fragment f.
template <int NP, class T>
__device__ __forceinline__ Parts<T, NP> parts_at(const T* frags, int elems, int f, int lane)
{
    Parts<T, NP> a;
#pragma unroll
    for (int n = 0; n < NP; ++n) a.p[n] = frag_nat(frags + n * elems + f * 512 + lane * 8, 0, 0, 0, 0);
    return a;
}

// Eight elements of a fragment as NP parts, `step` elements apart.
template <int NP, class T>
__device__ __forceinline__ void store_fragment(T* at, int64_t step, f32x4 lo, f32x4 hi)
{
    const Parts<T, NP> x = parts_of<T, NP>(lo, hi);
#pragma unroll
    for (int n = 0; n < NP; ++n) *reinterpret_cast<Vec8<T>*>(at + n * step) = x.p[n];
}

// ---- the inverse of a unit lower triangular matrix -----------------------

// fp32 product of two 16-row, 16-column blocks of LDS matrices (rows of LD):
// acc + a[.., 0 .. K) b[0 .. K, ..), on the matrix cores.
template <int LD, int K>
__device__ __forceinline__ f32x4 block_product(const float* a, const float* b, f32x4 acc, int lane)
{
    const int lr = lane & 15, gq = lane >> 4;
#pragma unroll
    for (int k = 0; k < K; k += 4)
        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[lr * LD + k + gq], b[(k + gq) * LD + lr], acc, 0, 0, 0);
    return acc;
}
template <int LD>
__device__ __forceinline__ void store_block(float* at, f32x4 x, int lane)
{
#pragma unroll
    for (int r = 0; r < 4; ++r) at[((lane >> 4) * 4 + r) * LD + (lane & 15)] = x[r];
}

// Row length of the inversion's matrices: rows start at 16 bytes, and 16 rows
// in different banks.
constexpr int inverse_stride(int c) { return c + 4; }

// m <- (I + m)^-1, m strictly lower triangular, fp32 in LDS with rows of
// inverse_stride(C). Of m only the entries below the diagonal are read, and the
// inverse's upper right quarter is not written. The diagonal 8 x 8 blocks by
// substitution (a column of one of them a lane of the first wave), then thrice
// twice as large blocks from two: [[A, 0], [M, B]]^-1 has -B^-1 M A^-1 in its
// corner. Substitution keeps the error at the size of the result's entries; a
// product of powers (I - m)(I + m^2).. would not, since the powers of m can be
// far larger than its inverse. Each block takes the place of the part of m that
// it was made from. `tmp`: 32 x 32, the same rows. THREADS = 4 C.
template <int C>
__device__ __forceinline__ void invert_unit_lower(float* m, float* tmp, int wave, int lane)
{
    constexpr int NB = C / 16, LD = inverse_stride(C);
    if (wave == 0 && lane < C) {
        const int b0 = lane / 8 * 8, col = lane % 8;
        const float* d = m + b0 * (LD + 1);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float s = i == col ? 1.f : 0.f;
#pragma unroll
            for (int j = 0; j < i; ++j) s -= d[i * LD + j] * x[j];
            x[i] = s;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) m[(b0 + i) * LD + b0 + col] = x[i];
    }
    // zero above the diagonal within the 32 x 32 blocks
    {
        const int r = lane / 8, c = lane % 8;
        m[(wave * 16 + r) * LD + wave * 16 + 8 + c] = 0.f;
        if (wave % 2 == 0) store_block<LD>(m + wave * 16 * LD + (wave + 1) * 16, f32x4{}, lane);
    }
    __syncthreads();
    {
        // 8 -> 16: wave w makes the corner of diagonal block w, an element a lane
        const int r = lane / 8, c = lane % 8, b0 = wave * 16;
        float y = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) y += m[(b0 + 8 + r) * LD + b0 + k] * m[(b0 + k) * LD + b0 + c];
        tmp[(wave * 8 + r) * LD + c] = y;
        __syncthreads();
        y = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) y -= m[(b0 + 8 + r) * LD + b0 + 8 + k] * tmp[(wave * 8 + k) * LD + c];
        m[(b0 + 8 + r) * LD + b0 + c] = y;
    }
    __syncthreads();
    // 16 -> 32: wave w < NB / 2 makes block (2 w + 1, 2 w)
    const int a = wave * 2;
    if (wave < NB / 2)
        store_block<LD>(tmp + wave * 16 * LD,
                        block_product<LD, 16>(m + (a + 1) * 16 * LD + a * 16, m + a * 16 * (LD + 1), f32x4{}, lane), lane);
    __syncthreads();
    if (wave < NB / 2)
        store_block<LD>(m + (a + 1) * 16 * LD + a * 16,
                        -block_product<LD, 16>(m + (a + 1) * 16 * (LD + 1), tmp + wave * 16 * LD, f32x4{}, lane), lane);
    __syncthreads();
    if constexpr (NB == 4) {
        // 32 -> 64: four blocks, one a wave
        const int bi = wave >> 1, bj = wave & 1;
        store_block<LD>(tmp + bi * 16 * LD + bj * 16,
                        block_product<LD, 32>(m + (32 + bi * 16) * LD, m + bj * 16, f32x4{}, lane), lane);
        __syncthreads();
        store_block<LD>(m + (32 + bi * 16) * LD + bj * 16,
                        -block_product<LD, 32>(m + (32 + bi * 16) * LD + 32, tmp + bj * 16, f32x4{}, lane), lane);
        __syncthreads();
    }
}

// Gate factors of a chunk in the workspace: e^G, e^(G_C - G), beta, and the sums
// of the decays (as logarithms to base 2) in two fp32 parts, C of each.
constexpr int kGateArrays = 5;

// Sums over a chunk in double, then split in two: the difference of two sums
// keeps fp32 accuracy however large they are.
template <int C>
__device__ __forceinline__ double scan_decays(double g, int lane)
{
#pragma unroll
    for (int d = 1; d < C; d *= 2) {
        const double o = __shfl_up(g, d, 64);
        if (lane >= d) g += o;
    }
    return g;
}
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
// e^(G_i - G_j)
__device__ __forceinline__ float decay(float hi_i, float lo_i, float hi_j, float lo_j)
{
    return exp2_fast((hi_i - hi_j) + (lo_i - lo_j));
}

template <class T>
__device__ __forceinline__ void zero_rows(const DeltaRows& r, int64_t first, int64_t last, int64_t step, int chunk,
                                          int heads, int dim, int tid, int threads)
{
    if (r.data == nullptr) return;
    T* p = static_cast<T*>(r.data);
    for (int64_t base = first; base < last; base += step)
        for (int i = tid; i < chunk * heads * dim; i += threads) {
            const int64_t row = base + i / (heads * dim);
            const int h = i / dim % heads, d = i % dim;
            if (row < last) p[row * r.ts + h * r.hs + d] = (T)0.f;
        }
}

__device__ __forceinline__ f32x4 gate4(const float* gate, int row) { return *reinterpret_cast<const f32x4*>(gate + row); }
// Row of tile t of a lower triangle's tiles in order: 0; 1, 1; 2, 2, 2; ...
__device__ __forceinline__ int tile_row(int t) { return t < 1 ? 0 : (t < 3 ? 1 : (t < 6 ? 2 : 3)); }

// LDS of the preparation: the matrix that is inverted takes the place of the K
// tile, which is done with before (Q's fragments come straight from memory).
// 18 KB for 128 key columns, seven workgroups a compute unit; four, with Q and
// the inverse in LDS too, measured the same. 8,544 chunks and heads with three
// parts of the inverse take 106 us: 565 MB, 5.3 TB/s (127 us when the inverse was
// written in the order of its rows, 8 bytes to a line).
template <class T, int DK>
struct PrepLds {
    static constexpr int C = kChunk<T, DK>, LK = lds_stride<T>(DK), LD = inverse_stride(C);
    static constexpr size_t tile = (size_t)C * LK * sizeof(T), matrix = (size_t)C * LD * sizeof(float);
    // block products: in the upper right quarter of a 64 x 64 matrix, behind a smaller one
    static constexpr size_t inverse = (C == 64 ? 1 : 2) * matrix;
    static constexpr size_t gate = tile > inverse ? tile : inverse, bytes = gate + 3 * C * sizeof(float);
};

// One workgroup for each (chunk slot, value head): gate factors, P and the
// inverse(s) to the workspace. The 16 x 16 tiles of K K^T and Q K^T up to the
// diagonal, row by row, go to the waves in turn.
template <class T, int DK, int NP, bool BWD>
__global__ __launch_bounds__((kChunk<T, DK> * 4)) void k_delta_prep(DeltaParams p)
{
    using S = PrepLds<T, DK>;
    constexpr int C = S::C, THREADS = C * 4, NB = C / 16, LK = S::LK, LD = S::LD, NF = kFine<T>;
    constexpr int NX = NP > NF ? NP : NF;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    T* ks = reinterpret_cast<T*>(smem);
    float* m = reinterpret_cast<float*>(smem);
    float* tmp = C == 64 ? m + 32 : m + C * LD;
    float* beta = reinterpret_cast<float*>(smem + S::gate);
    float* sum_hi = beta + C;
    float* sum_lo = sum_hi + C;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), gq = lane >> 4, lr = lane & 15;
    const int64_t slot = blockIdx.x / p.heads_v;
    const int h = blockIdx.x % p.heads_v, hk = h / (p.heads_v / p.heads_qk);
    const SlotInfo info = slot_info<C>(p.offsets, p.tokens, p.n_seqs, slot, lane);
    if (info.rows == 0) {
        if (p.zero_rest && info.beyond >= 0 && h == 0) {
            const int64_t begin = seq_begin(p.offsets, p.tokens, p.n_seqs, info.seq);
            const int64_t len = seq_length(p.offsets, p.tokens, p.n_seqs, info.seq, begin);
            const int64_t spare = p.n_slots - first_slot(begin, info.seq, C) - (len + C - 1) / C;
            const int64_t head = seq_begin(p.offsets, p.tokens, p.n_seqs, 0), at = info.beyond * C, step = spare * C;
            auto zero = [&](const DeltaRows& r, int heads, int dim) {
                zero_rows<T>(r, begin + len + at, p.tokens, step, C, heads, dim, tid, THREADS);
                zero_rows<T>(r, at, head, step, C, heads, dim, tid, THREADS);
            };
            auto zero_gates = [&](const DeltaRows& r) {
                if (!p.fp32_grads) return zero(r, p.heads_v, 1);
                zero_rows<float>(r, begin + len + at, p.tokens, step, C, p.heads_v, 1, tid, THREADS);
                zero_rows<float>(r, at, head, step, C, p.heads_v, 1, tid, THREADS);
            };
            if constexpr (BWD) {
                zero(p.dq, p.heads_qk, p.dim_k);
                zero(p.dk, p.heads_qk, p.dim_k);
                zero(p.dv, p.heads_v, p.dim_v);
                zero_gates(p.dg);
                zero_gates(p.dbeta);
            } else {
                zero(p.out, p.heads_v, p.dim_v);
            }
        }
        return;
    }
    const T* k0 = static_cast<const T*>(p.k.data) + info.row * p.k.ts + hk * p.k.hs;
    const T* q0 = static_cast<const T*>(p.q.data) + info.row * p.q.ts + hk * p.q.hs;
    const int64_t at = slot * p.heads_v + h;
    float g = 0.f, b = 0.f;
    if (wave == 0 && lane < info.rows) {
        if (p.g.data) g = clamp_decay(load_gate(p.g, info.row + lane, h, p.g_dtype));
        b = load_gate(p.beta, info.row + lane, h, p.beta_dtype);
    }
    TileRegs<T, C, DK, THREADS> kr;
    kr.load(k0, p.k.ts, info.rows, p.dim_k, tid);
    if (wave == 0) {
        const double sum = scan_decays<C>((double)g * 1.4426950408889634, lane);
        const double last = __shfl(sum, C - 1, 64);
        if (lane < C) {
            const float hi = (float)sum, lo = (float)(sum - (double)hi);
            beta[lane] = b;
            sum_hi[lane] = hi;
            sum_lo[lane] = lo;
            float* w = p.w_gate + at * kGateArrays * C;
            w[lane] = exp2_fast(hi);
            w[C + lane] = exp2_fast((float)(last - sum));
            w[2 * C + lane] = b;
            w[3 * C + lane] = hi;
            w[4 * C + lane] = lo;
        }
    }
    kr.store(ks, LK, tid);
    __syncthreads();

    // A tile's results run along i for the forward pass and along j for the
    // backward one, whichever makes a lane's four neighbours in P or its
    // transpose. m = L B.
    using F = Triangle<C>;
    constexpr int TILES = NB * (NB + 1) / 2, EACH = (TILES + NB - 1) / NB;
    T* wp = static_cast<T*>(p.w_p) + at * NF * F::elems;
    f32x4 low[BWD ? EACH : 1];      // B L
    f32x4 lb[EACH];                 // L B, for m once K is done with
    const auto q_rsrc = rows_rsrc(q0, p.q.ts * (int)sizeof(T), info.rows, whole_bytes<T>(p.dim_k));
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
        const int tile = e * NB + wave;
        if (tile >= TILES) break;
        const int it = tile_row(tile), jt = tile - it * (it + 1) / 2;
        f32x4 kk = {}, qk = {};
        Vec8<T> qf[DK / 32];
#pragma unroll
        for (int kb = 0; kb < DK / 32; ++kb) {
            const int row = it * 16 + lr, c = kb * 32 + gq * 8;
            qf[kb] = buffer_frag<T>(q_rsrc, row < info.rows && c < p.dim_k ? (row * (int)p.q.ts + c) * (int)sizeof(T) : kOutside,
                                    p.dim_k - c);
        }
#pragma unroll
        for (int kb = 0; kb < DK / 32; ++kb) {
            if (kSkip<T, DK> && kb * 32 >= p.dim_k) break;
            const Vec8<T> ki = frag_nat(ks, LK, it * 16, kb * 32, lane), kj = frag_nat(ks, LK, jt * 16, kb * 32, lane);
            kk = BWD ? mma(ki, kj, kk) : mma(kj, ki, kk);
            qk = BWD ? mma(qf[kb], kj, qk) : mma(kj, qf[kb], qk);
        }
        const int one = (BWD ? jt : it) * 16 + lr, four = (BWD ? it : jt) * 16 + gq * 4;
        const float hi = sum_hi[one], lo = sum_lo[one], b1 = beta[one];
        const f32x4 hi4 = gate4(sum_hi, four), lo4 = gate4(sum_lo, four), b4 = gate4(beta, four);
        f32x4 pij, mij;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = BWD ? four + r : one, j = BWD ? one : four + r;
            const float d = BWD ? decay(hi4[r], lo4[r], hi, lo) : decay(hi, lo, hi4[r], lo4[r]);
            pij[r] = i > j ? p.scale * d * qk[r] : (i == j ? p.scale * qk[r] : 0.f);
            mij[r] = i > j ? d * kk[r] : 0.f;
        }
        if constexpr (BWD) {
            low[e] = mij * b4;
            lb[e] = mij * b1;
            store_parts4<NF>(wp + F::upper_acc(one, four), F::elems, pij);
        } else {
            lb[e] = mij * b4;
            store_parts4<NF>(wp + F::lower_nat(one, four), F::elems, pij);
        }
    }
    // the zero tile beside each even diagonal tile, which its fragment holds
    if (wave % 2 == 0) {
        const int row = (BWD ? wave + 1 : wave) * 16 + lr, c = (BWD ? wave : wave + 1) * 16 + gq * 4;
        store_parts4<NF>(wp + (BWD ? F::upper_acc(row, c) : F::lower_nat(row, c)), F::elems, f32x4{});
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
        const int tile = e * NB + wave;
        if (tile >= TILES) break;
        const int it = tile_row(tile), jt = tile - it * (it + 1) / 2;
        if constexpr (BWD)
            store_block<LD>(m + it * 16 * LD + jt * 16, lb[e], lane);
        else
            *reinterpret_cast<f32x4*>(m + (it * 16 + lr) * LD + jt * 16 + gq * 4) = lb[e];
    }
    __syncthreads();

    invert_unit_lower<C>(m, tmp, wave, lane);
    T* wt = static_cast<T*>(p.w_t) + at * NX * F::elems;
    // fragment by fragment, so that a wave writes whole lines
    for (int i = tid; i < F::frags * 64; i += THREADS) {
        const int f = i / 64, kb = f >= NB, row = (kb ? f - 2 : f) * 16 + lr;
        const float* x = m + row * LD + kb * 32 + gq * 4;
        store_fragment<NX>(wt + f * 512 + lane * 8, F::elems, *reinterpret_cast<const f32x4*>(x),
                           *reinterpret_cast<const f32x4*>(x + 16));
    }
    if constexpr (BWD) {
        // the other inverse, of I + B L
        __syncthreads();
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const int tile = e * NB + wave;
            if (tile >= TILES) break;
            const int it = tile_row(tile), jt = tile - it * (it + 1) / 2;
            store_block<LD>(m + it * 16 * LD + jt * 16, low[e], lane);
        }
        __syncthreads();
        invert_unit_lower<C>(m, tmp, wave, lane);
        T* wtt = static_cast<T*>(p.w_tt) + at * NF * F::elems;
        for (int i = tid; i < F::frags * 64; i += THREADS) {
            const int f = i / 64, kb = f >= 2, row = (kb ? f - 2 : f) * 16 + lr;       // of the transposed
            const float* x = m + (kb * 32 + gq * 4) * LD + row;
            store_fragment<NF>(wtt + f * 512 + lane * 8, F::elems, f32x4{x[0], x[LD], x[2 * LD], x[3 * LD]},
                               f32x4{x[16 * LD], x[17 * LD], x[18 * LD], x[19 * LD]});
        }
    }
}

// ---- the scans --------------------------------------------------------------
//
// A workgroup goes through one sequence's chunks for NW x 16 columns of a value
// head. Its first NW waves carry the states, 16 columns each: what they do from
// chunk to chunk is the time that no parallelism takes away, so they do nothing
// else. NW more waves, one on each of the same SIMDs, bring the next chunk's
// tiles to LDS and work out the outputs of the last one from the states and u
// that were left in LDS. Two LDS buffers and one barrier a chunk. A chunk of 64
// tokens of a 128 x 128 head takes 1.8 us with two state-carrying waves (2.5 us with
// three parts) on half of the compute units, 2.3 us (3.2) on all of them, and 2.9 us
// (5.0) with four. (The same waves doing all of it took a third longer.)
// What bounds it is that chain of products, LDS reads and splittings; the matrix
// cores are busy for a third of it.

// LDS of a scan workgroup: KQ tiles of keys or queries, TP triangular matrices,
// the columns of V or dO and the gate factors; with OUT, the states and u on
// their way to the outputs.
template <class T, int DK, int NW, int KQ, int TP, bool OUT>
struct ScanLds {
    static constexpr int C = kChunk<T, DK>, LK = lds_stride<T>(DK), LC = lds_stride<T>(C), LV = lds_stride<T>(NW * 16);
    static constexpr size_t ks = 0, ts = ks + KQ * (size_t)C * LK * sizeof(T);
    static constexpr size_t vs = ts + TP * (size_t)Triangle<C>::elems * sizeof(T);
    static constexpr size_t gate = vs + (size_t)C * LV * sizeof(T), sx = gate + 3 * C * sizeof(float);
    static constexpr size_t ux = sx + (OUT ? (size_t)NW * 16 * LK * sizeof(T) : 0);
    static constexpr size_t buffer = ux + (OUT ? kFine<T> * (size_t)NW * 16 * LC * sizeof(T) : 0), bytes = 2 * buffer;
};

// Which columns of which sequence and head a workgroup goes through.
struct ScanPlace {
    int64_t seq, begin, len, slot0;
    int h, hk, first;       // first column of the workgroup
};
template <int C, int NW>
__device__ __forceinline__ bool scan_place(const DeltaParams& p, uint32_t block, ScanPlace* w)
{
    const uint32_t parts = (uint32_t)((p.dim_v + NW * 16 - 1) / (NW * 16));
    uint32_t group, part;
    xcd_split(block, parts, &group, &part);
    if (group >= (uint64_t)p.n_seqs * p.heads_v) return false;
    w->seq = group / p.heads_v;
    w->h = group % p.heads_v;
    w->hk = w->h / (p.heads_v / p.heads_qk);
    w->first = part * NW * 16;
    w->begin = seq_begin(p.offsets, p.tokens, p.n_seqs, w->seq);
    w->len = seq_length(p.offsets, p.tokens, p.n_seqs, w->seq, w->begin);
    w->slot0 = first_slot(w->begin, w->seq, C);
    return true;
}
// A (dim_k x dim_v) state's 16 columns, laid out as results: element [t][r] of
// a lane is row 16 t + 4 gq + r.
template <int DK>
__device__ __forceinline__ void load_state(f32x4 (&s)[DK / 16], const float* state, int dim_k, int dim_v, int col, int gq)
{
    // a resource over dim_k rows of the state, or over none
    const auto rsrc = rows_rsrc(state, (int64_t)dim_v * 4, state != nullptr ? dim_k : 1, state != nullptr ? dim_v * 4 : 0);
#pragma unroll
    for (int t = 0; t < DK / 16; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = t * 16 + gq * 4 + r;
            s[t][r] = buffer_load<float>(rsrc, col < dim_v && row < dim_k ? (row * dim_v + col) * 4 : kOutside);
        }
}
template <int DK, class T>
__device__ __forceinline__ void store_state(const f32x4 (&s)[DK / 16], T* state, int dim_k, int dim_v, int col, int gq)
{
    const auto rsrc = rows_rsrc(state, (int64_t)dim_v * (int)sizeof(T), dim_k, dim_v * (int)sizeof(T));
#pragma unroll
    for (int t = 0; t < DK / 16; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = t * 16 + gq * 4 + r;
            buffer_store<T>(rsrc, col < dim_v && row < dim_k ? (row * dim_v + col) * (int)sizeof(T) : kOutside, (T)s[t][r]);
        }
}
// Sixteen columns of R rows, laid out as results, in the workspace: 16 bytes a
// lane after the other, as the lanes hold them (TileRegs::store_columns puts
// them in order), so that every store is of whole lines. With a row for each
// column, 16 lines a store and a quarter of each, the stores were half of a
// chunk's time in the backward scan.
template <class T, int NP, int R, int NX>
__device__ __forceinline__ void store_columns(T* at, int64_t part, const Parts<T, NX> (&x)[R / 32], int group, int lane)
{
    T* to = at + (int64_t)group * 16 * R + lane * (16 / (int)sizeof(T));
#pragma unroll
    for (int n = 0; n < NP; ++n)
#pragma unroll
        for (int t = 0; t < R / 32; ++t) {
            if constexpr (sizeof(T) == 2) {
                *reinterpret_cast<Vec8<T>*>(to + n * part + t * 512) = x[t].p[n];
            } else {
                *reinterpret_cast<Vec4<T>*>(to + t * 512) = __builtin_shufflevector(x[t].p[n], x[t].p[n], 0, 1, 2, 3);
                *reinterpret_cast<Vec4<T>*>(to + t * 512 + 256) = __builtin_shufflevector(x[t].p[n], x[t].p[n], 4, 5, 6, 7);
            }
        }
}

// STORE: instead of the outputs, the states at the chunks' starts and U' go to
// the workspace (for the backward pass). NP: parts of the operands the state
// depends on.
template <class T, int DK, int NP, bool STORE, int NW>
__device__ __forceinline__ void delta_scan(const DeltaParams& p, uint32_t block, char* smem)
{
    constexpr int NF = kFine<T>, NX = NP > NF ? NP : NF;
    using L = ScanLds<T, DK, NW, 1, NX, !STORE>;
    constexpr int C = L::C, THREADS = NW * 64, NB = C / 16, LK = L::LK, LC = L::LC, LV = L::LV, NK = DK / 16;
    using F = Triangle<C>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % NW;
    const int gq = lane >> 4, lr = lane & 15;
    ScanPlace w;
    if (!scan_place<C, NW>(p, block, &w)) return;
    int64_t st;
    if (!slot_taken<2 * THREADS>(p.slots, p.n_states, w.seq, &st, threadIdx.x)) return;
    const int64_t state_at = (st * p.heads_v + w.h) * p.dim_k * p.dim_v;
    const int chunks = (int)((w.len + C - 1) / C);
    const int col0 = w.first + wave * 16, col = col0 + lr;
    auto rows_at = [&](int c) { return w.len - (int64_t)c * C < C ? (int)(w.len - (int64_t)c * C) : C; };
    auto place_at = [&](int c) { return (w.slot0 + c) * p.heads_v + w.h; };

    if (__builtin_amdgcn_readfirstlane(threadIdx.x) >= THREADS) {
        // tiles and outputs, which the other waves wait for at the barrier: first
        // on their SIMDs (packed prompts 440 us without, 428 with; the other way
        // round 460). The backward scan has no outputs here, and its states first.
        __builtin_amdgcn_s_setprio(2);
        const int tid = threadIdx.x - THREADS;
        const T* k0 = static_cast<const T*>(p.k.data) + w.begin * p.k.ts + w.hk * p.k.hs;
        const T* q0 = static_cast<const T*>(p.q.data) + w.begin * p.q.ts + w.hk * p.q.hs;
        const T* v0 = static_cast<const T*>(p.v.data) + w.begin * p.v.ts + w.h * p.v.hs + w.first;
        const int cols = p.dim_v - w.first < NW * 16 ? p.dim_v - w.first : NW * 16;
        TileRegs<T, C, DK, THREADS> kr;
        TileRegs<T, 1, NX * F::elems, THREADS> tr;
        TileRegs<T, C, NW * 16, THREADS> vr;
        TileRegs<float, 1, 3 * C, THREADS> gr;
        auto load = [&](int c) {
            const int rows = rows_at(c);
            kr.load(k0 + (int64_t)c * C * p.k.ts, p.k.ts, rows, p.dim_k, tid);
            tr.load(static_cast<const T*>(p.w_t) + place_at(c) * NX * F::elems, 0, 1, NX * F::elems, tid);
            vr.load(v0 + (int64_t)c * C * p.v.ts, p.v.ts, rows, cols, tid);
            gr.load(p.w_gate + place_at(c) * kGateArrays * C, 0, 1, 3 * C, tid);
        };
        auto store = [&](int c) {
            char* buffer = smem + (c & 1) * L::buffer;
            kr.store(reinterpret_cast<T*>(buffer + L::ks), LK, tid);
            tr.store(reinterpret_cast<T*>(buffer + L::ts), 0, tid);
            vr.store(reinterpret_cast<T*>(buffer + L::vs), LV, tid);
            gr.store(reinterpret_cast<float*>(buffer + L::gate), 0, tid);
        };
        if (chunks > 0) {
            load(0);
            store(0);
        }
        if (chunks > 1) load(1);
        // Outputs are shared out by token tiles, so that each of Q's and P's
        // rows is read once: MT token tiles, CT column tiles a wave
        constexpr int MT = NB > NW ? NB / NW : 1, CT = NB / MT;
        const int mt0 = wave * MT % NB, ct0 = wave * MT / NB * CT;
        Parts<T, 1> qf[DK / 32][MT];
        Parts<T, NF> pf[C / 32][MT];
        float eg[MT];
        for (int c = 0; c < chunks + (STORE ? 0 : 1); ++c) {
            __syncthreads();
            if constexpr (!STORE) {
                if (c > 0) {
                    // O transposed, so that a lane has four columns of one
                    // token: the state and u in the place of the left operand
                    const char* buffer = smem + ((c - 1) & 1) * L::buffer;
                    const T* sx = reinterpret_cast<const T*>(buffer + L::sx);
                    const T* ux = reinterpret_cast<const T*>(buffer + L::ux);
                    f32x4 o[CT][MT] = {};
                    // reads of the next products' operands ahead of the products
                    Parts<T, 1> sa[2][CT];
                    Parts<T, NF> ua[2][CT];
                    auto read_s = [&](int kb) {
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) sa[kb % 2][ct].p[0] = frag_nat(sx, LK, (ct0 + ct) * 16, kb * 32, lane);
                    };
                    auto read_u = [&](int kb) {
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                            for (int n = 0; n < NF; ++n)
                                ua[kb % 2][ct].p[n] = frag_nat(ux + n * NW * 16 * LC, LC, (ct0 + ct) * 16, kb * 32, lane);
                    };
                    read_s(0);
#pragma unroll
                    for (int kb = 0; kb < DK / 32; ++kb) {
                        if (kb + 1 < DK / 32)
                            read_s(kb + 1);
                        else
                            read_u(0);
                        if constexpr (MT == 1) __builtin_amdgcn_sched_barrier(0);
                        if (!kSkip<T, DK> || kb * 32 < p.dim_k)
#pragma unroll
                            for (int ct = 0; ct < CT; ++ct) mma_each<true>(qf[kb], sa[kb % 2][ct], o[ct]);
                        if constexpr (MT == 1) __builtin_amdgcn_sched_barrier(0);
                    }
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                        for (int m = 0; m < MT; ++m) o[ct][m] *= p.scale * eg[m];
#pragma unroll
                    for (int kb = 0; kb < C / 32; ++kb) {
                        if (kb + 1 < C / 32) read_u(kb + 1);
                        if constexpr (MT == 1) __builtin_amdgcn_sched_barrier(0);
                        if (2 * kb <= mt0 + MT - 1)       // P is lower triangular
#pragma unroll
                            for (int ct = 0; ct < CT; ++ct) mma_each<true>(pf[kb], ua[kb % 2][ct], o[ct]);
                    }
                    const int rows = rows_at(c - 1);
                    T* o0 = static_cast<T*>(p.out.data) + (w.begin + (int64_t)(c - 1) * C) * p.out.ts + w.h * p.out.hs;
                    const auto rsrc = rows_rsrc(o0, p.out.ts * (int)sizeof(T), rows, p.dim_v * (int)sizeof(T));
                    const int step = (int)p.out.ts * (int)sizeof(T);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const int row = (mt0 + m) * 16 + lr, oc = w.first + (ct0 + ct) * 16 + gq * 4;
                            const int to = row < rows && oc < p.dim_v ? row * step + oc * (int)sizeof(T) : kOutside;
                            const Vec4<T> y = __builtin_convertvector(o[ct][m], Vec4<T>);
                            if (p.out4) {
                                buffer_store(rsrc, to, y);
                            } else {
#pragma unroll
                                for (int r = 0; r < 4; ++r)
                                    buffer_store<T>(rsrc, oc + r < p.dim_v ? to + r * (int)sizeof(T) : kOutside, y[r]);
                            }
                        }
                }
                if (c < chunks) {
                    const int rows = rows_at(c);
                    const auto rsrc = rows_rsrc(q0 + (int64_t)c * C * p.q.ts, p.q.ts * (int)sizeof(T), rows,
                                                whole_bytes<T>(p.dim_k));
                    const T* wp = static_cast<const T*>(p.w_p) + place_at(c) * NF * F::elems;
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const int row = (mt0 + m) * 16 + lr;
#pragma unroll
                        for (int kb = 0; kb < DK / 32; ++kb) {
                            const int k = kb * 32 + gq * 8;
                            qf[kb][m].p[0] = buffer_frag<T>(
                                rsrc, row < rows && k < p.dim_k ? (row * (int)p.q.ts + k) * (int)sizeof(T) : kOutside,
                                p.dim_k - k);
                        }
                        eg[m] = p.w_gate[place_at(c) * kGateArrays * C + row];
                        // (above the diagonal: not kept, and 0)
#pragma unroll
                        for (int kb = 0; kb < C / 32; ++kb)
                            if (2 * kb <= mt0 + m)
                                pf[kb][m] = parts_at<NF>(wp, F::elems, F::lower(mt0 + m, kb), lane);
                            else
                                pf[kb][m] = Parts<T, NF>{};
                    }
                }
            }
            if (c + 1 < chunks) store(c + 1);
            if (c + 2 < chunks) load(c + 2);
        }
        return;
    }

    f32x4 s[NK];
    load_state<DK>(s, p.initial ? p.initial + state_at : nullptr, p.dim_k, p.dim_v, col, gq);
    // Split ahead, while the last update's products run, or, where the parts would
    // not fit the registers beside the state, when they are used.
    constexpr bool AHEAD = NK * NP <= 32;
    Parts<T, NP> sb[AHEAD ? DK / 32 : 1];
    auto split = [&](int kb) {
        if constexpr (AHEAD) sb[kb] = parts_of<T, NP>(s[2 * kb], s[2 * kb + 1]);
    };
    auto parts_of_state = [&](int kb) {
        if constexpr (AHEAD)
            return sb[kb];
        else
            return parts_of<T, NP>(s[2 * kb], s[2 * kb + 1]);
    };
#pragma unroll
    for (int kb = 0; kb < DK / 32; ++kb) split(kb);
    for (int c = 0; c < chunks; ++c) {
        char* buffer = smem + (c & 1) * L::buffer;
        const T* ks = reinterpret_cast<const T*>(buffer + L::ks);
        const T* ts = reinterpret_cast<const T*>(buffer + L::ts);
        const T* vs = reinterpret_cast<const T*>(buffer + L::vs);
        const float* gate = reinterpret_cast<const float*>(buffer + L::gate);
        if constexpr (STORE)
            if (col0 < p.dv_pad)
                store_columns<T, kStored<T>, DK>(static_cast<T*>(p.w_s) + place_at(c) * kStored<T> * DK * p.dv_pad,
                                                 (int64_t)DK * p.dv_pad, sb, col0 / 16, lane);
        __syncthreads();
        // X = V - diag(e^G) K S
        f32x4 x[NB] = {};
        Parts<T, 1> ka[2][NB];
        auto read_k = [&](int kb) {
#pragma unroll
            for (int mt = 0; mt < NB; ++mt) ka[kb % 2][mt].p[0] = frag_acc(ks, LK, mt * 16, kb * 32, lane);
        };
        read_k(0);
#pragma unroll
        for (int kb = 0; kb < DK / 32; ++kb) {
            if (kb + 1 < DK / 32) read_k(kb + 1);
            __builtin_amdgcn_sched_barrier(0);
            if (!kSkip<T, DK> || kb * 32 < p.dim_k) mma_each(ka[kb % 2], parts_of_state(kb), x);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (!STORE) {
            T* sx = reinterpret_cast<T*>(buffer + L::sx) + (wave * 16 + lr) * LK + gq * 4;
#pragma unroll
            for (int kb = 0; kb < DK / 32; ++kb) {
                const Vec8<T> y = parts_of_state(kb).p[0];
                *reinterpret_cast<Vec4<T>*>(sx + kb * 32) = __builtin_shufflevector(y, y, 0, 1, 2, 3);
                *reinterpret_cast<Vec4<T>*>(sx + kb * 32 + 16) = __builtin_shufflevector(y, y, 4, 5, 6, 7);
            }
        }
#pragma unroll
        for (int mt = 0; mt < NB; ++mt) {
            const Vec4<T> v = quad_tr(vs, LV, mt * 16, wave * 16, lane);
            x[mt] = __builtin_convertvector(v, f32x4) - gate4(gate, mt * 16 + gq * 4) * x[mt];
        }
        // U' = (I + L B)^-1 X; u = B U'
        f32x4 u[NB] = {};
#pragma unroll
        for (int kb = 0; kb < C / 32; ++kb) {
            Parts<T, NX> a[NB];
#pragma unroll
            for (int mt = 2 * kb; mt < NB; ++mt) a[mt] = parts_at<NX>(ts, F::elems, F::lower(mt, kb), lane);
            mma_each(a, parts_of<T, NX>(x[2 * kb], x[2 * kb + 1]), u, 2 * kb);
        }
        if constexpr (STORE)
            if (col0 < p.dv_pad) {
                Parts<T, NF> up[C / 32];
#pragma unroll
                for (int kb = 0; kb < C / 32; ++kb) up[kb] = parts_of<T, NF>(u[2 * kb], u[2 * kb + 1]);
                store_columns<T, NF, C>(static_cast<T*>(p.w_u) + place_at(c) * NF * C * p.dv_pad, (int64_t)C * p.dv_pad, up,
                                        col0 / 16, lane);
            }
#pragma unroll
        for (int mt = 0; mt < NB; ++mt) u[mt] *= gate4(gate, 2 * C + mt * 16 + gq * 4);
        if constexpr (!STORE) {
            T* ux = reinterpret_cast<T*>(buffer + L::ux) + (wave * 16 + lr) * LC + gq * 4;
#pragma unroll
            for (int mt = 0; mt < NB; ++mt) store_parts4<NF>(ux + mt * 16, NW * 16 * LC, u[mt]);
        }
        // S <- e^(G_C) S + K^T diag(e^(G_C - G)) u
#pragma unroll
        for (int mt = 0; mt < NB; ++mt) u[mt] *= gate4(gate, C + mt * 16 + gq * 4);
        const float keep = gate[C - 1];
#pragma unroll
        for (int t = 0; t < NK; ++t) s[t] *= keep;
#pragma unroll
        for (int kb = 0; kb < C / 32; ++kb) {
            const Parts<T, NX> ub = parts_of<T, NX>(u[2 * kb], u[2 * kb + 1]);
#pragma unroll
            for (int t0 = 0; t0 < NK; t0 += 4) {
                if (kSkip<T, DK> && t0 * 16 >= p.dim_k) break;
                Parts<T, 1> a[4];
                f32x4 acc[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    a[t].p[0] = frag_tr(ks, LK, kb * 32, (t0 + t) * 16, lane);
                    acc[t] = s[t0 + t];
                }
                mma_each(a, ub, acc);
#pragma unroll
                for (int t = 0; t < 4; ++t) s[t0 + t] = acc[t];
                // the next chunk's operands, while the other tiles' products run
                if (kb == C / 32 - 1)
#pragma unroll
                    for (int t = 0; t < 4; t += 2) split((t0 + t) / 2);
            }
        }
    }
    if constexpr (!STORE) {
        __syncthreads();      // the other waves' last chunk
        if (p.final_state != nullptr) store_state<DK>(s, p.final_state + state_at, p.dim_k, p.dim_v, col, gq);
    }
}

// ---- the backward scan -----------------------------------------------------
//
// With dS' the gradient at the chunk's end and dO given:
//   dU = P^T dO + diag(e^(G_C - G)) K dS'     Z = (I + B L)^-T dU     dX = B Z = dV
//   dS = e^(G_C) dS' + Q^T diag(scale e^G) dO - K^T diag(e^G) dX
// The same shape as the forward scan, from a sequence's last chunk to its
// first. Z and dS' go to the workspace; the next kernel, which has Z by rows,
// writes dV (16 two-byte stores a lane here were a third of a chunk's time).
// Both scans together move 580 MB for 2,096 chunks and heads of 128 x 128 in 146
// us, 4.0 TB/s: the memory bounds them, most of it the states and Z and U'.

template <class T, int DK, int ND, int NW>
__device__ __forceinline__ void delta_scan_back(const DeltaParams& p, uint32_t block, char* smem)
{
    constexpr int NF = kFine<T>;
    using L = ScanLds<T, DK, NW, 2, 2 * NF, false>;
    constexpr int C = L::C, THREADS = NW * 64, NB = C / 16, LK = L::LK, LV = L::LV, NK = DK / 16;
    using F = Triangle<C>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % NW;
    const int gq = lane >> 4, lr = lane & 15;
    ScanPlace w;
    if (!scan_place<C, NW>(p, block, &w)) return;
    const int64_t state_at = (w.seq * p.heads_v + w.h) * p.dim_k * p.dim_v;
    const int chunks = (int)((w.len + C - 1) / C);
    const int col0 = w.first + wave * 16, col = col0 + lr;
    auto rows_at = [&](int c) { return w.len - (int64_t)c * C < C ? (int)(w.len - (int64_t)c * C) : C; };
    auto place_at = [&](int c) { return (w.slot0 + c) * p.heads_v + w.h; };

    if (__builtin_amdgcn_readfirstlane(threadIdx.x) >= THREADS) {
        const int tid = threadIdx.x - THREADS;
        const T* k0 = static_cast<const T*>(p.k.data) + w.begin * p.k.ts + w.hk * p.k.hs;
        const T* q0 = static_cast<const T*>(p.q.data) + w.begin * p.q.ts + w.hk * p.q.hs;
        const T* o0 = static_cast<const T*>(p.d_out.data) + w.begin * p.d_out.ts + w.h * p.d_out.hs + w.first;
        const int cols = p.dim_v - w.first < NW * 16 ? p.dim_v - w.first : NW * 16;
        TileRegs<T, C, DK, THREADS> kr, qr;
        TileRegs<T, 1, NF * F::elems, THREADS> tr, pr;
        TileRegs<T, C, NW * 16, THREADS> orr;
        TileRegs<float, 1, 3 * C, THREADS> gr;
        auto load = [&](int c) {
            const int rows = rows_at(c);
            kr.load(k0 + (int64_t)c * C * p.k.ts, p.k.ts, rows, p.dim_k, tid);
            qr.load(q0 + (int64_t)c * C * p.q.ts, p.q.ts, rows, p.dim_k, tid);
            tr.load(static_cast<const T*>(p.w_tt) + place_at(c) * NF * F::elems, 0, 1, NF * F::elems, tid);
            pr.load(static_cast<const T*>(p.w_p) + place_at(c) * NF * F::elems, 0, 1, NF * F::elems, tid);
            orr.load(o0 + (int64_t)c * C * p.d_out.ts, p.d_out.ts, rows, cols, tid);
            gr.load(p.w_gate + place_at(c) * kGateArrays * C, 0, 1, 3 * C, tid);
        };
        auto store = [&](int c) {
            char* buffer = smem + (c & 1) * L::buffer;
            kr.store(reinterpret_cast<T*>(buffer + L::ks), LK, tid);
            qr.store(reinterpret_cast<T*>(buffer + L::ks) + C * LK, LK, tid);
            tr.store(reinterpret_cast<T*>(buffer + L::ts), 0, tid);
            pr.store(reinterpret_cast<T*>(buffer + L::ts) + NF * F::elems, 0, tid);
            orr.store(reinterpret_cast<T*>(buffer + L::vs), LV, tid);
            gr.store(reinterpret_cast<float*>(buffer + L::gate), 0, tid);
        };
        if (chunks > 0) {
            load(chunks - 1);
            store(chunks - 1);
        }
        if (chunks > 1) load(chunks - 2);
        for (int c = chunks - 1; c >= 0; --c) {
            __syncthreads();
            if (c > 0) store(c - 1);
            if (c > 1) load(c - 2);
        }
        return;
    }

    __builtin_amdgcn_s_setprio(2);
    f32x4 ds[NK];
    load_state<DK>(ds, p.d_final ? p.d_final + state_at : nullptr, p.dim_k, p.dim_v, col, gq);
    for (int c = chunks - 1; c >= 0; --c) {
        char* buffer = smem + (c & 1) * L::buffer;
        const T* ks = reinterpret_cast<const T*>(buffer + L::ks);
        const T* qs = ks + C * LK;
        const T* ts = reinterpret_cast<const T*>(buffer + L::ts);
        const T* ps = ts + NF * F::elems;
        const T* os = reinterpret_cast<const T*>(buffer + L::vs);
        const float* gate = reinterpret_cast<const float*>(buffer + L::gate);
        const int64_t at = place_at(c);
        Parts<T, ND> db[DK / 32];
#pragma unroll
        for (int kb = 0; kb < DK / 32; ++kb) db[kb] = parts_of<T, ND>(ds[2 * kb], ds[2 * kb + 1]);
        if (col0 < p.dv_pad)
            store_columns<T, ND, DK>(static_cast<T*>(p.w_ds) + at * ND * DK * p.dv_pad, (int64_t)DK * p.dv_pad, db,
                                     col0 / 16, lane);
        __syncthreads();
        // dU; dO is exact in T
        Vec4<T> d_o[NB];
#pragma unroll
        for (int mt = 0; mt < NB; ++mt) d_o[mt] = quad_tr(os, LV, mt * 16, wave * 16, lane);
        f32x4 z[NB] = {};
#pragma unroll
        for (int kb = 0; kb < DK / 32; ++kb) {
            Parts<T, 1> a[NB];
#pragma unroll
            for (int mt = 0; mt < NB; ++mt) a[mt].p[0] = frag_acc(ks, LK, mt * 16, kb * 32, lane);
            if (!kSkip<T, DK> || kb * 32 < p.dim_k) mma_each(a, db[kb], z);
        }
#pragma unroll
        for (int mt = 0; mt < NB; ++mt) z[mt] *= gate4(gate, C + mt * 16 + gq * 4);
#pragma unroll
        for (int kb = 0; kb < C / 32; ++kb) {
            Parts<T, NF> a[NB];
#pragma unroll
            for (int mt = 0; mt < 2 * kb + 2; ++mt) a[mt] = parts_at<NF>(ps, F::elems, F::upper(mt, kb), lane);
            mma_each(a, Parts<T, 1>{{__builtin_shufflevector(d_o[2 * kb], d_o[2 * kb + 1], 0, 1, 2, 3, 4, 5, 6, 7)}}, z, 0,
                     2 * kb + 2);
        }
        f32x4 y[NB] = {};
#pragma unroll
        for (int kb = 0; kb < C / 32; ++kb) {
            Parts<T, NF> a[NB];
#pragma unroll
            for (int mt = 0; mt < 2 * kb + 2; ++mt) a[mt] = parts_at<NF>(ts, F::elems, F::upper(mt, kb), lane);
            mma_each(a, parts_of<T, NF>(z[2 * kb], z[2 * kb + 1]), y, 0, 2 * kb + 2);
        }
        if (col0 < p.dv_pad) {
            Parts<T, NF> zp[C / 32];
#pragma unroll
            for (int kb = 0; kb < C / 32; ++kb) zp[kb] = parts_of<T, NF>(y[2 * kb], y[2 * kb + 1]);
            store_columns<T, NF, C>(static_cast<T*>(p.w_z) + at * NF * C * p.dv_pad, (int64_t)C * p.dv_pad, zp, col0 / 16, lane);
        }
        f32x4 e[NB];
#pragma unroll
        for (int mt = 0; mt < NB; ++mt) {
            const int row = mt * 16 + gq * 4;
            const f32x4 eg = gate4(gate, row);
            y[mt] *= -(eg * gate4(gate, 2 * C + row));
            e[mt] = __builtin_convertvector(d_o[mt], f32x4) * (p.scale * eg);
        }
        const float keep = gate[C - 1];
#pragma unroll
        for (int t = 0; t < NK; ++t) ds[t] *= keep;
#pragma unroll
        for (int kb = 0; kb < C / 32; ++kb) {
            const Parts<T, NF> eb = parts_of<T, NF>(e[2 * kb], e[2 * kb + 1]);
            // (in one part the initial state's gradient was off by 0.19 times a 16-bit
            // rounding at the median of 14 random calls, in two by 0.01; 3 us of a
            // training step's 460)
            const Parts<T, NF> yb = parts_of<T, NF>(y[2 * kb], y[2 * kb + 1]);
#pragma unroll
            for (int t0 = 0; t0 < NK; t0 += 4) {
                if (kSkip<T, DK> && t0 * 16 >= p.dim_k) break;
                Parts<T, 1> a[4], b[4];
                f32x4 acc[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    a[t].p[0] = frag_tr(qs, LK, kb * 32, (t0 + t) * 16, lane);
                    b[t].p[0] = frag_tr(ks, LK, kb * 32, (t0 + t) * 16, lane);
                    acc[t] = ds[t0 + t];
                }
                mma_each(a, eb, acc);
                mma_each(b, yb, acc);
#pragma unroll
                for (int t = 0; t < 4; ++t) ds[t0 + t] = acc[t];
            }
        }
    }
    if (p.d_initial != nullptr) {
        // (made unknown: else the places that load_state worked out are kept in
        // registers until here, and heads above 128 spill 112 bytes a lane)
        int here = col;
        asm volatile("" : "+v"(here));
        if (p.fp32_grads)
            store_state<DK>(ds, static_cast<float*>(p.d_initial) + state_at, p.dim_k, p.dim_v, here, gq);
        else
            store_state<DK>(ds, static_cast<T*>(p.d_initial) + state_at, p.dim_k, p.dim_v, here, gq);
    }
}

template <class T, int DK, int NP, int NW>
__global__ __launch_bounds__(NW * 128) DWS_TWO_WAVES void k_delta_scan(DeltaParams p)
{
    extern __shared__ __attribute__((aligned(16))) char smem[];
    delta_scan<T, DK, NP, false, NW>(p, blockIdx.x, smem);
}
// The backward pass's two scans, which do not need each other: half of the
// workgroups each, the longer ones first. Where there are fewer of them than
// compute units both run at once.
template <class T, int DK, int ND, int NW>
__global__ __launch_bounds__(NW * 128) DWS_TWO_WAVES void k_delta_scan_both(DeltaParams p)
{
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const uint32_t half = gridDim.x / 2;
    if (blockIdx.x < half)
        delta_scan_back<T, DK, ND, NW>(p, blockIdx.x, smem);
    else
        delta_scan<T, DK, kStored<T>, true, NW>(p, blockIdx.x - half, smem);
}

// ---- the gradients of q, k and the gates ------------------------------------
//
// Every chunk by itself, from the states, U', Z and dS' of the two scans:
//   dP = tril(dO U'^T) B                      M = -tril(Z U'^T, -1) B
//   W1 = scale D o dP                         W2 = B (D o M)
//   dQ = W1 K + scale diag(e^G) dO S^T
//   dK = W1^T Q + (W2 + W2^T) K + diag(e^(G_C - G)) B U' dS'^T - diag(e^G) B Z S^T
//   dV = B Z              dbeta_i = Z_i . U'_i
//   N = W1 o Q K^T + W2 o K K^T
//   dG_i = sum_j (N_ij - N_ji) + (scale e^G dO S^T)_i . q_i - (e^G B Z S^T)_i . k_i - w_i,
//          w_i = (e^(G_C - G) B U' dS'^T)_i . k_i;   dG_C also gets sum w + e^(G_C) <S, dS'>
//   dg_t = sum of dG_i from t to the chunk's end
// One workgroup for each (chunk slot, query/key head). A wave owns a row tile
// of 16 tokens and 64 of the key columns; the value heads
// that share the key head come in turn, so that their sums need no atomics and
// have one order. Blocks of 32 value columns of the workspace's arrays go through
// LDS, a row a column, where the transposing reads make operands of them. 2,096
// chunks and value heads of 128 x 128 take 177 us: 484 MB, which would take 90, but
// with all 256 registers of two waves a SIMD in use one block is in flight at a
// time, and a third of the time goes to waiting for it.

template <class T, int DK, int PARTS>
struct GradLds {
    static constexpr int C = kChunk<T, DK>, NB = C / 16, GROUPS = DK / 64, THREADS = NB * GROUPS * 64;
    static constexpr int LK = lds_stride<T>(DK), LC = lds_stride<T>(C), NF = kFine<T>, NS = kStored<T>, ND = PARTS;
    static constexpr size_t ks = 0, qs = ks + (size_t)C * LK * sizeof(T), w1 = qs + (size_t)C * LK * sizeof(T);
    static constexpr size_t w2 = w1 + (size_t)NF * C * LC * sizeof(T), w_end = w2 + (size_t)NF * C * LC * sizeof(T);
    // the blocks of 32 value columns are done with before W1 and W2 are written
    // (read transposed only: rows 32 bytes longer lie in different banks)
    static constexpr int LS = DK + 32 / (int)sizeof(T);
    static constexpr size_t st = w1, dst = st + (size_t)NS * 32 * LS * sizeof(T), ut = dst + (size_t)ND * 32 * LS * sizeof(T);
    static constexpr size_t zt = ut + (size_t)NF * 32 * LC * sizeof(T), z_end = zt + (size_t)NF * 32 * LC * sizeof(T);
    static constexpr size_t gate = w_end > z_end ? w_end : z_end;
    // floats behind: gate[5 C], row_part[GROUPS C], row_w[GROUPS C], d_beta[C], col_part[NB C], n_part[GROUPS C],
    // inner[THREADS / 64]
    static constexpr size_t bytes = gate + ((kGateArrays + 1 + 3 * GROUPS + NB) * C + 16) * sizeof(float);
};

// Over the 16 lanes of a group, by rotations within a row of lanes.
__device__ __forceinline__ float sum16(float x)
{
    auto turned = [](float y, auto n) {
        return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, y), 0x120 + decltype(n)::value, 0xf,
                                                                  0xf, true));
    };
    x += turned(x, std::integral_constant<int, 8>{});
    x += turned(x, std::integral_constant<int, 4>{});
    x += turned(x, std::integral_constant<int, 2>{});
    return x + turned(x, std::integral_constant<int, 1>{});
}
__device__ __forceinline__ float sum_groups(float x) // over the 4 groups
{
    x += __shfl_xor(x, 16, 64);
    return x + __shfl_xor(x, 32, 64);
}
// Eight elements of a row (at element `row` of the resource, -1: none), columns
// c .. c + 3 and c + 16 .. c + 19.
template <class T>
__device__ __forceinline__ void store_quads(__amdgpu_buffer_rsrc_t rsrc, bool whole, int row, int c, int dim, Vec8<T> x)
{
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int o = c + q * 16;
        const Vec4<T> y = q == 0 ? __builtin_shufflevector(x, x, 0, 1, 2, 3) : __builtin_shufflevector(x, x, 4, 5, 6, 7);
        if (whole) {
            buffer_store(rsrc, row >= 0 && o < dim ? (row + o) * (int)sizeof(T) : kOutside, y);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                buffer_store<T>(rsrc, row >= 0 && o + r < dim ? (row + o + r) * (int)sizeof(T) : kOutside, y[r]);
        }
    }
}

template <class T, int DK, int PARTS>
__global__ __launch_bounds__((GradLds<T, DK, PARTS>::THREADS)) DWS_TWO_WAVES void k_delta_grad(DeltaParams p)
{
    using L = GradLds<T, DK, PARTS>;
    constexpr int C = L::C, THREADS = L::THREADS, NB = L::NB, GROUPS = L::GROUPS, LK = L::LK, LC = L::LC, LS = L::LS, NF = L::NF, NS = L::NS, ND = L::ND;
    constexpr int NK = DK / 16 / GROUPS;             // key column tiles of a wave
    constexpr int NT = NB > GROUPS ? NB / GROUPS : 1;      // its column tiles of W1 and W2: grp, grp + GROUPS, ..
    extern __shared__ __attribute__((aligned(16))) char smem[];
    T* ks = reinterpret_cast<T*>(smem + L::ks);
    T* qs = reinterpret_cast<T*>(smem + L::qs);
    T* w1 = reinterpret_cast<T*>(smem + L::w1);
    T* w2 = reinterpret_cast<T*>(smem + L::w2);
    T* st = reinterpret_cast<T*>(smem + L::st);
    T* dst = reinterpret_cast<T*>(smem + L::dst);
    T* ut = reinterpret_cast<T*>(smem + L::ut);
    T* zt = reinterpret_cast<T*>(smem + L::zt);
    float* gate = reinterpret_cast<float*>(smem + L::gate);      // the workspace's factors
    float* row_part = gate + kGateArrays * C;                    // dG without column sums and w
    float* row_w = row_part + GROUPS * C;                        // w
    float* d_beta = row_w + GROUPS * C;
    float* col_part = d_beta + C;                                // [NB][C] column sums of N
    float* n_part = col_part + NB * C;                           // [GROUPS][C] row sums of N
    float* inner = n_part + GROUPS * C;                          // parts of <S, dS'>

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), gq = lane >> 4, lr = lane & 15;
    const int tile = wave % NB, grp = wave / NB, row0 = tile * 16, key0 = grp * 64;
    const int64_t slot = blockIdx.x / p.heads_qk;
    const int hk = blockIdx.x % p.heads_qk, share = p.heads_v / p.heads_qk;
    const SlotInfo info = slot_info<C>(p.offsets, p.tokens, p.n_seqs, slot, lane);
    if (info.rows == 0) return;
    const int rows = info.rows;

    TileRegs<T, 32, DK, THREADS> sr[NS], dsr[ND];
    TileRegs<T, 32, C, THREADS> ur[NF], zr[NF];
    Vec4<T> oa, ob;        // dO's row lr of this wave, 32 columns in acc order
    auto load = [&](int h, int c) {
        const int64_t at = slot * p.heads_v + h;
        const T* d_o = static_cast<const T*>(p.d_out.data) + info.row * p.d_out.ts + h * p.d_out.hs;
        const auto rsrc = rows_rsrc(d_o, p.d_out.ts * (int)sizeof(T), rows, whole_bytes<T>(p.dim_v));
        const int o0 = c + gq * 4, from = ((row0 + lr) * (int)p.d_out.ts + o0) * (int)sizeof(T);
        const bool in = row0 + lr < rows;
        oa = buffer_load<Vec4<T>>(rsrc, in && o0 < p.dim_v ? from : kOutside);
        ob = buffer_load<Vec4<T>>(rsrc, in && o0 + 16 < p.dim_v ? from + 16 * (int)sizeof(T) : kOutside);
#pragma unroll
        for (int n = 0; n < NS; ++n)
            sr[n].load(static_cast<const T*>(p.w_s) + ((at * NS + n) * p.dv_pad + c) * DK, DK, 32, DK, tid);
#pragma unroll
        for (int n = 0; n < ND; ++n)
            dsr[n].load(static_cast<const T*>(p.w_ds) + ((at * ND + n) * p.dv_pad + c) * DK, DK, 32, DK, tid);
#pragma unroll
        for (int n = 0; n < NF; ++n) {
            ur[n].load(static_cast<const T*>(p.w_u) + ((at * NF + n) * p.dv_pad + c) * C, C, 32, C, tid);
            zr[n].load(static_cast<const T*>(p.w_z) + ((at * NF + n) * p.dv_pad + c) * C, C, 32, C, tid);
        }
    };
    load(hk * share, 0);
    {
        TileRegs<T, C, DK, THREADS> kr, qr;
        kr.load(static_cast<const T*>(p.k.data) + info.row * p.k.ts + hk * p.k.hs, p.k.ts, rows, p.dim_k, tid);
        qr.load(static_cast<const T*>(p.q.data) + info.row * p.q.ts + hk * p.q.hs, p.q.ts, rows, p.dim_k, tid);
        kr.store(ks, LK, tid);
        qr.store(qs, LK, tid);
    }
    f32x4 dq[NK] = {}, dk[NK] = {};

    for (int m = 0; m < share; ++m) {
        const int h = hk * share + m;
        const int64_t at = slot * p.heads_v + h;
        for (int i = tid; i < kGateArrays * C; i += THREADS) gate[i] = p.w_gate[at * kGateArrays * C + i];

        const auto dv_rsrc = rows_rsrc(static_cast<T*>(p.dv.data) + info.row * p.dv.ts + h * p.dv.hs, p.dv.ts * (int)sizeof(T),
                                       rows, p.dim_v * (int)sizeof(T));
        f32x4 dp[NT] = {}, zu[NT] = {}, os[NK] = {}, zs[NK] = {}, us[NK] = {};
        float zdotu = 0.f, sds = 0.f;
        for (int c = 0; c < p.dv_pad; c += 32) {
            // (made unknown, so that the loop's addresses are worked out in each
            // turn: kept over the turns they take registers and spill, 190 us
            // instead of 178)
            int here = tid;
            asm volatile("" : "+v"(here));
            const int lane = here & 63, gq = lane >> 4, lr = lane & 15;
            Parts<T, 1> ao;
            ao.p[0] = __builtin_shufflevector(oa, ob, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
            for (int n = 0; n < NS; ++n) sr[n].store_columns(st + n * 32 * LS, LS, here);
#pragma unroll
            for (int n = 0; n < ND; ++n) dsr[n].store_columns(dst + n * 32 * LS, LS, here);
#pragma unroll
            for (int n = 0; n < NF; ++n) {
                ur[n].store_columns(ut + n * 32 * LC, LC, here);
                zr[n].store_columns(zt + n * 32 * LC, LC, here);
            }
            __syncthreads();
            if (c + 32 < p.dv_pad)
                load(h, c + 32);
            else if (m + 1 < share)
                load(h + 1, 0);
            __builtin_amdgcn_sched_barrier(0);
            const Parts<T, NF> az = parts_tr<NF>(zt, 32 * LC, LC, 0, row0, lane);
            const Parts<T, NF> au = parts_tr<NF>(ut, 32 * LC, LC, 0, row0, lane);
            if (grp == 0) {
                f32x8 dv = {};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float z = 0.f, u = 0.f;
#pragma unroll
                    for (int n = NF - 1; n >= 0; --n) {
                        z += (float)az.p[n][j];
                        u += (float)au.p[n][j];
                    }
                    zdotu += z * u;
                    dv[j] = gate[2 * C + row0 + lr] * z;
                }
                store_quads(dv_rsrc, p.dv4, row0 + lr < rows ? (row0 + lr) * (int)p.dv.ts : -1, c + gq * 4, p.dim_v,
                            __builtin_convertvector(dv, Vec8<T>));
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < NT; ++i)
                if (grp + i * GROUPS <= tile) {
                    const Parts<T, NF> b = parts_tr<NF>(ut, 32 * LC, LC, 0, (grp + i * GROUPS) * 16, lane);
                    dp[i] = mma(b, ao, dp[i]);
                    zu[i] = mma(b, az, zu[i]);
                }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < NK; ++t) {
                const Parts<T, NS> b = parts_tr<NS>(st, 32 * LS, LS, 0, key0 + t * 16, lane);
                const Parts<T, ND> d = parts_tr<ND>(dst, 32 * LS, LS, 0, key0 + t * 16, lane);
                os[t] = mma(ao, b, os[t]);
                zs[t] = mma(az, b, zs[t]);
                us[t] = mma(au, d, us[t]);
                if (t % NB == tile)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float x = 0.f, y = 0.f;
#pragma unroll
                        for (int n = NS - 1; n >= 0; --n) x += (float)b.p[n][j];
#pragma unroll
                        for (int n = ND - 1; n >= 0; --n) y += (float)d.p[n][j];
                        sds += x * y;
                    }
            }
            __syncthreads();
        }
        zdotu = sum_groups(zdotu);               // lane: row lr of the tile
        if (gq == 0 && grp == 0) d_beta[row0 + lr] = zdotu;
        sds = sum_groups(sum16(sds));
        if (lane == 0) inner[wave] = sds;

        // W1, W2 and N; Q K^T and K K^T once more. A lane has token i = lr of
        // the row tile and four tokens j
        float nrow = 0.f;
        const int i = row0 + lr;
        const float bi = gate[2 * C + i], hi = gate[3 * C + i], li = gate[4 * C + i];
#pragma unroll
        for (int e = 0; e < NT; ++e) {
            __builtin_amdgcn_sched_barrier(0);
            const int nt = grp + e * GROUPS, j0 = nt * 16 + gq * 4;
            if (nt >= NB) break;
            f32x4 a = {}, b = {}, ncol = {};
            if (nt <= tile) {
                f32x4 kk = {}, qk = {};
#pragma unroll
                for (int kb = 0; kb < DK; kb += 32) {
                    const Vec8<T> kj = frag_nat(ks, LK, nt * 16, kb, lane);
                    kk = mma(kj, frag_nat(ks, LK, row0, kb, lane), kk);
                    qk = mma(kj, frag_nat(qs, LK, row0, kb, lane), qk);
                }
                const f32x4 bj = gate4(gate, 2 * C + j0), hj = gate4(gate, 3 * C + j0), lj = gate4(gate, 4 * C + j0);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = j0 + r;
                    const float d = decay(hi, li, hj[r], lj[r]) * bj[r];
                    a[r] = i > j ? p.scale * d * dp[e][r] : (i == j ? p.scale * bj[r] * dp[e][r] : 0.f);
                    b[r] = i > j ? -bi * d * zu[e][r] : 0.f;
                    ncol[r] = i > j ? a[r] * qk[r] + b[r] * kk[r] : 0.f;     // N_ii cancels in dG
                    nrow += ncol[r];
                }
            }
            store_parts4<NF>(w1 + i * LC + j0, C * LC, a);
            store_parts4<NF>(w2 + i * LC + j0, C * LC, b);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float n = sum16(ncol[r]);
                if (lr == 0) col_part[tile * C + j0 + r] = n;
            }
        }
        nrow = sum_groups(nrow);
        if (gq == 0) n_part[grp * C + i] = nrow;
        __syncthreads();

        // the products with S, and their shares of dG
        f32x4 grow = {}, gw = {};
        const f32x4 eg4 = gate4(gate, row0 + gq * 4), eo4 = gate4(gate, C + row0 + gq * 4);
        const f32x4 b4 = gate4(gate, 2 * C + row0 + gq * 4);
#pragma unroll
        for (int t = 0; t < NK; ++t) {
            const f32x4 qv = __builtin_convertvector(quad_tr(qs, LK, row0, key0 + t * 16, lane), f32x4);
            const f32x4 kv = __builtin_convertvector(quad_tr(ks, LK, row0, key0 + t * 16, lane), f32x4);
            const f32x4 a1 = eg4 * p.scale * os[t], a2 = eg4 * b4 * zs[t], a3 = eo4 * b4 * us[t];
            dq[t] += a1;
            dk[t] += a3 - a2;
            grow += a1 * qv - a2 * kv;
            gw += a3 * kv;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float a = sum16(grow[r]), b = sum16(gw[r]);
            if (lr == 0) {
                row_part[grp * C + row0 + gq * 4 + r] = a;
                row_w[grp * C + row0 + gq * 4 + r] = b;
            }
        }
        // the products with K and Q: rows i of W1 and W2 for dQ and dK, columns for dK
#pragma unroll 1
        for (int kb = 0; kb < C / 32; ++kb) {
            const Parts<T, NF> a1 = parts_acc<NF>(w1, C * LC, LC, row0, kb * 32, lane);
            const Parts<T, NF> a2 = parts_acc<NF>(w2, C * LC, LC, row0, kb * 32, lane);
            const Parts<T, NF> b1 = parts_tr<NF>(w1, C * LC, LC, kb * 32, row0, lane);
            const Parts<T, NF> b2 = parts_tr<NF>(w2, C * LC, LC, kb * 32, row0, lane);
#pragma unroll
            for (int t = 0; t < NK; ++t) {
                const Parts<T, 1> kt = {{frag_tr(ks, LK, kb * 32, key0 + t * 16, lane)}};
                const Parts<T, 1> qt = {{frag_tr(qs, LK, kb * 32, key0 + t * 16, lane)}};
                dq[t] = mma(a1, kt, dq[t]);
                dk[t] = mma(b1, qt, dk[t]);
                dk[t] = mma(a2, kt, dk[t]);
                dk[t] = mma(b2, kt, dk[t]);
            }
        }
        __syncthreads();
        if (wave == 0) {
            float x = 0.f, w = 0.f;
            if (lane < C) {
#pragma unroll
                for (int i = 0; i < GROUPS; ++i) {
                    w += row_w[i * C + lane];
                    x += row_part[i * C + lane] + n_part[i * C + lane];
                }
                x -= w;
#pragma unroll
                for (int i = 0; i < NB; ++i) x -= col_part[i * C + lane];
            }
            float wsum = sum_groups(sum16(w)), in = 0.f;
#pragma unroll
            for (int i = 0; i < NB * GROUPS; ++i) in += inner[i];
            if (lane == C - 1) x += wsum + gate[C - 1] * in;
            // sums from each token to the chunk's end
#pragma unroll
            for (int d = 1; d < C; d *= 2) {
                const float o = __shfl_down(x, d, 64);
                if (lane + d < C) x += o;
            }
            if (lane < rows) {
                const int64_t g_at = (info.row + lane) * p.dg.ts + h * p.dg.hs;
                const int64_t b_at = (info.row + lane) * p.dbeta.ts + h * p.dbeta.hs;
                if (p.fp32_grads) {
                    if (p.dg.data) static_cast<float*>(p.dg.data)[g_at] = x;
                    static_cast<float*>(p.dbeta.data)[b_at] = d_beta[lane];
                } else {
                    if (p.dg.data) static_cast<T*>(p.dg.data)[g_at] = (T)x;
                    static_cast<T*>(p.dbeta.data)[b_at] = (T)d_beta[lane];
                }
            }
        }
        __syncthreads();
    }
    T* q0 = static_cast<T*>(p.dq.data) + info.row * p.dq.ts + hk * p.dq.hs;
    T* k0 = static_cast<T*>(p.dk.data) + info.row * p.dk.ts + hk * p.dk.hs;
    const auto q_rsrc = rows_rsrc(q0, p.dq.ts * (int)sizeof(T), rows, p.dim_k * (int)sizeof(T));
    const auto k_rsrc = rows_rsrc(k0, p.dk.ts * (int)sizeof(T), rows, p.dim_k * (int)sizeof(T));
#pragma unroll
    for (int t = 0; t < NK; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = row0 + gq * 4 + r, c = key0 + t * 16 + lr;
            const bool in = i < rows && c < p.dim_k;
            buffer_store<T>(q_rsrc, in ? (i * (int)p.dq.ts + c) * (int)sizeof(T) : kOutside, (T)dq[t][r]);
            buffer_store<T>(k_rsrc, in ? (i * (int)p.dk.ts + c) * (int)sizeof(T) : kOutside, (T)dk[t][r]);
        }
}

// ---- launches --------------------------------------------------------------

template <class K>
hipError_t launch_lds(K kernel, uint64_t blocks, int threads, size_t lds, const DeltaParams& p, hipStream_t stream)
{
    // more than 64 KiB of LDS has to be asked for, on the current device
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    kernel<<<dim3((uint32_t)blocks), dim3((uint32_t)threads), lds, stream>>>(p);
    return hipGetLastError();
}

// Rows that cannot be read 16 bytes at a time, copied to ones that can: padded
// to whole units, zero behind dim. 8,127 tokens of 8 key and 16 value heads of 128 x 128
// in bf16, one element off: 168 us forward instead of 113, 463 backward instead of 356,
// 18 us an array. It is for callers who cannot lay their rows out in whole units.
template <class T>
__global__ __launch_bounds__(256) void k_delta_pack(DeltaRows src, T* dst, int64_t tokens, int heads, int dim, int padded)
{
    const int64_t n = tokens * heads * padded;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / padded, t = row / heads;
        const int d = (int)(i - row * padded), h = (int)(row - t * heads);
        dst[i] = d < dim ? static_cast<const T*>(src.data)[t * src.ts + h * src.hs + d] : (T)0.f;
    }
}
template <class T>
hipError_t pack_rows(const DeltaPack& k, int64_t tokens, hipStream_t stream)
{
    if (k.n == 0 || tokens == 0) return hipSuccess;
    for (int i = 0; i < k.n; ++i) {
        const auto& r = k.rows[i];
        const int64_t blocks = (tokens * r.heads * r.padded + 255) / 256;
        k_delta_pack<T><<<dim3((uint32_t)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, stream>>>(
            r.src, static_cast<T*>(r.dst), tokens, r.heads, r.dim, r.padded);
    }
    return hipGetLastError();
}

inline uint64_t scan_blocks(const DeltaParams& p, int waves)
{
    const uint64_t parts = ((uint64_t)p.dim_v + waves * 16 - 1) / (waves * 16);
    const uint64_t groups = ((uint64_t)p.n_seqs * p.heads_v + 7) / 8 * 8;
    return groups * parts;
}
// 16-column waves of a scan workgroup: four share a chunk's tiles. Two, whose
// chunks take less time, as long as every workgroup still has a compute unit to
// itself: 8,192 tokens of 64 heads of 128 x 128 forward in 386 us with two and 440
// with four, of 72 heads 651 and 474; backward 711 and 787 with 32 heads, 1,136 and
// 1,020 with 48. (Sequences are counted, an empty one like a long one: their lengths
// are on the device.) And two for fp32 heads above 128, whose tiles and states leave
// LDS for no more.
template <class T, int DK>
constexpr int kMostWaves = sizeof(T) == 4 && DK > 128 ? 2 : 4;
constexpr uint64_t kComputeUnits = 256;

template <class T, int DK, int NP, int NW>
hipError_t launch_scan(const DeltaParams& p, hipStream_t stream)
{
    constexpr int NF = kFine<T>, NX = NP > NF ? NP : NF;
    return launch_lds(k_delta_scan<T, DK, NP, NW>, scan_blocks(p, NW), NW * 128, ScanLds<T, DK, NW, 1, NX, true>::bytes, p,
                      stream);
}
template <class T, int DK, int ND, int NW>
hipError_t launch_both(const DeltaParams& p, hipStream_t stream)
{
    // the backward scan's LDS, the larger one
    return launch_lds(k_delta_scan_both<T, DK, ND, NW>, 2 * scan_blocks(p, NW), NW * 128,
                      ScanLds<T, DK, NW, 2, 2 * kFine<T>, false>::bytes, p, stream);
}

template <class T, int DK, int NP>
hipError_t forward_dk(const DeltaParams& p, hipStream_t stream)
{
    constexpr int C = kChunk<T, DK>;
    const hipError_t e = launch_lds(k_delta_prep<T, DK, NP, false>, (uint64_t)p.n_slots * p.heads_v, C * 4,
                                    PrepLds<T, DK>::bytes, p, stream);
    if (e != hipSuccess) return e;
    if (scan_blocks(p, 2) <= kComputeUnits) return launch_scan<T, DK, NP, 2>(p, stream);
    return launch_scan<T, DK, NP, kMostWaves<T, DK>>(p, stream);
}
template <class T, int NP>
hipError_t forward_type(const DeltaParams& p, const DeltaPack& k, hipStream_t stream)
{
    const hipError_t e = pack_rows<T>(k, p.tokens, stream);
    if (e != hipSuccess) return e;
    switch (delta_padded_k(p.dim_k)) {
    case 64: return forward_dk<T, 64, NP>(p, stream);
    case 128: return forward_dk<T, 128, NP>(p, stream);
    default: return forward_dk<T, 256, NP>(p, stream);
    }
}

template <class T, int DK, int ND>
hipError_t backward_dk(const DeltaParams& p, hipStream_t stream)
{
    constexpr int C = kChunk<T, DK>;
    hipError_t e = launch_lds(k_delta_prep<T, DK, 1, true>, (uint64_t)p.n_slots * p.heads_v, C * 4,
                              PrepLds<T, DK>::bytes, p, stream);
    if (e != hipSuccess) return e;
    e = 2 * scan_blocks(p, 2) <= kComputeUnits ? launch_both<T, DK, ND, 2>(p, stream)
                                              : launch_both<T, DK, ND, kMostWaves<T, DK>>(p, stream);
    if (e != hipSuccess) return e;
    using L = GradLds<T, DK, ND>;
    return launch_lds(k_delta_grad<T, DK, ND>, (uint64_t)p.n_slots * p.heads_qk, L::THREADS, L::bytes, p, stream);
}
template <class T>
hipError_t backward_type(const DeltaParams& p, const DeltaPack& k, bool precise, hipStream_t stream)
{
    const hipError_t e = pack_rows<T>(k, p.tokens, stream);
    if (e != hipSuccess) return e;
    switch (delta_padded_k(p.dim_k)) {
    case 64: return precise ? backward_dk<T, 64, kFine<T>>(p, stream) : backward_dk<T, 64, kStoredGrad<T, 64>>(p, stream);
    case 128: return precise ? backward_dk<T, 128, kFine<T>>(p, stream) : backward_dk<T, 128, kStoredGrad<T, 128>>(p, stream);
    default: return backward_dk<T, 256, kStoredGrad<T, 256>>(p, stream);
    }
}

}  // namespace dws
