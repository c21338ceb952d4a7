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

namespace dws {

// Tokens of a chunk: 64, and 32 where a chunk's tiles twice over (the next
// chunk's arrive while this one is worked on) would not fit 160 KB of LDS.
template <class T, int DK>
constexpr int kChunk = sizeof(T) == 4 || DK > 128 ? 32 : 64;

// Parts of the 16-bit operands that are computed in fp32. With one part for
// all, bf16 outputs and gradients are off by 3.3e-3 to 4.9e-3 (2-norm), twice
// what rounding the result itself gives (1.7e-3). The arrays of a chunk's size,
// P, X, U', Z, dU, scale e^G dO, W1 and W2, make up nearly all of that; in two
// parts they leave at most 1.4 times the result's own rounding. So does the
// inverse: where keys repeat, its rows subtract neighbouring tokens from each
// other, and what is left is far smaller than its entries' rounding. S and dS,
// which are larger and cost the most products and bytes, add 0.5 times at most
// and keep one part.
template <class T>
constexpr int kFine = sizeof(T) == 4 ? 1 : 2;
// Parts of everything that a final state depends on, for fp32 accuracy.
template <class T>
constexpr int kPrecise = __is_same(T, bf16_t) ? 3 : kFine<T>;

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

// inv = (I + m)^-1, m strictly lower triangular, both fp32 in LDS with rows of
// C + 1. The diagonal 16 x 16 blocks by substitution (one wave each, a column a
// lane), then twice as large blocks from two: [[A, 0], [M, B]]^-1 has
// -B^-1 M A^-1 in its corner. Substitution keeps the error at the size of the
// result's entries; a product of powers (I - m)(I + m^2).. would not, since the
// powers of m can be far larger than its inverse. `tmp`: C x (C + 1).
template <int C>
__device__ __forceinline__ void invert_unit_lower(const float* m, float* inv, float* tmp, int wave, int lane)
{
    constexpr int NB = C / 16, LD = C + 1;
    const int col = lane & 15, gq = lane >> 4;
    {
        const float* d = m + wave * 16 * (LD + 1);
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == col ? 1.f : 0.f;
#pragma unroll
            for (int j = 0; j < i; ++j) s -= d[i * LD + j] * x[j];
            x[i] = s;
        }
        // four lanes have the same column: each stores a quarter of it
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i / 4 == gq) inv[(wave * 16 + i) * LD + wave * 16 + col] = x[i];
        for (int jb = wave + 1; jb < NB; ++jb) store_block<LD>(inv + wave * 16 * LD + jb * 16, f32x4{}, lane);
    }
    __syncthreads();
    // 16 -> 32: wave w < NB / 2 makes block (2 w + 1, 2 w)
    const int a = wave * 2;
    if (wave < NB / 2)
        store_block<LD>(tmp + a * 16 * LD, block_product<LD, 16>(m + (a + 1) * 16 * LD + a * 16, inv + a * 16 * (LD + 1), f32x4{}, lane), lane);
    __syncthreads();
    if (wave < NB / 2)
        store_block<LD>(inv + (a + 1) * 16 * LD + a * 16,
                        -block_product<LD, 16>(inv + (a + 1) * 16 * (LD + 1), tmp + a * 16 * LD, f32x4{}, lane), lane);
    __syncthreads();
    if constexpr (NB == 4) {
        // 32 -> 64: four blocks, one a wave
        const int bi = wave >> 1, bj = wave & 1;
        store_block<LD>(tmp + bi * 16 * LD + bj * 16,
                        block_product<LD, 32>(m + (32 + bi * 16) * LD, inv + bj * 16, f32x4{}, lane), lane);
        __syncthreads();
        store_block<LD>(inv + (32 + bi * 16) * LD + bj * 16,
                        -block_product<LD, 32>(inv + (32 + bi * 16) * LD + 32, tmp + bj * 16, f32x4{}, lane), lane);
        __syncthreads();
    }
}

// Sums of the chunk's log decays, in double: the differences of two sums of 64
// then keep fp32 accuracy however large the sums are.
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

// LDS of the preparation: the matrices of the inversion share their place with
// the K and Q tiles, which are done with before.
template <class T, int DK>
struct PrepLds {
    static constexpr int C = kChunk<T, DK>, LK = lds_stride<T>(DK), LD = C + 1;
    static constexpr size_t tiles = 2 * (size_t)C * LK * sizeof(T), inverse = 2 * (size_t)C * LD * sizeof(float);
    static constexpr size_t shared = tiles > inverse ? tiles : inverse;
    static constexpr size_t total = shared, beta = total + C * sizeof(double), m = beta + C * sizeof(float);
    static constexpr size_t bytes = m + (size_t)C * LD * sizeof(float);
};

// One workgroup for each (chunk slot, value head): gate factors, P and the
// inverse(s) to the workspace. Products over dim_k on the matrix cores, wave w
// owning the tokens 16 w .. 16 w + 15.
template <class T, int DK, int NP, bool BWD>
__global__ __launch_bounds__((kChunk<T, DK> * 4)) void k_delta_prep(DeltaParams p)
{
    using S = PrepLds<T, DK>;
    constexpr int C = S::C, THREADS = C * 4, NB = C / 16, LK = S::LK, LD = S::LD, NF = kFine<T>;
    constexpr int NX = NP > NF ? NP : NF;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    T* ks = reinterpret_cast<T*>(smem);
    T* qs = ks + C * LK;
    float* inv = reinterpret_cast<float*>(smem);
    float* tmp = inv + C * LD;
    double* total = reinterpret_cast<double*>(smem + S::total);
    float* beta = reinterpret_cast<float*>(smem + S::beta);
    float* m = reinterpret_cast<float*>(smem + S::m);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, gq = lane >> 4, lr = lane & 15;
    const int64_t slot = blockIdx.x / p.heads_v;
    const int h = blockIdx.x % p.heads_v, hk = h / (p.heads_v / p.heads_qk);
    const SlotInfo info = slot_info<C>(p.offsets, p.tokens, p.n_seqs, slot);
    if (info.rows == 0) {
        if (p.zero_tail && info.beyond >= 0 && h == 0) {
            const int64_t begin = seq_begin(p.offsets, p.tokens, p.n_seqs, info.seq);
            const int64_t len = seq_length(p.offsets, p.tokens, p.n_seqs, info.seq, begin);
            const int64_t spare = p.n_slots - first_slot(begin, info.seq, C) - (len + C - 1) / C;
            const int64_t first = begin + len + info.beyond * C, step = spare * C;
            if constexpr (BWD) {
                zero_rows<T>(p.dq, first, p.tokens, step, C, p.heads_qk, p.dim_k, tid, THREADS);
                zero_rows<T>(p.dk, first, p.tokens, step, C, p.heads_qk, p.dim_k, tid, THREADS);
                zero_rows<T>(p.dv, first, p.tokens, step, C, p.heads_v, p.dim_v, tid, THREADS);
                zero_rows<T>(p.dg, first, p.tokens, step, C, p.heads_v, 1, tid, THREADS);
                zero_rows<T>(p.dbeta, first, p.tokens, step, C, p.heads_v, 1, tid, THREADS);
            } else {
                zero_rows<T>(p.out, first, p.tokens, step, C, p.heads_v, p.dim_v, tid, THREADS);
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
    stage_tile<T, C, DK, THREADS>(ks, LK, k0, p.k.ts, info.rows, p.dim_k, p.vec, tid);
    stage_tile<T, C, DK, THREADS>(qs, LK, q0, p.q.ts, info.rows, p.dim_k, p.vec, tid);
    if (wave == 0) {
        const double sum = scan_decays<C>((double)g, lane);
        const double last = __shfl(sum, C - 1, 64);
        if (lane < C) {
            total[lane] = sum;
            beta[lane] = b;
            float* w = p.w_gate + at * 3 * C;
            w[lane] = expf((float)sum);
            w[C + lane] = expf((float)(last - sum));
            w[2 * C + lane] = b;
        }
    }
    __syncthreads();

    // row tile `wave` of K K^T and Q K^T, up to the diagonal. m = L B.
    T* wp = static_cast<T*>(p.w_p) + at * NF * C * C;
    f32x4 low[BWD ? NB : 1];      // B L
#pragma unroll
    for (int nt = 0; nt < NB; ++nt) {
        // P goes out four elements of a row a lane: its rows are tokens i
        // forward, j (P transposed) backward, the other token being the one
        // that runs along a lane's four results
        f32x4 kk = {}, qk = {};
        if (nt <= wave) {
#pragma unroll
            for (int kb = 0; kb < DK; kb += 32) {
                const Vec8<T> ki = frag_nat(ks, LK, wave * 16, kb, lane), kj = frag_nat(ks, LK, nt * 16, kb, lane);
                const Vec8<T> qi = frag_nat(qs, LK, wave * 16, kb, lane);
                kk = mma(ki, kj, kk);
                qk = BWD ? mma(qi, kj, qk) : mma(kj, qi, qk);
            }
        }
        f32x4 pij;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = wave * 16 + gq * 4 + r, j = nt * 16 + lr;
            const float d = i > j ? expf((float)(total[i] - total[j])) : 0.f;
            m[i * LD + j] = i > j ? d * beta[j] * kk[r] : 0.f;
            if constexpr (BWD) low[nt][r] = i > j ? d * beta[i] * kk[r] : 0.f;
            const int pi = BWD ? i : wave * 16 + lr, pj = BWD ? j : nt * 16 + gq * 4 + r;
            const float e = BWD ? d : (pi > pj ? expf((float)(total[pi] - total[pj])) : 0.f);
            pij[r] = pi > pj ? p.scale * e * qk[r] : (pi == pj ? p.scale * qk[r] : 0.f);
        }
        T* to = BWD ? wp + (nt * 16 + lr) * C + wave * 16 + gq * 4 : wp + (wave * 16 + lr) * C + nt * 16 + gq * 4;
        store_parts4<NF>(to, C * C, pij);
    }
    __syncthreads();

    invert_unit_lower<C>(m, inv, tmp, wave, lane);
    T* wt = static_cast<T*>(p.w_t) + at * NX * C * C;
    for (int i = tid; i < C * C / 4; i += THREADS) {
        const float* x = inv + i / (C / 4) * LD + i % (C / 4) * 4;
        store_parts4<NX>(wt + i * 4, C * C, f32x4{x[0], x[1], x[2], x[3]});
    }
    if constexpr (BWD) {
        // the other inverse, of I + B L
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < NB; ++nt)
#pragma unroll
            for (int r = 0; r < 4; ++r) m[(wave * 16 + gq * 4 + r) * LD + nt * 16 + lr] = low[nt][r];
        __syncthreads();
        invert_unit_lower<C>(m, inv, tmp, wave, lane);
        T* wtt = static_cast<T*>(p.w_tt) + at * NF * C * C;
        for (int i = tid; i < C * C / 4; i += THREADS) {
            const float* x = inv + i % (C / 4) * 4 * LD + i / (C / 4);
            store_parts4<NF>(wtt + i * 4, C * C, f32x4{x[0], x[LD], x[2 * LD], x[3 * LD]});
        }
    }
}

// ---- the forward scan ------------------------------------------------------

// LDS of a scan workgroup, two of each but for the tiles of a caller's arrays
// that cannot be read 16 bytes at a time.
template <class T, int DK, int KQ, int TP>
struct ScanLds {
    static constexpr int C = kChunk<T, DK>, LK = lds_stride<T>(DK), LC = lds_stride<T>(C);
    static constexpr size_t kq = KQ * (size_t)C * LK * sizeof(T), tp = TP * (size_t)C * LC * sizeof(T);
    static constexpr size_t buffer = kq + tp + 3 * C * sizeof(float), bytes = 2 * buffer;
};

// What the two scans share: which columns of which sequence and head a wave
// owns, and the state's transfer.
template <int NW>
struct ScanPlace {
    int64_t seq, begin, len, slot0;
    int h, hk, col0, col;
    bool mine;
};
template <int C, int NW>
__device__ __forceinline__ bool scan_place(const DeltaParams& p, int lane, int wave, ScanPlace<NW>* w)
{
    const uint32_t parts = (uint32_t)((p.dim_v + NW * 16 - 1) / (NW * 16));
    uint32_t group, part;
    xcd_split(blockIdx.x, parts, &group, &part);
    if (group >= (uint64_t)p.n_seqs * p.heads_v) return false;
    w->seq = group / p.heads_v;
    w->h = group % p.heads_v;
    w->hk = w->h / (p.heads_v / p.heads_qk);
    w->col0 = (part * NW + wave) * 16;
    w->col = w->col0 + (lane & 15);
    w->mine = w->col < p.dim_v;
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
// 16 columns of a chunk of a (tokens, dim) array, laid out as results.
template <class T, int NB>
struct ColumnRegs {
    // one element a register: two 16-bit ones in one would have to be put
    // together, and waited for, where they are loaded
    typedef typename Bits<sizeof(T)>::type BitsT;
    uint32_t x[NB * 4];

    __device__ __forceinline__ void load(const T* first, int64_t ts, int rows, int dim, int col, int gq)
    {
        const auto rsrc = rows_rsrc(first, ts * (int)sizeof(T), rows, dim * (int)sizeof(T));
        const int step = (int)ts * (int)sizeof(T);
#pragma unroll
        for (int i = 0; i < NB * 4; ++i) {
            const int row = i / 4 * 16 + gq * 4 + i % 4;
            x[i] = buffer_load<BitsT>(rsrc, col < dim && row < rows ? row * step + col * (int)sizeof(T) : kOutside);
        }
    }
    __device__ __forceinline__ f32x4 tile(int mt) const
    {
        f32x4 y;
#pragma unroll
        for (int r = 0; r < 4; ++r) y[r] = (float)__builtin_bit_cast(T, (BitsT)x[mt * 4 + r]);
        return y;
    }
};
// A state for the workspace, transposed: rows of DK, one a column of the value head.
template <class T, int DK>
__device__ __forceinline__ void store_columns(T* at, const f32x4 (&s)[DK / 16], int col, int dv_pad, int gq)
{
    if (col >= dv_pad) return;
    T* to = at + col * DK + gq * 4;
#pragma unroll
    for (int t = 0; t < DK / 16; ++t) *reinterpret_cast<Vec4<T>*>(to + t * 16) = __builtin_convertvector(s[t], Vec4<T>);
}
template <class T, int NF, int C>
__device__ __forceinline__ void store_columns(T* at, const f32x4 (&u)[C / 16], int col, int dv_pad, int gq)
{
    if (col >= dv_pad) return;
#pragma unroll
    for (int mt = 0; mt < C / 16; ++mt) store_parts4<NF>(at + col * C + mt * 16 + gq * 4, (int64_t)C * dv_pad, u[mt]);
}
__device__ __forceinline__ f32x4 gate4(const float* gate, int row) { return *reinterpret_cast<const f32x4*>(gate + row); }

// STORE: instead of the outputs, the states at the chunks' starts and U' go to
// the workspace (for the backward pass). NP: parts of the operands the state
// depends on. NW waves, 16 columns of the value head each. Two LDS buffers: the
// next chunk's tiles are written to one while the other is read, so a chunk
// needs one barrier, and the loads of the one after that are in flight.
template <class T, int DK, int NP, bool STORE, int NW>
__global__ __launch_bounds__(NW * 64) DWS_ONE_WAVE void k_delta_scan(DeltaParams p)
{
    constexpr int NF = kFine<T>, NX = NP > NF ? NP : NF;
    using L = ScanLds<T, DK, STORE ? 1 : 2, STORE ? NX : NX + NF>;
    constexpr int C = L::C, THREADS = NW * 64, NB = C / 16, LK = L::LK, LC = L::LC, NK = DK / 16;
    extern __shared__ __attribute__((aligned(16))) char smem[];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, gq = lane >> 4, lr = lane & 15;
    ScanPlace<NW> w;
    if (!scan_place<C, NW>(p, lane, wave, &w)) return;
    int64_t st;
    if (!slot_taken<THREADS>(p.slots, p.n_states, w.seq, &st, tid)) return;
    const int64_t state_at = (st * p.heads_v + w.h) * p.dim_k * p.dim_v;
    const T* k0 = static_cast<const T*>(p.k.data) + w.begin * p.k.ts + w.hk * p.k.hs;
    const T* q0 = static_cast<const T*>(p.q.data) + w.begin * p.q.ts + w.hk * p.q.hs;
    const T* v0 = static_cast<const T*>(p.v.data) + w.begin * p.v.ts + w.h * p.v.hs;

    TileRegs<T, C, DK, THREADS> kr, qr;
    TileRegs<T, NX * C, C, THREADS> tr;
    TileRegs<T, NF * C, C, THREADS> pr;
    TileRegs<float, 3, C, THREADS> gr;
    ColumnRegs<T, NB> vr;
    auto rows_at = [&](int64_t c0) { return w.len - c0 < C ? (int)(w.len - c0) : C; };
    // the chunk at c0, from global memory to registers
    auto load = [&](int64_t c0) {
        const int rows = rows_at(c0);
        const int64_t at = (w.slot0 + c0 / C) * p.heads_v + w.h;
        if (p.vec) {
            kr.load(k0 + c0 * p.k.ts, p.k.ts, rows, p.dim_k, tid);
            if constexpr (!STORE) qr.load(q0 + c0 * p.q.ts, p.q.ts, rows, p.dim_k, tid);
        }
        tr.load(static_cast<const T*>(p.w_t) + at * NX * C * C, C, NX * C, C, tid);
        if constexpr (!STORE) pr.load(static_cast<const T*>(p.w_p) + at * NF * C * C, C, NF * C, C, tid);
        gr.load(p.w_gate + at * 3 * C, C, 3, C, tid);
        vr.load(v0 + c0 * p.v.ts, p.v.ts, rows, p.dim_v, w.col, gq);
    };
    // and from there to an LDS buffer
    auto store = [&](int64_t c0, char* buffer) {
        T* ks = reinterpret_cast<T*>(buffer);
        T* ts = reinterpret_cast<T*>(buffer + L::kq);
        if (p.vec) {
            kr.store(ks, LK, tid);
            if constexpr (!STORE) qr.store(ks + C * LK, LK, tid);
        } else {
            const int rows = rows_at(c0);
            stage_elements<T, C, DK, THREADS>(ks, LK, k0 + c0 * p.k.ts, p.k.ts, rows, p.dim_k, tid);
            if constexpr (!STORE)
                stage_elements<T, C, DK, THREADS>(ks + C * LK, LK, q0 + c0 * p.q.ts, p.q.ts, rows, p.dim_k, tid);
        }
        tr.store(ts, LC, tid);
        if constexpr (!STORE) pr.store(ts + NX * C * LC, LC, tid);
        gr.store(reinterpret_cast<float*>(buffer + L::kq + L::tp), C, tid);
    };

    f32x4 s[NK];
    load_state<DK>(s, p.initial ? p.initial + state_at : nullptr, p.dim_k, p.dim_v, w.col, gq);
    if (w.len > 0) {
        load(0);
        store(0, smem);
    }
    int which = 0;
    for (int64_t c0 = 0; c0 < w.len; c0 += C, which ^= 1) {
        char* buffer = smem + which * L::buffer;
        const T* ks = reinterpret_cast<const T*>(buffer);
        const T* qs = ks + C * LK;
        const T* ts = reinterpret_cast<const T*>(buffer + L::kq);
        const T* ps = ts + NX * C * LC;
        const float* gate = reinterpret_cast<const float*>(buffer + L::kq + L::tp);
        f32x4 x[NB];
#pragma unroll
        for (int mt = 0; mt < NB; ++mt) x[mt] = vr.tile(mt);
        __syncthreads();
        const bool more = c0 + C < w.len;
        if (more) load(c0 + C);

        const int64_t at = (w.slot0 + c0 / C) * p.heads_v + w.h;
        if constexpr (STORE)
            store_columns<T, DK>(static_cast<T*>(p.w_s) + at * DK * p.dv_pad, s, w.col, p.dv_pad, gq);
        Parts<T, NP> sb[DK / 32];
#pragma unroll
        for (int kb = 0; kb < DK / 32; ++kb) sb[kb] = parts_of<T, NP>(s[2 * kb], s[2 * kb + 1]);
        // X = V - diag(e^G) K S
        {
            f32x4 acc[NB] = {};
#pragma unroll
            for (int kb = 0; kb < DK / 32; ++kb) {
                Parts<T, 1> a[NB];
#pragma unroll
                for (int mt = 0; mt < NB; ++mt) a[mt].p[0] = frag_acc(ks, LK, mt * 16, kb * 32, lane);
                mma_each(a, sb[kb], acc);
            }
#pragma unroll
            for (int mt = 0; mt < NB; ++mt) x[mt] -= gate4(gate, mt * 16 + gq * 4) * acc[mt];
        }
        // U' = (I + L B)^-1 X; u = B U'
        f32x4 u[NB] = {};
#pragma unroll
        for (int kb = 0; kb < C / 32; ++kb) {
            Parts<T, NX> a[NB];
#pragma unroll
            for (int mt = 2 * kb; mt < NB; ++mt) a[mt] = parts_acc<NX>(ts, C * LC, LC, mt * 16, kb * 32, lane);
            mma_each(a, parts_of<T, NX>(x[2 * kb], x[2 * kb + 1]), u, 2 * kb);
        }
        if constexpr (STORE)
            store_columns<T, NF, C>(static_cast<T*>(p.w_u) + at * NF * C * p.dv_pad, u, w.col, p.dv_pad, gq);
#pragma unroll
        for (int mt = 0; mt < NB; ++mt) u[mt] *= gate4(gate, 2 * C + mt * 16 + gq * 4);
        if constexpr (!STORE) {
            // O transposed, so that a lane has four columns of one token: the
            // state and u in the place of the left operand
            f32x4 o[NB] = {};
#pragma unroll
            for (int kb = 0; kb < DK / 32; ++kb) {
                Parts<T, 1> a[NB];
#pragma unroll
                for (int mt = 0; mt < NB; ++mt) a[mt].p[0] = frag_acc(qs, LK, mt * 16, kb * 32, lane);
                mma_each<true>(a, Parts<T, 1>{{sb[kb].p[0]}}, o);
            }
#pragma unroll
            for (int mt = 0; mt < NB; ++mt) o[mt] *= p.scale * gate[mt * 16 + lr];
#pragma unroll
            for (int kb = 0; kb < C / 32; ++kb) {
                Parts<T, NF> a[NB];
#pragma unroll
                for (int mt = 2 * kb; mt < NB; ++mt) a[mt] = parts_acc<NF>(ps, C * LC, LC, mt * 16, kb * 32, lane);
                mma_each<true>(a, parts_of<T, NF>(u[2 * kb], u[2 * kb + 1]), o, 2 * kb);
            }
            const int rows = rows_at(c0), c = w.col0 + gq * 4;
            T* o0 = static_cast<T*>(p.out.data) + (w.begin + c0) * p.out.ts + w.h * p.out.hs;
            const auto rsrc = rows_rsrc(o0, p.out.ts * (int)sizeof(T), rows, p.dim_v * (int)sizeof(T));
            const int step = (int)p.out.ts * (int)sizeof(T);
#pragma unroll
            for (int mt = 0; mt < NB; ++mt) {
                const int row = mt * 16 + lr, to = row < rows && c < p.dim_v ? row * step + c * (int)sizeof(T) : kOutside;
                const Vec4<T> y = __builtin_convertvector(o[mt], Vec4<T>);
                if (p.out4) {
                    buffer_store(rsrc, to, y);
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        buffer_store<T>(rsrc, c + r < p.dim_v ? to + r * (int)sizeof(T) : kOutside, y[r]);
                }
            }
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
            Parts<T, 1> a[NK];
#pragma unroll
            for (int t = 0; t < NK; ++t) a[t].p[0] = frag_tr(ks, LK, kb * 32, t * 16, lane);
            mma_each(a, ub, s);
        }
        if (more) store(c0 + C, smem + (which ^ 1) * L::buffer);
    }
    if (!STORE && p.final_state != nullptr) store_state<DK>(s, p.final_state + state_at, p.dim_k, p.dim_v, w.col, gq);
}

// ---- the backward scan -----------------------------------------------------
//
// With dS' the gradient at the chunk's end and dO given:
//   dU = P^T dO + diag(e^(G_C - G)) K dS'     Z = (I + B L)^-T dU     dX = B Z = dV
//   dS = e^(G_C) dS' + Q^T diag(scale e^G) dO - K^T diag(e^G) dX
// The same shape as the forward scan, from a sequence's last chunk to its
// first. Z and dS' go to the workspace, dV to its place.

template <class T, int DK, int NW>
__global__ __launch_bounds__(NW * 64) DWS_ONE_WAVE void k_delta_scan_back(DeltaParams p)
{
    constexpr int NF = kFine<T>;
    using L = ScanLds<T, DK, 2, 2 * NF>;
    constexpr int C = L::C, THREADS = NW * 64, NB = C / 16, LK = L::LK, LC = L::LC, NK = DK / 16;
    extern __shared__ __attribute__((aligned(16))) char smem[];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, gq = lane >> 4;
    ScanPlace<NW> w;
    if (!scan_place<C, NW>(p, lane, wave, &w)) return;
    const int64_t state_at = (w.seq * p.heads_v + w.h) * p.dim_k * p.dim_v;
    const T* k0 = static_cast<const T*>(p.k.data) + w.begin * p.k.ts + w.hk * p.k.hs;
    const T* q0 = static_cast<const T*>(p.q.data) + w.begin * p.q.ts + w.hk * p.q.hs;
    const T* o0 = static_cast<const T*>(p.d_out.data) + w.begin * p.d_out.ts + w.h * p.d_out.hs;

    TileRegs<T, C, DK, THREADS> kr, qr;
    TileRegs<T, NF * C, C, THREADS> tr, pr;
    TileRegs<float, 3, C, THREADS> gr;
    ColumnRegs<T, NB> orr;
    auto rows_at = [&](int64_t c0) { return w.len - c0 < C ? (int)(w.len - c0) : C; };
    auto load = [&](int64_t c0) {
        const int rows = rows_at(c0);
        const int64_t at = (w.slot0 + c0 / C) * p.heads_v + w.h;
        if (p.vec) {
            kr.load(k0 + c0 * p.k.ts, p.k.ts, rows, p.dim_k, tid);
            qr.load(q0 + c0 * p.q.ts, p.q.ts, rows, p.dim_k, tid);
        }
        tr.load(static_cast<const T*>(p.w_tt) + at * NF * C * C, C, NF * C, C, tid);
        pr.load(static_cast<const T*>(p.w_p) + at * NF * C * C, C, NF * C, C, tid);
        gr.load(p.w_gate + at * 3 * C, C, 3, C, tid);
        orr.load(o0 + c0 * p.d_out.ts, p.d_out.ts, rows, p.dim_v, w.col, gq);
    };
    auto store = [&](int64_t c0, char* buffer) {
        T* ks = reinterpret_cast<T*>(buffer);
        T* ts = reinterpret_cast<T*>(buffer + L::kq);
        if (p.vec) {
            kr.store(ks, LK, tid);
            qr.store(ks + C * LK, LK, tid);
        } else {
            const int rows = rows_at(c0);
            stage_elements<T, C, DK, THREADS>(ks, LK, k0 + c0 * p.k.ts, p.k.ts, rows, p.dim_k, tid);
            stage_elements<T, C, DK, THREADS>(ks + C * LK, LK, q0 + c0 * p.q.ts, p.q.ts, rows, p.dim_k, tid);
        }
        tr.store(ts, LC, tid);
        pr.store(ts + NF * C * LC, LC, tid);
        gr.store(reinterpret_cast<float*>(buffer + L::kq + L::tp), C, tid);
    };

    f32x4 ds[NK];
    load_state<DK>(ds, p.d_final ? p.d_final + state_at : nullptr, p.dim_k, p.dim_v, w.col, gq);
    const int64_t last = w.len > 0 ? (w.len - 1) / C * C : 0;
    if (w.len > 0) {
        load(last);
        store(last, smem);
    }
    int which = 0;
    for (int64_t c0 = last; c0 >= 0 && w.len > 0; c0 -= C, which ^= 1) {
        char* buffer = smem + which * L::buffer;
        const T* ks = reinterpret_cast<const T*>(buffer);
        const T* qs = ks + C * LK;
        const T* ts = reinterpret_cast<const T*>(buffer + L::kq);
        const T* ps = ts + NF * C * LC;
        const float* gate = reinterpret_cast<const float*>(buffer + L::kq + L::tp);
        f32x4 d_o[NB];
#pragma unroll
        for (int mt = 0; mt < NB; ++mt) d_o[mt] = orr.tile(mt);
        __syncthreads();
        if (c0 > 0) load(c0 - C);

        const int64_t at = (w.slot0 + c0 / C) * p.heads_v + w.h;
        store_columns<T, DK>(static_cast<T*>(p.w_ds) + at * DK * p.dv_pad, ds, w.col, p.dv_pad, gq);
        // dU
        f32x4 z[NB] = {};
#pragma unroll
        for (int kb = 0; kb < DK / 32; ++kb) {
            Parts<T, 1> a[NB];
#pragma unroll
            for (int mt = 0; mt < NB; ++mt) a[mt].p[0] = frag_acc(ks, LK, mt * 16, kb * 32, lane);
            mma_each(a, parts_of<T, 1>(ds[2 * kb], ds[2 * kb + 1]), z);
        }
#pragma unroll
        for (int mt = 0; mt < NB; ++mt) z[mt] *= gate4(gate, C + mt * 16 + gq * 4);
#pragma unroll
        for (int kb = 0; kb < C / 32; ++kb) {
            Parts<T, NF> a[NB];
#pragma unroll
            for (int mt = 0; mt < 2 * kb + 2; ++mt) a[mt] = parts_acc<NF>(ps, C * LC, LC, mt * 16, kb * 32, lane);
            mma_each(a, parts_of<T, 1>(d_o[2 * kb], d_o[2 * kb + 1]), z, 0, 2 * kb + 2);      // dO is exact in T
        }
        f32x4 y[NB] = {};
#pragma unroll
        for (int kb = 0; kb < C / 32; ++kb) {
            Parts<T, NF> a[NB];
#pragma unroll
            for (int mt = 0; mt < 2 * kb + 2; ++mt) a[mt] = parts_acc<NF>(ts, C * LC, LC, mt * 16, kb * 32, lane);
            mma_each(a, parts_of<T, NF>(z[2 * kb], z[2 * kb + 1]), y, 0, 2 * kb + 2);
        }
        store_columns<T, NF, C>(static_cast<T*>(p.w_z) + at * NF * C * p.dv_pad, y, w.col, p.dv_pad, gq);
        const int rows = rows_at(c0);
        T* dv0 = static_cast<T*>(p.dv.data) + (w.begin + c0) * p.dv.ts + w.h * p.dv.hs;
        const auto rsrc = rows_rsrc(dv0, p.dv.ts * (int)sizeof(T), rows, p.dim_v * (int)sizeof(T));
        const int step = (int)p.dv.ts * (int)sizeof(T);
#pragma unroll
        for (int mt = 0; mt < NB; ++mt) {
            const int row = mt * 16 + gq * 4;
            y[mt] *= gate4(gate, 2 * C + row);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                buffer_store<T>(rsrc, w.mine && row + r < rows ? (row + r) * step + w.col * (int)sizeof(T) : kOutside,
                                (T)y[mt][r]);
            const f32x4 eg = gate4(gate, row);
            y[mt] *= -eg;
            d_o[mt] *= p.scale * eg;
        }
        const float keep = gate[C - 1];
#pragma unroll
        for (int t = 0; t < NK; ++t) ds[t] *= keep;
#pragma unroll
        for (int kb = 0; kb < C / 32; ++kb) {
            Parts<T, 1> a[NK];
#pragma unroll
            for (int t = 0; t < NK; ++t) a[t].p[0] = frag_tr(qs, LK, kb * 32, t * 16, lane);
            mma_each(a, parts_of<T, NF>(d_o[2 * kb], d_o[2 * kb + 1]), ds);
#pragma unroll
            for (int t = 0; t < NK; ++t) a[t].p[0] = frag_tr(ks, LK, kb * 32, t * 16, lane);
            mma_each(a, parts_of<T, 1>(y[2 * kb], y[2 * kb + 1]), ds);
        }
        if (c0 > 0) store(c0 - C, smem + (which ^ 1) * L::buffer);
    }
    if (p.d_initial != nullptr)
        store_state<DK>(ds, static_cast<T*>(p.d_initial) + state_at, p.dim_k, p.dim_v, w.col, gq);
}

// ---- the gradients of q, k and the gates ------------------------------------
//
// Every chunk by itself, from the states, U', Z and dS' of the two scans:
//   dP = tril(dO U'^T) B                      M = -tril(Z U'^T, -1) B
//   W1 = scale D o dP                         W2 = B (D o M)
//   dQ = W1 K + scale diag(e^G) dO S^T
//   dK = W1^T Q + (W2 + W2^T) K + diag(e^(G_C - G)) B U' dS'^T - diag(e^G) B Z S^T
//   dbeta_i = Z_i . U'_i
//   N = W1 o Q K^T + W2 o K K^T
//   dG_i = sum_j (N_ij - N_ji) + (scale e^G dO S^T)_i . q_i - (e^G B Z S^T)_i . k_i - w_i,
//          w_i = (e^(G_C - G) B U' dS'^T)_i . k_i;   dG_C also gets sum w + e^(G_C) <S, dS'>
//   dg_t = sum of dG_i from t to the chunk's end
// One workgroup for each (chunk slot, query/key head). A wave owns a row tile
// of 16 tokens and 128 of the key columns (all, or half of 256); the value heads
// that share the key head come in turn, so that their sums need no atomics and
// have one order. The workspace's arrays have a row a value column: blocks of 32
// go through LDS, where the transposing reads make operands of them.

template <class T, int DK>
struct GradLds {
    static constexpr int C = kChunk<T, DK>, NB = C / 16, GROUPS = DK > 128 ? DK / 128 : 1, THREADS = NB * GROUPS * 64;
    static constexpr int LK = lds_stride<T>(DK), LC = lds_stride<T>(C), NF = kFine<T>;
    static constexpr size_t total = 0, ks = C * sizeof(double), qs = ks + (size_t)C * LK * sizeof(T);
    static constexpr size_t w1 = qs + (size_t)C * LK * sizeof(T), w2 = w1 + (size_t)NF * C * LC * sizeof(T);
    static constexpr size_t st = w2 + (size_t)NF * C * LC * sizeof(T), dst = st + (size_t)32 * LK * sizeof(T);
    static constexpr size_t ut = dst + (size_t)32 * LK * sizeof(T), zt = ut + (size_t)NF * 32 * LC * sizeof(T);
    static constexpr size_t gate = zt + (size_t)NF * 32 * LC * sizeof(T);
    // floats behind: gate[3 C], row_part[GROUPS C], row_w[GROUPS C], d_beta[C], col_part[NB C], inner[THREADS / 64]
    static constexpr size_t bytes = gate + ((4 + 2 * GROUPS + NB) * C + 16) * sizeof(float);
};

__device__ __forceinline__ float sum16(float x)      // over the 16 lanes of a group
{
#pragma unroll
    for (int d = 1; d < 16; d *= 2) x += __shfl_xor(x, d, 64);
    return x;
}
__device__ __forceinline__ float sum_groups(float x) // over the 4 groups
{
    x += __shfl_xor(x, 16, 64);
    return x + __shfl_xor(x, 32, 64);
}

template <class T, int DK>
__global__ __launch_bounds__((GradLds<T, DK>::THREADS)) DWS_ONE_WAVE void k_delta_grad(DeltaParams p)
{
    using L = GradLds<T, DK>;
    constexpr int C = L::C, THREADS = L::THREADS, NB = L::NB, GROUPS = L::GROUPS, LK = L::LK, LC = L::LC, NF = L::NF;
    constexpr int NK = DK / 16 / GROUPS;             // key column tiles of a wave
    extern __shared__ __attribute__((aligned(16))) char smem[];
    double* total = reinterpret_cast<double*>(smem);
    T* ks = reinterpret_cast<T*>(smem + L::ks);
    T* qs = reinterpret_cast<T*>(smem + L::qs);
    T* w1 = reinterpret_cast<T*>(smem + L::w1);
    T* w2 = reinterpret_cast<T*>(smem + L::w2);
    T* st = reinterpret_cast<T*>(smem + L::st);
    T* dst = reinterpret_cast<T*>(smem + L::dst);
    T* ut = reinterpret_cast<T*>(smem + L::ut);
    T* zt = reinterpret_cast<T*>(smem + L::zt);
    float* gate = reinterpret_cast<float*>(smem + L::gate);      // e^G, e^(G_C - G), beta
    float* row_part = gate + 3 * C;                              // dG without column sums and w
    float* row_w = row_part + GROUPS * C;                        // w
    float* d_beta = row_w + GROUPS * C;
    float* col_part = d_beta + C;                                // [NB][C] column sums of N
    float* inner = col_part + NB * C;                            // parts of <S, dS'>

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, gq = lane >> 4, lr = lane & 15;
    const int tile = wave % NB, grp = wave / NB, row0 = tile * 16, key0 = grp * 128;
    const int64_t slot = blockIdx.x / p.heads_qk;
    const int hk = blockIdx.x % p.heads_qk, share = p.heads_v / p.heads_qk;
    const SlotInfo info = slot_info<C>(p.offsets, p.tokens, p.n_seqs, slot);
    if (info.rows == 0) return;
    const int rows = info.rows;

    TileRegs<T, 32, DK, THREADS> sr, dsr;
    TileRegs<T, 32, C, THREADS> ur[NF], zr[NF];
    auto load = [&](int64_t at, int c) {
        sr.load(static_cast<const T*>(p.w_s) + (at * p.dv_pad + c) * DK, DK, 32, DK, tid);
        dsr.load(static_cast<const T*>(p.w_ds) + (at * p.dv_pad + c) * DK, DK, 32, DK, tid);
#pragma unroll
        for (int n = 0; n < NF; ++n) {
            ur[n].load(static_cast<const T*>(p.w_u) + ((at * NF + n) * p.dv_pad + c) * C, C, 32, C, tid);
            zr[n].load(static_cast<const T*>(p.w_z) + ((at * NF + n) * p.dv_pad + c) * C, C, 32, C, tid);
        }
    };
    load(slot * p.heads_v + hk * share, 0);
    stage_tile<T, C, DK, THREADS>(ks, LK, static_cast<const T*>(p.k.data) + info.row * p.k.ts + hk * p.k.hs, p.k.ts, rows,
                                  p.dim_k, p.vec, tid);
    stage_tile<T, C, DK, THREADS>(qs, LK, static_cast<const T*>(p.q.data) + info.row * p.q.ts + hk * p.q.hs, p.q.ts, rows,
                                  p.dim_k, p.vec, tid);
    f32x4 dq[NK] = {}, dk[NK] = {};

    for (int m = 0; m < share; ++m) {
        const int h = hk * share + m;
        const int64_t at = slot * p.heads_v + h;
        for (int i = tid; i < 3 * C; i += THREADS) gate[i] = p.w_gate[at * 3 * C + i];
        if (wave == 0) {
            const float g = lane < rows && p.g.data ? clamp_decay(load_gate(p.g, info.row + lane, h, p.g_dtype)) : 0.f;
            const double t = scan_decays<C>((double)g, lane);
            if (lane < C) total[lane] = t;
        }

        const T* d_o = static_cast<const T*>(p.d_out.data) + info.row * p.d_out.ts + h * p.d_out.hs;
        const auto o_rsrc = rows_rsrc(d_o, p.d_out.ts * (int)sizeof(T), rows, p.dim_v * (int)sizeof(T));
        const int o_at = (row0 + lr) * (int)p.d_out.ts;
        f32x4 dp[NB] = {}, zu[NB] = {}, os[NK] = {}, zs[NK] = {}, us[NK] = {};
        float zdotu = 0.f, sds = 0.f;
        for (int c = 0; c < p.dv_pad; c += 32) {
            // dO's rows of this wave, 32 columns in acc order
            Parts<T, 1> ao;
            if (p.vec) {
                const int o0 = c + gq * 4, o1 = o0 + 16;
                const bool in = row0 + lr < rows;
                const Vec4<T> a = buffer_load<Vec4<T>>(o_rsrc, in && o0 < p.dim_v ? (o_at + o0) * (int)sizeof(T) : kOutside);
                const Vec4<T> b = buffer_load<Vec4<T>>(o_rsrc, in && o1 < p.dim_v ? (o_at + o1) * (int)sizeof(T) : kOutside);
                ao.p[0] = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int o = c + gq * 4 + j % 4 + j / 4 * 16;
                    ao.p[0][j] = buffer_load<T>(o_rsrc, row0 + lr < rows && o < p.dim_v ? (o_at + o) * (int)sizeof(T) : kOutside);
                }
            }
            sr.store(st, LK, tid);
            dsr.store(dst, LK, tid);
#pragma unroll
            for (int n = 0; n < NF; ++n) {
                ur[n].store(ut + n * 32 * LC, LC, tid);
                zr[n].store(zt + n * 32 * LC, LC, tid);
            }
            __syncthreads();
            if (c + 32 < p.dv_pad)
                load(at, c + 32);
            else if (m + 1 < share)
                load(at + 1, 0);
            const Parts<T, NF> az = parts_tr<NF>(zt, 32 * LC, LC, 0, row0, lane);
            const Parts<T, NF> au = parts_tr<NF>(ut, 32 * LC, LC, 0, row0, lane);
            if (grp == 0)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float z = 0.f, u = 0.f;
#pragma unroll
                    for (int n = NF - 1; n >= 0; --n) {
                        z += (float)az.p[n][j];
                        u += (float)au.p[n][j];
                    }
                    zdotu += z * u;
                }
#pragma unroll
            for (int nt = 0; nt < NB; ++nt)
                if (nt <= tile && nt % GROUPS == grp) {
                    const Parts<T, NF> b = parts_tr<NF>(ut, 32 * LC, LC, 0, nt * 16, lane);
                    dp[nt] = mma(ao, b, dp[nt]);
                    zu[nt] = mma(az, b, zu[nt]);
                }
#pragma unroll
            for (int t = 0; t < NK; ++t) {
                const Parts<T, 1> b = {{frag_tr(st, LK, 0, key0 + t * 16, lane)}};
                const Parts<T, 1> d = {{frag_tr(dst, LK, 0, key0 + t * 16, lane)}};
                os[t] = mma(ao, b, os[t]);
                zs[t] = mma(az.p[0], b, zs[t]);
                us[t] = mma(au, d, us[t]);
                if (t % NB == tile)
#pragma unroll
                    for (int j = 0; j < 8; ++j) sds += (float)b.p[0][j] * (float)d.p[0][j];
            }
            __syncthreads();
        }
        zdotu = sum_groups(zdotu);               // lane: row lr of the tile
        if (gq == 0 && grp == 0) d_beta[row0 + lr] = zdotu;
        sds = sum_groups(sum16(sds));
        if (lane == 0) inner[wave] = sds;

        // W1, W2 and N; Q K^T and K K^T once more
        float nrow[4] = {};
#pragma unroll
        for (int nt = 0; nt < NB; ++nt) {
            if (nt % GROUPS != grp) continue;
            const int j = nt * 16 + lr;
            float ncol = 0.f;
            f32x4 kk = {}, qk = {};
            if (nt <= tile) {
#pragma unroll
                for (int kb = 0; kb < DK; kb += 32) {
                    const Vec8<T> b = frag_nat(ks, LK, nt * 16, kb, lane);
                    kk = mma(frag_nat(ks, LK, row0, kb, lane), b, kk);
                    qk = mma(frag_nat(qs, LK, row0, kb, lane), b, qk);
                }
            }
            const float bj = gate[2 * C + j];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = row0 + gq * 4 + r;
                const float d = i > j ? expf((float)(total[i] - total[j])) : (i == j ? 1.f : 0.f);
                const float a = i >= j ? p.scale * d * bj * dp[nt][r] : 0.f;
                const float b = i > j ? -gate[2 * C + i] * d * bj * zu[nt][r] : 0.f;
                store_parts<NF>(w1 + i * LC + j, C * LC, a);
                store_parts<NF>(w2 + i * LC + j, C * LC, b);
                const float n = i > j ? a * qk[r] + b * kk[r] : 0.f;     // N_ii cancels in dG
                nrow[r] += n;
                ncol += n;
            }
            ncol = sum_groups(ncol);
            if (gq == 0) col_part[tile * C + j] = ncol;
        }
        __syncthreads();

        // the products with S, and their shares of dG
        float grow[4] = {}, gw[4] = {};
#pragma unroll
        for (int t = 0; t < NK; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = row0 + gq * 4 + r, c = key0 + t * 16 + lr;
                const float qv = (float)qs[i * LK + c], kv = (float)ks[i * LK + c];
                const float b = gate[2 * C + i];
                const float a1 = p.scale * gate[i] * os[t][r], a2 = gate[i] * b * zs[t][r];
                const float a3 = gate[C + i] * b * us[t][r];
                dq[t][r] += a1;
                dk[t][r] += a3 - a2;
                grow[r] += a1 * qv - a2 * kv;
                gw[r] += a3 * kv;
            }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float a = sum16(grow[r] + nrow[r]), b = sum16(gw[r]);
            if (lr == 0) {
                row_part[grp * C + row0 + gq * 4 + r] = a;
                row_w[grp * C + row0 + gq * 4 + r] = b;
            }
        }
        // the products with K and Q: rows i of W1 and W2 for dQ and dK, columns for dK
#pragma unroll
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
                    x += row_part[i * C + lane];
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
                if (p.dg.data)
                    static_cast<T*>(p.dg.data)[(info.row + lane) * p.dg.ts + h * p.dg.hs] = (T)x;
                static_cast<T*>(p.dbeta.data)[(info.row + lane) * p.dbeta.ts + h * p.dbeta.hs] = (T)d_beta[lane];
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

inline uint64_t scan_blocks(const DeltaParams& p, int waves)
{
    const uint64_t parts = ((uint64_t)p.dim_v + waves * 16 - 1) / (waves * 16);
    const uint64_t groups = ((uint64_t)p.n_seqs * p.heads_v + 7) / 8 * 8;
    return groups * parts;
}

template <class T, int DK, int NP>
hipError_t forward_dk(const DeltaParams& p, hipStream_t stream)
{
    constexpr int C = kChunk<T, DK>, NW = 4, NF = kFine<T>, NX = NP > NF ? NP : NF;
    hipError_t e = launch_lds(k_delta_prep<T, DK, NP, false>, (uint64_t)p.n_slots * p.heads_v, C * 4,
                              PrepLds<T, DK>::bytes, p, stream);
    if (e != hipSuccess) return e;
    return launch_lds(k_delta_scan<T, DK, NP, false, NW>, scan_blocks(p, NW), NW * 64, ScanLds<T, DK, 2, NX + NF>::bytes,
                      p, stream);
}
template <class T, int NP>
hipError_t forward_type(const DeltaParams& p, hipStream_t stream)
{
    switch (delta_padded_k(p.dim_k)) {
    case 64: return forward_dk<T, 64, NP>(p, stream);
    case 128: return forward_dk<T, 128, NP>(p, stream);
    default: return forward_dk<T, 256, NP>(p, stream);
    }
}

template <class T, int DK>
hipError_t backward_dk(const DeltaParams& p, hipStream_t stream)
{
    constexpr int C = kChunk<T, DK>, NW = 4;
    hipError_t e = launch_lds(k_delta_prep<T, DK, 1, true>, (uint64_t)p.n_slots * p.heads_v, C * 4,
                              PrepLds<T, DK>::bytes, p, stream);
    if (e != hipSuccess) return e;
    e = launch_lds(k_delta_scan<T, DK, 1, true, NW>, scan_blocks(p, NW), NW * 64, ScanLds<T, DK, 1, kFine<T>>::bytes, p,
                   stream);
    if (e != hipSuccess) return e;
    e = launch_lds(k_delta_scan_back<T, DK, NW>, scan_blocks(p, NW), NW * 64, ScanLds<T, DK, 2, 2 * kFine<T>>::bytes, p, stream);
    if (e != hipSuccess) return e;
    return launch_lds(k_delta_grad<T, DK>, (uint64_t)p.n_slots * p.heads_qk, GradLds<T, DK>::THREADS,
                      GradLds<T, DK>::bytes, p, stream);
}
template <class T>
hipError_t backward_type(const DeltaParams& p, hipStream_t stream)
{
    switch (delta_padded_k(p.dim_k)) {
    case 64: return backward_dk<T, 64>(p, stream);
    case 128: return backward_dk<T, 128>(p, stream);
    default: return backward_dk<T, 256>(p, stream);
    }
}

}  // namespace dws
