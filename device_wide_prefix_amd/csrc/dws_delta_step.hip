// The recurrent gated delta rule: a few tokens for each sequence of a batch,
// each sequence's state read from the pool once and written back once.
//
// With a = e^g, and S the state before the token:
//   u = beta (v - a S^T k);   S <- a S + k u^T;   o = scale S^T q = scale (a S^T q + (k . q) u)
// so one pass over S gives both S^T k and S^T q, and only S itself is written.
// Bound by the state's bytes: 8 dim_k dim_v for each head and sequence, however many
// tokens it has.
#include "dws_delta_device.hpp"

namespace dws {
namespace {

constexpr int kStepThreads = 256;
constexpr int kStepMaxK = 256;

__device__ __forceinline__ float load_as_float(const void* p, int64_t at, int dtype)
{
    if (dtype == DWS_FLOAT32) return static_cast<const float*>(p)[at];
    if (dtype == DWS_BFLOAT16) return (float)static_cast<const bf16_t*>(p)[at];
    return (float)static_cast<const f16_t*>(p)[at];
}
__device__ __forceinline__ void store_as(void* p, int64_t at, int dtype, float x)
{
    if (dtype == DWS_FLOAT32)
        static_cast<float*>(p)[at] = x;
    else if (dtype == DWS_BFLOAT16)
        static_cast<bf16_t*>(p)[at] = (bf16_t)x;
    else
        static_cast<f16_t*>(p)[at] = (f16_t)x;
}

// One workgroup: CBL * VW columns of one (sequence, value head). A row of the
// block is read by CBL lanes, VW columns each; thread group rg holds rows
// rg, rg + GROUPS, ... in registers for all of the sequence's tokens.
template <int VW, int CBL, int RPT, bool NT>
__global__ __launch_bounds__(kStepThreads) void k_delta_step(DeltaStepParams p)
{
    constexpr int GROUPS = kStepThreads / CBL, CB = CBL * VW, WAVES = kStepThreads / 64;
    typedef float VecF __attribute__((ext_vector_type(VW)));
    __shared__ float kq[2][kStepMaxK];
    __shared__ float part[2][WAVES][CB];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int cl = tid % CBL, rg = tid / CBL;
    const uint32_t parts = (uint32_t)(p.dim_v + CB - 1) / CB;
    const int cb = blockIdx.x % parts;
    const int64_t rest = blockIdx.x / parts;
    const int h = (int)(rest % p.heads_v), hk = h / (p.heads_v / p.heads_qk);
    const int64_t seq = rest / p.heads_v;
    const int c0 = cb * CB + cl * VW;

    const int64_t begin = seq_begin(p.offsets, p.tokens, p.n_seqs, seq);
    const int64_t len = seq_length(p.offsets, p.tokens, p.n_seqs, seq, begin);
    if (len == 0) return;
    int64_t st;
    if (!slot_taken<kStepThreads>(p.slots, p.n_states, seq, &st, tid)) return;
    float* s0 = p.state + (st * p.heads_v + h) * p.dim_k * p.dim_v + c0;

    VecF s[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int row = rg + i * GROUPS;
        s[i] = VecF{};
        const VecF* at = reinterpret_cast<const VecF*>(s0 + (int64_t)row * p.dim_v);
        if (row < p.dim_k && c0 < p.dim_v) s[i] = NT ? __builtin_nontemporal_load(at) : *at;
    }
    for (int64_t t = begin; t < begin + len; ++t) {
        for (int i = tid; i < kStepMaxK; i += kStepThreads) {
            const bool in = i < p.dim_k;
            kq[0][i] = in ? load_as_float(p.k.data, t * p.k.ts + hk * p.k.hs + i, p.dtype) : 0.f;
            kq[1][i] = in ? load_as_float(p.q.data, t * p.q.ts + hk * p.q.hs + i, p.dtype) : 0.f;
        }
        const float a = p.g.data ? expf(clamp_decay(load_gate(p.g, t, h, p.g_dtype))) : 1.f;
        const float beta = load_gate(p.beta, t, h, p.beta_dtype);
        __syncthreads();
        float sk[VW] = {}, sq[VW] = {}, dot = 0.f;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int row = rg + i * GROUPS;
            const float k = kq[0][row], q = kq[1][row];
            dot += k * q;
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                s[i][j] *= a;
                sk[j] += s[i][j] * k;
                sq[j] += s[i][j] * q;
            }
        }
        // over the row groups: the lanes of a wave that hold the same columns, then the waves
#pragma unroll
        for (int d = CBL; d < 64; d *= 2) {
            dot += __shfl_xor(dot, d, 64);
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                sk[j] += __shfl_xor(sk[j], d, 64);
                sq[j] += __shfl_xor(sq[j], d, 64);
            }
        }
        __shared__ float dots[WAVES];
        if (lane < CBL) {
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                part[0][wave][lane * VW + j] = sk[j];
                part[1][wave][lane * VW + j] = sq[j];
            }
        }
        if (lane == 0) dots[wave] = dot;
        __syncthreads();
        float u[VW];
        dot = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) dot += dots[w];
#pragma unroll
        for (int j = 0; j < VW; ++j) {
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                x += part[0][w][cl * VW + j];
                y += part[1][w][cl * VW + j];
            }
            const bool in = c0 + j < p.dim_v;
            const float v = in ? load_as_float(p.v.data, t * p.v.ts + h * p.v.hs + c0 + j, p.dtype) : 0.f;
            u[j] = beta * (v - x);
            if (rg == 0 && in) store_as(p.out.data, t * p.out.ts + h * p.out.hs + c0 + j, p.dtype, p.scale * (y + dot * u[j]));
        }
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const float k = kq[0][rg + i * GROUPS];
#pragma unroll
            for (int j = 0; j < VW; ++j) s[i][j] += k * u[j];
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int row = rg + i * GROUPS;
        VecF* at = reinterpret_cast<VecF*>(s0 + (int64_t)row * p.dim_v);
        if (row < p.dim_k && c0 < p.dim_v) {
            if (NT)
                __builtin_nontemporal_store(s[i], at);
            else
                *at = s[i];
        }
    }
}

// Zeros to the rows of out before the first sequence and behind the last.
__global__ __launch_bounds__(kStepThreads) void k_delta_step_rest(DeltaStepParams p)
{
    const int64_t first = seq_begin(p.offsets, p.tokens, p.n_seqs, 0), last = seq_begin(p.offsets, p.tokens, p.n_seqs, p.n_seqs - 1);
    const int64_t end = last + seq_length(p.offsets, p.tokens, p.n_seqs, p.n_seqs - 1, last);
    const int64_t rest = first + p.tokens - end;
    for (int64_t r = blockIdx.x; r < rest; r += gridDim.x) {
        const int64_t row = r < first ? r : end + (r - first);
        for (int i = threadIdx.x; i < p.heads_v * p.dim_v; i += kStepThreads)
            store_as(p.out.data, row * p.out.ts + i / p.dim_v * p.out.hs + i % p.dim_v, p.dtype, 0.f);
    }
}

template <int VW, int CBL, bool NT = false>
hipError_t launch(const DeltaStepParams& p, hipStream_t stream)
{
    constexpr int GROUPS = kStepThreads / CBL, CB = CBL * VW;
    const uint64_t blocks = (uint64_t)p.n_seqs * p.heads_v * (((uint64_t)p.dim_v + CB - 1) / CB);
    const dim3 grid((uint32_t)blocks), threads(kStepThreads);
    switch (delta_padded_k(p.dim_k)) {
    case 64: k_delta_step<VW, CBL, 64 / GROUPS, NT><<<grid, threads, 0, stream>>>(p); break;
    case 128: k_delta_step<VW, CBL, 128 / GROUPS, NT><<<grid, threads, 0, stream>>>(p); break;
    default: k_delta_step<VW, CBL, 256 / GROUPS, NT><<<grid, threads, 0, stream>>>(p); break;
    }
    return hipGetLastError();
}

}  // namespace

// A workgroup takes as many of a head's columns as it has, 128 at most: whole
// rows of 512 bytes, and one sum over the rows for all of them (16 sequences of
// 32 heads of 128 x 128: 14.1 us against 17.6 us with 32 columns; four tokens for
// 64 of them 68 against 109; 64 x 64 heads with their 64 columns 17.5 against
// 25.2 with 32 and 40.5 with 128). With fewer heads than compute units it takes
// 32, which spreads them over more (one sequence of 32 heads 6.1 us against 8.6).
// States of 128 MB and more, half of the last-level cache, will not be there at
// the next step, with a model's other layers in between: they go past it (128
// sequences, three pools in turn: 105 us, 5.0 TB/s, against 117 us).
hipError_t launch_delta_step(const DeltaStepParams& p, bool vec4, hipStream_t stream)
{
    if (p.zero_rest && p.offsets != nullptr) {      // equal shares leave no rows
        k_delta_step_rest<<<dim3((uint32_t)(p.tokens < 1024 ? p.tokens : 1024)), dim3(kStepThreads), 0, stream>>>(p);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    constexpr int64_t kComputeUnits = 256, kPast = (int64_t)128 << 20;
    const int64_t heads = p.n_seqs * p.heads_v;
    if (!vec4) return launch<1, 32>(p, stream);
    if (p.dim_v <= 32 || heads < kComputeUnits) return launch<4, 8>(p, stream);
    const bool past = heads * p.dim_k * p.dim_v * 4 >= kPast;
    if (p.dim_v <= 64) return past ? launch<4, 16, true>(p, stream) : launch<4, 16>(p, stream);
    return past ? launch<4, 32, true>(p, stream) : launch<4, 32>(p, stream);
}

}  // namespace dws
