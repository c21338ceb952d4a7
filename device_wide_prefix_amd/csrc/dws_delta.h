// Host-side interface between the delta rule's C entry points
// (dws_delta_abi.cpp) and its kernels. Not installed; not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dws_scan.h"

namespace dws {

// Head dimensions the chunk kernels are built for; others run zero-padded.
constexpr int delta_padded_k(int dim_k) { return dim_k <= 64 ? 64 : (dim_k <= 128 ? 128 : 256); }
// Tokens of a chunk (kChunk of the kernels, which says why).
constexpr int delta_chunk(int dtype, int dim_k) { return dtype == DWS_FLOAT32 || dim_k > 128 ? 32 : 64; }
// Columns of a value head are laid out in the workspace in whole 32s.
constexpr int delta_padded_v(int dim_v) { return (dim_v + 31) / 32 * 32; }
// Elements of a triangular matrix's fragments (Triangle in the kernels).
constexpr int delta_triangle(int chunk) { return (chunk == 64 ? 6 : 2) * 512; }

// Parts (numbers of the input type whose sum is the value) of the operands
// computed in fp32: those of a chunk's size, the states and the states' gradients
// that the backward pass keeps, and all that a final state depends on.
constexpr int delta_fine_parts(int dtype) { return dtype == DWS_FLOAT32 ? 1 : 2; }
constexpr int delta_state_parts(int dtype) { return delta_fine_parts(dtype); }
constexpr int delta_state_grad_parts(int dtype, int dim_k, bool precise)
{
    return precise || dim_k > 128 ? delta_fine_parts(dtype) : 1;
}
constexpr int delta_precise_parts(int dtype) { return dtype == DWS_BFLOAT16 ? 3 : delta_fine_parts(dtype); }

// One (tokens, heads, dim) operand: strides in elements, dim contiguous.
struct DeltaRows {
    void* data;
    int64_t ts, hs;
};

// What every delta-rule kernel is given (by value).
struct DeltaParams {
    int64_t tokens, n_seqs;
    const int64_t* offsets;      // n_seqs + 1, or null: tokens / n_seqs each
    int heads_qk, heads_v, dim_k, dim_v, dv_pad;
    float scale;
    int g_dtype, beta_dtype;
    int out4, dv4;               // out's (dv's) rows are whole, aligned units of four elements
    DeltaRows q, k, v, g, beta, out;
    const float* initial;        // (n_seqs or n_states, heads_v, dim_k, dim_v)
    float* final_state;
    const int* slots;
    int64_t n_states;
    // backward
    DeltaRows d_out, dq, dk, dv, dg, dbeta;
    const float* d_final;
    void* d_initial;
    int fp32_grads;              // dg, dbeta and d_initial are fp32, else of the input type
    int zero_rest;               // zero the output rows in no sequence
    // workspace
    int64_t n_slots;             // chunk slots: tokens / chunk + n_seqs + 1 (the last ones empty)
    float* w_gate;               // [slot][head][5][chunk]: gate factors (kGateArrays in the kernels)
    // triangular matrices as operand fragments (Triangle in the kernels)
    void* w_t;                   // [slot][head][parts][frags]: (I + L diag(beta))^-1
    void* w_p;                   // [slot][head][fine][frags]: P (forward), its transpose (backward)
    void* w_tt;                  // [slot][head][fine][frags]: transpose of (I + diag(beta) L)^-1 (backward)
    // 16 columns of the value head after the other (store_columns in the kernels)
    void* w_s;                   // [slot][head][state parts][dv_pad / 16][16 x padded dim_k]: states at the chunks' starts
    void* w_u;                   // [slot][head][fine][dv_pad / 16][16 x chunk]: U'
    void* w_z;                   // [slot][head][fine][dv_pad / 16][16 x chunk]: Z
    void* w_ds;                  // [slot][head][state grad parts][dv_pad / 16][16 x padded dim_k]: state gradients at the chunks' ends
};

// Arrays that are copied to the workspace first, since their rows are not whole
// 16-byte units; the parameters name the copies.
struct DeltaPack {
    struct {
        DeltaRows src;
        void* dst;
        int heads, dim, padded;
    } rows[4];
    int n;
};

// Per-type launchers (dws_delta_{bf16,f16,f32}.hip). `precise`: the states have
// fp32 accuracy, as a final one that is wanted has to; backward, the states'
// gradients enter the products in as many parts as the states.
hipError_t launch_delta_forward_bf16(const DeltaParams& p, const DeltaPack& k, bool precise, hipStream_t stream);
hipError_t launch_delta_forward_f16(const DeltaParams& p, const DeltaPack& k, bool precise, hipStream_t stream);
hipError_t launch_delta_forward_f32(const DeltaParams& p, const DeltaPack& k, bool precise, hipStream_t stream);
hipError_t launch_delta_backward_bf16(const DeltaParams& p, const DeltaPack& k, bool precise, hipStream_t stream);
hipError_t launch_delta_backward_f16(const DeltaParams& p, const DeltaPack& k, bool precise, hipStream_t stream);
hipError_t launch_delta_backward_f32(const DeltaParams& p, const DeltaPack& k, bool precise, hipStream_t stream);

struct DeltaStepParams {
    int64_t tokens, n_seqs;
    const int64_t* offsets;
    int heads_qk, heads_v, dim_k, dim_v;
    float scale;
    int dtype, g_dtype, beta_dtype;
    DeltaRows q, k, v, g, beta, out;
    float* state;
    const int* slots;
    int64_t n_states;
    int zero_rest;
};
hipError_t launch_delta_step(const DeltaStepParams& p, bool vec4, hipStream_t stream);

}  // namespace dws
