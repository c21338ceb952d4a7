// C entry points of the gated delta rule: argument checks, workspace layout
// and dispatch. The contract is in include/dws_scan.h.
#include "dws_scan.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <new>

#include "dws_delta.h"

namespace {

using namespace dws;

constexpr int kMaxDim = 256;
constexpr int kMaxHeads = 65535;
constexpr int64_t kMaxTokens = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxStride = (int64_t)1 << 40;
// a chunk of 64 rows spans less than 2^30 bytes, for 32-bit offsets
constexpr int64_t kMaxTokenStride = (int64_t)1 << 22;
// a launch holds fewer than 2^32 threads
constexpr uint64_t kMaxThreads = ((uint64_t)1 << 32) - 1;

dws_status status_of(hipError_t e)
{
    if (e == hipSuccess) return DWS_OK;
    if (e == hipErrorOutOfMemory || e == hipErrorMemoryAllocation) return DWS_ERR_OOM;
    return DWS_ERR_HIP;
}

size_t size_of(int dtype)
{
    return dtype == DWS_FLOAT32 ? 4 : (dtype == DWS_FLOAT16 || dtype == DWS_BFLOAT16 ? 2 : 0);
}

// Byte ranges of a call's operands, to refuse outputs that overlap others.
struct Ranges {
    struct One {
        uintptr_t begin, end;
        bool written;
    };
    One r[32];
    int n = 0;

    dws_status add(const void* ptr, unsigned __int128 bytes, bool written, size_t align)
    {
        if (bytes == 0) return DWS_OK;
        if (ptr == nullptr) return DWS_ERR_INVALID_ARG;
        const uintptr_t b = reinterpret_cast<uintptr_t>(ptr);
        if (b % align) return DWS_ERR_MISALIGNED;
        if (bytes > ((unsigned __int128)1 << 50) || b + (uintptr_t)bytes < b) return DWS_ERR_INVALID_ARG;
        r[n++] = {b, b + (uintptr_t)bytes, written};
        return DWS_OK;
    }
    bool overlap() const
    {
        for (int i = 0; i < n; ++i)
            for (int j = 0; j < i; ++j)
                if ((r[i].written || r[j].written) && r[i].begin < r[j].end && r[j].begin < r[i].end) return true;
        return false;
    }
};

// A (tokens, heads, dim) operand. Written ones must not name an element twice.
dws_status add_rows(Ranges* ranges, const dws_rows& a, int64_t tokens, int heads, int dim, int dtype, bool written,
                    DeltaRows* out)
{
    *out = {a.data, a.token_stride, a.head_stride};
    if (tokens == 0) return DWS_OK;
    const int64_t ts = a.token_stride, hs = a.head_stride;
    if (ts < 0 || hs < 0 || ts > kMaxStride || hs > kMaxStride) return DWS_ERR_INVALID_ARG;
    if (tokens > 1 && ts >= kMaxTokenStride) return DWS_ERR_UNSUPPORTED;
    if (written) {
        const __int128 heads_span = (__int128)(heads - 1) * hs + dim, token_span = (__int128)(tokens - 1) * ts + dim;
        const bool by_token = (heads == 1 || hs >= dim) && (tokens == 1 || ts >= heads_span);
        const bool by_head = (tokens == 1 || ts >= dim) && (heads == 1 || hs >= token_span);
        if (!by_token && !by_head) return DWS_ERR_INVALID_ARG;
    }
    const unsigned __int128 span =
        (unsigned __int128)(tokens - 1) * (uint64_t)ts + (unsigned __int128)(heads - 1) * (uint64_t)hs + dim;
    return ranges->add(a.data, span * size_of(dtype), written, size_of(dtype));
}

// Whether the rows are whole, aligned units of `bytes` bytes.
bool whole_units(const DeltaRows& a, int dim, int dtype, int bytes)
{
    const int64_t v = bytes / (int64_t)size_of(dtype);
    return reinterpret_cast<uintptr_t>(a.data) % bytes == 0 && dim % v == 0 && a.ts % v == 0 && a.hs % v == 0;
}

// Operand i of q, k, v, d_out: whether its rows have to be copied, and the
// copy's row length, whole 16-byte units.
struct Packed {
    bool needed;
    int heads, dim, padded;
};
Packed packed_of(const dws_delta_rule_args* a, int i)
{
    const dws_rows& r = i == 0 ? a->q : (i == 1 ? a->k : (i == 2 ? a->v : a->out_grad));
    const int dim = i < 2 ? a->dim_k : a->dim_v, unit = 16 / (int)size_of(a->dtype);
    const bool whole = whole_units({r.data, r.token_stride, r.head_stride}, dim, a->dtype, 16);
    return {a->tokens > 0 && !whole, i < 2 ? a->heads_qk : a->heads_v, dim, (dim + unit - 1) / unit * unit};
}

struct Sizes {
    size_t gate, t, p, tt, s, u, z, ds, pack[4];    // offsets
    size_t bytes;
    int64_t n_slots;
};

dws_status check_shape(const dws_delta_rule_args* a)
{
    if (a == nullptr) return DWS_ERR_INVALID_ARG;
    if (size_of(a->dtype) == 0 || a->tokens < 0 || a->n_seqs < 1) return DWS_ERR_INVALID_ARG;
    if (a->options & ~(DWS_DELTA_FP32_GRADS | DWS_DELTA_PRECISE)) return DWS_ERR_INVALID_ARG;
    if (a->heads_qk < 1 || a->heads_v < 1 || a->dim_k < 1 || a->dim_v < 1) return DWS_ERR_INVALID_ARG;
    if (a->heads_v % a->heads_qk != 0) return DWS_ERR_INVALID_ARG;
    if (a->d_offsets == nullptr && a->tokens % a->n_seqs != 0) return DWS_ERR_INVALID_ARG;
    if (a->dim_k > kMaxDim || a->dim_v > kMaxDim || a->heads_v > kMaxHeads) return DWS_ERR_UNSUPPORTED;
    if (a->tokens > kMaxTokens || a->n_seqs > kMaxTokens) return DWS_ERR_UNSUPPORTED;
    // one workgroup of at most 256 threads for each chunk slot and value head,
    // and scan workgroups of 16 columns at least
    const uint64_t slots = (uint64_t)a->tokens / delta_chunk(a->dtype, a->dim_k) + (uint64_t)a->n_seqs + 1;
    if (slots * (uint64_t)a->heads_v > kMaxThreads / 256) return DWS_ERR_UNSUPPORTED;
    if (((uint64_t)a->n_seqs * a->heads_v + 8) * 16 > kMaxThreads / 512) return DWS_ERR_UNSUPPORTED;
    return DWS_OK;
}

// Workspace arrays of a call, each at a multiple of 256 bytes. The caller's
// sizes have passed check_shape. The counts of parts are the kernels'. `precise`:
// as the launchers'.
Sizes workspace_of(const dws_delta_rule_args* a, bool backward, bool precise)
{
    Sizes z{};
    const size_t c = (size_t)delta_chunk(a->dtype, a->dim_k), e = size_of(a->dtype);
    const size_t dk = (size_t)delta_padded_k(a->dim_k), dv = (size_t)delta_padded_v(a->dim_v);
    z.n_slots = a->tokens / (int64_t)c + a->n_seqs + 1;
    const size_t fine = (size_t)delta_fine_parts(a->dtype);
    const size_t n = (size_t)z.n_slots * (size_t)a->heads_v;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t was = at;
        at += (bytes + 255) / 256 * 256;
        return was;
    };
    z.gate = take(n * 5 * c * sizeof(float));
    const size_t tri = (size_t)delta_triangle((int)c) * e;
    z.t = take(n * tri * (precise && !backward ? (size_t)delta_precise_parts(a->dtype) : fine));
    z.p = take(n * tri * fine);
    if (backward) {
        z.tt = take(n * tri * fine);
        z.s = take(n * dk * dv * e * (size_t)delta_state_parts(a->dtype));
        z.u = take(n * c * dv * e * fine);
        z.z = take(n * c * dv * e * fine);
        z.ds = take(n * dk * dv * e * (size_t)delta_state_grad_parts(a->dtype, a->dim_k, precise));
    }
    const int kinds = backward ? 4 : 3;
    for (int i = 0; i < kinds; ++i) {
        const Packed k = packed_of(a, i);
        z.pack[i] = at;
        if (k.needed) take((size_t)a->tokens * k.heads * k.padded * e);
    }
    z.bytes = at;
    return z;
}

// Points the parameters at the copies of rows that are not whole 16-byte units.
void pack(const dws_delta_rule_args* a, const Sizes& z, bool backward, DeltaParams* p, DeltaPack* k)
{
    DeltaRows* rows[] = {&p->q, &p->k, &p->v, &p->d_out};
    for (int i = 0; i < (backward ? 4 : 3); ++i) {
        const Packed of = packed_of(a, i);
        if (!of.needed) continue;
        auto& r = k->rows[k->n++];
        r = {*rows[i], static_cast<char*>(a->d_workspace) + z.pack[i], of.heads, of.dim, of.padded};
        *rows[i] = {r.dst, (int64_t)of.heads * of.padded, of.padded};
    }
}

bool is_precise(const dws_delta_rule_args* a, bool backward)
{
    return a->dtype != DWS_FLOAT32 && ((!backward && a->d_final_state != nullptr) || (a->options & DWS_DELTA_PRECISE) != 0);
}

// The operands that both directions read, and the launch's parameters.
dws_status common(const dws_delta_rule_args* a, Ranges* r, DeltaParams* p)
{
    if (dws_status st = check_shape(a); st != DWS_OK) return st;
    if (size_of(a->beta_dtype) == 0 || (a->g.data != nullptr && size_of(a->g_dtype) == 0)) return DWS_ERR_INVALID_ARG;
    p->tokens = a->tokens;
    p->n_seqs = a->n_seqs;
    p->offsets = reinterpret_cast<const int64_t*>(a->d_offsets);
    p->heads_qk = a->heads_qk;
    p->heads_v = a->heads_v;
    p->dim_k = a->dim_k;
    p->dim_v = a->dim_v;
    p->dv_pad = delta_padded_v(a->dim_v);
    p->scale = a->scale;
    p->g_dtype = a->g_dtype;
    p->beta_dtype = a->beta_dtype;
    dws_status st = add_rows(r, a->q, a->tokens, a->heads_qk, a->dim_k, a->dtype, false, &p->q);
    if (st == DWS_OK) st = add_rows(r, a->k, a->tokens, a->heads_qk, a->dim_k, a->dtype, false, &p->k);
    if (st == DWS_OK) st = add_rows(r, a->v, a->tokens, a->heads_v, a->dim_v, a->dtype, false, &p->v);
    if (st == DWS_OK && a->g.data != nullptr)
        st = add_rows(r, a->g, a->tokens, a->heads_v, 1, a->g_dtype, false, &p->g);
    if (st == DWS_OK) st = add_rows(r, a->beta, a->tokens, a->heads_v, 1, a->beta_dtype, false, &p->beta);
    if (st == DWS_OK && a->d_offsets != nullptr)
        st = r->add(a->d_offsets, (unsigned __int128)(a->n_seqs + 1) * 8, false, 8);
    return st;
}

unsigned __int128 state_bytes(const dws_delta_rule_args* a, int64_t count, size_t size)
{
    return (unsigned __int128)(uint64_t)count * (uint64_t)a->heads_v * (uint64_t)a->dim_k * (uint64_t)a->dim_v * size;
}

// Slots, and the states they pick from: *count states at each state pointer.
dws_status check_slots(const dws_delta_rule_args* a, Ranges* r, int64_t* count)
{
    *count = a->n_seqs;
    if (a->d_slots == nullptr) return DWS_OK;
    if (a->n_states < 1) return DWS_ERR_INVALID_ARG;
    if (a->n_states > kMaxTokens) return DWS_ERR_UNSUPPORTED;
    *count = a->n_states;
    return r->add(a->d_slots, (unsigned __int128)a->n_seqs * 4, false, 4);
}

dws_status forward_entry(const dws_delta_rule_args* a, hipStream_t stream)
{
    Ranges r;
    DeltaParams p{};
    dws_status st = common(a, &r, &p);
    if (st == DWS_OK) st = add_rows(&r, a->out, a->tokens, a->heads_v, a->dim_v, a->dtype, true, &p.out);
    int64_t states = 0;
    if (st == DWS_OK) st = check_slots(a, &r, &states);
    if (st == DWS_OK && a->d_initial_state != nullptr && a->d_initial_state != a->d_final_state)
        st = r.add(a->d_initial_state, state_bytes(a, states, 4), false, 4);
    if (st == DWS_OK && a->d_final_state != nullptr) st = r.add(a->d_final_state, state_bytes(a, states, 4), true, 4);
    if (st != DWS_OK) return st;
    const bool precise = is_precise(a, false);
    const Sizes z = workspace_of(a, false, precise);
    if (a->d_workspace == nullptr || a->workspace_bytes < z.bytes) return DWS_ERR_INVALID_ARG;
    if ((st = r.add(a->d_workspace, z.bytes, true, 256)) != DWS_OK) return st;
    if (r.overlap()) return DWS_ERR_OVERLAP;
    p.out4 = whole_units(p.out, a->dim_v, a->dtype, 4 * (int)size_of(a->dtype));
    p.initial = a->d_initial_state;
    p.final_state = a->d_final_state;
    p.slots = a->d_slots;
    p.n_states = states;
    p.zero_rest = a->zero_rest;
    p.n_slots = z.n_slots;
    char* w = static_cast<char*>(a->d_workspace);
    p.w_gate = reinterpret_cast<float*>(w + z.gate);
    p.w_t = w + z.t;
    p.w_p = w + z.p;
    DeltaPack k{};
    pack(a, z, false, &p, &k);
    switch (a->dtype) {
    case DWS_BFLOAT16: return status_of(launch_delta_forward_bf16(p, k, precise, stream));
    case DWS_FLOAT16: return status_of(launch_delta_forward_f16(p, k, precise, stream));
    default: return status_of(launch_delta_forward_f32(p, k, precise, stream));
    }
}

dws_status backward_entry(const dws_delta_rule_args* a, hipStream_t stream)
{
    Ranges r;
    DeltaParams p{};
    dws_status st = common(a, &r, &p);
    if (st == DWS_OK && a->d_slots != nullptr) st = DWS_ERR_UNSUPPORTED;
    if (st == DWS_OK) st = add_rows(&r, a->out_grad, a->tokens, a->heads_v, a->dim_v, a->dtype, false, &p.d_out);
    if (st == DWS_OK) st = add_rows(&r, a->q_grad, a->tokens, a->heads_qk, a->dim_k, a->dtype, true, &p.dq);
    if (st == DWS_OK) st = add_rows(&r, a->k_grad, a->tokens, a->heads_qk, a->dim_k, a->dtype, true, &p.dk);
    if (st == DWS_OK) st = add_rows(&r, a->v_grad, a->tokens, a->heads_v, a->dim_v, a->dtype, true, &p.dv);
    if (st != DWS_OK) return st;
    p.fp32_grads = a->options & DWS_DELTA_FP32_GRADS;
    const int narrow = p.fp32_grads ? (int)DWS_FLOAT32 : a->dtype;      // of the gates' and the states' gradients
    const size_t e = size_of(narrow);
    if (a->g_grad.data != nullptr) {
        st = a->g.data == nullptr ? DWS_ERR_INVALID_ARG
                                  : add_rows(&r, a->g_grad, a->tokens, a->heads_v, 1, narrow, true, &p.dg);
    }
    if (st == DWS_OK) st = add_rows(&r, a->beta_grad, a->tokens, a->heads_v, 1, narrow, true, &p.dbeta);
    if (st == DWS_OK && a->d_initial_state != nullptr)
        st = r.add(a->d_initial_state, state_bytes(a, a->n_seqs, 4), false, 4);
    if (st == DWS_OK && a->d_final_grad != nullptr) st = r.add(a->d_final_grad, state_bytes(a, a->n_seqs, 4), false, 4);
    if (st == DWS_OK && a->d_initial_grad != nullptr)
        st = r.add(a->d_initial_grad, state_bytes(a, a->n_seqs, e), true, e);
    if (st != DWS_OK) return st;
    const bool precise = is_precise(a, true);
    const Sizes z = workspace_of(a, true, precise);
    // the gradients' workgroups have up to 512 threads
    if ((uint64_t)z.n_slots * (uint64_t)a->heads_qk > kMaxThreads / 512) return DWS_ERR_UNSUPPORTED;
    if (a->d_workspace == nullptr || a->workspace_bytes < z.bytes) return DWS_ERR_INVALID_ARG;
    if ((st = r.add(a->d_workspace, z.bytes, true, 256)) != DWS_OK) return st;
    if (r.overlap()) return DWS_ERR_OVERLAP;
    p.dv4 = whole_units(p.dv, a->dim_v, a->dtype, 4 * (int)size_of(a->dtype));
    p.initial = a->d_initial_state;
    p.d_final = a->d_final_grad;
    p.d_initial = a->d_initial_grad;
    p.zero_rest = a->zero_rest;
    p.n_slots = z.n_slots;
    char* w = static_cast<char*>(a->d_workspace);
    p.w_gate = reinterpret_cast<float*>(w + z.gate);
    p.w_t = w + z.t;
    p.w_p = w + z.p;
    p.w_tt = w + z.tt;
    p.w_s = w + z.s;
    p.w_u = w + z.u;
    p.w_z = w + z.z;
    p.w_ds = w + z.ds;
    DeltaPack k{};
    pack(a, z, true, &p, &k);
    switch (a->dtype) {
    case DWS_BFLOAT16: return status_of(launch_delta_backward_bf16(p, k, precise, stream));
    case DWS_FLOAT16: return status_of(launch_delta_backward_f16(p, k, precise, stream));
    default: return status_of(launch_delta_backward_f32(p, k, precise, stream));
    }
}

dws_status step_entry(const dws_delta_rule_args* a, hipStream_t stream)
{
    Ranges r;
    DeltaParams c{};
    dws_status st = common(a, &r, &c);
    DeltaStepParams p{};
    if (st == DWS_OK) st = add_rows(&r, a->out, a->tokens, a->heads_v, a->dim_v, a->dtype, true, &p.out);
    int64_t states = 0;
    if (st == DWS_OK) st = check_slots(a, &r, &states);
    if (st == DWS_OK && (a->d_final_state == nullptr || a->d_initial_state != a->d_final_state)) st = DWS_ERR_INVALID_ARG;
    if (st == DWS_OK) st = r.add(a->d_final_state, state_bytes(a, states, 4), true, 4);
    if (st != DWS_OK) return st;
    if (r.overlap()) return DWS_ERR_OVERLAP;
    if (a->tokens == 0) return DWS_OK;
    p.tokens = c.tokens;
    p.n_seqs = c.n_seqs;
    p.offsets = c.offsets;
    p.heads_qk = c.heads_qk;
    p.heads_v = c.heads_v;
    p.dim_k = c.dim_k;
    p.dim_v = c.dim_v;
    p.scale = c.scale;
    p.dtype = a->dtype;
    p.g_dtype = c.g_dtype;
    p.beta_dtype = c.beta_dtype;
    p.q = c.q;
    p.k = c.k;
    p.v = c.v;
    p.g = c.g;
    p.beta = c.beta;
    p.state = a->d_final_state;
    p.slots = a->d_slots;
    p.n_states = states;
    p.zero_rest = a->zero_rest;
    const bool vec4 = a->dim_v % 4 == 0 && (reinterpret_cast<uintptr_t>(a->d_final_state) & 15u) == 0;
    return status_of(launch_delta_step(p, vec4, stream));
}

template <class F>
dws_status guarded(F f)
{
    try {
        return f();
    } catch (const std::bad_alloc&) {
        return DWS_ERR_OOM;
    } catch (...) {
        return DWS_ERR_HIP;
    }
}

}  // namespace

extern "C" {

dws_status dws_delta_rule_workspace(const dws_delta_rule_args* args, int backward, size_t* bytes)
{
    if (bytes == nullptr) return DWS_ERR_INVALID_ARG;
    if (dws_status st = check_shape(args); st != DWS_OK) return st;
    *bytes = workspace_of(args, backward != 0, is_precise(args, backward != 0)).bytes;
    return DWS_OK;
}

dws_status dws_delta_rule(const dws_delta_rule_args* args, hipStream_t stream)
{
    return guarded([&] { return forward_entry(args, stream); });
}

dws_status dws_delta_rule_backward(const dws_delta_rule_args* args, hipStream_t stream)
{
    return guarded([&] { return backward_entry(args, stream); });
}

dws_status dws_delta_rule_step(const dws_delta_rule_args* args, hipStream_t stream)
{
    return guarded([&] { return step_entry(args, stream); });
}

}  // extern "C"
