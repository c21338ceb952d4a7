// C entry points of the beam selection: argument checks, workspace layout and
// dispatch. The contract is in include/dws_scan.h.
#include "dws_scan.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <new>

#include "dws_abi_arrays.h"
#include "dws_beam.h"

namespace {

using namespace dws;

constexpr int64_t kMaxCount = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int64_t kMaxGrid = (((int64_t)1 << 32) - 1) / 512;     // workgroups of at most 512 threads in a launch

size_t size_of(int dtype)
{
    return dtype == DWS_FLOAT32 ? 4 : (dtype == DWS_FLOAT16 || dtype == DWS_BFLOAT16 ? 2 : 0);
}

struct Sizes {
    int64_t splits;
    size_t stat, bytes;
};
dws_status sizes_of(const dws_beam_args* a, Sizes* z)
{
    if (a == nullptr || size_of(a->dtype) == 0 || a->batch < 0 || a->beams < 1 || a->vocab < 1 || a->k < 1)
        return DWS_ERR_INVALID_ARG;
    if (a->beams > kMaxBeams || a->k > kMaxBest || a->vocab > kMaxCount || a->batch > kMaxCount / a->beams)
        return DWS_ERR_UNSUPPORTED;
    if (a->k > a->beams * a->vocab) return DWS_ERR_INVALID_ARG;
    const int64_t rows = a->batch * a->beams;
    z->splits = beam_splits(rows > 0 ? rows : 1, a->vocab);
    if (rows * z->splits > kMaxGrid) return DWS_ERR_UNSUPPORTED;
    z->stat = ((size_t)(rows * z->splits * a->k) * 8 + 255) / 256 * 256;
    z->bytes = z->stat + (size_t)(rows * z->splits) * sizeof(BeamStat);
    return DWS_OK;
}

dws_status select_entry(const dws_beam_args* a, hipStream_t stream)
{
    Sizes z{};
    dws_status st = sizes_of(a, &z);
    if (st != DWS_OK) return st;
    if (a->batch_stride < 0 || a->beam_stride < 0 || a->batch_stride > kMaxStride || a->beam_stride > kMaxStride)
        return DWS_ERR_INVALID_ARG;
    if (a->d_finished != nullptr && (a->end_token < 0 || a->end_token >= a->vocab)) return DWS_ERR_INVALID_ARG;
    if (a->d_rows != nullptr && a->k != a->beams) return DWS_ERR_INVALID_ARG;
    if (a->batch == 0) return DWS_OK;
    const int64_t e = (int64_t)size_of(a->dtype), n = a->batch * a->beams, out = a->batch * a->k;
    Arrays arrays;
    const Strided logits{{a->batch_stride * e, a->beam_stride * e, 0}, {a->batch, a->beams, 1}, a->vocab * e};
    st = arrays.add(a->d_logits, logits, false, (size_t)e);
    if (st == DWS_OK) st = arrays.add(a->d_scores, n * 4, false, 4);
    if (st == DWS_OK && a->d_finished != nullptr) st = arrays.add(a->d_finished, n, false, 1);
    if (st == DWS_OK) st = arrays.add(a->d_out_scores, out * 4, true, 4);
    if (st == DWS_OK) st = arrays.add(a->d_parents, out * 4, true, 4);
    if (st == DWS_OK) st = arrays.add(a->d_tokens, out * 4, true, 4);
    if (a->d_rows != nullptr) {
        if (st == DWS_OK) st = arrays.add(a->d_rows, n * 4, false, 4);
        if (st == DWS_OK) st = arrays.add(a->d_out_rows, n * 4, true, 4);
        if (st == DWS_OK) st = arrays.add(a->d_src, n * 4, true, 4);
        if (st == DWS_OK) st = arrays.add(a->d_dst, n * 4, true, 4);
    }
    if (st != DWS_OK) return st;
    if (a->d_workspace == nullptr || a->workspace_bytes < z.bytes) return DWS_ERR_INVALID_ARG;
    if ((st = arrays.add(a->d_workspace, (int64_t)z.bytes, true, 256)) != DWS_OK) return st;
    if (arrays.overlap()) return DWS_ERR_OVERLAP;
    BeamParams p{};
    p.logits = a->d_logits;
    p.batch = a->batch;
    p.beams = a->beams;
    p.vocab = a->vocab;
    p.batch_stride = a->batch_stride;
    p.beam_stride = a->beam_stride;
    p.k = a->k;
    p.splits = (int)z.splits;
    p.scores = a->d_scores;
    p.finished = a->d_finished;
    p.end_token = a->end_token;
    p.rows = a->d_rows;
    p.out_scores = a->d_out_scores;
    p.parents = a->d_parents;
    p.tokens = a->d_tokens;
    p.out_rows = a->d_out_rows;
    p.src = a->d_src;
    p.dst = a->d_dst;
    p.best = static_cast<uint64_t*>(a->d_workspace);
    p.stat = reinterpret_cast<BeamStat*>(static_cast<char*>(a->d_workspace) + z.stat);
    const hipError_t r = launch_beam_select(p, a->dtype, stream);
    return r == hipSuccess ? DWS_OK : DWS_ERR_HIP;
}

}  // namespace

extern "C" {

dws_status dws_beam_select_workspace(const dws_beam_args* args, size_t* bytes)
{
    if (bytes == nullptr) return DWS_ERR_INVALID_ARG;
    Sizes z{};
    const dws_status st = sizes_of(args, &z);
    if (st == DWS_OK) *bytes = z.bytes;
    return st;
}

dws_status dws_beam_select(const dws_beam_args* args, hipStream_t stream)
{
    try {
        return select_entry(args, stream);
    } catch (const std::bad_alloc&) {
        return DWS_ERR_OOM;
    } catch (...) {
        return DWS_ERR_HIP;
    }
}

}  // extern "C"
