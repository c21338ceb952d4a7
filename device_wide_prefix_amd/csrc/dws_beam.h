// Host-side interface between the C entry points of the beam selection
// (dws_beam_abi.cpp) and its kernels. Not installed; not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dws_scan.h"

namespace dws {

constexpr int kMaxBeams = 64;
constexpr int kMaxBest = 64;            // one a lane
constexpr int kBeamBlock = 512;         // logits that a wave takes at a time, eight a lane

// A stretch of a beam's logits: the sum of their exponentials is sum e^top.
struct BeamStat {
    double sum;
    float top;
    int pad;
};

constexpr int kBeamWaves = 8;           // of a workgroup that reads logits

// Workgroups that a beam's logits are shared out to: as many as give 512 in all, two a
// compute unit, but at least one block for each of a workgroup's waves. More cost more
// than they spread: with 1,024, 512 rows of 131,071 logits take 46 us instead of 42,
// and 160 rows of 50,001 take 36 instead of 28.
constexpr int64_t beam_splits(int64_t rows, int64_t vocab)
{
    const int64_t most = (vocab + kBeamWaves * kBeamBlock - 1) / (kBeamWaves * kBeamBlock), want = (512 + rows - 1) / rows;
    const int64_t n = want < most ? want : most;
    return n < 1 ? 1 : (n > 64 ? 64 : n);
}

struct BeamParams {
    const void* logits;
    int64_t batch, beams, vocab, batch_stride, beam_stride;
    int k, splits;
    const float* scores;
    const unsigned char* finished;
    int64_t end_token;
    const int* rows;
    float* out_scores;
    int* parents;
    int* tokens;
    int* out_rows;
    int* src;
    int* dst;
    // workspace
    uint64_t* best;         // [batch * beams][splits][k], descending; 0 where there are fewer
    BeamStat* stat;         // [batch * beams][splits]
};
hipError_t launch_beam_select(const BeamParams& p, int dtype, hipStream_t stream);

}  // namespace dws
