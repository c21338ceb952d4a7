// Beam search's selection: the k best of score[beam] + log softmax(logits[beam])
// [token] over a request's beams and the vocabulary.
//
// Within a beam the order is that of the logits, so one pass over them (their bytes
// bound it) finds both the sum of the exponentials and the k largest; only the k of
// each beam are then compared across beams, in fp64. The k-th largest of the lanes'
// maxima of what a workgroup reads first is a border that k logits are not below:
// few of the rest are above it. Those are put down as they come, and a wave sorts
// them, 64 at a time, into the best so far, one a lane.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dws_beam.h"
#include "dws_cache_device.hpp"

namespace dws {
namespace {

typedef __bf16 bf16_t;
typedef _Float16 f16_t;
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef u32x4_t Loose __attribute__((aligned(2)));      // at any address that elements have

constexpr int kEach = kBeamBlock / 64;      // logits of a lane's chunk
constexpr double kLog2eD = 1.4426950408889634074;

// A logit and its token as a number: larger for larger logits, then for lower
// tokens; never 0.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t token)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.f);       // -0 as 0
    const uint32_t ordered = u & 0x80000000u ? ~u : u | 0x80000000u;
    return (uint64_t)ordered << 32 | (uint32_t)~token;
}
__device__ __forceinline__ float logit_of(uint64_t key)
{
    const uint32_t u = (uint32_t)(key >> 32);
    return __builtin_bit_cast(float, u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
// Of a key's upper half; -infinity where there is no key.
__device__ __forceinline__ float border_of(uint32_t ordered)
{
    return ordered == 0 ? -__builtin_inff() : logit_of((uint64_t)ordered << 32);
}
__device__ __forceinline__ uint64_t lane_of(uint64_t x, int lane)
{
    return (uint64_t)__builtin_amdgcn_readlane((uint32_t)(x >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((uint32_t)x, lane);
}

// The value of the lane whose number differs in bit D, without a trip through the LDS.
template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t x)
{
    return __builtin_amdgcn_update_dpp(x, x, CTRL, 0xf, 0xf, false);
}
template <int D>
__device__ __forceinline__ uint32_t across(uint32_t x, int lane)
{
    if constexpr (D == 1) return moved<0xb1>(x);                // lanes 1 0 3 2 of four
    if constexpr (D == 2) return moved<0x4e>(x);                // 2 3 0 1
    if constexpr (D == 4) return moved<0x1b>(moved<0x141>(x));  // eight backwards, then four backwards
    if constexpr (D == 8) return moved<0x128>(x);               // sixteen turned by eight
    if constexpr (D == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        return lane & 16 ? r[0] : r[1];
    }
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return lane & 32 ? r[0] : r[1];
}
template <int D>
__device__ __forceinline__ uint64_t across(uint64_t x, int lane)
{
    return (uint64_t)across<D>((uint32_t)(x >> 32), lane) << 32 | across<D>((uint32_t)x, lane);
}
__device__ __forceinline__ uint64_t reversed(uint64_t x, int lane)
{
    return (uint64_t)(uint32_t)__shfl((int)(x >> 32), 63 - lane, 64) << 32 | (uint32_t)__shfl((int)x, 63 - lane, 64);
}

// One step of a descending bitonic network: of two lanes the lower (`up`: the
// upper) one keeps the larger.
template <int D, class U>
__device__ __forceinline__ U exchange(U x, int lane, bool up)
{
    const U y = across<D>(x, lane);
    const bool larger = ((lane & D) == 0) != up;
    return (x > y) == larger ? x : y;
}
template <int D, class U>
__device__ __forceinline__ U steps_down(U x, int lane, bool up)
{
    x = exchange<D>(x, lane, up);
    if constexpr (D > 1) x = steps_down<D / 2>(x, lane, up);
    return x;
}
template <class U>
__device__ __forceinline__ U sorted(U x, int lane)
{
    x = steps_down<1>(x, lane, lane & 2);
    x = steps_down<2>(x, lane, lane & 4);
    x = steps_down<4>(x, lane, lane & 8);
    x = steps_down<8>(x, lane, lane & 16);
    x = steps_down<16>(x, lane, lane & 32);
    return steps_down<32>(x, lane, false);
}
// The 64 best of two descending lists, the second given backwards.
template <class U>
__device__ __forceinline__ U merged(U x, U backwards, int lane)
{
    return steps_down<32>(x > backwards ? x : backwards, lane, false);
}

template <class T>
struct Stretch {
    static constexpr int VEC = 16 / sizeof(T), LOADS = kEach / VEC;
    typedef T Vec __attribute__((ext_vector_type(VEC)));
    u32x4_t raw[LOADS];

    // Eight elements of a row, which may start anywhere: with chunks that went by
    // addresses, rows of equal logits would be summed in different orders, and equal
    // beams would not tie.
    __device__ __forceinline__ void load(const T* from)
    {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) raw[i] = *(const __attribute__((address_space(1))) Loose*)(from + i * VEC);
    }
    // The first `count` of them; -infinity for the others.
    __device__ __forceinline__ void load(const T* from, int count)
    {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            Vec x;
#pragma unroll
            for (int j = 0; j < VEC; ++j) x[j] = i * VEC + j < count ? from[i * VEC + j] : (T)-__builtin_inff();
            raw[i] = __builtin_bit_cast(u32x4_t, x);
        }
    }
    // (of those that are numbers, if there are any)
    __device__ __forceinline__ float largest() const
    {
        float top = get(0);
#pragma unroll
        for (int j = 1; j < kEach; ++j) top = fmaxf(top, get(j));
        return top;
    }
    __device__ __forceinline__ float get(int j) const
    {
        // (in bits: from conversions the compiler makes a maximum with a rounding at each step)
        if constexpr (__is_same(T, bf16_t)) {
            const uint32_t pair = raw[j / VEC][j % VEC / 2];
            return __builtin_bit_cast(float, j % 2 ? pair & 0xffff0000u : pair << 16);
        }
        return (float)__builtin_bit_cast(Vec, raw[j / VEC])[j % VEC];
    }
};

// A float in the order of the keys' upper halves; NaN as 0, below everything.
__device__ __forceinline__ uint32_t ordered_of(float x)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.f);
    return x != x ? 0 : (u & 0x80000000u ? ~u : u | 0x80000000u);
}

// 512 rows of 131,071 bf16 logits take 37 us, 3.7 TB/s, where a copy reaches 5.3:
// each logit costs ten instructions' time beside its bytes, four of them its
// exponential.
// A wave's code runs once over little data, so it is kept short: with the sorting
// in each step's code (138 KB) the same took 52 us.
template <class T>
__global__ __launch_bounds__(64 * kBeamWaves) void k_beam_rows(BeamParams p)
{
    constexpr int AHEAD = sizeof(T) == 2 ? 4 : 2;       // blocks in flight
    constexpr float kLog2e = 1.44269502162933349609f, kLog2eRest = 1.9259629911266e-8f;      // log2(e) in two parts
    __shared__ uint64_t lists[kBeamWaves][64];
    __shared__ BeamStat stats[kBeamWaves];
    __shared__ float tops[kBeamWaves][64];
    __shared__ uint64_t found[kBeamWaves][64 + kBeamBlock];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t r = blockIdx.x / p.splits;
    const int split = blockIdx.x % p.splits;
    const T* row = static_cast<const T*>(p.logits) + r / p.beams * p.batch_stride + r % p.beams * p.beam_stride;
    // whole blocks, and what is behind the last one, which is the last wave's
    const int blocks = (int)(p.vocab / kBeamBlock), per = (blocks + p.splits - 1) / p.splits;
    const int end = split * per + per < blocks ? split * per + per : blocks;
    const int rest = split == p.splits - 1 && wave == kBeamWaves - 1 ? (int)(p.vocab % kBeamBlock) - lane * kEach : 0;

    // The loads of the loop are always made: after one that may not have been, a wait is for all that are under way.
    Stretch<T> x[AHEAD], tail;
    int block = split * per + wave;
    auto at = [&](int block) { return row + ((int64_t)(block < blocks ? block : blocks - 1) * 64 + lane) * kEach; };
    float top = -__builtin_inff();          // (NaN stays out of it)
    tail.load(row + ((int64_t)blocks * 64 + lane) * kEach, rest);
    if (block < end) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) x[i].load(at(block + i * kBeamWaves));
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (block + i * kBeamWaves < end) top = fmaxf(top, x[i].largest());
    }
    if (rest > 0) top = fmaxf(top, tail.largest());

    // the k-th largest of 64 maxima of eight lanes: as good as that of all the lanes, and one a lane
    tops[wave][lane] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kBeamWaves; ++i) top = fmaxf(top, tops[i][lane]);
    float border = border_of(__builtin_amdgcn_readlane(sorted(ordered_of(top), lane), p.k - 1));

    // Sums are of exp(x - m); m follows the largest x at a distance that keeps them finite.
    float m = -__builtin_inff(), limit = -__builtin_inff();
    double sum = 0.;
    uint64_t key = 0;                       // lane i: the i-th best so far
    int count = 0;                          // of those put down since

    // Takes up what was put down, but for less than 64, or all.
    auto sort_in = [&](bool all) {
        wave_sync();
        int at = 0;
        while (count - at >= 64 || (all && at < count)) {
            const uint64_t y = at + lane < count ? found[wave][at + lane] : 0;
            key = merged(key, reversed(sorted(y, lane), lane), lane);
            at += 64;
        }
        const uint64_t rest = at + lane < count ? found[wave][at + lane] : 0;
        wave_sync();
        found[wave][lane] = rest;
        count = count > at ? count - at : 0;
        if (lane >= p.k) key = 0;
        const uint32_t least = lane_of(key, p.k - 1) >> 32;
        if (least != 0) border = fmaxf(border, border_of(least + 1));
    };
    auto take = [&](const Stretch<T>& x, int block, int left) {
        float v[kEach];
#pragma unroll
        for (int j = 0; j < kEach; ++j) v[j] = x.get(j);
        const float top = x.largest();
        if (__ballot(top > limit)) {
            const float now = top > limit ? top : m;
            sum *= now == m ? 1. : (double)__builtin_amdgcn_exp2f((m - now) * kLog2e);
            limit = top > limit ? top + 32.f : limit;
            m = now;
        }
        const float from = m == -__builtin_inff() ? 0.f : m;
        float part = 0.f;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const float d = v[j] - from;
            part += __builtin_amdgcn_exp2f(__builtin_fmaf(d, kLog2e, d * kLog2eRest));
        }
        sum += (double)part;

        if (!__ballot(top >= border)) return;
        const uint32_t first = ((uint32_t)block * 64 + lane) * kEach;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const bool above = v[j] >= border && j < left;
            const uint64_t with = __ballot(above);
            if (with == 0) continue;
            if (above) {
                const int at = __builtin_amdgcn_mbcnt_hi((uint32_t)(with >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)with, 0));
                found[wave][count + at] = key_of(v[j], first + j);
            }
            count += __popcll(with);
        }
        // (k logits of these and earlier blocks keep out later ones that equal them)
        if (count >= 64) sort_in(false);
    };

    for (; block < end; block += AHEAD * kBeamWaves) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (block + i * kBeamWaves < end) take(x[i], block + i * kBeamWaves, kEach);
            x[i].load(at(block + (i + AHEAD) * kBeamWaves));
        }
    }
    if (__ballot(rest > 0)) take(tail, blocks, rest);
    if (count > 0) sort_in(true);

    // the wave's sum, then the workgroup's
    top = m;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
    sum = m == -__builtin_inff() ? sum : sum * exp2(((double)m - (double)top) * kLog2eD);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
    lists[wave][lane] = key;
    if (lane == 0) stats[wave] = {sum, top, 0};
    for (int n = 1; n < kBeamWaves; n <<= 1) {
        __syncthreads();
        if (wave % (2 * n) == 0) {
            key = merged(key, lists[wave + n][63 - lane], lane);
            lists[wave][lane] = key;
        }
    }
    if (wave != 0) return;
    const int64_t out = r * p.splits + split;
    if (lane < p.k) p.best[out * p.k + lane] = key;
    const BeamStat mine = stats[lane & (kBeamWaves - 1)];
    float all = mine.top;
    static_assert(kBeamWaves == 8, "lanes of a sum");
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) all = fmaxf(all, __shfl_xor(all, d, 64));
    double total = mine.top == -__builtin_inff() ? mine.sum : mine.sum * exp2(((double)mine.top - (double)all) * kLog2eD);
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) total += __shfl_xor(total, d, 64);
    if (lane == 0) p.stat[out] = {total, all, 0};
}

// A continuation as a number: its score's order in the upper 52 bits, below them
// (larger first) beam * 64 + its place among the beam's. Scores that differ by less
// than 2^-40 of themselves are equal by that; what they are the logarithm of has an
// error of 2^-23 already, and the same for equal beams.
static_assert(kMaxBeams * kMaxBest <= 4096, "twelve bits");
__device__ __forceinline__ uint64_t continuation(double score, uint32_t place)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, score + 0.);
    const uint64_t ordered = u >> 63 ? ~u : u | 1ull << 63;
    return (ordered & ~4095ull) | (4095 - place);
}
__device__ __forceinline__ double score_of(uint64_t x)
{
    x &= ~4095ull;
    return __builtin_bit_cast(double, x >> 63 ? x & ~(1ull << 63) : ~x & ~4095ull);
}

// One workgroup a request, one wave a beam at a time. A chain of steps that wait for
// one another: 5 us for 8 beams, 12 for 32 beams in 4 stretches each.
constexpr int kJoinWaves = 16;
__global__ __launch_bounds__(64 * kJoinWaves) void k_beam_join(BeamParams p)
{
    __shared__ int token[kMaxBeams][kMaxBest];
    __shared__ uint64_t lists[kJoinWaves][64];
    __shared__ int owner[64], nth[64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int64_t b = blockIdx.x;
    uint64_t best = 0;
    const int own_row = p.rows != nullptr && lane < p.beams ? p.rows[b * p.beams + lane] : 0;
    for (int w = wave; w < p.beams; w += waves) {
        const int64_t r = b * p.beams + w;
        // at most 64 stretches, one a lane
        const BeamStat mine = lane < p.splits ? p.stat[r * p.splits + lane] : BeamStat{0., -__builtin_inff(), 0};
        const float score = p.scores[r];
        const bool open = p.finished == nullptr || p.finished[r] == 0;
        const uint64_t* from = p.best + r * p.splits * p.k;
        uint64_t key = lane < p.k ? from[lane] : 0;
        for (int i = 1; i < p.splits; i += 4) {
            uint64_t next[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                next[j] = i + j < p.splits && 63 - lane < p.k ? from[(int64_t)(i + j) * p.k + 63 - lane] : 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (lane_of(next[j], 63) > lane_of(key, p.k - 1)) key = merged(key, next[j], lane);
        }
        float top = mine.top;
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
        double sum = mine.top == -__builtin_inff() ? mine.sum : mine.sum * exp2(((double)mine.top - (double)top) * kLog2eD);
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
        const double norm = (double)top + log2(sum) / kLog2eD;
        // (a finished beam goes on by its score, whatever its logits are)
        const bool alive = __builtin_fabsf(score) < __builtin_inff() && (!open || __builtin_fabs(norm) < __builtin_inf());
        uint64_t x = 0;
        int64_t t = lane;
        if (alive && open) {
            t = key != 0 ? (int64_t)(uint32_t)~(uint32_t)key : p.vocab;
            x = continuation((double)score + ((double)logit_of(key) - norm), w * 64 + lane);
        } else if (alive) {
            t = lane == 0 ? p.end_token : lane - 1 + (lane - 1 >= p.end_token);
            x = continuation(lane == 0 ? (double)score : -__builtin_inf(), w * 64 + lane);
        } else {
            x = continuation(-__builtin_inf(), w * 64 + lane);
        }
        if (t >= p.vocab || lane >= p.k) x = 0;
        token[w][lane] = (int)t;
        best = w == wave ? x : merged(best, reversed(x, lane), lane);
    }
    for (int n = 1; n < waves; n <<= 1) {
        lists[wave][lane] = best;
        __syncthreads();
        if (wave % (2 * n) == 0 && wave + n < waves) best = merged(best, lists[wave + n][63 - lane], lane);
        __syncthreads();
    }
    __syncthreads();
    if (wave != 0) return;
    const bool in = best != 0;
    const int place = in ? 4095 - (int)(best & 4095) : 0, parent = place / 64;
    if (lane < p.k) {
        p.out_scores[b * p.k + lane] = in ? (float)score_of(best) : -__builtin_inff();
        p.parents[b * p.k + lane] = parent;
        p.tokens[b * p.k + lane] = in ? token[parent][place % 64] : 0;
    }
    if (p.rows == nullptr) return;
    // k == beams: lane c is continuation c, and beam c
    const uint64_t earlier = lane == 0 ? 0 : ~0ull >> (64 - lane);
    owner[lane] = 64;
    wave_sync();
    if (lane < p.k) atomicMin(&owner[parent], lane);
    wave_sync();
    const bool first = lane < p.k && owner[parent] == lane;
    const uint64_t ended = __ballot(lane < p.beams && owner[lane] == 64), again = __ballot(lane < p.k && !first);
    // the n-th further continuation gets the n-th beam that ends: there are as many of each
    if (ended >> lane & 1) nth[__popcll(ended & earlier)] = lane;
    wave_sync();
    const int kept = __shfl(own_row, parent, 64);
    const int taken = __shfl(own_row, first || lane >= p.k ? parent : nth[__popcll(again & earlier)], 64);
    if (lane < p.k) {
        const int64_t at = b * p.beams;
        p.out_rows[at + lane] = taken;
        p.src[at + lane] = first ? -1 : kept;
        p.dst[at + lane] = first ? -1 : taken;
    }
}

}  // namespace

hipError_t launch_beam_select(const BeamParams& p, int dtype, hipStream_t stream)
{
    const unsigned grid = (unsigned)(p.batch * p.beams * p.splits);
    if (dtype == DWS_FLOAT32)
        k_beam_rows<float><<<grid, 64 * kBeamWaves, 0, stream>>>(p);
    else if (dtype == DWS_BFLOAT16)
        k_beam_rows<bf16_t><<<grid, 64 * kBeamWaves, 0, stream>>>(p);
    else
        k_beam_rows<f16_t><<<grid, 64 * kBeamWaves, 0, stream>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int waves = p.beams < kJoinWaves ? (int)p.beams : kJoinWaves;
    k_beam_join<<<(unsigned)p.batch, 64 * waves, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace dws
