// Beam search's selection: the k best of score[beam] + log softmax(logits[beam])
// [token] over a request's beams and the vocabulary.
//
// Within a beam the order is that of the logits, so one pass over them (their bytes
// bound it) finds both the sum of the exponentials and the k largest; only the k of
// each beam are then compared across beams, in fp64. A wave keeps the best so far
// sorted, one a lane; a block of logits is looked at again only if one of them is
// above the k-th, which happens k log(blocks) times.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dws_beam.h"

namespace dws {
namespace {

typedef __bf16 bf16_t;
typedef _Float16 f16_t;
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kEach = kBeamBlock / 64;      // logits of a lane's chunk

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
__device__ __forceinline__ uint64_t lane_of(uint64_t x, int lane)
{
    return (uint64_t)__builtin_amdgcn_readlane((uint32_t)(x >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((uint32_t)x, lane);
}

// One step of a descending bitonic network: of two lanes the lower (`up`: the
// upper) one keeps the larger.
__device__ __forceinline__ uint64_t exchange(uint64_t x, int lane, int d, bool up)
{
    const uint64_t y = __shfl_xor(x, d, 64);
    const bool larger = ((lane & d) == 0) != up;
    return (x > y) == larger ? x : y;
}
__device__ __forceinline__ uint64_t sorted(uint64_t x, int lane)
{
#pragma unroll
    for (int n = 2; n <= 64; n <<= 1)
#pragma unroll
        for (int d = n / 2; d > 0; d >>= 1) x = exchange(x, lane, d, (lane & n) != 0 && n < 64);
    return x;
}
// The 64 best of two descending lists, the second given backwards.
__device__ __forceinline__ uint64_t merged(uint64_t x, uint64_t backwards, int lane)
{
    x = x > backwards ? x : backwards;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x = exchange(x, lane, d, false);
    return x;
}

template <class T>
struct Stretch {
    static constexpr int VEC = 16 / sizeof(T), LOADS = kEach / VEC;
    typedef T Vec __attribute__((ext_vector_type(VEC)));
    u32x4_t raw[LOADS];

    // Elements first .. first + 7 of a row, which may start anywhere: with chunks that
    // went by addresses, rows of equal logits would be summed in different orders, and
    // equal beams would not tie.
    __device__ __forceinline__ void load(const T* row, int64_t first, int64_t vocab)
    {
        if (first + kEach <= vocab) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) __builtin_memcpy(&raw[i], row + first + i * VEC, 16);
        } else {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                Vec x;
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const int64_t e = first + i * VEC + j;
                    x[j] = e < vocab ? row[e] : (T)-__builtin_inff();
                }
                raw[i] = __builtin_bit_cast(u32x4_t, x);
            }
        }
    }
    __device__ __forceinline__ float get(int j) const { return (float)__builtin_bit_cast(Vec, raw[j / VEC])[j % VEC]; }
};

template <class T>
__global__ __launch_bounds__(64 * kWaves) void k_beam_rows(BeamParams p)
{
    constexpr int AHEAD = sizeof(T) == 2 ? 4 : 2;       // blocks in flight
    __shared__ uint64_t lists[kWaves][64];
    __shared__ BeamStat stats[kWaves];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t r = blockIdx.x / p.splits;
    const int split = blockIdx.x % p.splits;
    const T* row = static_cast<const T*>(p.logits) + r / p.beams * p.batch_stride + r % p.beams * p.beam_stride;
    const int64_t blocks = (p.vocab + kBeamBlock - 1) / kBeamBlock;
    const int64_t per = (blocks + p.splits - 1) / p.splits;
    const int64_t end = split * per + per < blocks ? split * per + per : blocks;

    float m = -__builtin_inff();
    double sum = 0.;
    uint64_t key = 0, least = 0;            // lane i: the i-th best; the k-th
    float border = -__builtin_inff();       // its logit
    bool full = false;

    auto take = [&](const Stretch<T>& x, int64_t block) {
        const int64_t first = (block * 64 + lane) * kEach;
        const int count = p.vocab - first < kEach ? (int)(p.vocab - first) : kEach;             // may be negative
        float v[kEach];
#pragma unroll
        for (int j = 0; j < kEach; ++j) v[j] = x.get(j);
        float top = v[0];
#pragma unroll
        for (int j = 1; j < kEach; ++j) top = fmaxf(top, v[j]);
        if (__ballot(top > m)) {
            const float now = fmaxf(m, top);
            sum *= now == m ? 1. : (double)__builtin_amdgcn_exp2f((m - now) * 1.44269504088896f);
            m = now;
        }
        // exp(x - m) as 2^y: log2(e) in two parts, since a common error of all terms would not average out
        const float base = m == -__builtin_inff() ? 0.f : m;
        float part = 0.f;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const float d = v[j] - base;
            part += __builtin_amdgcn_exp2f(__builtin_fmaf(d, 1.44269502162933349609f, d * 1.9259629911266e-8f));
        }
        sum += (double)part;

        if (!__ballot(full ? top > border : count > 0)) return;
        uint64_t mine[kEach];
#pragma unroll
        for (int j = 0; j < kEach; ++j)
            mine[j] = j < count && v[j] == v[j] ? key_of(v[j], (uint32_t)(first + j)) : 0;
        if (least == 0 && lane_of(key, 0) == 0) {
            // the first block: the lanes' best ones, sorted, are most of the list
            uint64_t best = 0;
#pragma unroll
            for (int j = 0; j < kEach; ++j) best = mine[j] > best ? mine[j] : best;
#pragma unroll
            for (int j = 0; j < kEach; ++j) mine[j] = mine[j] == best ? 0 : mine[j];
            key = sorted(best, lane);
            if (lane >= p.k) key = 0;
            least = lane_of(key, p.k - 1);
        }
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            uint64_t left = __ballot(mine[j] > least);
            while (left != 0) {
                const int from_lane = __builtin_ctzll(left);
                const uint64_t x = lane_of(mine[j], from_lane);
                const int place = __popcll(__ballot(key > x));
                const uint64_t up = __shfl_up(key, 1, 64);
                key = lane < place ? key : (lane == place ? x : up);
                if (lane >= p.k) key = 0;
                least = lane_of(key, p.k - 1);
                left &= left - 1;
                left &= __ballot(mine[j] > least);
            }
        }
        full = least != 0;
        border = full ? logit_of(least) : -__builtin_inff();
    };

    Stretch<T> x[AHEAD];
    int64_t block = split * per + wave;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (block + i * kWaves < end) x[i].load(row, ((block + i * kWaves) * 64 + lane) * kEach, p.vocab);
    while (block < end) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (block >= end) break;
            const Stretch<T> now = x[i];
            const int64_t next = block + AHEAD * kWaves;
            if (next < end) x[i].load(row, (next * 64 + lane) * kEach, p.vocab);
            take(now, block);
            block += kWaves;
        }
    }

    // the wave's sum, then the workgroup's
    float top = m;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
    sum = m == -__builtin_inff() ? sum : sum * exp((double)m - (double)top);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
    lists[wave][lane] = key;
    if (lane == 0) stats[wave] = {sum, top, 0};
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (int w = 1; w < kWaves; ++w) key = merged(key, lists[w][63 - lane], lane);
    const int64_t out = r * p.splits + split;
    if (lane < p.k) p.best[out * p.k + lane] = key;
    if (lane == 0) {
        float all = stats[0].top;
        for (int w = 1; w < kWaves; ++w) all = fmaxf(all, stats[w].top);
        double total = 0.;
        for (int w = 0; w < kWaves; ++w)
            total += stats[w].top == -__builtin_inff() ? stats[w].sum : stats[w].sum * exp((double)stats[w].top - (double)all);
        p.stat[out] = {total, all, 0};
    }
}

// A continuation: its score, and beam * 64 + its place among the beam's, which
// breaks ties.
struct Best {
    double score;
    uint32_t tie;
};
__device__ __forceinline__ bool before(const Best& a, const Best& b)
{
    return a.score > b.score || (a.score == b.score && a.tie < b.tie);
}
__device__ __forceinline__ Best merged(Best x, Best backwards, int lane)
{
    if (before(backwards, x)) x = backwards;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const Best y{__shfl_xor(x.score, d, 64), (uint32_t)__shfl_xor((int)x.tie, d, 64)};
        if (((lane & d) == 0) == before(y, x)) x = y;
    }
    return x;
}

// One workgroup a request, one wave a beam at a time.
constexpr int kJoinWaves = 8;
__global__ __launch_bounds__(64 * kJoinWaves) void k_beam_join(BeamParams p)
{
    __shared__ int token[kMaxBeams][kMaxBest];
    __shared__ Best lists[kJoinWaves][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int64_t b = blockIdx.x;
    const double none = -__builtin_inf();
    Best best{none, 0xffffffffu};
    for (int w = wave; w < p.beams; w += waves) {
        const int64_t r = b * p.beams + w;
        // at most 64 stretches, one a lane
        const BeamStat mine = lane < p.splits ? p.stat[r * p.splits + lane] : BeamStat{0., -__builtin_inff(), 0};
        float top = mine.top;
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
        double sum = mine.top == -__builtin_inff() ? mine.sum : mine.sum * exp((double)mine.top - (double)top);
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
        const float score = p.scores[r];
        const double norm = (double)top + log(sum);
        const bool alive = __builtin_fabs(norm) < __builtin_inf() && __builtin_fabsf(score) < __builtin_inff();
        Best x{none, (uint32_t)(w * 64 + lane)};
        int64_t t = lane;
        if (alive && (p.finished == nullptr || p.finished[r] == 0)) {
            const uint64_t* from = p.best + r * p.splits * p.k;
            uint64_t key = lane < p.k ? from[lane] : 0;
            for (int i = 1; i < p.splits; ++i) {
                const uint64_t next = 63 - lane < p.k ? from[(int64_t)i * p.k + 63 - lane] : 0;
                if (lane_of(next, 63) > lane_of(key, p.k - 1)) key = merged(key, next, lane);
            }
            t = key != 0 ? (int64_t)(uint32_t)~(uint32_t)key : p.vocab;
            if (key != 0) x.score = (double)score + ((double)logit_of(key) - norm);
        } else if (alive) {
            t = lane == 0 ? p.end_token : lane - 1 + (lane - 1 >= p.end_token);
            if (lane == 0) x.score = score;
        }
        if (t >= p.vocab || lane >= p.k) x = Best{none, 0xffffffffu};
        token[w][lane] = (int)t;
        const Best back{__shfl(x.score, 63 - lane, 64), (uint32_t)__shfl((int)x.tie, 63 - lane, 64)};
        best = merged(best, back, lane);
    }
    for (int n = 1; n < waves; n <<= 1) {
        lists[wave][lane] = best;
        __syncthreads();
        if (wave % (2 * n) == 0 && wave + n < waves) best = merged(best, lists[wave + n][63 - lane], lane);
        __syncthreads();
    }
    __syncthreads();
    if (wave != 0) return;
    const bool in = lane < p.k && best.tie != 0xffffffffu;
    const int parent = in ? (int)(best.tie / 64) : 0;
    if (lane < p.k) {
        p.out_scores[b * p.k + lane] = (float)best.score;
        p.parents[b * p.k + lane] = parent;
        p.tokens[b * p.k + lane] = in ? token[parent][best.tie % 64] : 0;
    }
    if (p.rows == nullptr) return;
    // k == beams: lane c is continuation c, and beam c
    const uint64_t earlier = lane == 0 ? 0 : ~0ull >> (64 - lane);
    bool first = false, ends = false;
    for (int w = 0; w < p.beams; ++w) {
        const uint64_t with = __ballot(lane < p.k && parent == w);
        if (parent == w) first = (with & earlier) == 0;
        if (lane == w) ends = with == 0;
    }
    const uint64_t ended = __ballot(lane < p.beams && ends), again = __ballot(lane < p.k && !first);
    // the n-th further continuation gets the n-th beam that ends: there are as many of each
    const int rank = __popcll(again & earlier);
    uint64_t left = ended;
    for (int i = 0; i < rank; ++i) left &= left - 1;
    if (lane < p.k) {
        const int64_t at = b * p.beams;
        const int kept = p.rows[at + parent];
        const int now = first || left == 0 ? kept : p.rows[at + __builtin_ctzll(left)];
        p.out_rows[at + lane] = now;
        p.src[at + lane] = first ? -1 : kept;
        p.dst[at + lane] = first ? -1 : now;
    }
}

}  // namespace

hipError_t launch_beam_select(const BeamParams& p, int dtype, hipStream_t stream)
{
    const unsigned grid = (unsigned)(p.batch * p.beams * p.splits);
    if (dtype == DWS_FLOAT32)
        k_beam_rows<float><<<grid, 64 * kWaves, 0, stream>>>(p);
    else if (dtype == DWS_BFLOAT16)
        k_beam_rows<bf16_t><<<grid, 64 * kWaves, 0, stream>>>(p);
    else
        k_beam_rows<f16_t><<<grid, 64 * kWaves, 0, stream>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int waves = p.beams < kJoinWaves ? (int)p.beams : kJoinWaves;
    k_beam_join<<<(unsigned)p.batch, 64 * waves, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace dws
