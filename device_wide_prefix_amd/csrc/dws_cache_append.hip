// Keys and values of new tokens into the pages of a cache, keys and queries
// turned by their positions on the way:
//   (a, b) -> (a cos x - b sin x, a sin x + b cos x),  x = position * freqs[pair]
// Each byte is read once and written once, so memory bounds large calls (16,384
// tokens) and the chain of dependent loads (offset, row, length, page) small ones.
// One wave takes a token: it finds the token's place with one trip to memory a
// link, works out the angles once for all heads, and then streams the heads.
#include "dws_cache_device.hpp"

namespace dws {
namespace {

constexpr int kMaxPairs = 128;

// cos and sin of position * freq. A product of a 31-bit and a 24-bit number has up to 55
// bits, and 2^-53 of far positions' angles is several units of fp32: so the angle and
// 1 / (2 pi) are two fp64 numbers each, and the whole turns go before anything is rounded.
// The rest of the rounding to fp32 enters through the first order, so that both are as good
// as fp32 holds them, however far the position.
__device__ __forceinline__ float2 turn_of(int position, float freq)
{
    constexpr double kTurn = 0.15915494309189535, kTurnRest = -9.839338337591243e-18;    // 1 / (2 pi)
    const double angle = (double)position * (double)freq;
    const double angle_rest = __builtin_fma((double)position, (double)freq, -angle);
    const double turns = __builtin_fma(angle, kTurn, -rint(angle * kTurn));
    const double half = 2.0 * (turns + __builtin_fma(angle, kTurnRest, angle_rest * kTurn));     // half turns, -1 .. 1
    const float x = (float)half;
    const float rest = (float)(half - (double)x) * 3.14159265358979f;
    float s, c;
    sincospif(x, &s, &c);
    return make_float2(__builtin_fmaf(-rest, s, c), __builtin_fmaf(rest, c, s));
}

// E: elements of a load, a whole 16 bytes or one. A unit is what a lane turns at
// a time: E pairs (E / 2 adjacent ones), or E elements that stay as they are.
template <class T, int E, bool ADJACENT>
struct Unit {
    typedef T Vec __attribute__((ext_vector_type(E)));
    static constexpr bool kTwo = !ADJACENT || E == 1;       // a pair's halves come in two loads
    static constexpr int kPairs = E == 1 ? 1 : (ADJACENT ? E / 2 : E);

    Vec a, b;
    __device__ __forceinline__ void load(const T* src, int u, int turned, int pairs)
    {
        if (u < turned) {
            if constexpr (E == 1) {
                a = src[ADJACENT ? 2 * u : u];
                b = src[ADJACENT ? 2 * u + 1 : u + pairs];
            } else if constexpr (ADJACENT) {
                a = *reinterpret_cast<const Vec*>(src + u * E);
            } else {
                a = *reinterpret_cast<const Vec*>(src + u * E);
                b = *reinterpret_cast<const Vec*>(src + pairs + u * E);
            }
        } else {
            a = *reinterpret_cast<const Vec*>(src + 2 * pairs + (u - turned) * E);
        }
    }
    __device__ __forceinline__ void store(T* dst, int u, int turned, int pairs, const float2* turn)
    {
        if (u >= turned) {
            *reinterpret_cast<Vec*>(dst + 2 * pairs + (u - turned) * E) = a;
            return;
        }
        if constexpr (E > 1 && ADJACENT) {
#pragma unroll
            for (int j = 0; j < E / 2; ++j) {
                const float2 t = turn[u * (E / 2) + j];
                const float x = (float)a[2 * j], y = (float)a[2 * j + 1];
                a[2 * j] = (T)(x * t.x - y * t.y);
                a[2 * j + 1] = (T)(x * t.y + y * t.x);
            }
            *reinterpret_cast<Vec*>(dst + u * E) = a;
        } else {
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const float2 t = turn[u * E + j];
                const float x = (float)a[j], y = (float)b[j];
                a[j] = (T)(x * t.x - y * t.y);
                b[j] = (T)(x * t.y + y * t.x);
            }
            if constexpr (E == 1) {
                dst[ADJACENT ? 2 * u : u] = a[0];
                dst[ADJACENT ? 2 * u + 1 : u + pairs] = b[0];
            } else {
                *reinterpret_cast<Vec*>(dst + u * E) = a;
                *reinterpret_cast<Vec*>(dst + pairs + u * E) = b;
            }
        }
    }
};

// A lane's place in heads of `size` units each, 64 units further at a step.
struct Place {
    int head, unit;
    int heads_step, units_step, size;
    __device__ __forceinline__ Place(int size, int lane) : size(size)
    {
        head = lane / size;
        unit = lane - head * size;
        heads_step = 64 / size;
        units_step = 64 - heads_step * size;
    }
    __device__ __forceinline__ void next()
    {
        head += heads_step;
        unit += units_step;
        if (unit >= size) {
            unit -= size;
            ++head;
        }
    }
};

template <class T, int E, bool ADJACENT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_pages_append(AppendParams p)
{
    __shared__ float2 turns[WAVES][kMaxPairs];
    typedef typename Unit<T, E, ADJACENT>::Vec Vec;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * WAVES + wave;
    if (t >= p.c.tokens) return;
    const KvView& c = p.c;

    int64_t first = 0, count = 0;
    const int64_t seq = seq_of(c, t, &first, &count, lane);
    bool in = seq >= 0;
    int64_t row = in ? (c.rows != nullptr ? c.rows[seq] : seq) : -1;
    in = in && row >= 0 && row < c.n_rows && (p.granted == nullptr || p.granted[seq] != 0);
    const int64_t length = in ? c.lengths[row] : 0;
    if (in && c.rows != nullptr) {
        bool again = false;
        for (int64_t j = lane; j < seq; j += 4 * 64) {
            int other[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) other[u] = c.rows[j + u * 64 < seq ? j + u * 64 : seq];
#pragma unroll
            for (int u = 0; u < 4; ++u) again |= j + u * 64 < seq && other[u] == (int)row;
        }
        in = __ballot(again) == 0;
    }
    in = in && count <= length && length <= c.max_pages * c.page_tokens;
    T* q_out = static_cast<T*>(p.q_out.data) + t * p.q_out.ts;
    if (!in) {
        if (p.zero_rest)
            for (int64_t u = lane; u < (int64_t)p.heads_q * c.dim_k; u += 64)
                q_out[u / c.dim_k * p.q_out.hs + u % c.dim_k] = (T)0.f;
        return;
    }
    const int at = (int)(length - count + (t - first));
    const int page = c.table[row * c.max_pages + at / c.page_tokens], place = at % c.page_tokens;
    const bool write = page >= 0 && page < c.n_pages;

    float2* turn = turns[wave];
    if (p.pairs > 0) {
        const int position = p.positions != nullptr ? p.positions[t] : at;
        for (int j = lane; j < p.pairs; j += 64) turn[j] = turn_of(position, p.freqs[j]);
    }
    wave_sync();

    const T* q = static_cast<const T*>(p.q.data) + t * p.q.ts;
    const T* k = static_cast<const T*>(p.k.data) + t * p.k.ts;
    const T* v = static_cast<const T*>(p.v.data) + t * p.v.ts;
    T* keys = static_cast<T*>(c.keys.data) + page * c.keys.ps + place * c.keys.ts;
    T* values = static_cast<T*>(c.values.data) + page * c.values.ps + place * c.values.ts;

    // queries, then keys; four units in flight a lane
    const int turned = p.pairs / Unit<T, E, ADJACENT>::kPairs;
    const int heads = p.heads_q + (write ? c.heads : 0);
    Place at_unit(turned + (c.dim_k - 2 * p.pairs) / E, lane);
    while (at_unit.head < heads) {
        Unit<T, E, ADJACENT> unit[4];
        const T* src[4];
        T* dst[4];
        int which[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int h = at_unit.head, hk = h - p.heads_q;
            which[i] = at_unit.unit;
            src[i] = hk < 0 ? q + h * p.q.hs : k + hk * p.k.hs;
            dst[i] = h >= heads ? nullptr : (hk < 0 ? q_out + h * p.q_out.hs : keys + hk * c.keys.hs);
            if (dst[i] != nullptr) unit[i].load(src[i], which[i], turned, p.pairs);
            at_unit.next();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (dst[i] != nullptr) unit[i].store(dst[i], which[i], turned, p.pairs, turn);
    }
    if (!write) return;
    Place at_value(c.dim_v / E, lane);
    while (at_value.head < c.heads) {
        Vec x[4];
        T* dst[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            dst[i] = at_value.head < c.heads ? values + at_value.head * c.values.hs + at_value.unit * E : nullptr;
            if (dst[i] != nullptr) x[i] = *reinterpret_cast<const Vec*>(v + at_value.head * p.v.hs + at_value.unit * E);
            at_value.next();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (dst[i] != nullptr) *reinterpret_cast<Vec*>(dst[i]) = x[i];
    }
}

template <class T, int E, int WAVES>
void launch_as(const AppendParams& p, hipStream_t stream)
{
    const dim3 grid((unsigned)((p.c.tokens + WAVES - 1) / WAVES)), block(64 * WAVES);
    if (p.adjacent)
        k_pages_append<T, E, true, WAVES><<<grid, block, 0, stream>>>(p);
    else
        k_pages_append<T, E, false, WAVES><<<grid, block, 0, stream>>>(p);
}
template <class T>
void launch_of(const AppendParams& p, hipStream_t stream)
{
    // workgroups of one wave while that leaves compute units with few tokens
    constexpr int E = 16 / sizeof(T);
    if (p.c.tokens < 4096) {
        if (p.whole)
            launch_as<T, E, 1>(p, stream);
        else
            launch_as<T, 1, 1>(p, stream);
    } else {
        if (p.whole)
            launch_as<T, E, 4>(p, stream);
        else
            launch_as<T, 1, 4>(p, stream);
    }
}

}  // namespace

hipError_t launch_pages_append(const AppendParams& p, int dtype, hipStream_t stream)
{
    if (dtype == DWS_FLOAT32)
        launch_of<float>(p, stream);
    else if (dtype == DWS_BFLOAT16)
        launch_of<bf16_t>(p, stream);
    else
        launch_of<f16_t>(p, stream);
    return hipGetLastError();
}

}  // namespace dws
