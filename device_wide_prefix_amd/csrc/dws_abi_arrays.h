// A call's arrays, to refuse written ones that meet others. Host only.
#pragma once

#include "dws_scan.h"

#include <stdint.h>

namespace dws {

constexpr int64_t kMaxArrayBytes = (int64_t)1 << 50;

// Up to three strided dimensions around a run of `run` bytes; strides and
// counts in bytes and elements. A plain range has none.
struct Strided {
    int64_t stride[3] = {0, 0, 0};
    int64_t count[3] = {1, 1, 1};
    int64_t run = 0;

    __int128 span() const
    {
        __int128 s = run;
        for (int i = 0; i < 3; ++i) s += (__int128)(count[i] - 1) * stride[i];
        return s;
    }
    // Whether no byte is named twice.
    bool distinct() const
    {
        bool used[3] = {false, false, false};
        __int128 inner = run;
        for (int n = 0; n < 3; ++n) {
            int best = -1;
            for (int i = 0; i < 3; ++i)
                if (!used[i] && (best < 0 || stride[i] < stride[best])) best = i;
            used[best] = true;
            if (count[best] <= 1) continue;
            if ((__int128)stride[best] < inner) return false;
            inner += (__int128)(count[best] - 1) * stride[best];
        }
        return true;
    }
    // Bytes modulo `period` that are touched: all lie in [0, result), or -1 if
    // that cannot be said.
    __int128 within(int64_t period) const
    {
        __int128 s = run;
        for (int i = 0; i < 3; ++i)
            if (count[i] > 1 && stride[i] % period != 0) s += (__int128)(count[i] - 1) * stride[i];
        return s <= period ? s : -1;
    }
};

struct Arrays {
    struct One {
        uintptr_t begin, end;
        bool written;
        Strided shape;
    };
    One r[24];
    int n = 0;

    dws_status add(const void* ptr, const Strided& shape, bool written, size_t align)
    {
        if (ptr == nullptr) return DWS_ERR_INVALID_ARG;
        const uintptr_t b = reinterpret_cast<uintptr_t>(ptr);
        if (b % align) return DWS_ERR_MISALIGNED;
        const __int128 bytes = shape.span();
        if (bytes > kMaxArrayBytes || b + (uintptr_t)bytes < b) return DWS_ERR_INVALID_ARG;
        if (written && !shape.distinct()) return DWS_ERR_INVALID_ARG;
        r[n++] = {b, b + (uintptr_t)bytes, written, shape};
        return DWS_OK;
    }
    dws_status add(const void* ptr, int64_t bytes, bool written, size_t align)
    {
        if (bytes == 0) return DWS_OK;
        Strided s;
        s.run = bytes;
        return add(ptr, s, written, align);
    }
    // Two arrays whose ranges meet are still apart where both repeat with one
    // period and lie beside each other within it: parts of one projection's rows,
    // keys and values of one pool.
    static bool beside(const One& a, const One& b)
    {
        for (int i = 0; i < 3; ++i) {
            const int64_t p = a.shape.stride[i];
            if (a.shape.count[i] <= 1 || p <= 0) continue;
            const __int128 wa = a.shape.within(p), wb = b.shape.within(p);
            if (wa < 0 || wb < 0) continue;
            const bool up = b.begin >= a.begin;
            const int64_t far = (int64_t)((up ? b.begin - a.begin : a.begin - b.begin) % (uintptr_t)p);
            const int64_t d = up || far == 0 ? far : p - far;
            if (d >= wa && d + wb <= p) return true;
        }
        return false;
    }
    // Whether runs of two arrays with the same strides and counts meet, b beginning d
    // bytes behind a: in the dimensions from the widest one on, `order`, each wider than
    // all behind it, only the two places next to d can be as near as that.
    static bool meet(__int128 d, const Strided& a, const Strided& b, const int* order, int n)
    {
        if (n == 3) return d < a.run && -d < b.run;
        const __int128 s = a.stride[order[n]], c = a.count[order[n]];
        if (c <= 1) return meet(d, a, b, order, n + 1);
        __int128 k = d / s;
        if (k * s > d) --k;
        for (int i = 0; i < 2; ++i, ++k)
            if (k > -c && k < c && meet(d - k * s, a, b, order, n + 1)) return true;
        return false;
    }
    static bool interleaved(const One& a, const One& b)
    {
        Strided widest = a.shape;
        widest.run = a.shape.run > b.shape.run ? a.shape.run : b.shape.run;
        if (!widest.distinct()) return false;
        for (int i = 0; i < 3; ++i)
            if (a.shape.count[i] != b.shape.count[i] || (a.shape.count[i] > 1 && (a.shape.stride[i] != b.shape.stride[i] || a.shape.stride[i] <= 0)))
                return false;
        int order[3] = {0, 1, 2};
        for (int i = 0; i < 2; ++i)
            for (int j = 0; j < 2 - i; ++j)
                if (a.shape.stride[order[j]] < a.shape.stride[order[j + 1]]) {
                    const int t = order[j];
                    order[j] = order[j + 1];
                    order[j + 1] = t;
                }
        const __int128 d = (__int128)b.begin - (__int128)a.begin;
        return !meet(d, a.shape, b.shape, order, 0);
    }
    bool overlap() const
    {
        for (int i = 0; i < n; ++i)
            for (int j = 0; j < i; ++j)
                if ((r[i].written || r[j].written) && r[i].begin < r[j].end && r[j].begin < r[i].end &&
                    !beside(r[i], r[j]) && !beside(r[j], r[i]) && !interleaved(r[i], r[j]))
                    return true;
        return false;
    }
};

}  // namespace dws
