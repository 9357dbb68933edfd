// Whether strided tensors share memory: host checks of the decode operators, plain C++.
#pragma once

#include <cstdint>

namespace ks {

// Runs of `run` contiguous bytes, repeated along up to three axes. Counts are at least 1, strides are
// in bytes and not negative; an axis of one entry, or of stride 0, adds no bytes.
struct Strided {
    const void *p;
    int64_t run;
    int64_t count[3];
    int64_t stride[3];
    int64_t step(int k) const { return count[k] > 1 ? stride[k] : 0; }
};

// The axes by falling stride (the larger of both tensors').
struct StridedOrder {
    int axis[3] = {0, 1, 2};
    StridedOrder(const Strided &x, const Strided &y) {
        auto key = [&](int k) { return x.step(k) > y.step(k) ? x.step(k) : y.step(k); };
        for (int i = 0; i < 2; ++i)
            for (int j = 0; j < 2 - i; ++j)
                if (key(axis[j]) < key(axis[j + 1])) {
                    const int t = axis[j];
                    axis[j] = axis[j + 1];
                    axis[j + 1] = t;
                }
    }
};

// Bytes from the first to past the last of the axes from order.axis[at] on.
inline int64_t strided_span(const Strided &v, const StridedOrder &o, int at = 0) {
    int64_t n = v.run;
    for (int i = at; i < 3; ++i) n += (v.count[o.axis[i]] - 1) * v.step(o.axis[i]);
    return n;
}

// Whether a tensor's runs are apart: each axis steps over all that lies within it.
inline bool strided_rows_apart(const Strided &v) {
    const StridedOrder o(v, v);
    for (int i = 0; i < 3; ++i)
        if (v.count[o.axis[i]] > 1 && v.step(o.axis[i]) < strided_span(v, o, i + 1)) return false;
    return true;
}

// The same for what the axes from `at` on make of x and of y, which begins d bytes behind x. Along an
// axis that both step alike, y's entry lies d - i * step behind x's for some distance i of their
// indices, and few such distances bring them near each other: those are looked into, so that parts of
// one tensor that alternate at any level come out apart. Different steps: what lies between the first
// and last byte counts as shared.
inline bool strided_cross(const Strided &x, const Strided &y, const StridedOrder &o, int at, int64_t d) {
    if (d >= strided_span(x, o, at) || -d >= strided_span(y, o, at)) return false;
    if (at == 3) return true;
    const int k = o.axis[at];
    const int64_t sx = x.step(k), sy = y.step(k), s = sx > sy ? sx : sy;
    if (s == 0) return strided_cross(x, y, o, at + 1, d);
    if (sx && sy && sx != sy) return true;
    const int64_t nx = strided_span(x, o, at + 1), ny = strided_span(y, o, at + 1);
    const int64_t lowest = sy ? 1 - y.count[k] : 0, highest = sx ? x.count[k] - 1 : 0;
    // -ny < d - i s < nx
    auto floor_div = [](int64_t a, int64_t b) { return a / b - (a % b < 0); };
    int64_t first = floor_div(d - nx, s) + 1, last = -floor_div(-(d + ny), s) - 1;
    if (first < lowest) first = lowest;
    if (last > highest) last = highest;
    if (last - first > 8) return true;  // axes that do not nest
    for (int64_t i = first; i <= last; ++i)
        if (strided_cross(x, y, o, at + 1, d - i * s)) return true;
    return false;
}

// Whether two tensors share a byte. Spans are below 2^62 bytes.
inline bool strided_cross(const Strided &x, const Strided &y) {
    const StridedOrder o(x, y);
    const uintptr_t px = (uintptr_t)x.p, py = (uintptr_t)y.p;
    if (py >= px ? py - px >= (uintptr_t)strided_span(x, o) : px - py >= (uintptr_t)strided_span(y, o)) return false;
    return strided_cross(x, y, o, 0, py >= px ? (int64_t)(py - px) : -(int64_t)(px - py));
}

}  // namespace ks
