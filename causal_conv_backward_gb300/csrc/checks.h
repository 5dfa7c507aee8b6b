// checks.h - argument checks that the entry points share: shapes, strides,
// alignment, workspaces, and outputs that overlap what a call reads.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <initializer_list>

#include "plan.h"

namespace mcc1d {

constexpr int64_t kMaxS = (int64_t)1 << 31, kMaxB = 65535, kMaxH = (int64_t)1 << 20, kMaxGrid = 0x7FFFFFFF;

inline bool shape_ok(int64_t S, int64_t B, int64_t H)
{
    return S >= 1 && S <= kMaxS - 4096 && B >= 1 && B <= kMaxB && H >= 1 && H <= kMaxH;
}

template <int N>
bool strides_ok(const int64_t (&s)[N])
{
    for (int i = 0; i < N; ++i)
        if (s[i] < 0)
            return false;
    return true;
}

// Every pointer on its element's size (null passes).
inline bool on2(std::initializer_list<const void *> ps)
{
    for (const void *p : ps)
        if ((uintptr_t)p & 1u)
            return false;
    return true;
}

inline bool on4(std::initializer_list<const void *> ps)
{
    for (const void *p : ps)
        if ((uintptr_t)p & 3u)
            return false;
    return true;
}

inline int32_t check_workspace(const void *ws, uint64_t have, uint64_t need)
{
    if (need == 0)
        return kOk;
    if (!ws)
        return kErrNull;
    if ((uintptr_t)ws & 15u)
        return kErrInvalid;
    return have < need ? kErrWorkspace : kOk;
}

// What a call reads: rows of `row` bytes at `at`, repeated `count` times `step`
// bytes apart along up to three axes. Dense memory is one row. Null is nothing.
struct Region {
    struct Axis {
        int64_t count;
        uint64_t step;
    };
    uintptr_t at;
    uint64_t row;
    int axes;
    Axis axis[3];       // by falling step

    Region(const void *p, int64_t bytes) : at((uintptr_t)p), row(p ? (uint64_t)bytes : 0), axes(0) {}
    // rows of n elements of `size` bytes, strides in elements
    Region(const void *p, int64_t n, std::initializer_list<Axis> a, uint64_t size = 2)
        : at((uintptr_t)p), row(p ? size * (uint64_t)n : 0), axes(0)
    {
        for (const Axis &x : a)
            if (x.count > 1 && x.step > 0)
                axis[axes++] = {x.count, size * x.step};
        std::sort(axis, axis + axes, [](const Axis &x, const Axis &y) { return x.step > y.step; });
    }
    // Whether a byte of lo..hi-1 is read.
    bool meets(uintptr_t lo, uintptr_t hi) const { return row > 0 && lo < hi && meets(lo, hi, 0, at); }

private:
    bool meets(uintptr_t lo, uintptr_t hi, int k, uintptr_t from) const
    {
        if (k >= axes || k >= 3)
            return from < hi && from + row > lo;
        uint64_t inner = row;       // from an index of axis k to the end of its last row
        for (int j = k + 1; j < axes; ++j)
            inner += (uint64_t)(axis[j].count - 1) * axis[j].step;
        if (from >= hi)
            return false;
        const uint64_t first = lo >= from + inner ? (lo - from - inner) / axis[k].step + 1 : 0;
        const uint64_t last = std::min<uint64_t>((uint64_t)axis[k].count - 1, (hi - 1 - from) / axis[k].step);
        for (uint64_t i = first; i <= last; ++i)
            if (meets(lo, hi, k + 1, from + i * axis[k].step))
                return true;
        return false;
    }
};

// What a call writes: dense memory.
struct Written {
    uintptr_t lo, hi;
    Written(const void *p, int64_t bytes) : lo((uintptr_t)p), hi(p ? lo + (uint64_t)bytes : lo) {}
    bool meets(const Written &w) const { return lo < hi && w.lo < w.hi && lo < w.hi && w.lo < hi; }
};

// No output on an input or on another output.
inline int32_t apart(std::initializer_list<Written> out, std::initializer_list<Region> in)
{
    for (const Written *o = out.begin(); o != out.end(); ++o) {
        for (const Written *q = out.begin(); q != o; ++q)
            if (o->meets(*q))
                return kErrInvalid;
        for (const Region &r : in)
            if (r.meets(o->lo, o->hi))
                return kErrInvalid;
    }
    return kOk;
}

}  // namespace mcc1d
