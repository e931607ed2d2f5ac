// host_checks.h -- argument checks that the C entry points share.
#pragma once

#include <stdint.h>

#include <initializer_list>

namespace {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A range of memory a call reads or writes (null: none).
struct Range {
    const void *p;
    int64_t bytes;
};
inline bool meet(const Range &a, const Range &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.bytes > 0 && b.bytes > 0 &&
           (x < y ? y - x < (uintptr_t)a.bytes : x - y < (uintptr_t)b.bytes);
}
// Whether each of outs is apart from every one of ins and from the other outs.
inline bool apart(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (const Range *o = outs.begin(); o != outs.end(); ++o) {
        for (const Range &i : ins)
            if (meet(*o, i)) return false;
        for (const Range *p = o + 1; p != outs.end(); ++p)
            if (meet(*o, *p)) return false;
    }
    return true;
}

}  // namespace
