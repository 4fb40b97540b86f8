// plan_util.h -- host helpers of the entry points that keep plans over
// separate tensors: error reports, alignment and overlap checks, the guard
// against C++ exceptions, and the key of the stochastic rounding.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <new>
#include <vector>

#include "fp_internal.h"

namespace fpk {
namespace {

fp_status bad(fp_status st, const char* fmt, ...) {
    char text[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    return report_error(st, text);
}

fp_status device_error(hipError_t e, const char* what) {
    return bad(FP_ERR_DEVICE, "%s: %s", what, hipGetErrorString(e));
}

bool on(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Bytes [lo, hi) of a buffer.
struct Span {
    uintptr_t lo, hi;
    bool operator<(const Span& o) const { return lo < o.lo; }
};

Span span_of(const void* p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, a + (uintptr_t)bytes};
}

bool meet(const Span& a, const Span& b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

// Sorted, disjoint spans that cover the same bytes (touching ones joined).
std::vector<Span> joined(std::vector<Span> v) {
    std::sort(v.begin(), v.end());
    std::vector<Span> r;
    for (const Span& s : v) {
        if (s.lo >= s.hi) continue;
        if (!r.empty() && s.lo <= r.back().hi) r.back().hi = std::max(r.back().hi, s.hi);
        else r.push_back(s);
    }
    return r;
}

bool meets_any(const Span& a, const std::vector<Span>& sorted) {
    if (a.lo >= a.hi) return false;
    auto it = std::upper_bound(sorted.begin(), sorted.end(), a);
    if (it != sorted.end() && meet(a, *it)) return true;
    return it != sorted.begin() && meet(a, *(it - 1));
}

// Runs `f`; no C++ exception leaves an entry point.
template <class F>
fp_status guarded(F f) {
    try {
        return f();
    } catch (const std::bad_alloc&) {
        return bad(FP_ERR_DEVICE, "out of host memory");
    } catch (...) {
        return bad(FP_ERR_DEVICE, "unexpected host error");
    }
}

// The stochastic rounding's key: the seed through two rounds of
// multiplication, so that seeds that count steps give unrelated keys.  The
// first multiplier is 2^64 over the golden ratio; the second, with the shifts by
// 32 around it, is the published 64-bit integer mixer known as degski's.
uint32_t key_of(uint64_t seed) {
    uint64_t z = seed * 0x9E3779B97F4A7C15ull;
    z ^= z >> 32;
    z *= 0xD6E8FEB86659FD93ull;
    return (uint32_t)(z ^ (z >> 32));
}

}  // namespace
}  // namespace fpk
