// Small helpers of the C entry points: argument checks and the profiler range
// every entry point opens.
#pragma once

#include <math.h>
#include <nvtx3/nvToolsExt.h>
#include <stdint.h>

namespace sa {

struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
};

inline bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Memory an argument covers: `rows` runs of `bytes`, `stride` bytes apart; none
// where it is NULL.
struct Span {
    const void* p;
    long long bytes, rows, stride;
    Span(const void* p, long long bytes, long long rows = 1, long long stride = 1)
        : p(p), bytes(bytes), rows(rows), stride(stride) {}
};

// Whether a and b have a byte in common.  Two that are both in runs, with unlike
// strides, are compared as if a had no gaps.
inline bool overlap(Span a, Span b) {
    if (a.p == nullptr || b.p == nullptr) return false;
    if (a.rows > 1 && b.rows > 1 && a.stride != b.stride) a = Span(a.p, (a.rows - 1) * a.stride + a.bytes);
    if (a.rows > 1 && b.rows == 1) {
        const Span t = a;
        a = b;
        b = t;
    }
    const long long at = (long long)(reinterpret_cast<uintptr_t>(a.p) - reinterpret_cast<uintptr_t>(b.p));
    // run j of b against run i of a, k = j - i: the first k whose run of b ends past a's first byte
    const long long past = at - b.bytes;
    long long k = (past >= 0 ? past / b.stride : -((b.stride - 1 - past) / b.stride)) + 1;
    if (k < 1 - a.rows) k = 1 - a.rows;
    return k < b.rows && k * b.stride - at < a.bytes;
}

inline float resolve_scale(float scale, int d) { return scale > 0.f ? scale : (float)(1.0 / sqrt((double)d)); }

}  // namespace sa
