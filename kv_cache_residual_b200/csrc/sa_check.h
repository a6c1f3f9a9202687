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

inline float resolve_scale(float scale, int d) { return scale > 0.f ? scale : (float)(1.0 / sqrt((double)d)); }

}  // namespace sa
