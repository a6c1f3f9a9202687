// Device code the paged cache's kernels share: where a slot's row lies, which
// slots a query sees, and the even split of all units' tiles over the CTAs.
#pragma once

#include "sa_common.cuh"
#include "sa_paged.h"

namespace sa {

__device__ __forceinline__ int pg_length(const PagedView& c, int b) {
    return min(max(__ldg(c.lengths + b), 0), c.cap);
}

// newest position of sequence b
__device__ __forceinline__ int pg_newest(const PagedView& c, int b, int len) {
    return (c.seen != nullptr ? __ldg(c.seen + b) : len) - 1;
}

__device__ __forceinline__ int pg_col(const PagedView& c, int slot) {
    return c.shift >= 0 ? slot >> c.shift : slot / c.page;
}

// element offset of (slot, head), its page read from the table before, or -1
// where that is not one of the pool
__device__ __forceinline__ long long pg_offset(const PagedView& c, int page, int g, int slot) {
    if ((unsigned)page >= (unsigned)c.n_pages) return -1;
    const int row = c.shift >= 0 ? slot & (c.page - 1) : slot % c.page;
    return (long long)page * c.ps + (long long)g * c.hs + (long long)row * c.rs;
}

// the same for the sequence whose table row is `trow`
__device__ __forceinline__ long long pg_row(const PagedView& c, const int32_t* trow, int g, int slot) {
    return pg_offset(c, __ldg(trow + pg_col(c, slot)), g, slot);
}

// The slots a query reads, as a list without gaps: all of [0, len), or, where
// slots are positions, the sink [0, s_eff) and the window [len - w, len).
// With positions of their own (pos) every slot is listed and masked one by one.
struct PgList {
    int len, s_eff, n;       // slots in use, listed slots before the gap, listed slots
    __device__ __forceinline__ int slot(int t) const { return t < s_eff ? t : t + (len - n); }
};

__device__ __forceinline__ PgList pg_list(const PagedView& c, int b, int sink, int local) {
    PgList l;
    l.len = pg_length(c, b);
    l.s_eff = l.n = l.len;
    if (local > 0 && c.pos == nullptr) {
        l.s_eff = min(sink, l.len);
        l.n = l.s_eff + min(local, l.len - l.s_eff);
    }
    return l;
}

// The even split: sequence b has tiles(b) tiles in each of its `per` units;
// all T tiles, in order (sequence, unit, tile), are cut into N ranges [T i / N,
// T (i + 1) / N).  Every CTA reads all the lengths and sums them, so that no
// host code or earlier kernel has to know them.
struct PgSplit {
    long long T;
    int N;
    __device__ __forceinline__ long long begin(int i) const { return T * i / N; }
    // the range that tile t lies in
    __device__ __forceinline__ int owner(long long t) const { return (int)(((t + 1) * N - 1) / T); }
};

struct PgCursor {
    int b, sub, tile;        // sequence, unit within it, tile within the unit
    long long unit0;         // flat index of the unit's first tile
};

// Sets split and the cursor of CTA i's first tile (every thread of the CTA
// calls; NT threads).  min_tiles: fewest tiles worth a CTA.  Returns false
// where the CTA has no tiles.
template <int NT, typename F>
__device__ __forceinline__ bool pg_locate(int B, int per, int min_tiles, int i, F tiles, PgSplit& sp, PgCursor& cur,
                                          long long& t0, long long& t1) {
    constexpr int W = NT / 32;
    __shared__ long long s_warp[W];
    __shared__ long long s_base;
    __shared__ int s_b;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int each = (B + NT - 1) / NT;
    const int b0 = min(B, (int)threadIdx.x * each), b1 = min(B, b0 + each);
    long long sum = 0;
    for (int b = b0; b < b1; ++b) sum += tiles(b);
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const long long y = s_warp[w];
        if (w < warp) before += y;
        all += y;
    }
    before += inc - sum;
    sp.T = all * per;
    const long long most = sp.T / min_tiles;
    sp.N = (int)(most < 1 ? 1 : (most < (long long)gridDim.x ? most : (long long)gridDim.x));
    if (i >= sp.N) return false;               // uniform over the CTA
    t0 = sp.begin(i);
    t1 = sp.begin(i + 1);
    if (t0 >= before * per && t0 < (before + sum) * per) {      // this thread's sequences hold t0
        long long base = before;
        int b = b0;
        for (;; ++b) {
            const int n = tiles(b);
            if (t0 < (base + n) * per) break;
            base += n;
        }
        s_b = b;
        s_base = base;
    }
    __syncthreads();
    cur.b = s_b;
    const int n = tiles(cur.b);
    const long long r = t0 - s_base * per;
    cur.sub = (int)(r / n);
    cur.tile = (int)(r - (long long)cur.sub * n);
    cur.unit0 = t0 - cur.tile;
    return true;
}

}  // namespace sa
