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
    return (int)((__umulhi((unsigned)slot, c.pmul) + (unsigned)slot) >> c.pshr);
}

// element offset of (slot, head), its page read from the table before, or -1
// where that is not one of the pool
__device__ __forceinline__ long long pg_offset(const PagedView& c, int page, int g, int slot) {
    if ((unsigned)page >= (unsigned)c.n_pages) return -1;
    const int row = slot - pg_col(c, slot) * c.page;
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

// The even split: sequence b has tiles(b) tiles in each of its `per` units; all
// tiles, in order (sequence, unit, tile), are cut into N ranges, the first
// T % N of them one longer.  A unit costs a CTA more than its tiles (queries,
// table, merge, hand-in), so every unit counts `extra` tiles more, before its
// own; T < 2^31 is their number with these.  Every CTA reads all the lengths
// and sums them, so that no host code or earlier kernel has to know them.
struct PgSplit {
    unsigned q, r;           // T / N, T % N
    int extra;
    __device__ __forceinline__ unsigned begin(unsigned i) const { return i * q + min(i, r); }
    // the range that tile t lies in
    __device__ __forceinline__ unsigned owner(unsigned t) const {
        const unsigned longer = r * (q + 1);
        return t < longer ? t / (q + 1) : r + (t - longer) / q;
    }
};

struct PgCursor {
    int b, sub, tile;        // sequence, unit within it, tile within the unit, its extra ones first
    unsigned unit0;          // flat index of the unit's first tile
};

// Sets split, the cursor of CTA i's first tile and its range [t0, t1) (every
// thread of the CTA calls; NT threads).  The extra tiles are at most a quarter
// of a CTA's own.  Returns false where the CTA has no tiles.
template <int NT, typename F>
__device__ __forceinline__ bool pg_locate(int B, int per, int extra, unsigned i, F tiles, PgSplit& sp, PgCursor& cur,
                                          unsigned& t0, unsigned& t1) {
    constexpr int W = NT / 32;
    __shared__ unsigned s_warp[W];
    __shared__ unsigned s_base;
    __shared__ int s_b;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int each = (B + NT - 1) / NT;
    const int b0 = min(B, (int)threadIdx.x * each), b1 = min(B, b0 + each);
    unsigned sum = 0;
    for (int b = b0; b < b1; ++b) sum += tiles(b);
    unsigned inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    unsigned before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const unsigned y = s_warp[w];
        if (w < warp) before += y;
        all += y;
    }
    before += inc - sum;
    const unsigned N = min(all * (unsigned)per, gridDim.x);
    if (i >= N) return false;                  // uniform over the CTA
    const int E = min(extra, (int)(all * (unsigned)per / N) / 4);
    const unsigned T = (all + (unsigned)(E * B)) * per;
    sp.extra = E;
    sp.q = T / N;
    sp.r = T - sp.q * N;
    t0 = sp.begin(i);
    t1 = sp.begin(i + 1);
    before += E * b0;
    sum += E * (b1 - b0);
    if (t0 >= before * per && t0 < (before + sum) * per) {      // this thread's sequences hold t0
        unsigned base = before;
        int b = b0;
        for (; b < b1 - 1; ++b) {
            const unsigned n = tiles(b) + E;
            if (t0 < (base + n) * per) break;
            base += n;
        }
        s_b = b;
        s_base = base;
    }
    __syncthreads();
    cur.b = s_b;
    const unsigned n = tiles(cur.b) + E, x = t0 - s_base * per;
    cur.sub = min((int)(x / n), per - 1);
    cur.tile = (int)(x - cur.sub * n);
    cur.unit0 = t0 - cur.tile;
    return true;
}

}  // namespace sa
