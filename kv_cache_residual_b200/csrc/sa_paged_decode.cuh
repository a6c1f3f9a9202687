// Device code shared by the paged decode kernels: logits, records of partial
// units and their join.
#pragma once

#include "sa_paged.cuh"

namespace sa {

struct PgDecodeIo {
    PagedView c;
    const void* q;
    long long q_stride;
    const float* slopes;
    float* out;
    float* lse;
    float* lse2;             // with weights: log2 of the rows' masses
    float* x;                // with weights: logits (log2) [B, Hq, ldx] of the listed slots, or null
    float* rec;              // two records per CTA
    unsigned* cnt;           // completion tickets, one per unit
    float softcap, cap_in;   // c, scale / c
    float factor;            // log2(e) times the scale, or times c
    int sink, local, ldx, extra;
};

// A logit in log2 units less `ref`: factor c - slope2 dist - ref, with c the dot
// product, or its tanh where logits are capped (tanhf: 2 ulp, so that a capped
// logit is as exact as the dot product).  Taking ref (the running maximum) off
// inside the fused operations leaves no rounding of the size of the logit.
__device__ __forceinline__ float pg_cap(const PgDecodeIo& io, float dot) {
    return io.softcap > 0.f ? tanhf(dot * io.cap_in) : dot;
}
__device__ __forceinline__ float pg_logit(const PgDecodeIo& io, float c, float slope2, float dist, float ref) {
    return fmaf(-slope2, dist, fmaf(c, io.factor, -ref));
}

// What a lane reads of a listed slot: its page, and its position where slots
// have positions of their own.  Only loads here, so that they can be issued
// well ahead of pg_see.
struct PgRaw {
    int slot, page, pos;
};

__device__ __forceinline__ PgRaw pg_fetch(const PgDecodeIo& io, const PgList& ls, const int32_t* trow,
                                          const int32_t* prow, int y, int end) {
    PgRaw r{0, -1, 0};
    if (y < end) {
        r.slot = ls.slot(y);
        r.page = __ldg(trow + pg_col(io.c, r.slot));
        if (prow != nullptr) r.pos = __ldg(prow + r.slot);
    }
    return r;
}

// the slot's row offset (-1: not visible) and its distance from the newest position
__device__ __forceinline__ long long pg_see(const PgDecodeIo& io, const PgRaw& r, bool own_pos, int g, int newest,
                                            float& dist) {
    const int p = own_pos ? r.pos : r.slot;
    const long long away = (long long)newest - p;
    dist = (float)away;
    if (own_pos && io.local > 0 && !(p < io.sink || away < io.local)) return -1;
    return pg_offset(io.c, r.page, g, r.slot);
}

// Records of a unit, in split order: its first CTA's second record, then the
// first records of the CTAs after it.
__device__ __forceinline__ float* pg_rec(float* rec, int floats, int cta, bool begins) {
    return rec + (size_t)(2 * cta + (begins ? 1 : 0)) * floats;
}

// a head's log of its mass L 2^M
__device__ __forceinline__ void pg_write_lse(const PgDecodeIo& io, size_t qh, float M, float L) {
    constexpr float kLn2Rest = -1.9046543e-9f;     // ln 2 - kLn2
    if (io.lse != nullptr) io.lse[qh] = L == 0.f ? -INFINITY : fmaf(M, kLn2, fmaf(M, kLn2Rest, logf(L)));
    if (io.x != nullptr) io.lse2[qh] = L == 0.f ? -INFINITY : M + log2f(L);
}

// 1 / L, and 0 where nothing is seen (out = A inv: one rounding more than A / L)
__device__ __forceinline__ float pg_inv(float L) { return L == 0.f ? 0.f : 1.f / L; }

// A row's element, its sum of values A times inv = pg_inv(L).  Matrix products of
// parts make NaN of an infinite value (zero parts, the parts of an infinity, a
// weight that underflows), so where the row's weights are numbers and the sum is
// not, a mark is left for pg_not_finite, and the unit noted in `odd` (shared: the
// first and the last).
constexpr unsigned kPgMark = 0x7fc0a11fu;          // a NaN that no operation makes
__device__ __forceinline__ float pg_element(float A, float inv, int unit, int* odd) {
    const float y = A * inv;
    if (y == y) return y;
    if (inv == 0.f) return 0.f;                    // nothing seen, or every weight 0
    if (inv != inv) return y;
    atomicMin(odd, unit);
    atomicMax(odd + 1, unit);
    return __uint_as_float(kPgMark);
}

// The unit's last CTA joins its n records (fixed order) and writes the rows of
// its gh <= 8 heads from h0 on.  Thread (column, part): a column is four dims of
// a head, and the records are cut into as many parts as there are threads for;
// a part's first records are on their way before the weights are known.
// f: shared scratch of kPgJoinFloats floats; unit, odd: as pg_element.  All threads
// call.
constexpr int kPgJoin = 10;                // records of a part in flight
// the heads' m and l, then [head][record] weights, then over them the parts' sums (a float4 per thread)
constexpr int kPgJoinFloats = 8 * (kPgSlots + 2);

template <int D, int NT>
__device__ __forceinline__ void pg_join(const PgDecodeIo& io, int first, int n, size_t qh0, int h0, int gh, float* f,
                                        int unit, int* odd) {
    const int hu = io.c.hu, floats = hu * (2 + D);
    float* sM = f;
    float* sL = f + 8;
    float* w = f + 16;                         // [head][record] weights 2^(m - M)
    float4* sums = reinterpret_cast<float4*>(w);
    static_assert(16 + 4 * NT <= kPgJoinFloats, "the parts' sums lie over the weights");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float* rest = pg_rec(io.rec, floats, first, false) + h0;         // record s > 0: 2 s records on
    const float* begin = pg_rec(io.rec, floats, first, true) + h0;
    auto rec = [&](int s) { return s == 0 ? begin : rest + (size_t)(2 * s) * floats; };
    const int cols = gh * (D / 4);
    const int parts = max(1, NT / cols), part = threadIdx.x / cols;        // part >= parts: none
    const int each = (n + parts - 1) / parts;
    // a thread's column and records in pass c0 over the columns; the first ones
    // are on their way before the weights are known
    int h, e, s0, s1;
    bool mine;
    float4 a[kPgJoin];
    auto place = [&](int c0) {
        const int col = parts > 1 ? threadIdx.x % cols : c0 + threadIdx.x;
        h = col / (D / 4);
        e = (col % (D / 4)) * 4;
        s0 = parts > 1 ? part * each : 0;
        s1 = min(n, s0 + each);
        mine = col < cols && (parts == 1 || part < parts);
    };
    auto load = [&](int s) {
#pragma unroll
        for (int j = 0; j < kPgJoin; ++j)
            if (mine && s + j < s1) a[j] = __ldcg(reinterpret_cast<const float4*>(rec(s + j) - h0 + 2 * hu + (h0 + h) * D + e));
    };
    place(0);
    load(s0);
#pragma unroll 1
    for (int x = warp; x < gh; x += NT / 32) {
        // the first 32 records' m and l at once
        float m = lane < n ? __ldcg(rec(lane) + x) : -INFINITY, l = lane < n ? __ldcg(rec(lane) + hu + x) : 0.f;
        float M = m;
#pragma unroll 1
        for (int s = lane; s < n;) {
            w[x * n + s] = m;
            s += 32;
            if (s < n) {
                m = __ldcg(rec(s) + x);
                M = (m > M || m != m) ? m : M; // NaN stays
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float y = __shfl_xor_sync(0xffffffffu, M, o);
            M = (y > M || y != y) ? y : M;
        }
        float L = 0.f;
#pragma unroll 1
        for (int s = lane; s < n;) {
            const float q = w[x * n + s], y = q == -INFINITY ? 0.f : ex2(q - M);
            w[x * n + s] = y;
            L = fmaf(l, y, L);
            s += 32;
            if (s < n) l = __ldcg(rec(s) + hu + x);
        }
        L = group_sum<32>(L);
        if (lane == 0) {
            sM[x] = M;
            sL[x] = pg_inv(L);
            pg_write_lse(io, qh0 + x, M, L);
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int c0 = 0; c0 < cols; c0 += NT) {
        if (c0 > 0) {
            place(c0);
            load(s0);
        }
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int s = s0; mine && s < s1; s += kPgJoin) {
            if (s > s0) load(s);
#pragma unroll
            for (int j = 0; j < kPgJoin; ++j) {
                if (s + j < s1) {
                    const float y = w[h * n + s + j];
                    A.x = fmaf(a[j].x, y, A.x);
                    A.y = fmaf(a[j].y, y, A.y);
                    A.z = fmaf(a[j].z, y, A.z);
                    A.w = fmaf(a[j].w, y, A.w);
                }
            }
        }
        if (parts > 1) {
            __syncthreads();
            if (mine) sums[threadIdx.x] = A;
            __syncthreads();
            for (int p = 1; part == 0 && p < parts; ++p) {
                const float4 B = sums[p * cols + threadIdx.x];
                A.x += B.x; A.y += B.y; A.z += B.z; A.w += B.w;
            }
        }
        if (mine && (parts == 1 || part == 0)) {
            const float inv = sL[h];
            *reinterpret_cast<float4*>(io.out + (qh0 + h) * D + e) =
                make_float4(pg_element(A.x, inv, unit, odd), pg_element(A.y, inv, unit, odd),
                            pg_element(A.z, inv, unit, odd), pg_element(A.w, inv, unit, odd));
        }
    }
}

}  // namespace sa
