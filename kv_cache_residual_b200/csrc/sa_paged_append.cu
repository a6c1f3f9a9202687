// Append to the paged cache: new key and value rows into their slots.
//
// A pure copy: every byte read once and written once.  One warp takes 32 * UN
// 16-byte chunks of a token's key row (all heads, one after another) and the
// same chunks of its value row, all loads before the first store and before the
// search of where they go.  Bound: the launch for a step's single tokens (2.9 us
// for 32), HBM for prompts (24.7 thousand tokens of 4 KB: 29.7 us, 0.89 of the
// copy rate; eight tokens a warp with their searches side by side: 33 us).
#include "sa_paged.cuh"

namespace sa {

template <typename T, int D, int UN>
__global__ void __launch_bounds__(kThreads)
k_paged_append(PagedAppendArgs a, int parts, long long items) {
    constexpr int EPC = Geom<T, D>::EPC, CPR = Geom<T, D>::CPR;
    const PagedView& c = a.c;
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (item >= items) return;
    const int i = (int)(item / parts), part = (int)(item - (long long)i * parts);
    // the rows first: they do not wait for the search of where they go
    const int n = c.Hkv * CPR;
    const T* kn = static_cast<const T*>(a.k_new) + (long long)i * a.token_stride;
    const T* vn = static_cast<const T*>(a.v_new) + (long long)i * a.token_stride;
    uint4 wk[UN], wv[UN];
#pragma unroll
    for (int j = 0; j < UN; ++j) {
        const int x = part * 32 * UN + j * 32 + lane;
        if (x < n) {
            const long long o = (long long)(x / CPR) * a.head_stride + (x % CPR) * EPC;
            wk[j] = ld_stream16(kn + o);
            wv[j] = ld_stream16(vn + o);
        }
    }
    // the token's sequence, and how many of its tokens come from this one on
    int b = i, left = 1;
    if (a.start != nullptr) {
        int lo = 0, hi = c.B;                  // the last b with start[b] <= i, below B
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(a.start + mid) <= i) lo = mid; else hi = mid;
        }
        b = lo;
        left = __ldg(a.start + b + 1) - i;
        if (__ldg(a.start + b) > i || left <= 0) return;
    }
    const int len = pg_length(c, b);
    const int slot = len - left;
    if (slot < 0) return;
    if (part == 0 && (a.pos != nullptr || a.weight != nullptr)) {
        for (int g = lane; g < c.Hkv; g += 32) {
            const size_t w = ((size_t)b * c.Hkv + g) * c.ldw + slot;
            if (a.pos != nullptr) a.pos[w] = pg_newest(c, b, len) + 1 - left;
            if (a.weight != nullptr) a.weight[w] = 0.f;
        }
    }
    const long long row = pg_row(c, c.table + (size_t)b * c.max_pages, 0, slot);
    if (row < 0) return;
    T* k = static_cast<T*>(const_cast<void*>(c.k)) + row;
    T* v = static_cast<T*>(const_cast<void*>(c.v)) + row;
#pragma unroll
    for (int j = 0; j < UN; ++j) {
        const int x = part * 32 * UN + j * 32 + lane;
        if (x < n) {
            const long long o = (long long)(x / CPR) * c.hs + (x % CPR) * EPC;
            *reinterpret_cast<uint4*>(k + o) = wk[j];
            *reinterpret_cast<uint4*>(v + o) = wv[j];
        }
    }
}

template <typename T, int D>
static cudaError_t append_t(const PagedDims& d, const PagedAppendArgs& a, cudaStream_t s) {
    constexpr int CPR = Geom<T, D>::CPR;
    // few tokens: one chunk per lane, so that a step's rows spread over as many
    // warps as there are; many: four, for the loads in flight
    const int n = d.Hkv * CPR;
    const bool few = (long long)a.n_new * cdiv(n, 32) <= 148 * 32;
    const int parts = cdiv(n, few ? 32 : 128);
    const long long items = (long long)a.n_new * parts;
    const unsigned grid = (unsigned)((items + kWarps - 1) / kWarps);
    if (few) k_paged_append<T, D, 1><<<grid, kThreads, 0, s>>>(a, parts, items);
    else k_paged_append<T, D, 4><<<grid, kThreads, 0, s>>>(a, parts, items);
    return cudaGetLastError();
}

cudaError_t launch_paged_append(const PagedDims& d, const PagedAppendArgs& a, cudaStream_t s) {
    if (d.bf16) return d.d == 128 ? append_t<__nv_bfloat16, 128>(d, a, s) : append_t<__nv_bfloat16, 64>(d, a, s);
    return d.d == 128 ? append_t<float, 128>(d, a, s) : append_t<float, 64>(d, a, s);
}

}  // namespace sa
