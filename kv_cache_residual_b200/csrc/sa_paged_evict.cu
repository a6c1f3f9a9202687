// Eviction from the paged cache by accumulated attention weight.
//
// Per unit (sequence, KV head): the slots ranked by (protected, weight desc,
// slot asc); the first n' = min(len, budget) stay.  The kept slots at or past
// n' move into the freed slots before it, so sources and destinations never
// meet and the rows move in place, in any order, in one pass.
//
// One cluster of CTAs per unit, each over a slice of the slots: 32-bit keys
// in shared memory, four 8-bit radix passes whose histograms are summed over
// the cluster through distributed shared memory, ranks by ballots and prefix
// sums in slot order, then the moves.  Bound: HBM for the moved rows; for
// small evictions the chain of cluster barriers.
#include <cooperative_groups.h>

#include "sa_paged.cuh"

namespace cg = cooperative_groups;

namespace sa {

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvKeys = 48 * 1024;     // most keys of a slice kept in shared memory

// Order of the slots: larger keys stay.  Protected slots first, then the
// weights as ordered integers (-0 and +0 alike), NaN as -inf.
__device__ __forceinline__ uint32_t ev_key(float w, bool always) {
    if (always) return 0xffffffffu;
    if (w != w) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);       // -0 + 0 = +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <typename T, int D>
__global__ void __launch_bounds__(kEvThreads)
k_paged_evict(PagedEvictArgs a, int slice_keys, int moves, int32_t* lists) {
    extern __shared__ uint32_t s_key[];
    __shared__ uint32_t s_hist[4][256];
    __shared__ uint32_t s_part[8];
    __shared__ uint32_t s_digit, s_above, s_equal;
    __shared__ uint32_t s_cnt[3];                      // equal keys, freed slots, late kept slots of this slice
    __shared__ uint32_t s_w[2][kEvWarps];

    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), CL = (int)cl.num_blocks();
    const PagedView& c = a.c;
    const int u = blockIdx.x / CL, b = u / c.Hkv, g = u - b * c.Hkv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int len = pg_length(c, b), keep = min(len, a.budget);
    const size_t row = (size_t)u * c.ldw;
    const float* W = a.weight + row;
    const int32_t* P = c.pos == nullptr ? nullptr : c.pos + row;
    if (threadIdx.x == 0 && rank == 0 && g == 0) a.lengths_out[b] = keep;
    const int slice = (len + CL - 1) / CL;
    const int lo = min(len, rank * slice), hi = min(len, lo + slice);
    if (len <= a.budget) {                             // nothing to evict: the whole cluster leaves
        for (int s = lo + threadIdx.x; s < hi; s += kEvThreads) {
            a.weight_out[row + s] = W[s];
            a.pos_out[row + s] = P == nullptr ? s : P[s];
        }
        return;
    }
    const long long newest = pg_newest(c, b, len);
    // crowded: more slots hold protected positions than may stay (positions given
    // twice), so that the weights decide among those alone
    bool crowded = false;
    auto make_key = [&](int s) -> uint32_t {
        const long long p = P == nullptr ? s : __ldg(P + s);
        const bool always = p < a.sink || newest - p < a.local;
        return crowded ? (always ? ev_key(__ldg(W + s), false) : 0u) : ev_key(__ldg(W + s), always);
    };
    const bool cached = hi - lo <= slice_keys;
    auto key = [&](int s) -> uint32_t { return cached ? s_key[s - lo] : make_key(s); };
    uint32_t prefix, need, equal;
    for (;;) {
        for (int x = threadIdx.x; x < 4 * 256; x += kEvThreads) (&s_hist[0][0])[x] = 0u;
        if (cached)
            for (int s = lo + threadIdx.x; s < hi; s += kEvThreads) s_key[s - lo] = make_key(s);
        __syncthreads();

        // ---- the smallest kept key: keep-th largest, one digit at a time ----------
        uint32_t mask = 0u;
        prefix = 0u;
        need = (uint32_t)keep;
        equal = 0u;
        for (int d = 0; d < 4; ++d) {
            const int sh = 24 - 8 * d;
            for (int s = lo + threadIdx.x; s < hi; s += kEvThreads) {
                const uint32_t k = key(s);
                if ((k & mask) == prefix) atomicAdd(&s_hist[d][(k >> sh) & 255u], 1u);
            }
            cl.sync();
            // thread t < 256: digit 255 - t over the whole unit, then an inclusive scan
            uint32_t n = 0u, inc = 0u;
            if (threadIdx.x < 256) {
                for (int r = 0; r < CL; ++r) n += cl.map_shared_rank(&s_hist[d][0], r)[255 - threadIdx.x];
                inc = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += y;
                }
                if (lane == 31) s_part[warp] = inc;
            }
            __syncthreads();
            if (threadIdx.x < 256) {
                for (int w = 0; w < warp; ++w) inc += s_part[w];
                if (inc >= need && inc - n < need) {       // exactly one digit
                    s_digit = 255u - threadIdx.x;
                    s_above = inc - n;
                    s_equal = n;
                }
            }
            __syncthreads();
            prefix |= s_digit << sh;
            mask |= 255u << sh;
            need -= s_above;
            equal = s_equal;
        }
        if (crowded || prefix != 0xffffffffu || need == equal) break;
        crowded = true;
        cl.sync();                                     // the histograms have been read by all
    }
    // slots with a larger key stay; of the `equal` slots with key == prefix the
    // first `need`

    // ---- ranks in slot order ---------------------------------------------------------
    // warp w takes a run of the slice, 32 slots at a time
    const int run = ((hi - lo + kEvWarps - 1) / kEvWarps + 31) & ~31;
    const int w0 = min(hi, lo + warp * run), w1 = min(hi, w0 + run);
    if (threadIdx.x < 3) s_cnt[threadIdx.x] = 0u;
    uint32_t eq_rank = 0u;                             // equal keys in slots before this warp's run
    __syncthreads();
    if (need < equal) {
        uint32_t n = 0u;
        for (int s = w0 + lane; s < w1; s += 32) n += key(s) == prefix ? 1u : 0u;
        n = __reduce_add_sync(0xffffffffu, n);
        if (lane == 0) s_w[0][warp] = n;
        __syncthreads();
        if (threadIdx.x == 0) {
            uint32_t t = 0u;
            for (int w = 0; w < kEvWarps; ++w) t += s_w[0][w];
            s_cnt[0] = t;
        }
        cl.sync();
        for (int r = 0; r < rank; ++r) eq_rank += *cl.map_shared_rank(&s_cnt[0], r);
        for (int w = 0; w < warp; ++w) eq_rank += s_w[0][w];
        __syncthreads();
    }
    // calls f(slot, kept) for the warp's slots, 32 at a time, kept meaningful where slot < w1
    auto each = [&](auto f) {
        uint32_t eq = eq_rank;
        for (int s0 = w0; s0 < w1; s0 += 32) {
            const int s = s0 + lane;
            const uint32_t k = s < w1 ? key(s) : 0u;
            bool stays = s < w1 && k > prefix;
            const bool tie = s < w1 && k == prefix;
            const unsigned ties = __ballot_sync(0xffffffffu, tie);
            if (tie) stays = need == equal || eq + __popc(ties & ((1u << lane) - 1u)) < need;
            eq += __popc(ties);
            f(s, s < w1, stays);
        }
    };
    uint32_t nh = 0u, nl = 0u;
    each([&](int s, bool in, bool stays) {
        nh += __popc(__ballot_sync(0xffffffffu, in && s < keep && !stays));
        nl += __popc(__ballot_sync(0xffffffffu, in && s >= keep && stays));
    });
    if (lane == 0) { s_w[0][warp] = nh; s_w[1][warp] = nl; }
    __syncthreads();
    if (threadIdx.x < 2) {
        uint32_t t = 0u;
        for (int w = 0; w < kEvWarps; ++w) t += s_w[threadIdx.x][w];
        s_cnt[1 + threadIdx.x] = t;
    }
    cl.sync();
    uint32_t hole = 0u, late = 0u, total = 0u;
    for (int r = 0; r < CL; ++r) {
        const uint32_t* q = cl.map_shared_rank(&s_cnt[0], r);
        const uint32_t h = q[1], l = q[2];
        total += h;
        if (r < rank) { hole += h; late += l; }
    }
    for (int w = 0; w < warp; ++w) { hole += s_w[0][w]; late += s_w[1][w]; }
    int32_t* holes = lists + (size_t)u * 2 * moves;
    int32_t* lates = holes + moves;
    each([&](int s, bool in, bool stays) {
        const bool h = in && s < keep && !stays, l = in && s >= keep && stays;
        const unsigned mh = __ballot_sync(0xffffffffu, h), ml = __ballot_sync(0xffffffffu, l);
        const unsigned below = (1u << lane) - 1u;
        if (h) holes[hole + __popc(mh & below)] = s;
        if (l) lates[late + __popc(ml & below)] = s;
        hole += __popc(mh);
        late += __popc(ml);
        if (in && s < keep && stays) {
            a.weight_out[row + s] = W[s];
            a.pos_out[row + s] = P == nullptr ? s : P[s];
        }
    });
    cl.sync();                                         // the lists are whole; no CTA reads another's memory from here

    // ---- the moves --------------------------------------------------------------------
    using Gm = Geom<T, D>;
    constexpr int CPR = Gm::CPR, EPC = Gm::EPC, NG = Gm::GPW * kEvWarps;
    constexpr int UN = 4;
    const int li = threadIdx.x % CPR, grp = threadIdx.x / CPR;
    const int32_t* trow = c.table + (size_t)b * c.max_pages;
    T* K = static_cast<T*>(const_cast<void*>(c.k)) + li * EPC;
    T* V = static_cast<T*>(const_cast<void*>(c.v)) + li * EPC;
    for (int m0 = (rank * NG + grp) * UN; m0 < (int)total; m0 += CL * NG * UN) {
        uint4 wk[UN], wv[UN];
        long long to[UN];
#pragma unroll
        for (int j = 0; j < UN; ++j) {
            to[j] = -1;
            if (m0 + j < (int)total) {
                const int src = __ldcg(lates + m0 + j), dst = __ldcg(holes + m0 + j);
                const long long from = pg_row(c, trow, g, src);
                to[j] = from < 0 ? -1 : pg_row(c, trow, g, dst);
                if (to[j] >= 0) {
                    wk[j] = ld_stream16(K + from);
                    wv[j] = ld_stream16(V + from);
                }
                if (li == 0) {
                    a.weight_out[row + dst] = W[src];
                    a.pos_out[row + dst] = P == nullptr ? src : P[src];
                }
            }
        }
#pragma unroll
        for (int j = 0; j < UN; ++j) {
            if (to[j] >= 0) {
                *reinterpret_cast<uint4*>(K + to[j]) = wk[j];
                *reinterpret_cast<uint4*>(V + to[j]) = wv[j];
            }
        }
    }
}

PagedEvictPlan paged_evict_plan(const PagedDims& d, int budget) {
    PagedEvictPlan p;
    // few units: more CTAs each, up to the portable eight
    p.cluster = 1;
    while (p.cluster < 8 && (long long)d.U() * p.cluster < 148 * 2 && d.cap / p.cluster > 1024) p.cluster *= 2;
    const int slice = cdiv(d.cap, p.cluster);
    p.slice_max = slice < kEvKeys ? slice : kEvKeys;
    const int past = d.cap > budget ? d.cap - budget : 0;
    p.moves = past < budget ? past : budget;
    if (p.moves < 1) p.moves = 1;
    p.off_list = 0;
    p.bytes = align256(sizeof(int32_t) * 2 * (size_t)d.U() * p.moves);
    return p;
}

template <typename T, int D>
static cudaError_t evict_t(const PagedDims& d, const PagedEvictPlan& p, const PagedEvictArgs& a, cudaStream_t s) {
    static std::atomic<unsigned long long> opted{0};
    cudaError_t e = opt_in_smem(k_paged_evict<T, D>, (size_t)kEvKeys * 4, opted);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)d.U() * p.cluster);
    cfg.blockDim = dim3(kEvThreads);
    cfg.dynamicSmemBytes = (size_t)p.slice_max * 4;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_paged_evict<T, D>, a, p.slice_max, p.moves,
                              reinterpret_cast<int32_t*>(a.ws + p.off_list));
}

cudaError_t launch_paged_evict(const PagedDims& d, const PagedEvictPlan& p, const PagedEvictArgs& a, cudaStream_t s) {
    if (d.bf16) return d.d == 128 ? evict_t<__nv_bfloat16, 128>(d, p, a, s) : evict_t<__nv_bfloat16, 64>(d, p, a, s);
    return d.d == 128 ? evict_t<float, 128>(d, p, a, s) : evict_t<float, 64>(d, p, a, s);
}

}  // namespace sa
