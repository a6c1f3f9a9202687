// Eviction from the paged cache by accumulated attention weight.
//
// Per unit (sequence, KV head): the slots ranked by (protected, weight desc,
// slot asc); the first n' = min(len, budget) stay.  The kept slots at or past
// n' move into the freed slots before it, so sources and destinations never
// meet and the rows move in place, in any order, in one pass.
//
// k_evict_select: one cluster of CTAs per unit, each over a slice of the slots.
// One pass over the weights makes 32-bit keys (in shared memory, or in the
// workspace where a slice is too long) and writes the outputs of the slots that
// may stay in place.  Then radix digits of 11, 11 and 10 bits until the digits'
// prefix alone tells who stays (22 bits mostly do): a histogram per CTA, of
// which the cluster reads 64 coarse sums and then the 32 bins of one of them
// through distributed shared memory.  Ranks by prefix sums in slot order; out
// come the lists of freed and of late kept slots.  Bound: the chain of barriers
// and the latency of the weights (4112 slots of 256 units: 13 us; 32K of 64: 20
// us; 128K of 8: 24 us, and 27 with clusters of sixteen).
// k_evict_move: the rows, split evenly over the GPU whatever the units'
// counts.  Bound: HBM, each moved row read once and written once (402 MB in 66 us,
// 0.95 of the copy rate).
#include <cooperative_groups.h>

#include "sa_paged.cuh"

namespace cg = cooperative_groups;

namespace sa {

constexpr int kEvThreads = 512;
constexpr int kEvBins = 2048, kEvCoarse = 64;
constexpr int kEvUn = 2;               // quads of slots a thread reads at once
constexpr int kEvKeys = 40 * 1024;     // most keys of a slice kept in shared memory,
constexpr int kEvKeysTwo = 21 * 1024;  // and where two CTAs share an SM
constexpr int kEvMoveThreads = 256;
constexpr int kEvMoveUn = 4;           // rows a lane group reads at once

constexpr uint32_t kEvZero = 0x80000000u;      // the key of 0; next to it, with its top digit, lie the subnormals

// Order of the slots: larger keys stay.  Protected slots first, then the
// weights as ordered integers (-0 and +0 alike), NaN as -inf.
__device__ __forceinline__ uint32_t ev_key(float w, bool always) {
    if (always) return 0xffffffffu;
    if (w != w) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);       // -0 + 0 = +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <int CL>
__device__ __forceinline__ void ev_sync() {
    if constexpr (CL == 1) __syncthreads();
    else cg::this_cluster().sync();
}

template <int CL, typename T>
__device__ __forceinline__ const T* ev_peer(T* p, int rank) {
    if constexpr (CL == 1) return p;
    else return cg::this_cluster().map_shared_rank(p, rank);
}

// four slots from s on, s a multiple of 4 (vec: the row is aligned)
template <typename T4, typename T>
__device__ __forceinline__ void ev_load(T (&x)[4], const T* row, int s, int end, bool vec) {
    if (vec && s + 4 <= end) {
        const T4 y = __ldg(reinterpret_cast<const T4*>(row + s));
        x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = s + i < end ? __ldg(row + s + i) : T(0);
    }
}
template <typename T4, typename T>
__device__ __forceinline__ void ev_store(const T (&x)[4], T* row, int s, int end, bool vec) {
    if (vec && s + 4 <= end) {
        *reinterpret_cast<T4*>(row + s) = T4{x[0], x[1], x[2], x[3]};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (s + i < end) row[s + i] = x[i];
    }
}

template <int CL>
__global__ void __launch_bounds__(kEvThreads, 2)
k_evict_select(PagedEvictArgs a, int moves, int32_t* lists, int32_t* counts, uint32_t* far_keys, int far_row) {
    constexpr int NT = kEvThreads, kW = NT / 32;
    extern __shared__ __align__(16) uint32_t s_mem[];
    uint32_t* s_hist = s_mem;                          // [3][kEvBins]
    __shared__ __align__(8) uint32_t s_coarse[3][kEvCoarse];
    __shared__ uint32_t s_digit, s_above, s_equal, s_zeros, s_tiny;
    // kept for their keys, keys equal to the last one kept, and the same of slots before `keep`
    __shared__ uint32_t s_w[4][kW], s_cnt[4];

    const PagedView& c = a.c;
    const int u = blockIdx.x / CL, rank = blockIdx.x % CL, b = u / c.Hkv, g = u - b * c.Hkv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int len = pg_length(c, b), keep = min(len, a.budget);
    const size_t row = (size_t)u * c.ldw;
    const float* W = a.weight + row;
    const int32_t* P = c.pos == nullptr ? nullptr : c.pos + row;
    float* Wo = a.weight_out + row;
    int32_t* Po = a.pos_out + row;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(W) | reinterpret_cast<uintptr_t>(P) |
                           reinterpret_cast<uintptr_t>(Wo) | reinterpret_cast<uintptr_t>(Po);
    const bool vec = (bits & 15) == 0;
    if (threadIdx.x == 0 && rank == 0) {
        if (g == 0) a.lengths_out[b] = keep;
        if (len <= a.budget) counts[u] = 0;
    }
    const int slice = ((len + CL - 1) / CL + 31) & ~31;
    const int lo = min(len, rank * slice), hi = min(len, lo + slice);
    cudaTriggerProgrammaticLaunchCompletion();         // the moves' CTAs may come and wait
    const bool evicts = len > a.budget;
    const long long newest = pg_newest(c, b, len);
    uint32_t* keys = far_keys == nullptr ? s_mem + 3 * kEvBins : far_keys + (size_t)u * far_row + lo;
    // crowded: more slots hold protected positions than may stay (positions given
    // twice), so that the weights decide among those alone
    bool crowded = false;

    // ---- the digits of the smallest kept key ------------------------------------------
    // slots with key & mask > prefix stay; of the `equal` slots with key & mask
    // == prefix the first `need`
    uint32_t prefix, mask, need, equal;
    for (;;) {
        constexpr int kStep = 4 * kEvUn * NT;
        float w[2][kEvUn][4];
        int p[2][kEvUn][4];
        auto load = [&](int k, int s0) {
#pragma unroll
            for (int j = 0; j < kEvUn; ++j) {
                const int s = s0 + j * 4 * NT;
                if (s < hi) {
                    ev_load<float4>(w[k][j], W, s, hi, vec);
                    if (P != nullptr) ev_load<int4>(p[k][j], P, s, hi, vec);
                }
            }
        };
        load(0, lo + 4 * threadIdx.x);
        if (threadIdx.x == 0) s_tiny = 0u;
        for (int x = threadIdx.x; x < 3 * kEvBins / 4; x += NT)
            reinterpret_cast<uint4*>(s_hist)[x] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
#pragma unroll 1
        for (int s0 = lo + 4 * threadIdx.x; s0 < hi; s0 += kStep) {
            load(1, s0 + kStep);
#pragma unroll
            for (int j = 0; j < kEvUn; ++j) {
                const int s = s0 + j * 4 * NT;
                if (s < hi) {
                    int q[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) q[i] = P == nullptr ? s + i : p[0][j][i];
                    // a freed slot's are written over by the move into it
                    ev_store<float4>(w[0][j], Wo, s, min(keep, hi), vec);
                    ev_store<int4>(q, Po, s, min(keep, hi), vec);
                    if (evicts) {
                        uint32_t k[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const bool always = q[i] < a.sink || newest - q[i] < a.local;
                            k[i] = crowded && !always ? 0u : ev_key(w[0][j][i], always && !crowded);
                            // past the slice 0, which is no weight's key and never the last one kept
                            if (s + i < hi) atomicAdd(s_hist + (k[i] >> 21), 1u); else k[i] = 0u;
                            if (k[i] - kEvZero - 1u < (1u << 21) - 1u) s_tiny = 1u;
                        }
                        *reinterpret_cast<uint4*>(keys + s - lo) = make_uint4(k[0], k[1], k[2], k[3]);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kEvUn; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) { w[0][j][i] = w[1][j][i]; p[0][j][i] = p[1][j][i]; }
        }
        if (!evicts) return;                           // the whole cluster
        __syncthreads();
        mask = prefix = equal = 0u;
        need = (uint32_t)keep;
#pragma unroll 1
        for (int d = 0; d < 3 && need != equal; ++d) {
            const int sh = d == 0 ? 21 : (d == 1 ? 10 : 0);
            const uint32_t bins = d == 2 ? 1023u : 2047u;
            uint32_t* h = s_hist + d * kEvBins;
            if (d > 0) {
                for (int s0 = 4 * threadIdx.x; s0 < hi - lo; s0 += kStep) {
                    uint4 k[kEvUn];
#pragma unroll
                    for (int j = 0; j < kEvUn; ++j) {
                        const int s = s0 + j * 4 * NT;
                        k[j] = s < hi - lo ? *reinterpret_cast<const uint4*>(keys + s) : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int j = 0; j < kEvUn; ++j) {
                        if ((k[j].x & mask) == prefix) atomicAdd(h + ((k[j].x >> sh) & bins), 1u);
                        if ((k[j].y & mask) == prefix) atomicAdd(h + ((k[j].y >> sh) & bins), 1u);
                        if ((k[j].z & mask) == prefix) atomicAdd(h + ((k[j].z >> sh) & bins), 1u);
                        if ((k[j].w & mask) == prefix) atomicAdd(h + ((k[j].w >> sh) & bins), 1u);
                    }
                }
                __syncthreads();
            }
            for (int x = warp; x < kEvCoarse; x += kW) {
                const uint32_t n = __reduce_add_sync(0xffffffffu, h[x * 32 + lane]);
                if (lane == 0) s_coarse[d][x] = n;
            }
            ev_sync<CL>();
            if (warp == 0) {
                // from the top: lane l has coarse bins 63 - 2 l and 62 - 2 l of the unit
                uint32_t q0 = 0u, q1 = 0u;
#pragma unroll
                for (int r = 0; r < CL; ++r) {
                    const uint2 y = *reinterpret_cast<const uint2*>(ev_peer<CL>(&s_coarse[d][0], r) + 62 - 2 * lane);
                    q0 += y.y;
                    q1 += y.x;
                }
                uint32_t inc = q0 + q1;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += y;
                }
                // the first lane that reaches `need` has the bin
                const int at = __ffs(__ballot_sync(0xffffffffu, inc >= need)) - 1;
                uint32_t above = __shfl_sync(0xffffffffu, inc - q0 - q1, at);
                const uint32_t first = __shfl_sync(0xffffffffu, q0, at);
                int x = 63 - 2 * at;
                if (above + first < need) { above += first; --x; }
                uint32_t n = 0u;                       // lane l: bin 31 - l of coarse bin x
#pragma unroll
                for (int r = 0; r < CL; ++r) n += ev_peer<CL>(h, r)[x * 32 + 31 - lane];
                inc = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += y;
                }
                const int bin = __ffs(__ballot_sync(0xffffffffu, above + inc >= need)) - 1;
                // where the last one kept has the weight 0 (a new token's) and nothing
                // but zeros shares its digit, the key is known
                bool tiny = false;
                if (lane < CL) tiny = *ev_peer<CL>(&s_tiny, lane) != 0u;
                tiny = __any_sync(0xffffffffu, tiny);
                if (lane == bin) {
                    s_zeros = d == 0 && !tiny && (uint32_t)(x * 32 + 31 - lane) == kEvZero >> 21 ? 1u : 0u;
                    s_digit = (uint32_t)(x * 32 + 31 - lane);
                    s_above = above + inc - n;
                    s_equal = n;
                }
            }
            __syncthreads();
            prefix |= s_digit << sh;
            mask |= bins << sh;
            need -= s_above;
            equal = s_equal;
            if (s_zeros != 0u) {
                mask = 0xffffffffu;
                break;
            }
        }
        // more protected slots than may stay: only the protected have this key
        if (crowded || prefix != 0xffffffffu || need == equal) break;
        crowded = true;
        ev_sync<CL>();                                 // the histograms have been read by all
    }

    // ---- ranks in slot order ---------------------------------------------------------
    // Kept before slot s: those with a larger key, and of the equal ones the first
    // `need`, so prefix counts of both kinds give every slot's place: a freed slot
    // s < keep is number s - kept(s), a late kept one number kept(s) - kept(keep).
    // warp w takes a run of the slice, 128 slots at a time, four in a row a lane
    const int run = ((hi - lo + kW - 1) / kW + 127) & ~127;
    const int w0 = min(hi, lo + warp * run), w1 = min(hi, w0 + run);
    auto quad = [&](int s0, uint32_t (&k)[4]) {        // masked keys; past the run 0, below every prefix
        const int s = s0 + 4 * lane;
        const uint4 y = s < w1 ? *reinterpret_cast<const uint4*>(keys + s - lo) : make_uint4(0u, 0u, 0u, 0u);
        k[0] = y.x & mask; k[1] = y.y & mask; k[2] = y.z & mask; k[3] = y.w & mask;
    };
    uint32_t n[4] = {0u, 0u, 0u, 0u};
#pragma unroll 2
    for (int s0 = w0; s0 < w1; s0 += 128) {
        uint32_t k[4];
        quad(s0, k);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool early = s0 + 4 * lane + i < keep;
            n[0] += k[i] > prefix ? 1u : 0u;
            n[1] += k[i] == prefix ? 1u : 0u;
            n[2] += k[i] > prefix && early ? 1u : 0u;
            n[3] += k[i] == prefix && early ? 1u : 0u;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) n[i] = __reduce_add_sync(0xffffffffu, n[i]);
    if (lane < 4) s_w[lane][warp] = lane == 0 ? n[0] : lane == 1 ? n[1] : lane == 2 ? n[2] : n[3];
    __syncthreads();
    if (warp < 4) {
        const uint32_t t = __reduce_add_sync(0xffffffffu, lane < kW ? s_w[warp][lane] : 0u);
        if (lane == 0) s_cnt[warp] = t;
    }
    ev_sync<CL>();
    uint32_t gt = 0u, eq = 0u, gt1 = 0u, eq1 = 0u;
#pragma unroll
    for (int r = 0; r < CL; ++r) {
        const uint32_t* q = ev_peer<CL>(&s_cnt[0], r);
        gt += r < rank ? q[0] : 0u;
        eq += r < rank ? q[1] : 0u;
        gt1 += q[2];
        eq1 += q[3];
    }
#pragma unroll
    for (int w = 0; w < kW; ++w) {
        gt += w < warp ? s_w[0][w] : 0u;
        eq += w < warp ? s_w[1][w] : 0u;
    }
    const uint32_t kept1 = gt1 + min(need, eq1);       // kept(keep)
    if (threadIdx.x == 0 && rank == 0) counts[u] = keep - (int32_t)kept1;
    int32_t* holes = lists + (size_t)u * 2 * moves;
    int32_t* lates = holes + moves;
#pragma unroll 1
    for (int s0 = w0; s0 < w1; s0 += 128) {
        uint32_t k[4], own = 0u;                       // larger keys in the low half, ties in the high one
        quad(s0, k);
#pragma unroll
        for (int i = 0; i < 4; ++i) own += k[i] > prefix ? 1u : k[i] == prefix ? 0x10000u : 0u;
        uint32_t inc = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        uint32_t g = gt + ((inc - own) & 0xffffu), ties = eq + ((inc - own) >> 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = s0 + 4 * lane + i;
            const bool above = k[i] > prefix, tie = k[i] == prefix;
            const bool stays = above || (tie && ties < need);
            const uint32_t kept = g + min(need, ties);
            if (s < keep && s < w1 && !stays) holes[s - (int)kept] = s;
            if (s >= keep && stays) lates[kept - kept1] = s;
            g += above ? 1u : 0u;
            ties += tie ? 1u : 0u;
        }
        const uint32_t all = __shfl_sync(0xffffffffu, inc, 31);
        gt += all & 0xffffu;
        eq += all >> 16;
    }
    if constexpr (CL > 1) ev_sync<CL>();               // no CTA leaves while another reads its memory
}

// Warp x of a unit: its moves [32 x, 32 x + 32), whose places the lanes look up
// one each, so that the chain count, lists, table is walked once for 32 rows.
template <typename T, int D>
__global__ void __launch_bounds__(kEvMoveThreads, 1)       // 80 registers, three CTAs per SM: more of them slow each other down
k_evict_move(PagedEvictArgs a, int chunks, int moves, const int32_t* lists, const int32_t* counts) {
    using Gm = Geom<T, D>;
    constexpr int CPR = Gm::CPR, EPC = Gm::EPC, GPW = Gm::GPW, UN = kEvMoveUn;
    const PagedView& c = a.c;
    const int lane = threadIdx.x & 31, li = lane % CPR, gsub = lane / CPR;
    const int x = blockIdx.x * (kEvMoveThreads / 32) + (threadIdx.x >> 5), u = x / chunks;
    const int b = u / c.Hkv, g = u - b * c.Hkv, m = (x - u * chunks) * 32 + lane;
    cudaGridDependencySynchronize();                   // the lists
    if (u >= c.B * c.Hkv) return;
    const int n = __ldcg(counts + u);
    if (m - lane >= n) return;
    const size_t row = (size_t)u * c.ldw;
    const int32_t* lates = lists + (size_t)u * 2 * moves + moves;
    const int32_t* trow = c.table + (size_t)b * c.max_pages;
    long long from = -1, to = -1;
    if (m < n) {
        const int s = __ldcg(lates + m), d = __ldcg(lates + m - moves);
        from = pg_row(c, trow, g, s);
        to = pg_row(c, trow, g, d);
        if (to < 0) from = -1;
        a.weight_out[row + d] = __ldg(a.weight + row + s);
        a.pos_out[row + d] = c.pos == nullptr ? s : __ldg(c.pos + row + s);
    }
    T* K = static_cast<T*>(const_cast<void*>(c.k)) + li * EPC;
    T* V = static_cast<T*>(const_cast<void*>(c.v)) + li * EPC;
    const int end = min(32, n - (m - lane));
#pragma unroll 1
    for (int j0 = 0; j0 < end; j0 += GPW * UN) {
        uint4 wk[UN], wv[UN];
        long long f[UN];
#pragma unroll
        for (int j = 0; j < UN; ++j) {
            f[j] = __shfl_sync(0xffffffffu, from, j0 + j * GPW + gsub);
            if (f[j] >= 0) {
                wk[j] = ld_stream16(K + f[j]);
                wv[j] = ld_stream16(V + f[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < UN; ++j) {
            const long long t = __shfl_sync(0xffffffffu, to, j0 + j * GPW + gsub);
            if (f[j] >= 0) {
                *reinterpret_cast<uint4*>(K + t) = wk[j];
                *reinterpret_cast<uint4*>(V + t) = wv[j];
            }
        }
    }
}

PagedEvictPlan paged_evict_plan(const PagedDims& d, int budget) {
    PagedEvictPlan p;
    // few units: more CTAs each, up to the portable eight, as long as all are
    // resident at once (two per SM)
    p.cluster = 1;
    while (p.cluster < 8 && (long long)d.U() * p.cluster * 2 <= 148 * 2 && d.cap / p.cluster > 1024) p.cluster *= 2;
    // Longer slices than two CTAs of an SM have room for keep their keys in the
    // workspace, or the clusters above would come in two waves (32 units of 256K to
    // 64K: 260 us, 227 with the keys there; 16 units 203 and 196).  In shared memory
    // all the same: with CTAs on half the SMs at most (8 units of 256K: 107 us, 114
    // in the workspace), and units of one CTA (256 of 32K to 16 less: 51.7, 53.0).
    const int slice = (cdiv(d.cap, p.cluster) + 31) & ~31;
    const bool alone = p.cluster == 1 || d.U() * p.cluster * 2 <= 148;
    p.near_keys = slice <= (alone ? kEvKeys : kEvKeysTwo) ? slice : 0;
    const int past = d.cap > budget ? d.cap - budget : 0;
    p.moves = past < budget ? past : budget;
    size_t off = 0;
    p.off_count = off; off = align256(off + sizeof(int32_t) * (size_t)d.U());
    p.off_list = off;  off = align256(off + sizeof(int32_t) * 2 * (size_t)d.U() * p.moves);
    p.off_keys = off;  if (p.near_keys == 0) off = align256(off + sizeof(uint32_t) * (size_t)d.U() * ((d.cap + 31) & ~31));
    p.bytes = off;
    return p;
}

template <int CL>
static cudaError_t select_t(const PagedDims& d, const PagedEvictPlan& p, const PagedEvictArgs& a, cudaStream_t s) {
    static std::atomic<unsigned long long> opted{0};
    const cudaError_t e = opt_in_smem(k_evict_select<CL>, (size_t)(3 * kEvBins + kEvKeys) * 4, opted);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)d.U() * CL);
    cfg.blockDim = dim3(kEvThreads);
    cfg.dynamicSmemBytes = (size_t)(3 * kEvBins + p.near_keys) * 4;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CL;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CL > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_evict_select<CL>, a, p.moves,
                              reinterpret_cast<int32_t*>(a.ws + p.off_list), reinterpret_cast<int32_t*>(a.ws + p.off_count),
                              p.near_keys > 0 ? nullptr : reinterpret_cast<uint32_t*>(a.ws + p.off_keys),
                              (d.cap + 31) & ~31);
}

template <typename T, int D>
static cudaError_t move_t(const PagedDims& d, const PagedEvictPlan& p, const PagedEvictArgs& a, cudaStream_t s) {
    const int chunks = cdiv(p.moves, 32);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((long long)d.U() * chunks + kEvMoveThreads / 32 - 1) / (kEvMoveThreads / 32)));
    cfg.blockDim = dim3(kEvMoveThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_evict_move<T, D>, a, chunks, p.moves,
                              static_cast<const int32_t*>(reinterpret_cast<int32_t*>(a.ws + p.off_list)),
                              static_cast<const int32_t*>(reinterpret_cast<int32_t*>(a.ws + p.off_count)));
}

cudaError_t launch_paged_evict(const PagedDims& d, const PagedEvictPlan& p, const PagedEvictArgs& a, cudaStream_t s) {
    const cudaError_t e = p.cluster == 1 ? select_t<1>(d, p, a, s) : p.cluster == 2 ? select_t<2>(d, p, a, s)
                        : p.cluster == 4 ? select_t<4>(d, p, a, s) : select_t<8>(d, p, a, s);
    if (e != cudaSuccess || p.moves == 0) return e;    // no sequence can be longer than the budget
    if (d.bf16) return d.d == 128 ? move_t<__nv_bfloat16, 128>(d, p, a, s) : move_t<__nv_bfloat16, 64>(d, p, a, s);
    return d.d == 128 ? move_t<float, 128>(d, p, a, s) : move_t<float, 64>(d, p, a, s);
}

}  // namespace sa
