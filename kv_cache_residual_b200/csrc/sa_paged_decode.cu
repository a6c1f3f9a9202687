// Decode attention of one query per sequence over the paged cache.
//
//   x_hs = cap(scale q_h . k_s) - slope_h (newest - pos_s)
//   out_h = sum_s softmax_s(x_hs) v_s          (one pass, running maximum and sum)
//
// A unit is a KV head of a sequence with up to eight of its query heads.  All
// units' 64-slot tiles are split evenly over two CTAs per SM (sa_paged.cuh), so
// ragged batches, one long sequence and many short ones load the GPU alike; a
// unit cut by the split is joined by the last of its CTAs to finish.
//
// k_paged_tc (bf16): matrix instructions.  k_paged_cc (fp32): CUDA cores.
#include "sa_paged_decode.cuh"
#include "sa_tc.cuh"

namespace sa {

// tiles of a unit of sequence b: at least one, so that an empty row is written
#define SA_PG_TILES(io) \
    [&](int b) { return max(1, (pg_list((io).c, b, (io).sink, (io).local).n + kPgTile - 1) / kPgTile); }

// What a CTA needs of the unit its cursor is in: [tile, end) are its tiles, none
// where its range ends among the extra ones.
template <typename T, int D>
struct PgUnit {
    PgList ls;
    int b, g, nt, tile, end, s1, newest, gh, head0;   // s1: the end of its list entries; gh heads from head0 on
    size_t qh0;
    const T* q;
    const int32_t* trow;
    const int32_t* prow;                           // positions, or null where they are not needed or the slots
    __device__ __forceinline__ PgUnit(const PgDecodeIo& io, const PgSplit& sp, const PgCursor& cur, unsigned left) {
        const PagedView& c = io.c;
        b = cur.b;
        g = cur.sub / c.nhb;
        const int hb = cur.sub - g * c.nhb;
        ls = pg_list(c, b, io.sink, io.local);
        nt = max(1, (ls.n + kPgTile - 1) / kPgTile);
        tile = max(0, cur.tile - sp.extra);
        end = max(0, (int)min((unsigned)(nt + sp.extra), cur.tile + left) - sp.extra);
        s1 = min(ls.n, end * kPgTile);
        newest = pg_newest(c, b, ls.len);
        head0 = g * c.G + hb * c.hu;
        gh = min(c.hu, c.G - hb * c.hu);
        qh0 = (size_t)b * c.Hq + head0;
        q = static_cast<const T*>(io.q) + (long long)b * io.q_stride + (long long)head0 * D;
        trow = c.table + (size_t)b * c.max_pages;
        prow = c.pos == nullptr || (io.local == 0 && io.slopes == nullptr)
                   ? nullptr : c.pos + ((size_t)b * c.Hkv + g) * c.ldw;
    }
    __device__ __forceinline__ float slope2(const PgDecodeIo& io, int h) const {
        return h < gh && io.slopes != nullptr ? __ldg(io.slopes + head0 + h) * kLog2e : 0.f;
    }
};

// This CTA's part of a unit: written out where the CTA has the whole unit, else
// a record, which the last CTA of the unit joins with the others.
template <typename T, int D>
struct PgPart {
    bool whole;
    float* rec;
    __device__ __forceinline__ PgPart(const PgDecodeIo& io, const PgUnit<T, D>& u)
        : whole(u.tile == 0 && u.end == u.nt), rec(pg_rec(io.rec, io.c.hu * (2 + D), blockIdx.x, u.tile == 0)) {}
    // accumulator A of dim e of head h, mass L relative to 2^M
    __device__ __forceinline__ void put(const PgDecodeIo& io, const PgUnit<T, D>& u, int h, int e, float A, float M,
                                        float L) const {
        if (whole) {
            io.out[(u.qh0 + h) * D + e] = A * pg_inv(L);
            if (e == 0) pg_write_lse(io, u.qh0 + h, M, L);
        } else {
            rec[2 * io.c.hu + h * D + e] = A;
            if (e == 0) { rec[h] = M; rec[io.c.hu + h] = L; }
        }
    }
};

// after all have put: the unit's last CTA joins.  All threads call; f as pg_join.
template <typename T, int D, int NT>
__device__ __forceinline__ void pg_hand_in(const PgDecodeIo& io, const PgSplit& sp, const PgCursor& cur,
                                           const PgUnit<T, D>& u, const PgPart<T, D>& part, float* f) {
    if (part.whole) return;
    const unsigned own0 = cur.unit0 + sp.extra;
    const int first = (int)sp.owner(own0), n = (int)sp.owner(own0 + u.nt - 1) - first + 1;
    unsigned* cnt = io.cnt + (size_t)cur.b * io.c.Hkv * io.c.nhb + cur.sub;
    if (last_cta_of_unit(cnt, n)) {
#pragma unroll 1
        for (int h0 = 0; h0 < u.gh; h0 += 8) {
            pg_join<D, NT>(io, first, n, u.qh0 + h0, h0, min(8, u.gh - h0), f);
            __syncthreads();
        }
        reset_counter(cnt);
    }
}

// the cursor's unit that is left, the next one; t0 moves along.  False at the range's end.
template <typename T, int D>
__device__ __forceinline__ bool pg_next(const PgDecodeIo& io, const PgSplit& sp, PgCursor& cur, PgUnit<T, D>& u,
                                        unsigned& t0, unsigned t1) {
    const int n = u.nt + sp.extra;
    t0 += n - cur.tile;                            // past t1 where the unit goes on in another CTA
    if (t0 >= t1) return false;
    cur.unit0 += n;
    cur.tile = 0;
    if (++cur.sub == io.c.Hkv * io.c.nhb) { cur.sub = 0; ++cur.b; }
    u = PgUnit<T, D>(io, sp, cur, t1 - t0);
    return u.end > u.tile;                         // none of its own: then the range ends there
}

// ---- bf16: matrix instructions --------------------------------------------------
// A warp takes 16 of a tile's slots through a ring of its own (cp.async, rows
// padded by 16 bytes for ldmatrix), with no barrier among warps until the unit
// ends:
//   S   = Q K^T     A = the unit's queries, B = 16 key rows (ldmatrix)
//   O^T += V^T P^T  A = value rows (ldmatrix.trans), B = the weights: the layout
//                   of S's accumulators is that of B's fragments, so weights
//                   never move between lanes
// Lane (r = lane / 4, t = lane % 4) holds row r (and r + 8 where HB = 16) of S at
// slots 2t, 2t+1, 8+2t, 9+2t, and dims 16 i + r, + 8 of heads 2t, 2t+1 of O^T.
// Weights are fp32: they enter as three bf16 parts (24 bits), so that the only
// rounding below 32 bits is the cache's own.  With up to four heads rows 4..7
// repeat rows 0..3 and two of the parts share one instruction.  The maximum is
// moved only when a logit passes it by 8 (2^8 in the sums): one vote per step.
constexpr int kPtThreads = 256;
constexpr int kPtWarps = kPtThreads / 32;
constexpr int kPtStep = kPtWarps * 16;          // list entries of a step of the CTA

template <int D>
struct PgStage {
    static constexpr int kPitch = 2 * D + 16;
    static constexpr int kBytes = 2 * 16 * kPitch + 16 * 4;      // K rows, V rows, distances
    static constexpr int kStages = D == 128 ? 3 : 5;             // with the scratch, what an SM has room for
    static constexpr int kRing = kPtWarps * kStages * kBytes;
    static constexpr int kAcc = kPtWarps * 4 * (D + 4);          // floats: four heads' states of the warps
    static constexpr int kScratch = kAcc > kPgJoinFloats ? kAcc : kPgJoinFloats;
    static constexpr size_t kSmem = kRing + 4 * (size_t)kScratch;
};

__device__ __forceinline__ void pg_cp16(uint32_t s, const void* g, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(s), "l"(g), "r"(ok ? 16 : 0) : "memory");
}

// p = hi + mid + lo, bf16 each
__device__ __forceinline__ void split3(float p0, float p1, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
    const float2 hf = __bfloat1622float2(h);
    tc::split_bf2(p0 - hf.x, p1 - hf.y, mid, lo);
    hi = *reinterpret_cast<const uint32_t*>(&h);
}

template <int D, int HB>
__global__ void __launch_bounds__(kPtThreads, 1)
k_paged_tc(PgDecodeIo io) {
    using T = __nv_bfloat16;
    using St = PgStage<D>;
    constexpr int S = St::kStages, P = St::kPitch;
    constexpr int KS = D / 16, MT = D / 16;
    constexpr int CPR = D / 8, RPI = 32 / CPR;                   // chunks per row, rows per copy instruction
    constexpr int R = HB == 16 ? 2 : 1;                          // query rows per lane
    constexpr int LD = D + 4;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float s_ml[kPtWarps][HB][2];
    const PagedView& c = io.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, t = lane & 3;
    const int per = c.Hkv * c.nhb;
    unsigned char* ring = smem + warp * S * St::kBytes;
    float* scratch = reinterpret_cast<float*>(smem + St::kRing);
    const uint32_t ring_u = tc::smem_u32(ring);
    const T* K = static_cast<const T*>(c.k) + (lane % CPR) * 8;
    const T* V = static_cast<const T*>(c.v) + (lane % CPR) * 8;
    PgSplit sp;
    PgCursor cur;
    unsigned t0, t1;
    cudaTriggerProgrammaticLaunchCompletion();                   // the weights' kernel may come and wait
    if (!pg_locate<kPtThreads>(c.B, per, io.extra, blockIdx.x, SA_PG_TILES(io), sp, cur, t0, t1)) return;

    int head[R], stage = 0;                                       // ring stage of the unit's first step
    uint32_t qa[KS][2 * R];
    float sl[R];
    PgRaw ahead;
    int row0, n = 0;                                              // this warp's steps: 16 list entries from row0 + i kPtStep
    PgUnit<T, D> u(io, sp, cur, t1 - t0), done = u;               // the unit at hand, the one before it
    PgCursor at = cur;                                            // of `done`
    float m[R], l[R], o[R][MT][4];                                // maxima, masses, accumulators of the unit

    auto fetch = [&](int i) {
        return pg_fetch(io, u.ls, u.trow, u.prow, row0 + i * kPtStep + (lane & 15), i < n ? u.s1 : 0);
    };
    auto issue = [&](int i, const PgRaw& raw) {
        float dist;
        const long long off = pg_see(io, raw, u.prow != nullptr, u.g, u.newest, dist);
        const int at = (stage + i) % S * St::kBytes;
        if (lane < 16) *reinterpret_cast<float*>(ring + at + 32 * P + 4 * lane) = off >= 0 ? dist : INFINITY;
#pragma unroll
        for (int j = 0; j < 16 / RPI; ++j) {
            const int row = j * RPI + lane / CPR;
            const long long o = __shfl_sync(0xffffffffu, off, row);
            const uint32_t to = ring_u + at + row * P + (lane % CPR) * 16;
            pg_cp16(to, K + (o < 0 ? 0 : o), o >= 0);
            pg_cp16(to + 16 * P, V + (o < 0 ? 0 : o), o >= 0);
        }
    };
    // a unit's queries and the copies of its first steps; runs while the unit
    // before it is handed in
    auto begin = [&]() {
        stage = (stage + n) % S;
        row0 = u.tile * kPgTile + warp * 16;
        n = u.s1 > row0 ? (u.s1 - row0 + kPtStep - 1) / kPtStep : 0;
        PgRaw raw[S - 1];
#pragma unroll
        for (int i = 0; i < S - 1; ++i) raw[i] = fetch(i);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            head[k] = HB == 4 ? (r & 3) : r + 8 * k;
            sl[k] = u.slope2(io, head[k]);
            const T* q = u.q + (size_t)head[k] * D + 2 * t;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                qa[ks][k] = head[k] < u.gh ? __ldg(reinterpret_cast<const unsigned*>(q + ks * 16)) : 0u;
                qa[ks][R + k] = head[k] < u.gh ? __ldg(reinterpret_cast<const unsigned*>(q + ks * 16 + 8)) : 0u;
            }
        }
#pragma unroll
        for (int i = 0; i < S - 1; ++i) {
            if (i < n) issue(i, raw[i]);
            tc::cp_commit();
        }
        ahead = fetch(S - 1);
    };
#pragma unroll 1
    for (bool handed = true, more = u.end > u.tile;;) {
        if (more) begin();
        if (!handed) {
            const PgPart<T, D> part(io, done);
#pragma unroll
            for (int k = 0; k < R; ++k) {
                l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
                l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
                if (t == 0 && (HB != 4 || r < 4)) {
                    s_ml[warp][(HB == 4 ? r & 3 : r + 8 * k)][0] = m[k];
                    s_ml[warp][(HB == 4 ? r & 3 : r + 8 * k)][1] = l[k];
                }
            }
            // four heads at a time through the scratch
#pragma unroll
            for (int hq = 0; hq < HB / 4; ++hq) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float y = o[hq / 2][mt][j];
                        if (HB == 4) y += __shfl_xor_sync(0xffffffffu, y, 2);        // its parts' two columns
                        if (t / 2 == (hq & 1))
                            scratch[(warp * 4 + (2 * t + (j & 1)) % 4) * LD + mt * 16 + r + (j >> 1) * 8] = y;
                    }
                __syncthreads();
                for (int x = threadIdx.x; x < 4 * D; x += kPtThreads) {
                    const int h4 = x / D, e = x - h4 * D, h = 4 * hq + h4;
                    if (h >= done.gh) break;
                    float M = -INFINITY, A = 0.f, L = 0.f;
#pragma unroll
                    for (int w = 0; w < kPtWarps; ++w) M = fmaxf(M, s_ml[w][h][0]);
#pragma unroll
                    for (int w = 0; w < kPtWarps; ++w) {
                        const float mw = s_ml[w][h][0];
                        const float f = mw == -INFINITY ? 0.f : ex2(mw - M);
                        A = fmaf(scratch[(w * 4 + h4) * LD + e], f, A);
                        L = fmaf(s_ml[w][h][1], f, L);
                    }
                    part.put(io, done, h, e, A, M, L);
                }
                __syncthreads();
            }
            pg_hand_in<T, D, kPtThreads>(io, sp, at, done, part, scratch);
        }
        if (!more) break;
        __syncthreads();                                          // the scratch has been read
#pragma unroll
        for (int k = 0; k < R; ++k) {
            m[k] = -INFINITY;
            l[k] = 0.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[k][mt][j] = 0.f;
        }
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            __syncwarp();                                         // stage i - 1 has been read by all lanes
            if (i + S - 1 < n) issue(i + S - 1, ahead);
            tc::cp_commit();
            ahead = fetch(i + S);
            tc::cp_wait<S - 1>();
            __syncwarp();
            const int at = (stage + i) % S * St::kBytes;
            const uint32_t kt = ring_u + at, vt = kt + 16 * P;
            const float* dist = reinterpret_cast<const float*>(ring + at + 32 * P);
            float s[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[h][j] = 0.f;
#pragma unroll
            for (int kp = 0; kp < KS / 2; ++kp)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t b[4];
                    tc::ldsm4(kt + (h * 8 + (lane & 7)) * P + (kp * 32 + (lane >> 3) * 8) * 2, b);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t (&a)[2 * R] = qa[2 * kp + e];
                        tc::mma_bf16(s[h], a[0], R == 2 ? a[1] : 0u, a[R], R == 2 ? a[2 * R - 1] : 0u, b[2 * e], b[2 * e + 1]);
                    }
                }
            // logits of this lane's rows and slots (2t, 2t+1, 8+2t, 9+2t)
            float x[R][4];
            const float2 d0 = *reinterpret_cast<const float2*>(dist + 2 * t);
            const float2 d1 = *reinterpret_cast<const float2*>(dist + 8 + 2 * t);
            const float dd[4] = {d0.x, d0.y, d1.x, d1.y};
            bool rises = false;
#pragma unroll
            for (int k = 0; k < R; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[k][j] = dd[j] == INFINITY ? -INFINITY : pg_logit(io, s[j >> 1][2 * k + (j & 1)], sl[k], dd[j]);
                    rises |= x[k][j] > m[k] + 8.f;
                }
            if (io.x != nullptr) {
                const int y = row0 + i * kPtStep + 2 * t;
#pragma unroll
                for (int k = 0; k < R; ++k)
                    if (head[k] < u.gh && (HB != 4 || r < 4)) {
                        float* xs = io.x + (u.qh0 + head[k]) * io.ldx + y;      // rows of whole tiles: both pairs fit
                        *reinterpret_cast<float2*>(xs) = make_float2(x[k][0], x[k][1]);
                        *reinterpret_cast<float2*>(xs + 8) = make_float2(x[k][2], x[k][3]);
                    }
            }
            if (__any_sync(0xffffffffu, rises)) {
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    float mx = fmaxf(fmaxf(x[k][0], x[k][1]), fmaxf(x[k][2], x[k][3]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    mx = fmaxf(mx, m[k]);
                    const float sc = m[k] == -INFINITY ? 0.f : ex2(m[k] - mx);
                    m[k] = mx;
                    l[k] *= sc;
                    const float c0 = __shfl_sync(0xffffffffu, sc, 8 * t), c1 = __shfl_sync(0xffffffffu, sc, 8 * t + 4);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        o[k][mt][0] *= c0;
                        o[k][mt][1] *= c1;
                        o[k][mt][2] *= c0;
                        o[k][mt][3] *= c1;
                    }
                }
            }
            uint32_t b[R][3][2];                                  // parts of the weights, slots 2t.. and 8 + 2t..
#pragma unroll
            for (int k = 0; k < R; ++k) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[k][j] = x[k][j] == -INFINITY ? 0.f : ex2(x[k][j] - m[k]);
                    l[k] += x[k][j];
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    split3(x[k][2 * h], x[k][2 * h + 1], b[k][0][h], b[k][1][h], b[k][2][h]);
                    if (HB == 4 && r >= 4) { b[k][0][h] = b[k][1][h]; b[k][2][h] = 0u; }
                }
            }
            const uint32_t va = vt + ((lane & 7) + ((lane >> 4) & 1) * 8) * P + ((lane >> 3) & 1) * 16;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                uint32_t a[4];
                tc::ldsm4t(va + mt * 32, a);
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    tc::mma_bf16(o[k][mt], a[0], a[1], a[2], a[3], b[k][0][0], b[k][0][1]);
                    if (HB != 4) tc::mma_bf16(o[k][mt], a[0], a[1], a[2], a[3], b[k][1][0], b[k][1][1]);
                    tc::mma_bf16(o[k][mt], a[0], a[1], a[2], a[3], b[k][2][0], b[k][2][1]);
                }
            }
        }
        __syncwarp();
        // the unit is done: its successor's first copies go out before it is handed in
        done = u;
        at = cur;
        handed = false;
        more = pg_next(io, sp, cur, u, t0, t1);
    }
    tc::cp_wait<0>();
}

// ---- fp32: CUDA cores --------------------------------------------------------------
// A lane group reads UN cache rows at a time (16-byte loads; the table a step
// ahead).  Their UN GB dot products are summed across the group's W lanes by
// halves, so that they end spread over the lanes: a lane caps, masks and
// exponentiates its own, and the weights come back by shuffles.
template <int GB>
struct PgCc {
    static constexpr int UN = GB == 8 ? 2 : 4;
};

template <int D, int GB>
__global__ void __launch_bounds__(kThreads, 2)
k_paged_cc(PgDecodeIo io) {
    using T = float;
    using Gm = Geom<T, D>;
    constexpr int EPC = Gm::EPC, W = Gm::CPR, GPW = Gm::GPW, NG = Gm::NG, UN = PgCc<GB>::UN;
    // dot product x = row GB + head: the lanes x DUP / NPL .. of the group, their register x % NPL
    constexpr int NV = UN * GB, NPL = NV > W ? NV / W : 1, DUP = NV < W ? W / NV : 1;
    constexpr int JS = GB * DUP / NPL;         // lanes from a row to the next
    static_assert(JS >= 1, "a lane's dot products are of one row");
    __shared__ float sm[kWarps * GB * (D + 2)];
    __shared__ float s_own[GB * (D + 2)];
    __shared__ __align__(16) float s_join[kPgJoinFloats];
    const PagedView& c = io.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int li = lane % W, gsub = lane / W, lane0 = lane - li;
    const int row = li / JS, head0 = li * NPL / DUP % GB;      // of this lane's dot products
    const int per = c.Hkv * c.nhb;
    PgSplit sp;
    PgCursor cur;
    unsigned t0, t1;
    cudaTriggerProgrammaticLaunchCompletion();
    if (!pg_locate<kThreads>(c.B, per, io.extra, blockIdx.x, SA_PG_TILES(io), sp, cur, t0, t1)) return;

    PgUnit<T, D> u(io, sp, cur, t1 - t0);
#pragma unroll 1
    for (bool more = u.end > u.tile; more;) {
        const T* K = static_cast<const T*>(c.k) + li * EPC;
        const T* V = static_cast<const T*>(c.v) + li * EPC;
        const bool own_pos = u.prow != nullptr;
        float qv[GB][EPC], sl[NPL];
        PgRaw raw[UN];
        int wt = u.tile * kPgTile + warp * UN * GPW;
#pragma unroll
        for (int j = 0; j < UN; ++j) raw[j] = pg_fetch(io, u.ls, u.trow, u.prow, wt + j * GPW + gsub, u.s1);
#pragma unroll
        for (int h = 0; h < GB; ++h) {
            if (h < u.gh) {
                unpack<T>(ld_nc16(u.q + (size_t)h * D + li * EPC), qv[h]);
            } else {
#pragma unroll
                for (int e = 0; e < EPC; ++e) qv[h][e] = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i) sl[i] = u.slope2(io, head0 + i);
        float m[NPL], l[NPL];
        Online<GB, EPC> os;
        os.init();
#pragma unroll
        for (int i = 0; i < NPL; ++i) { m[i] = -INFINITY; l[i] = 0.f; }
#pragma unroll 1
        for (; wt < u.s1; wt += UN * NG) {
            uint4 wk[UN], wv[UN];
            float dist = 0.f;
            bool seen = false;                                 // of this lane's row
#pragma unroll
            for (int j = 0; j < UN; ++j) {
                float dj;
                const long long off = pg_see(io, raw[j], own_pos, u.g, u.newest, dj);
                wk[j] = off >= 0 ? ld_stream16(K + off) : make_uint4(0, 0, 0, 0);
                wv[j] = off >= 0 ? ld_stream16(V + off) : make_uint4(0, 0, 0, 0);
                if (row == j) { dist = dj; seen = off >= 0; }
            }
            const int y = wt + row * GPW + gsub;
#pragma unroll
            for (int j = 0; j < UN; ++j)
                raw[j] = pg_fetch(io, u.ls, u.trow, u.prow, wt + UN * NG + j * GPW + gsub, u.s1);
            float v[NV];
#pragma unroll
            for (int j = 0; j < UN; ++j) {
                float kf[EPC];
                unpack<T>(wk[j], kf);
#pragma unroll
                for (int h = 0; h < GB; ++h) {
                    float x = 0.f;
#pragma unroll
                    for (int e = 0; e < EPC; ++e) x = fmaf(qv[h][e], kf[e], x);
                    v[j * GB + h] = x;
                }
            }
            // sums over the group's lanes: while a lane has several, it gives half away
#pragma unroll
            for (int off = W / 2, n = NV; off > 0; off >>= 1) {
                if (n > 1) {
                    n >>= 1;
                    const bool up = (li & off) != 0;
#pragma unroll
                    for (int i = 0; i < n; ++i) {
                        const float give = up ? v[i] : v[i + n];
                        v[i] = (up ? v[i + n] : v[i]) + __shfl_xor_sync(0xffffffffu, give, off);
                    }
                } else {
                    v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
                }
            }
            bool rises = false;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                v[i] = seen ? pg_logit(io, v[i], sl[i], dist) : -INFINITY;
                rises |= v[i] > m[i] + 8.f;
                if (io.x != nullptr && li % DUP == 0 && head0 + i < u.gh && y < u.s1)
                    io.x[(u.qh0 + head0 + i) * io.ldx + y] = v[i];
            }
            if (__any_sync(0xffffffffu, rises)) {
                float sc[NPL];
#pragma unroll
                for (int i = 0; i < NPL; ++i) {
                    float mx = fmaxf(m[i], v[i]);
#pragma unroll
                    for (int off = JS; off < W; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                    sc[i] = m[i] == -INFINITY ? 0.f : ex2(m[i] - mx);
                    l[i] *= sc[i];
                    m[i] = mx;
                }
#pragma unroll
                for (int h = 0; h < GB; ++h) {
                    const float f = __shfl_sync(0xffffffffu, sc[h % NPL], lane0 + h * DUP / NPL);
#pragma unroll
                    for (int e = 0; e < EPC; ++e) os.acc[h][e] *= f;
                }
            }
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                v[i] = v[i] == -INFINITY ? 0.f : ex2(v[i] - m[i]);         // e^-inf: no weight
                l[i] += v[i];
            }
#pragma unroll
            for (int j = 0; j < UN; ++j) {
                float vf[EPC];
                unpack<T>(wv[j], vf);
#pragma unroll
                for (int h = 0; h < GB; ++h) {
                    const int x = j * GB + h;
                    const float p = __shfl_sync(0xffffffffu, v[x % NPL], lane0 + x * DUP / NPL);
#pragma unroll
                    for (int e = 0; e < EPC; ++e) os.acc[h][e] = fmaf(p, vf[e], os.acc[h][e]);
                }
            }
        }
        // the rows' sums, then every head's state in every lane of the group
#pragma unroll
        for (int i = 0; i < NPL; ++i)
#pragma unroll
            for (int off = JS; off < W; off <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
#pragma unroll
        for (int h = 0; h < GB; ++h) {
            os.m[h] = __shfl_sync(0xffffffffu, m[h % NPL], lane0 + h * DUP / NPL);
            os.l[h] = __shfl_sync(0xffffffffu, l[h % NPL], lane0 + h * DUP / NPL);
        }
        warp_merge<GB, EPC, W>(os);
        cta_merge_store<GB, EPC, W, D>(os, sm, s_own);         // m[GB], l[GB], acc[GB][D]
        const PgPart<T, D> part(io, u);
        for (int x = threadIdx.x; x < u.gh * D; x += kThreads) {
            const int h = x / D, e = x - h * D;
            part.put(io, u, h, e, s_own[2 * GB + x], s_own[h], s_own[GB + h]);
        }
        pg_hand_in<T, D, kThreads>(io, sp, cur, u, part, s_join);
        __syncthreads();
        more = pg_next(io, sp, cur, u, t0, t1);
    }
}

// weight_out = weight + the step's attention weights summed over the group's
// heads, from the logits the decode left and the rows' masses.  Four slots per
// thread, four heads' loads of each at once; bound: HBM (or L2, where the logits
// still are) for 4 G + 8 bytes a slot.
constexpr int kPgWUn = 4;
constexpr int kPgWTile = kThreads * kPgWUn;        // slots per CTA step

__global__ void __launch_bounds__(kThreads)
k_paged_weights(PgDecodeIo io, const float* weight, float* weight_out) {
    const PagedView& c = io.c;
    auto tiles = [&](int b) { return max(1, (pg_length(c, b) + kPgWTile - 1) / kPgWTile); };
    PgSplit sp;
    PgCursor cur;
    unsigned t0, t1;
    const bool any = pg_locate<kThreads>(c.B, c.Hkv, 0, blockIdx.x, tiles, sp, cur, t0, t1);
    cudaGridDependencySynchronize();               // the logits and masses
    if (!any) return;
    for (unsigned t = t0; t < t1; ++t) {
        const int b = cur.b, g = cur.sub;
        const PgList ls = pg_list(c, b, io.sink, io.local);
        const size_t u = (size_t)b * c.Hkv + g, row = u * c.ldw;
        const size_t qh0 = (size_t)b * c.Hq + (size_t)g * c.G;
        const int gap = ls.len - ls.n, first = cur.tile * kPgWTile + threadIdx.x;
        float p[kPgWUn], w[kPgWUn];
        int y[kPgWUn];                             // list entry, -1: not listed
#pragma unroll
        for (int j = 0; j < kPgWUn; ++j) {
            const int slot = first + j * kThreads;
            y[j] = slot >= ls.len ? -1 : slot < ls.s_eff ? slot : slot >= ls.s_eff + gap ? slot - gap : -1;
            w[j] = slot < ls.len && weight != nullptr ? weight[row + slot] : 0.f;
            p[j] = 0.f;
        }
        for (int h = 0; h < c.G; h += 4) {
            float x[4][kPgWUn], l2[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                l2[k] = h + k < c.G ? __ldcg(io.lse2 + qh0 + h + k) : 0.f;
                const float* xs = io.x + (qh0 + h + k) * io.ldx;
#pragma unroll
                for (int j = 0; j < kPgWUn; ++j) x[k][j] = h + k < c.G && y[j] >= 0 ? __ldcg(xs + y[j]) : -INFINITY;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int j = 0; j < kPgWUn; ++j) p[j] += x[k][j] == -INFINITY ? 0.f : ex2(x[k][j] - l2[k]);
        }
#pragma unroll
        for (int j = 0; j < kPgWUn; ++j) {
            const int slot = first + j * kThreads;
            if (slot < ls.len) weight_out[row + slot] = w[j] + p[j];
        }
        const int nt = tiles(b);
        if (++cur.tile == nt) {
            cur.tile = 0;
            if (++cur.sub == c.Hkv) { cur.sub = 0; ++cur.b; }
        }
    }
}

template <int D, int HB>
static cudaError_t tc_launch(const PagedDecodePlan& p, const PgDecodeIo& io, cudaStream_t s) {
    static std::atomic<unsigned long long> opted{0};
    constexpr size_t smem = PgStage<D>::kSmem;
    const cudaError_t e = opt_in_smem(k_paged_tc<D, HB>, smem, opted);
    if (e != cudaSuccess) return e;
    k_paged_tc<D, HB><<<p.grid, kPtThreads, smem, s>>>(io);
    return cudaGetLastError();
}

template <int D>
static cudaError_t decode_launch(const PagedDims& d, const PagedDecodePlan& p, const PgDecodeIo& io, cudaStream_t s) {
    if (d.bf16) {
        if (d.G <= 4) return tc_launch<D, 4>(p, io, s);
        return d.G <= 8 ? tc_launch<D, 8>(p, io, s) : tc_launch<D, 16>(p, io, s);
    }
    if (d.G == 1) k_paged_cc<D, 1><<<p.grid, kThreads, 0, s>>>(io);
    else if (d.G == 2) k_paged_cc<D, 2><<<p.grid, kThreads, 0, s>>>(io);
    else if (d.G <= 4) k_paged_cc<D, 4><<<p.grid, kThreads, 0, s>>>(io);
    else k_paged_cc<D, 8><<<p.grid, kThreads, 0, s>>>(io);
    return cudaGetLastError();
}

cudaError_t launch_paged_decode(const PagedDims& d, const PagedDecodePlan& p, const PagedDecodeArgs& a,
                                cudaStream_t s) {
    PgDecodeIo io;
    io.c = a.c;
    io.q = a.q;
    io.q_stride = a.q_stride;
    io.slopes = a.slopes;
    io.out = a.out;
    io.lse = a.lse;
    const bool weights = a.weight_out != nullptr;
    io.lse2 = weights ? reinterpret_cast<float*>(a.ws + p.off_lse) : nullptr;
    io.x = weights ? reinterpret_cast<float*>(a.ws + p.off_x) : nullptr;
    io.rec = reinterpret_cast<float*>(a.ws + p.off_rec);
    io.cnt = reinterpret_cast<unsigned*>(a.ws + p.off_cnt);
    io.scale = a.scale;
    io.qscale = a.scale * kLog2e;
    io.softcap = a.softcap;
    io.cap_in = a.softcap > 0.f ? a.scale / a.softcap : 0.f;
    io.cap_out = a.softcap * kLog2e;
    io.sink = a.sink;
    io.local = a.local;
    io.ldx = p.ldx;
    io.extra = p.extra;
    const cudaError_t e = d.d == 128 ? decode_launch<128>(d, p, io, s) : decode_launch<64>(d, p, io, s);
    if (e != cudaSuccess || !weights) return e;
    const long long steps = (long long)d.U() * ((d.cap + kPgWTile - 1) / kPgWTile);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(steps < 148 * 8 ? steps : 148 * 8));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_paged_weights, io, a.weight, a.weight_out);
}

}  // namespace sa
