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

// What a CTA needs of the unit its cursor is in.
template <typename T, int D>
struct PgUnit {
    PgList ls;
    int b, g, nt, end, s1, newest, gh, head0;      // tiles, this CTA's end among them, its last list entry, heads
    size_t qh0;
    const T* q;
    const int32_t* trow;
    const int32_t* prow;                           // positions, or null where they are not needed or the slots
    __device__ __forceinline__ PgUnit(const PgDecodeIo& io, const PgCursor& cur, long long left) {
        const PagedView& c = io.c;
        b = cur.b;
        g = cur.sub / c.nhb;
        const int hb = cur.sub - g * c.nhb;
        ls = pg_list(c, b, io.sink, io.local);
        nt = max(1, (ls.n + kPgTile - 1) / kPgTile);
        end = (int)min((long long)nt, cur.tile + left);
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

// Hands in this CTA's part of a unit, own = m[HB], l[HB], acc[HB][D] in shared
// memory: written out where the CTA has the whole unit, else a record, and the
// last CTA of the unit joins them (f: hu (n + 2) floats).  All threads call.
template <typename T, int D, int HB, int NT>
__device__ void pg_hand_in(const PgDecodeIo& io, const PgSplit& sp, const PgCursor& cur, const PgUnit<T, D>& u,
                           const float* own, float* f) {
    const int gh = u.gh, hu = io.c.hu;
    if (cur.tile == 0 && u.end == u.nt) {
        for (int x = threadIdx.x; x < gh * D; x += NT) {
            const int h = x / D, e = x - h * D;
            pg_write<D>(io, u.qh0 + h, e, own[2 * HB + x], own[h], own[HB + h]);
        }
        return;
    }
    float* r = pg_rec(io.rec, hu * (2 + D), blockIdx.x, cur.tile == 0);
    for (int x = threadIdx.x; x < gh * (D + 2); x += NT) {
        if (x < gh) r[x] = own[x];
        else if (x < 2 * gh) r[hu + x - gh] = own[HB + x - gh];
        else r[2 * hu + x - 2 * gh] = own[2 * HB + x - 2 * gh];
    }
    const int first = sp.owner(cur.unit0), n = sp.owner(cur.unit0 + u.nt - 1) - first + 1;
    unsigned* cnt = io.cnt + (size_t)cur.b * io.c.Hkv * io.c.nhb + cur.sub;
    if (last_cta_of_unit(cnt, n)) {
        pg_join<D, NT>(io, first, n, u.qh0, gh, f);
        reset_counter(cnt);
    }
}

__device__ __forceinline__ void pg_next(PgCursor& cur, int per, int nt) {
    cur.unit0 += nt;
    cur.tile = 0;
    if (++cur.sub == per) { cur.sub = 0; ++cur.b; }
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
constexpr int kPtThreads = 128;
constexpr int kPtWarps = kPtThreads / 32;

template <int D>
struct PgStage {
    static constexpr int kPitch = 2 * D + 16;
    static constexpr int kBytes = 2 * 16 * kPitch + 16 * 4;      // K rows, V rows, distances
    static constexpr int kStages = D == 128 ? 3 : 6;             // 8 KB of rows in flight per warp and stage pair
};

template <int D, int HB>
__host__ __device__ constexpr size_t pg_tc_smem() {
    const size_t ring = (size_t)kPtWarps * PgStage<D>::kStages * PgStage<D>::kBytes;
    // over the ring: the warps' states, the CTA's, or the join's weights
    const size_t merge = sizeof(float) * ((size_t)kPtWarps * HB * (D + 4 + 2) + HB * (D + 2));
    const size_t join = sizeof(float) * (HB == 16 ? 16 : 8) * (kPgSlots + 2);
    const size_t m = merge > join ? merge : join;
    return ring > m ? ring : m;
}

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
__global__ void __launch_bounds__(kPtThreads, 2)
k_paged_tc(PgDecodeIo io) {
    using St = PgStage<D>;
    constexpr int S = St::kStages, P = St::kPitch;
    constexpr int KS = D / 16, MT = D / 16;
    constexpr int CPR = D / 8, RPI = 32 / CPR;                   // chunks per row, rows per copy instruction
    constexpr int R = HB == 16 ? 2 : 1;                          // query rows per lane
    extern __shared__ __align__(16) unsigned char smem[];
    const PagedView& c = io.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, t = lane & 3;
    const int per = c.Hkv * c.nhb;
    unsigned char* ring = smem + (size_t)warp * S * St::kBytes;
    const uint32_t ring_u = tc::smem_u32(ring);
    PgSplit sp;
    PgCursor cur;
    long long t0, t1;
    if (!pg_locate<kPtThreads>(c.B, per, io.min_tiles, blockIdx.x, SA_PG_TILES(io), sp, cur, t0, t1)) return;

    while (t0 < t1) {
        const PgUnit<__nv_bfloat16, D> u(io, cur, t1 - t0);
        const __nv_bfloat16* K = static_cast<const __nv_bfloat16*>(c.k) + (lane % CPR) * 8;
        const __nv_bfloat16* V = static_cast<const __nv_bfloat16*>(c.v) + (lane % CPR) * 8;
        // this warp's steps: 16 list entries from row0 + i kPgTile
        const int row0 = cur.tile * kPgTile + warp * 16;
        const int n = u.s1 > row0 ? (u.s1 - row0 + kPgTile - 1) / kPgTile : 0;
        const bool own_pos = u.prow != nullptr;
        auto fetch = [&](int i) { return pg_fetch(io, u.ls, u.trow, u.prow, row0 + i * kPgTile + (lane & 15), i < n ? u.s1 : 0); };
        auto issue = [&](int i, const PgRaw& raw) {
            float dist;
            const long long off = pg_see(io, raw, own_pos, u.g, u.newest, dist);
            const uint32_t base = ring_u + (uint32_t)(i % S) * St::kBytes;
            if (lane < 16)
                *reinterpret_cast<float*>(ring + (i % S) * St::kBytes + 32 * P + 4 * lane) = off >= 0 ? dist : INFINITY;
#pragma unroll
            for (int j = 0; j < 16 / RPI; ++j) {
                const int row = j * RPI + lane / CPR;
                const long long o = __shfl_sync(0xffffffffu, off, row);
                const uint32_t at = base + row * P + (lane % CPR) * 16;
                pg_cp16(at, K + (o < 0 ? 0 : o), o >= 0);
                pg_cp16(at + 16 * P, V + (o < 0 ? 0 : o), o >= 0);
            }
        };
        {
            PgRaw raw[S - 1];
#pragma unroll
            for (int i = 0; i < S - 1; ++i) raw[i] = fetch(i);
#pragma unroll
            for (int i = 0; i < S - 1; ++i) {
                if (i < n) issue(i, raw[i]);
                tc::cp_commit();
            }
        }
        PgRaw ahead = fetch(S - 1);

        uint32_t qa[KS][2 * R];
        float sl[R], m[R], l[R], o[R][MT][4];
        int head[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            head[k] = HB == 4 ? (r & 3) : r + 8 * k;
            sl[k] = u.slope2(io, head[k]);
            const __nv_bfloat16* q = u.q + (size_t)head[k] * D + 2 * t;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                qa[ks][k] = head[k] < u.gh ? *reinterpret_cast<const uint32_t*>(q + ks * 16) : 0u;
                qa[ks][R + k] = head[k] < u.gh ? *reinterpret_cast<const uint32_t*>(q + ks * 16 + 8) : 0u;
            }
            m[k] = -INFINITY;
            l[k] = 0.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[k][mt][j] = 0.f;
        }

        for (int i = 0; i < n; ++i) {
            __syncwarp();                                         // stage i - 1 has been read by all lanes
            if (i + S - 1 < n) issue(i + S - 1, ahead);
            tc::cp_commit();
            ahead = fetch(i + S);
            tc::cp_wait<S - 1>();
            __syncwarp();
            const uint32_t kt = ring_u + (uint32_t)(i % S) * St::kBytes, vt = kt + 16 * P;
            const float* dist = reinterpret_cast<const float*>(ring + (i % S) * St::kBytes + 32 * P);
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
                const int y = row0 + i * kPgTile + 2 * t;
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
        tc::cp_wait<0>();
        __syncthreads();                                          // the ring is free: states over it

        constexpr int LD = D + 4;
        float* acc = reinterpret_cast<float*>(smem);              // [warp][HB][LD]
        float* ml = acc + kPtWarps * HB * LD;                     // [warp][HB][2]
        float* own = ml + kPtWarps * HB * 2;                      // m[HB], l[HB], acc[HB][D]
#pragma unroll
        for (int k = 0; k < R; ++k) {
            l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
            l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
            if (t == 0 && (HB != 4 || r < 4)) {
                ml[(warp * HB + head[k]) * 2] = m[k];
                ml[(warp * HB + head[k]) * 2 + 1] = l[k];
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float y = o[k][mt][j];
                    if (HB == 4) y += __shfl_xor_sync(0xffffffffu, y, 2);
                    const int h = 2 * t + (j & 1) + 8 * k;
                    if (HB != 4 || t < 2) acc[(warp * HB + h) * LD + mt * 16 + r + (j >> 1) * 8] = y;
                }
        }
        __syncthreads();
        for (int x = threadIdx.x; x < u.gh * D; x += kPtThreads) {
            const int h = x / D, e = x - h * D;
            float M = -INFINITY, A = 0.f, L = 0.f;
#pragma unroll
            for (int w = 0; w < kPtWarps; ++w) M = fmaxf(M, ml[(w * HB + h) * 2]);
#pragma unroll
            for (int w = 0; w < kPtWarps; ++w) {
                const float mw = ml[(w * HB + h) * 2];
                const float f = mw == -INFINITY ? 0.f : ex2(mw - M);
                A = fmaf(acc[(w * HB + h) * LD + e], f, A);
                L = fmaf(ml[(w * HB + h) * 2 + 1], f, L);
            }
            own[2 * HB + x] = A;
            if (e == 0) { own[h] = M; own[HB + h] = L; }
        }
        __syncthreads();
        // the join's scratch lies over the warps' states: own has been written out by then
        pg_hand_in<__nv_bfloat16, D, HB, kPtThreads>(io, sp, cur, u, own, acc);
        __syncthreads();
        t0 += u.end - cur.tile;
        pg_next(cur, per, u.nt);
    }
}

// ---- fp32: CUDA cores --------------------------------------------------------------
// A lane group reads one cache row per step (16-byte loads, four rows in
// flight) and keeps the unit's states in registers.
template <int D, int GB>
__global__ void __launch_bounds__(kThreads, 2)
k_paged_cc(PgDecodeIo io) {
    using T = float;
    using Gm = Geom<T, D>;
    constexpr int EPC = Gm::EPC, CPR = Gm::CPR, GPW = Gm::GPW, NG = Gm::NG;
    constexpr int UN = 4;                      // rows in flight per lane group
    __shared__ float sm[kWarps * GB * (D + 2)];
    __shared__ float s_own[GB * (D + 2)];
    __shared__ float s_join[8 * (kPgSlots + 2)];
    const PagedView& c = io.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int li = lane % CPR, gsub = lane / CPR;
    const int per = c.Hkv * c.nhb;
    PgSplit sp;
    PgCursor cur;
    long long t0, t1;
    if (!pg_locate<kThreads>(c.B, per, io.min_tiles, blockIdx.x, SA_PG_TILES(io), sp, cur, t0, t1)) return;

    while (t0 < t1) {
        const PgUnit<T, D> u(io, cur, t1 - t0);
        const T* K = static_cast<const T*>(c.k) + li * EPC;
        const T* V = static_cast<const T*>(c.v) + li * EPC;
        float qv[GB][EPC], sl[GB];
#pragma unroll
        for (int h = 0; h < GB; ++h) {
            sl[h] = u.slope2(io, h);
            if (h < u.gh) {
                unpack<T>(ld_nc16(u.q + (size_t)h * D + li * EPC), qv[h]);
            } else {
#pragma unroll
                for (int e = 0; e < EPC; ++e) qv[h][e] = 0.f;
            }
        }
        Online<GB, EPC> os;
        os.init();
        for (int wt = cur.tile * kPgTile + warp * UN * GPW; wt < u.s1; wt += UN * NG) {
            uint4 wk[UN], wv[UN];
            float dist[UN];
            bool ok[UN];
#pragma unroll
            for (int j = 0; j < UN; ++j) {
                const PgRaw raw = pg_fetch(io, u.ls, u.trow, u.prow, wt + j * GPW + gsub, u.s1);
                const long long off = pg_see(io, raw, u.prow != nullptr, u.g, u.newest, dist[j]);
                ok[j] = off >= 0;
                wk[j] = ok[j] ? ld_stream16(K + off) : make_uint4(0, 0, 0, 0);
                wv[j] = ok[j] ? ld_stream16(V + off) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < UN; ++j) {
                const int y = wt + j * GPW + gsub;
                float kf[EPC], vf[EPC];
                unpack<T>(wk[j], kf);
                unpack<T>(wv[j], vf);
#pragma unroll
                for (int h = 0; h < GB; ++h) {
                    float x = 0.f;
#pragma unroll
                    for (int e = 0; e < EPC; ++e) x = fmaf(qv[h][e], kf[e], x);
                    x = pg_logit(io, group_sum<CPR>(x), sl[h], dist[j]);
                    if (ok[j] && x != -INFINITY) os.add(h, x, vf);       // e^-inf: no weight
                    if (io.x != nullptr && li == h % CPR && h < u.gh && y < u.s1)
                        io.x[(u.qh0 + h) * io.ldx + y] = ok[j] ? x : -INFINITY;
                }
            }
        }
        warp_merge<GB, EPC, CPR>(os);
        cta_merge_store<GB, EPC, CPR, D>(os, sm, s_own);         // m[GB], l[GB], acc[GB][D]
        pg_hand_in<T, D, GB, kThreads>(io, sp, cur, u, s_own, s_join);
        __syncthreads();
        t0 += u.end - cur.tile;
        pg_next(cur, per, u.nt);
    }
}

// weight_out = weight + the step's attention weights summed over the group's
// heads, from the logits the decode left and the rows' masses.  One thread per
// slot; bound: HBM (or L2, where the logits still are) for 4 G + 8 bytes a slot.
constexpr int kPgWTile = 1024;         // slots per CTA step

__global__ void __launch_bounds__(kThreads)
k_paged_weights(PgDecodeIo io, const float* weight, float* weight_out) {
    const PagedView& c = io.c;
    auto tiles = [&](int b) { return max(1, (pg_length(c, b) + kPgWTile - 1) / kPgWTile); };
    PgSplit sp;
    PgCursor cur;
    long long t0, t1;
    if (!pg_locate<kThreads>(c.B, c.Hkv, 1, blockIdx.x, tiles, sp, cur, t0, t1)) return;
    for (long long t = t0; t < t1; ++t) {
        const int b = cur.b, g = cur.sub;
        const PgList ls = pg_list(c, b, io.sink, io.local);
        const size_t u = (size_t)b * c.Hkv + g;
        const float* xs = io.x + ((size_t)b * c.Hq + (size_t)g * c.G) * io.ldx;
        const float* l2 = io.lse2 + (size_t)b * c.Hq + (size_t)g * c.G;
        const int s1 = min(ls.len, (cur.tile + 1) * kPgWTile), gap = ls.len - ls.n;
        for (int slot = cur.tile * kPgWTile + threadIdx.x; slot < s1; slot += kThreads) {
            float p = 0.f;
            if (slot < ls.s_eff || slot >= ls.s_eff + gap) {
                const float* x = xs + (slot < ls.s_eff ? slot : slot - gap);
#pragma unroll 4
                for (int h = 0; h < c.G; ++h) {
                    const float y = __ldcg(x + (size_t)h * io.ldx);
                    p += y == -INFINITY ? 0.f : ex2(y - __ldg(l2 + h));
                }
            }
            const size_t w = u * c.ldw + slot;
            weight_out[w] = (weight == nullptr ? 0.f : weight[w]) + p;
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
    constexpr size_t smem = pg_tc_smem<D, HB>();
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
    io.min_tiles = 1;
    io.ldx = p.ldx;
    const cudaError_t e = d.d == 128 ? decode_launch<128>(d, p, io, s) : decode_launch<64>(d, p, io, s);
    if (e != cudaSuccess || !weights) return e;
    const long long steps = (long long)d.U() * ((d.cap + kPgWTile - 1) / kPgWTile);
    const unsigned grid = (unsigned)(steps < 148 * 8 ? steps : 148 * 8);
    k_paged_weights<<<grid, kThreads, 0, s>>>(io, a.weight, a.weight_out);
    return cudaGetLastError();
}

}  // namespace sa
