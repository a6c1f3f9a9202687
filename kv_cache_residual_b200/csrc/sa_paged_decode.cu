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
// k_paged_cc: the CUDA-core pass.  A lane group reads one cache row per step
// (16-byte loads, four rows in flight) and keeps the unit's states in
// registers.  Bound: HBM for the rows.
#include "sa_paged_decode.cuh"

namespace sa {

template <typename T, int D, int GB>
__global__ void __launch_bounds__(kThreads, 2)
k_paged_cc(PgDecodeIo io) {
    using Gm = Geom<T, D>;
    constexpr int EPC = Gm::EPC, CPR = Gm::CPR, GPW = Gm::GPW, NG = Gm::NG;
    constexpr int UN = 4;                      // rows in flight per lane group
    __shared__ float sm[kWarps * GB * (D + 2)];
    __shared__ float s_own[GB * (D + 2)];
    __shared__ float s_join[kPgHeads * kPgSlots + 2 * kPgHeads];
    const PagedView& c = io.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int li = lane % CPR, gsub = lane / CPR;
    const int per = c.Hkv * c.nhb;
    auto tiles = [&](int b) { return max(1, (pg_list(c, b, io.sink, io.local).n + kPgTile - 1) / kPgTile); };
    PgSplit sp;
    PgCursor cur;
    long long t0, t1;
    if (!pg_locate<kThreads>(c.B, per, io.min_tiles, blockIdx.x, tiles, sp, cur, t0, t1)) return;

    long long t = t0;
    while (t < t1) {
        const int b = cur.b, g = cur.sub / c.nhb, hb = cur.sub - g * c.nhb;
        const PgList ls = pg_list(c, b, io.sink, io.local);
        const int nt = max(1, (ls.n + kPgTile - 1) / kPgTile);
        const int end = (int)min((long long)nt, cur.tile + (t1 - t));
        const int newest = pg_newest(c, b, ls.len);
        const int gh = min(kPgHeads, c.G - hb * kPgHeads);
        const size_t qh0 = (size_t)b * c.Hq + (size_t)g * c.G + hb * kPgHeads;
        const T* qg = static_cast<const T*>(io.q) + (long long)b * io.q_stride + (long long)(g * c.G + hb * kPgHeads) * D;
        const int32_t* trow = c.table + (size_t)b * c.max_pages;
        const T* K = static_cast<const T*>(c.k) + li * EPC;
        const T* V = static_cast<const T*>(c.v) + li * EPC;
        float* xs = io.x == nullptr ? nullptr : io.x + ((size_t)b * c.Hkv + g) * c.cap * c.G + hb * kPgHeads;

        float qv[GB][EPC], sl[GB];
#pragma unroll
        for (int h = 0; h < GB; ++h) {
            const bool ok = h < gh;
            sl[h] = (ok && io.slopes != nullptr) ? __ldg(io.slopes + g * c.G + hb * kPgHeads + h) * kLog2e : 0.f;
            if (ok) {
                unpack<T>(ld_nc16(qg + (size_t)h * D + li * EPC), qv[h]);
            } else {
#pragma unroll
                for (int e = 0; e < EPC; ++e) qv[h][e] = 0.f;
            }
        }
        Online<GB, EPC> os;
        os.init();
        const int s1 = min(ls.n, end * kPgTile);
        for (int wt = cur.tile * kPgTile + warp * UN * GPW; wt < s1; wt += UN * NG) {
            uint4 wk[UN], wv[UN];
            float dist[UN];
            bool ok[UN];
#pragma unroll
            for (int j = 0; j < UN; ++j) {
                const int y = wt + j * GPW + gsub;
                long long off = -1;
                if (y < s1) off = pg_see(io, trow, b, g, ls.slot(y), newest, dist[j]);
                ok[j] = off >= 0;
                wk[j] = ok[j] ? ld_stream16(K + off) : make_uint4(0, 0, 0, 0);
                wv[j] = ok[j] ? ld_stream16(V + off) : make_uint4(0, 0, 0, 0);
                if (!ok[j]) dist[j] = 0.f;
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
                    if (xs != nullptr && li == h % CPR && h < gh && y < s1)
                        xs[(size_t)y * c.G + h] = ok[j] ? x : -INFINITY;
                }
            }
        }
        warp_merge<GB, EPC, CPR>(os);
        cta_merge_store<GB, EPC, CPR, D>(os, sm, s_own);         // m[GB], l[GB], acc[GB][D]
        const long long uend = cur.unit0 + nt;
        if (cur.tile == 0 && end == nt) {
            for (int x = threadIdx.x; x < gh * D; x += kThreads) {
                const int h = x / D, e = x - h * D;
                pg_write<D>(io, qh0 + h, e, s_own[2 * GB + x], s_own[h], s_own[GB + h]);
            }
            __syncthreads();
        } else {
            float* r = pg_rec(io.rec, kPgHeads * (2 + D), blockIdx.x, cur.tile == 0);
            for (int x = threadIdx.x; x < gh * (D + 2); x += kThreads) {
                if (x < gh) r[x] = s_own[x];
                else if (x < 2 * gh) r[kPgHeads + x - gh] = s_own[GB + x - gh];
                else r[2 * kPgHeads + x - 2 * gh] = s_own[2 * GB + x - 2 * gh];
            }
            const int first = sp.owner(cur.unit0), n = sp.owner(uend - 1) - first + 1;
            unsigned* cnt = io.cnt + (size_t)b * per + cur.sub;
            if (last_cta_of_unit(cnt, n)) {
                pg_join<D, kThreads>(io, kPgHeads * (2 + D), first, n, qh0, gh, s_join);
                reset_counter(cnt);
            }
            __syncthreads();
        }
        t += end - cur.tile;
        cur.unit0 = uend;
        cur.tile = 0;
        if (++cur.sub == per) { cur.sub = 0; ++cur.b; }
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
        const float* xs = io.x + u * c.cap * c.G;
        const float* l2 = io.lse2 + (size_t)b * c.Hq + (size_t)g * c.G;
        const int s1 = min(ls.len, (cur.tile + 1) * kPgWTile);
        for (int slot = cur.tile * kPgWTile + threadIdx.x; slot < s1; slot += kThreads) {
            float p = 0.f;
            const int gap = ls.len - ls.n;
            if (slot < ls.s_eff || slot >= ls.s_eff + gap) {
                const float* x = xs + (size_t)(slot < ls.s_eff ? slot : slot - gap) * c.G;
                if ((c.G & 3) == 0) {
                    for (int h = 0; h < c.G; h += 4) {
                        const float4 y = __ldcg(reinterpret_cast<const float4*>(x + h));
                        p += y.x == -INFINITY ? 0.f : ex2(y.x - __ldg(l2 + h));
                        p += y.y == -INFINITY ? 0.f : ex2(y.y - __ldg(l2 + h + 1));
                        p += y.z == -INFINITY ? 0.f : ex2(y.z - __ldg(l2 + h + 2));
                        p += y.w == -INFINITY ? 0.f : ex2(y.w - __ldg(l2 + h + 3));
                    }
                } else {
                    for (int h = 0; h < c.G; ++h) {
                        const float y = __ldcg(x + h);
                        p += y == -INFINITY ? 0.f : ex2(y - __ldg(l2 + h));
                    }
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

template <typename T, int D>
static cudaError_t decode_launch(const PagedDims& d, const PagedDecodePlan& p, const PgDecodeIo& io, cudaStream_t s) {
    if (d.G == 1) k_paged_cc<T, D, 1><<<p.grid, kThreads, 0, s>>>(io);
    else if (d.G == 2) k_paged_cc<T, D, 2><<<p.grid, kThreads, 0, s>>>(io);
    else if (d.G <= 4) k_paged_cc<T, D, 4><<<p.grid, kThreads, 0, s>>>(io);
    else k_paged_cc<T, D, 8><<<p.grid, kThreads, 0, s>>>(io);
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
    cudaError_t e;
    if (d.bf16) e = d.d == 128 ? decode_launch<__nv_bfloat16, 128>(d, p, io, s) : decode_launch<__nv_bfloat16, 64>(d, p, io, s);
    else e = d.d == 128 ? decode_launch<float, 128>(d, p, io, s) : decode_launch<float, 64>(d, p, io, s);
    if (e != cudaSuccess || !weights) return e;
    const long long steps = (long long)d.U() * ((d.cap + kPgWTile - 1) / kPgWTile);
    const unsigned grid = (unsigned)(steps < 148 * 8 ? steps : 148 * 8);
    k_paged_weights<<<grid, kThreads, 0, s>>>(io, a.weight, a.weight_out);
    return cudaGetLastError();
}

}  // namespace sa
