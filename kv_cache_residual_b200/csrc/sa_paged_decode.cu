// Decode attention of one query per sequence over the paged cache.
//
//   x_hs = cap(scale q_h . k_s) - slope_h (newest - pos_s)
//   out_h = sum_s softmax_s(x_hs) v_s          (one pass, running maximum and sum)
//
// A unit is a KV head of a sequence with up to eight (bf16: sixteen) of its
// query heads.  All units' 64-slot tiles are split evenly over one CTA per SM
// (sa_paged.cuh), so ragged batches, one long sequence and many short ones load
// the GPU alike; a unit cut by the split is joined by the last of its CTAs to
// finish.  Bound: HBM for the rows; for few of them the chain lengths, table,
// rows, record, ticket, join.  Measured (bf16, 32 / 8 heads of 128): 32 x 32K
// 690 to 719 us, 0.92 to 0.96 of the copy rate; 1 x 32K 34.5 us of which the rows
// are 20; 1 x 2K in fp32 10.5 us.
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
    int index;                                     // of the unit, and of its first own tile
    unsigned own0;
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
        index = b * c.Hkv * c.nhb + cur.sub;
        own0 = cur.unit0 + sp.extra;
        qh0 = (size_t)b * c.Hq + head0;
        q = static_cast<const T*>(io.q) + (long long)b * io.q_stride + (long long)head0 * D;
        trow = c.table + (size_t)b * c.max_pages;
        prow = c.pos == nullptr || (io.local == 0 && io.slopes == nullptr)
                   ? nullptr : c.pos + ((size_t)b * c.Hkv + g) * c.ldw;
    }
    __device__ __forceinline__ bool any() const { return end > tile; }
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
    // accumulator A of dim e of head h, mass L relative to 2^M; odd: as pg_element
    __device__ __forceinline__ void put(const PgDecodeIo& io, const PgUnit<T, D>& u, int h, int e, float A, float M,
                                        float L, int* odd) const {
        if (whole) {
            io.out[(u.qh0 + h) * D + e] = pg_element(A, pg_inv(L), u.index, odd);
            if (e == 0) pg_write_lse(io, u.qh0 + h, M, L);
        } else {
            rec[2 * io.c.hu + h * D + e] = A;
            if (e == 0) { rec[h] = M; rec[io.c.hu + h] = L; }
        }
    }
};

// The marked elements of a unit, by the formula: a value that is not finite
// decides its dim's sum whatever the finite ones are, so what matters is which
// kinds of them a head's weights meet (an infinity times a weight of exactly zero
// is NaN).  The lanes of a row read its value chunks, eight rows at once, and
// where one is not finite the row's logits, a chunk each.
template <typename T, int D, int NT>
__device__ __forceinline__ void pg_not_finite(const PgDecodeIo& io, int unit, unsigned* kinds) {
    constexpr int EPC = 16 / (int)sizeof(T), CPR = D / EPC, ROWS = NT / CPR, RPW = 32 / CPR, UN = 8;
    constexpr unsigned kPos = 1u, kNeg = 2u, kNan = 4u;
    const int per = io.c.Hkv * io.c.nhb;
    const int lane = threadIdx.x & 31, at = (lane % CPR) * EPC;
    const T* K = static_cast<const T*>(io.c.k) + at;
    const T* V = static_cast<const T*>(io.c.v) + at;
    const PgUnit<T, D> u(io, PgSplit{0u, 0u, 0}, PgCursor{unit / per, unit % per, 0, 0u}, 1u);
    float* out = io.out + u.qh0 * D;
    bool marked = false;
    for (int x = threadIdx.x; x < u.gh * D; x += NT) {
        kinds[x] = 0u;
        marked |= __float_as_uint(out[x]) == kPgMark;
    }
    if (!__syncthreads_or(marked)) return;
#pragma unroll 1
    for (int y0 = (threadIdx.x >> 5) * RPW; y0 < u.ls.n; y0 += ROWS * UN) {        // the warp's rows
        PgRaw raw[UN];
        long long off[UN];
        float dist[UN];
        uint4 w[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i)
            raw[i] = pg_fetch(io, u.ls, u.trow, u.prow, y0 + i * ROWS + lane / CPR, u.ls.n);
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            off[i] = pg_see(io, raw[i], u.prow != nullptr, u.g, u.newest, dist[i]);
            w[i] = off[i] >= 0 ? *reinterpret_cast<const uint4*>(V + off[i]) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            float v[EPC], a[EPC], k[EPC];
            bool odd = false;
            unpack<T>(w[i], v);
#pragma unroll
            for (int j = 0; j < EPC; ++j) odd |= !(fabsf(v[j]) < INFINITY);
            if (!__any_sync(0xffffffffu, odd)) continue;
            unpack<T>(off[i] >= 0 ? *reinterpret_cast<const uint4*>(K + off[i]) : make_uint4(0u, 0u, 0u, 0u), k);
#pragma unroll 1
            for (int h = 0; h < u.gh; ++h) {
                unpack<T>(__ldg(reinterpret_cast<const uint4*>(u.q + (size_t)h * D + at)), a);
                float dot = 0.f;
#pragma unroll
                for (int j = 0; j < EPC; ++j) dot = fmaf(a[j], k[j], dot);
                dot = group_sum<CPR>(dot);
                const bool none = pg_logit(io, pg_cap(io, dot), u.slope2(io, h), dist[i], 0.f) == -INFINITY;
#pragma unroll
                for (int j = 0; j < EPC; ++j)
                    if (!(fabsf(v[j]) < INFINITY))
                        atomicOr(kinds + h * D + at + j, none || v[j] != v[j] ? kNan : v[j] > 0.f ? kPos : kNeg);
            }
        }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < u.gh * D; x += NT) {
        if (__float_as_uint(out[x]) == kPgMark)        // no kind: finite values whose sum has overflowed
            out[x] = kinds[x] == kPos ? INFINITY : kinds[x] == kNeg ? -INFINITY : NAN;
    }
    __syncthreads();
}

// The same for units [first, last]: this CTA has written both, and so all between,
// which lie whole in its range.  Called at the CTA's end, out of line, so that the
// pass keeps its registers: it and the elements' check cost short units
// a little and long ones nothing (64 sequences of up to 300 tokens 25.7 -> 26.4 us,
// 32 x 32K 674); one infinity in 128K slots takes 2.6 ms.  All threads call.
template <typename T, int D, int NT>
__device__ __noinline__ void pg_marked(const PgDecodeIo& io, int first, int last, unsigned* kinds) {
#pragma unroll 1
    for (int unit = first; unit <= last; ++unit) pg_not_finite<T, D, NT>(io, unit, kinds);
}

// after all have put: the unit's last CTA joins.  All threads call; f, odd as pg_join.
template <typename T, int D, int NT>
__device__ __forceinline__ void pg_hand_in(const PgDecodeIo& io, const PgSplit& sp, const PgUnit<T, D>& u,
                                           const PgPart<T, D>& part, float* f, int* odd) {
    if (part.whole) return;
    const int first = (int)sp.owner(u.own0), n = (int)sp.owner(u.own0 + u.nt - 1) - first + 1;
    unsigned* cnt = io.cnt + u.index;
    if (last_cta_of_unit(cnt, n)) {
#pragma unroll 1
        for (int h0 = 0; h0 < u.gh; h0 += 8) {
            pg_join<D, NT>(io, first, n, u.qh0 + h0, h0, min(8, u.gh - h0), f, u.index, odd);
            __syncthreads();
        }
        reset_counter(cnt);
    }
}

// Moves the cursor from its unit, nt tiles long, to the next; t0 moves along.
// False at the range's end.
__device__ __forceinline__ bool pg_next(const PgDecodeIo& io, const PgSplit& sp, PgCursor& cur, int nt, unsigned& t0,
                                        unsigned t1) {
    const int n = nt + sp.extra;
    t0 += n - cur.tile;                            // past t1 where the unit goes on in another CTA
    if (t0 >= t1) return false;
    cur.unit0 += n;
    cur.tile = 0;
    if (++cur.sub == io.c.Hkv * io.c.nhb) { cur.sub = 0; ++cur.b; }
    return cur.b < io.c.B;
}

// ---- the pass --------------------------------------------------------------------
// A warp takes 16 slots of a step through a ring of its own (cp.async, padded
// rows), with no barrier among warps until the unit ends:
//   S   = Q K^T     A = the unit's queries, B = 16 key rows
//   O^T += V^T P^T  A = value rows, B = the weights: the layout of S's
//                   accumulators is that of B's fragments, so weights never
//                   move between lanes
// Lane (r = lane / 4, t = lane % 4) holds row r (and r + 8 where HB = 16) of S at
// slots 2t, 2t+1, 8+2t, 9+2t, and of O^T 2 MT dims of heads 2t, 2t+1.
//
// What is fp32 enters as three bf16 parts of 8 bits each, cut off the top, so
// that nothing is rounded on the way in: the weights always, and with fp32
// caches queries, keys and values too.  Cut off, a middle part reaches 2^-7 of
// the number and a last one 2^-15.  Of the nine products the last with the last
// is left out (2^-30), and of the two of a middle and a last part (2^-22 of the
// product at most, 0.34 x 2^-24 on average over normal numbers, each with the
// product's sign): the last of a query with the middle of a key; the middle of a
// value with the last of a weight and, with more than four heads, the last of a
// value with the middle of a weight.  Errors stay below the plain fp32 form's
// (0.65 of them over 30 random cases), whose roundings are as large.  (Either way
// the tensor pipe is under a fifth busy, so mma.sync will do.)  With up
// to four heads rows 4..7 repeat rows 0..3 and two of the weights' parts share
// one instruction.  The maximum is moved only when a logit passes it by 8 (2^8
// in the sums): one vote per step.
template <typename T, int D>
struct PgTc {
    static constexpr bool kBf16 = sizeof(T) == 2;
    // fp32 rows: as many warps as a stage ahead leaves room for (16 x 8K, 4 heads
    // of 128: 284 us with 4 warps and 3 stages, 256 with 6 and 2)
    static constexpr int kWarps = !kBf16 && D == 128 ? 6 : 8, kThreads = kWarps * 32;
    static constexpr int kStep = kWarps * 16;                    // list entries of a step of the CTA
    // row pitches without bank conflicts: bf16, ldmatrix; fp32, a lane's four
    // dims of row r (K), of rows 2t, 2t+1, .. (V)
    static constexpr int kPitchK = kBf16 ? 2 * D + 16 : 4 * D + 64, kPitchV = kBf16 ? 2 * D + 16 : 4 * D + 16;
    static constexpr int kV = 16 * kPitchK, kDist = kV + 16 * kPitchV, kBytes = kDist + 16 * 4;
    // one stage ahead of the one at hand is enough with eight warps (32 x 32K 688
    // us, 702 with two ahead, four warps and more stages 830 and up)
    static constexpr int kStages = !kBf16 || D == 128 ? 2 : 4;
    static constexpr int kRing = kWarps * kStages * kBytes;
    static constexpr int kAcc = kWarps * 4 * (D + 4);            // floats: four heads' states of the warps
    static constexpr int kScratch = kAcc > kPgJoinFloats ? kAcc : kPgJoinFloats;
    static constexpr size_t kSmem = kRing + 4 * (size_t)kScratch;
    static_assert((kBf16 ? 16 : 8) * D <= kScratch, "pg_not_finite: a word for each element of a unit");
};

__device__ __forceinline__ void pg_cp16(uint32_t s, const void* g, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(s), "l"(g), "r"(ok ? 16 : 0) : "memory");
}

// d = a b on the matrix unit, from zero.  A matrix instruction cuts its sum off
// where fp32 ends instead of rounding it, which over many adds up on one side
// (8e-6 of the output after 32K rows), so sums begin anew every few instructions
// and are added up by ordinary additions.
__device__ __forceinline__ void pg_mma0(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// x = hi + mid + lo exactly, 8 bits each, a pair of x to a register
__device__ __forceinline__ void pg_split(float x0, float x1, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    const uint32_t a = __float_as_uint(x0), b = __float_as_uint(x1);
    hi = __byte_perm(a, b, 0x7632);
    const float r0 = x0 - __uint_as_float(a & 0xffff0000u), r1 = x1 - __uint_as_float(b & 0xffff0000u);
    const uint32_t c = __float_as_uint(r0), d = __float_as_uint(r1);
    mid = __byte_perm(c, d, 0x7632);
    lo = __byte_perm(__float_as_uint(r0 - __uint_as_float(c & 0xffff0000u)),
                     __float_as_uint(r1 - __uint_as_float(d & 0xffff0000u)), 0x7632);
}

// The queries of a lane's rows as A fragments, and S for 16 key rows.
template <typename T, int D, int HB>
struct PgQ;

template <int D, int HB>
struct PgQ<__nv_bfloat16, D, HB> {
    static constexpr int KS = D / 16, R = HB == 16 ? 2 : 1;
    uint32_t a[KS][2 * R];
    __device__ __forceinline__ void load(const __nv_bfloat16* q, const int (&head)[R], int gh) {
        const int t = threadIdx.x & 3;
#pragma unroll
        for (int k = 0; k < R; ++k)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const __nv_bfloat16* p = q + (size_t)head[k] * D + ks * 16 + 2 * t;
                a[ks][k] = head[k] < gh ? __ldg(reinterpret_cast<const unsigned*>(p)) : 0u;
                a[ks][R + k] = head[k] < gh ? __ldg(reinterpret_cast<const unsigned*>(p + 8)) : 0u;
            }
    }
    __device__ __forceinline__ void ready() {}
    __device__ __forceinline__ void dots(const unsigned char* rows, float (&x)[R][4]) const {
        constexpr int P = PgTc<__nv_bfloat16, D>::kPitchK;
        const int lane = threadIdx.x & 31;
        const uint32_t kt = tc::smem_u32(rows);
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
                float z[4];
                const uint32_t (&q0)[2 * R] = a[2 * kp], (&q1)[2 * R] = a[2 * kp + 1];
                pg_mma0(z, q0[0], R == 2 ? q0[1] : 0u, q0[R], R == 2 ? q0[2 * R - 1] : 0u, b[0], b[1]);
                tc::mma_bf16(z, q1[0], R == 2 ? q1[1] : 0u, q1[R], R == 2 ? q1[2 * R - 1] : 0u, b[2], b[3]);
#pragma unroll
                for (int j = 0; j < 2 * R; ++j) s[h][j] += z[j];
            }
#pragma unroll
        for (int k = 0; k < R; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[k][j] = s[j >> 1][2 * k + (j & 1)];
    }
};

// fp32: rows 0..7 of A are the top parts, rows 8..15 the middle ones, and the
// bottom ones an A of their own.  A chunk's 16 dims are dealt so that a lane's
// two pairs are the four dims from 4t on.
template <int D, int HB>
struct PgQ<float, D, HB> {
    static_assert(HB <= 8, "the parts of eight heads fill A");
    static constexpr int KS = D / 16, R = 1;
    float4 q[KS];
    uint32_t hm[KS][4], lo[KS][2];
    const float* src;                              // the row's query, or null: zeros
    __device__ __forceinline__ void load(const float* first, const int (&head)[1], int gh) {
        const int t = threadIdx.x & 3;
        src = head[0] < gh ? first + (size_t)head[0] * D : nullptr;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
            q[ks] = src != nullptr ? __ldg(reinterpret_cast<const float4*>(src + ks * 16 + 4 * t))
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ void ready() {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            pg_split(q[ks].x, q[ks].y, hm[ks][0], hm[ks][1], lo[ks][0]);
            pg_split(q[ks].z, q[ks].w, hm[ks][2], hm[ks][3], lo[ks][1]);
        }
    }
    __device__ __forceinline__ void dots(const unsigned char* rows, float (&x)[1][4]) const {
        constexpr int P = PgTc<float, D>::kPitchK;
        const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
        float s[2][2][4];                          // [slots][products of top parts with them, the others]
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[h][0][j] = s[h][1][j] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 k = *reinterpret_cast<const float4*>(rows + (h * 8 + r) * P + (ks * 16 + 4 * t) * 4);
                uint32_t b[3][2];
                pg_split(k.x, k.y, b[0][0], b[1][0], b[2][0]);
                pg_split(k.z, k.w, b[0][1], b[1][1], b[2][1]);
                float z[4];
                pg_mma0(z, hm[ks][0], hm[ks][1], hm[ks][2], hm[ks][3], b[0][0], b[0][1]);
                tc::mma_bf16(s[h][1], hm[ks][0], hm[ks][1], hm[ks][2], hm[ks][3], b[2][0], b[2][1]);
                tc::mma_bf16(s[h][1], lo[ks][0], 0u, lo[ks][1], 0u, b[0][0], b[0][1]);
                tc::mma_bf16(s[h][1], hm[ks][0], hm[ks][1], hm[ks][2], hm[ks][3], b[1][0], b[1][1]);
#pragma unroll
                for (int j = 0; j < 4; ++j) s[h][0][j] += z[j];
            }
        bool odd = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float (&y)[2][4] = s[j >> 1];
            x[0][j] = y[0][j & 1] + (y[0][2 + (j & 1)] + (y[1][j & 1] + y[1][2 + (j & 1)]));
            odd |= x[0][j] != x[0][j];
        }
        // the parts of an infinity are not numbers, nor is 0 times one: as the formula has it
        if (__any_sync(0xffffffffu, odd)) {
            float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
            for (int e = 0; e < D && src != nullptr; e += 4) {
                const float4 z = __ldg(reinterpret_cast<const float4*>(src + e));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 k = *reinterpret_cast<const float4*>(rows + ((j >> 1) * 8 + 2 * t + (j & 1)) * P + e * 4);
                    y[j] = fmaf(z.w, k.w, fmaf(z.z, k.z, fmaf(z.y, k.y, fmaf(z.x, k.x, y[j]))));
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) x[0][j] = y[j];
        }
    }
};

// O^T += V^T P^T for 16 value rows; w[k]: the weights of row k's slots.
template <typename T, int D, int HB>
__device__ __forceinline__ void pg_values(const unsigned char* rows, const float (&w)[HB == 16 ? 2 : 1][4],
                                          float (&o)[HB == 16 ? 2 : 1][D / 16][4]) {
    constexpr int R = HB == 16 ? 2 : 1, MT = D / 16, P = PgTc<T, D>::kPitchV;
    const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
    uint32_t b[R][3][2];                           // parts of the weights, slots 2t.. and 8 + 2t..
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            pg_split(w[k][2 * h], w[k][2 * h + 1], b[k][0][h], b[k][1][h], b[k][2][h]);
            if (HB == 4 && r >= 4) { b[k][0][h] = b[k][1][h]; b[k][2][h] = 0u; }
        }
    if constexpr (PgTc<T, D>::kBf16) {
        const uint32_t va = tc::smem_u32(rows) + ((lane & 7) + ((lane >> 4) & 1) * 8) * P + ((lane >> 3) & 1) * 16;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            uint32_t a[4];
            tc::ldsm4t(va + mt * 32, a);
#pragma unroll
            for (int k = 0; k < R; ++k) {
                float z[4];
                pg_mma0(z, a[0], a[1], a[2], a[3], b[k][2][0], b[k][2][1]);
                if (HB != 4) tc::mma_bf16(z, a[0], a[1], a[2], a[3], b[k][1][0], b[k][1][1]);
                tc::mma_bf16(z, a[0], a[1], a[2], a[3], b[k][0][0], b[k][0][1]);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[k][mt][j] += z[j];
            }
        }
    } else {
        // 32 dims at a time: a lane's four from 4r on are rows r, r + 8 of two tiles
#pragma unroll
        for (int c = 0; c < MT / 2; ++c) {
            float v[4][4];                         // slots 2t, 2t+1, 8+2t, 9+2t
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<float4*>(v[j]) = *reinterpret_cast<const float4*>(
                    rows + ((j >> 1) * 8 + 2 * t + (j & 1)) * P + (c * 32 + 4 * r) * 4);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t a[3][4];
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        pg_split(v[2 * h][2 * i + e], v[2 * h + 1][2 * i + e], a[0][e + 2 * h], a[1][e + 2 * h], a[2][e + 2 * h]);
                float z[4];
                pg_mma0(z, a[2][0], a[2][1], a[2][2], a[2][3], b[0][0][0], b[0][0][1]);
                tc::mma_bf16(z, a[0][0], a[0][1], a[0][2], a[0][3], b[0][2][0], b[0][2][1]);
                if (HB != 4) {
                    tc::mma_bf16(z, a[1][0], a[1][1], a[1][2], a[1][3], b[0][1][0], b[0][1][1]);
                    tc::mma_bf16(z, a[0][0], a[0][1], a[0][2], a[0][3], b[0][1][0], b[0][1][1]);
                }
                tc::mma_bf16(z, a[1][0], a[1][1], a[1][2], a[1][3], b[0][0][0], b[0][0][1]);
                tc::mma_bf16(z, a[0][0], a[0][1], a[0][2], a[0][3], b[0][0][0], b[0][0][1]);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[0][2 * c + i][j] += z[j];
            }
        }
    }
}

// dim of O^T's accumulator j of tile mt in lane row r
template <typename T, int D>
__device__ __forceinline__ int pg_dim(int mt, int r, int j) {
    return PgTc<T, D>::kBf16 ? mt * 16 + r + (j >> 1) * 8 : (mt >> 1) * 32 + 4 * r + (mt & 1) * 2 + (j >> 1);
}

template <typename T, int D, int HB>
__global__ void __launch_bounds__(PgTc<T, D>::kThreads, 1)
k_paged_decode(const __grid_constant__ PgDecodeIo io) {
    using Tc = PgTc<T, D>;
    constexpr int S = Tc::kStages, MT = D / 16, NW = Tc::kWarps, NT = Tc::kThreads;
    constexpr int EPC = 16 / (int)sizeof(T), CPR = D / EPC, RPI = 32 / CPR;     // chunks per row, rows per copy instruction
    constexpr int R = HB == 16 ? 2 : 1;                          // query rows per lane
    constexpr int LD = D + 4;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float s_ml[NW][HB][2];
    __shared__ int s_odd[2];                                     // the first and the last unit with marks
    const PagedView& c = io.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, t = lane & 3;
    unsigned char* ring = smem + warp * S * Tc::kBytes;
    float* scratch = reinterpret_cast<float*>(smem + Tc::kRing);
    const uint32_t ring_u = tc::smem_u32(ring);
    const T* K = static_cast<const T*>(c.k) + (lane % CPR) * EPC;
    const T* V = static_cast<const T*>(c.v) + (lane % CPR) * EPC;
    PgSplit sp;
    PgCursor cur;
    unsigned t0, t1;
    if (threadIdx.x == 0) { s_odd[0] = 0x7fffffff; s_odd[1] = -1; }
    cudaTriggerProgrammaticLaunchCompletion();                   // the weights' kernel may come and wait
    if (!pg_locate<NT>(c.B, c.Hkv * c.nhb, io.extra, blockIdx.x, SA_PG_TILES(io), sp, cur, t0, t1)) return;

    int head[R];
#pragma unroll
    for (int k = 0; k < R; ++k) head[k] = HB == 4 ? (r & 3) : r + 8 * k;
    PgUnit<T, D> u(io, sp, cur, t1 - t0), done = u;               // the unit at hand, the one before it
    bool more = u.any(), handed = true;
    PgQ<T, D, HB> q;
    float sl[R], m[R], l[R], o[R][MT][4];                         // slopes, maxima, masses, accumulators
    PgRaw first[S - 1], ahead;                                    // of the unit's first steps, of the next step
    int stage = 0;                                                // ring stage of the unit's first step

    // this warp's steps of a unit: 16 list entries from row0 + i kStep, i < n
    auto row0 = [&](const PgUnit<T, D>& x) { return x.tile * kPgTile + warp * 16; };
    auto steps = [&](const PgUnit<T, D>& x) { return x.s1 > row0(x) ? (x.s1 - row0(x) + Tc::kStep - 1) / Tc::kStep : 0; };
    auto fetch = [&](const PgUnit<T, D>& x, int i) {
        const int y = row0(x) + i * Tc::kStep;
        return pg_fetch(io, x.ls, x.trow, x.prow, y + (lane & 15), y < x.s1 ? x.s1 : 0);
    };
    auto issue = [&](int i, const PgRaw& raw) {
        float dist;
        const long long off = pg_see(io, raw, u.prow != nullptr, u.g, u.newest, dist);
        const int at = (stage + i) % S * Tc::kBytes;
        if (lane < 16) *reinterpret_cast<float*>(ring + at + Tc::kDist + 4 * lane) = off >= 0 ? dist : INFINITY;
#pragma unroll
        for (int j = 0; j < 16 / RPI; ++j) {
            const int row = j * RPI + lane / CPR;
            const long long p = __shfl_sync(0xffffffffu, off, row);
            const uint32_t to = ring_u + at + (lane % CPR) * 16;
            pg_cp16(to + row * Tc::kPitchK, K + (p < 0 ? 0 : p), p >= 0);
            pg_cp16(to + Tc::kV + row * Tc::kPitchV, V + (p < 0 ? 0 : p), p >= 0);
        }
    };
    if (more) {
#pragma unroll
        for (int i = 0; i < S - 1; ++i) first[i] = fetch(u, i);
    }
#pragma unroll 1
    for (;;) {
        const int n = more ? steps(u) : 0;
        if (more) {                                               // queries and first copies: on their way during the hand-in
            q.load(u.q, head, u.gh);
#pragma unroll
            for (int k = 0; k < R; ++k) sl[k] = u.slope2(io, head[k]);
#pragma unroll
            for (int i = 0; i < S - 1; ++i) {
                if (i < n) issue(i, first[i]);
                tc::cp_commit();
            }
            ahead = fetch(u, S - 1);
        }
        if (!handed) {
            const PgPart<T, D> part(io, done);
#pragma unroll
            for (int k = 0; k < R; ++k) {
                l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
                l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
                if (t == 0 && (HB != 4 || r < 4)) {
                    s_ml[warp][head[k]][0] = m[k];
                    s_ml[warp][head[k]][1] = l[k];
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
                            scratch[(warp * 4 + (2 * t + (j & 1)) % 4) * LD + pg_dim<T, D>(mt, r, j)] = y;
                    }
                __syncthreads();
                for (int x = threadIdx.x; x < 4 * D; x += NT) {
                    const int h4 = x / D, e = x - h4 * D, h = 4 * hq + h4;
                    if (h >= done.gh) break;
                    float M = -INFINITY, A = 0.f, L = 0.f;
#pragma unroll
                    for (int w = 0; w < NW; ++w) M = fmaxf(M, s_ml[w][h][0]);
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        const float mw = s_ml[w][h][0];
                        const float f = mw == -INFINITY ? 0.f : ex2(mw - M);
                        A = fmaf(scratch[(w * 4 + h4) * LD + e], f, A);
                        L = fmaf(s_ml[w][h][1], f, L);
                    }
                    part.put(io, done, h, e, A, M, L, s_odd);
                }
                __syncthreads();
            }
            pg_hand_in<T, D, NT>(io, sp, done, part, scratch, s_odd);
        }
        if (!more) break;
        __syncthreads();                                          // the scratch has been read
        done = u;
        handed = false;
        more = pg_next(io, sp, cur, done.nt, t0, t1);
        PgUnit<T, D> next = done;
        if (more) {
            next = PgUnit<T, D>(io, sp, cur, t1 - t0);
            more = next.any();
        }
        if (more) {                                               // its table entries, during this unit's rows
#pragma unroll
            for (int i = 0; i < S - 1; ++i) first[i] = fetch(next, i);
        }
        q.ready();
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
            ahead = fetch(u, i + S);
            tc::cp_wait<S - 1>();
            __syncwarp();
            const unsigned char* rows = ring + (stage + i) % S * Tc::kBytes;
            const float* dist = reinterpret_cast<const float*>(rows + Tc::kDist);
            // dot products of this lane's rows and slots (2t, 2t+1, 8+2t, 9+2t)
            float x[R][4];
            q.dots(rows, x);
            const float2 d0 = *reinterpret_cast<const float2*>(dist + 2 * t);
            const float2 d1 = *reinterpret_cast<const float2*>(dist + 8 + 2 * t);
            const float dd[4] = {d0.x, d0.y, d1.x, d1.y};
            // relative to the maximum so far, which is moved when one passes it by 8
            float p[R][4];
            bool rises = false;
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const float ref = m[k] == -INFINITY ? 0.f : m[k], over = m[k] == -INFINITY ? -INFINITY : 8.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[k][j] = pg_cap(io, x[k][j]);
                    p[k][j] = dd[j] == INFINITY ? -INFINITY : pg_logit(io, x[k][j], sl[k], dd[j], ref);
                    rises |= p[k][j] > over;
                }
            }
            if (io.x != nullptr) {
                const int y = row0(u) + i * Tc::kStep + 2 * t;
#pragma unroll
                for (int k = 0; k < R; ++k)
                    if (head[k] < u.gh && (HB != 4 || r < 4)) {
                        float* xs = io.x + (u.qh0 + head[k]) * io.ldx + y;      // rows of whole tiles: both pairs fit
                        float z[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            z[j] = dd[j] == INFINITY ? -INFINITY : pg_logit(io, x[k][j], sl[k], dd[j], 0.f);
                        *reinterpret_cast<float2*>(xs) = make_float2(z[0], z[1]);
                        *reinterpret_cast<float2*>(xs + 8) = make_float2(z[2], z[3]);
                    }
            }
            if (__any_sync(0xffffffffu, rises)) {
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    const float ref = m[k] == -INFINITY ? 0.f : m[k];
                    float mx = fmaxf(fmaxf(p[k][0], p[k][1]), fmaxf(p[k][2], p[k][3]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    mx = fmaxf(m[k], ref + mx);
                    const float sc = m[k] == -INFINITY ? 0.f : ex2(m[k] - mx);
                    m[k] = mx;
                    l[k] *= sc;
                    // none so far but -inf, or what is not a number and has to stay that
                    const float to = mx == -INFINITY ? 0.f : mx;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        p[k][j] = dd[j] == INFINITY ? -INFINITY : pg_logit(io, x[k][j], sl[k], dd[j], to);
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
#pragma unroll
            for (int k = 0; k < R; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    p[k][j] = p[k][j] == -INFINITY ? 0.f : ex2(p[k][j]);
                    l[k] += p[k][j];
                }
            pg_values<T, D, HB>(rows + Tc::kV, p, o);
        }
        __syncwarp();
        stage = (stage + n) % S;
        if (more) u = next;
    }
    tc::cp_wait<0>();
    __syncthreads();
    if (s_odd[1] >= 0) pg_marked<T, D, NT>(io, s_odd[0], s_odd[1], reinterpret_cast<unsigned*>(scratch));
}

// weight_out = weight + the step's attention weights summed over the group's
// heads, from the logits the decode left and the rows' masses.  A thread takes
// four slots in a row, as vectors where list and arrays are aligned alike.
// Bound: HBM (or L2, where the logits still are) for 4 G + 8 bytes a slot.
// One CTA per 1024 slots of the capacity: those past a length leave at once.
constexpr int kPgWTile = kThreads * 4;         // slots per CTA

__global__ void __launch_bounds__(kThreads)
k_paged_weights(PgDecodeIo io, int tiles, const float* weight, float* weight_out) {
    const PagedView& c = io.c;
    const bool aligned = ((reinterpret_cast<uintptr_t>(weight) | reinterpret_cast<uintptr_t>(weight_out)) & 15) == 0 &&
                         c.ldw % 4 == 0;
    const int unit = blockIdx.x / tiles, b = unit / c.Hkv, g = unit - b * c.Hkv;
    const int slot = (blockIdx.x - unit * tiles) * kPgWTile + 4 * threadIdx.x;
    const PgList ls = pg_list(c, b, io.sink, io.local);
    cudaGridDependencySynchronize();               // the logits and masses
    if (slot >= ls.len) return;
    const size_t row = (size_t)unit * c.ldw;
    const size_t qh0 = (size_t)b * c.Hq + (size_t)g * c.G;
    const int gap = ls.len - ls.n;
    const bool vec = aligned && gap == 0 && slot + 4 <= ls.len;
    float w[4], p[4] = {0.f, 0.f, 0.f, 0.f};
    int y[4];                                  // list entries, -1: not listed
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int s = slot + j;
        y[j] = s >= ls.len ? -1 : s < ls.s_eff ? s : s >= ls.s_eff + gap ? s - gap : -1;
        w[j] = 0.f;
    }
    if (weight != nullptr) {
        if (vec) {
            *reinterpret_cast<float4*>(w) = *reinterpret_cast<const float4*>(weight + row + slot);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (slot + j < ls.len) w[j] = weight[row + slot + j];
        }
    }
#pragma unroll 4
    for (int h = 0; h < c.G; ++h) {
        const float l2 = __ldcg(io.lse2 + qh0 + h);
        const float* xs = io.x + (qh0 + h) * io.ldx;
        float x[4];
        if (vec) {
            *reinterpret_cast<float4*>(x) = __ldcg(reinterpret_cast<const float4*>(xs + slot));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = y[j] >= 0 ? __ldcg(xs + y[j]) : -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] += x[j] == -INFINITY ? 0.f : ex2(x[j] - l2);
    }
    if (vec) {
        *reinterpret_cast<float4*>(weight_out + row + slot) = make_float4(w[0] + p[0], w[1] + p[1], w[2] + p[2], w[3] + p[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (slot + j < ls.len) weight_out[row + slot + j] = w[j] + p[j];
    }
}

template <typename T, int D, int HB>
static cudaError_t decode_launch(const PagedDecodePlan& p, const PgDecodeIo& io, cudaStream_t s) {
    using Tc = PgTc<T, D>;
    static std::atomic<unsigned long long> opted{0};
    const cudaError_t e = opt_in_smem(k_paged_decode<T, D, HB>, Tc::kSmem, opted);
    if (e != cudaSuccess) return e;
    k_paged_decode<T, D, HB><<<p.grid, Tc::kThreads, Tc::kSmem, s>>>(io);
    return cudaGetLastError();
}

template <int D>
static cudaError_t decode_heads(const PagedDims& d, const PagedDecodePlan& p, const PgDecodeIo& io, cudaStream_t s) {
    using B = __nv_bfloat16;
    if (d.bf16)
        return d.G <= 4 ? decode_launch<B, D, 4>(p, io, s) : d.G <= 8 ? decode_launch<B, D, 8>(p, io, s)
                                                                      : decode_launch<B, D, 16>(p, io, s);
    return d.G <= 4 ? decode_launch<float, D, 4>(p, io, s) : decode_launch<float, D, 8>(p, io, s);
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
    io.softcap = a.softcap;
    io.cap_in = a.softcap > 0.f ? a.scale / a.softcap : 0.f;
    io.factor = (a.softcap > 0.f ? a.softcap : a.scale) * kLog2e;
    io.sink = a.sink;
    io.local = a.local;
    io.ldx = p.ldx;
    io.extra = p.extra;
    const cudaError_t e = d.d == 128 ? decode_heads<128>(d, p, io, s) : decode_heads<64>(d, p, io, s);
    if (e != cudaSuccess || !weights) return e;
    const int tiles = cdiv(d.cap, kPgWTile);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)d.U() * tiles);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_paged_weights, io, tiles, a.weight, a.weight_out);
}

}  // namespace sa
