// Host-side plans and launchers of the paged cache's operators, and the
// arguments their kernels share.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "sa_internal.h"

namespace sa {

constexpr int kPgTile = 64;            // slots per tile: the unit of the split over a cache's length
constexpr int kPgSlots = 148;          // CTAs of the decode: one per SM

struct PagedDims {
    int B, Hq, Hkv, G, d;
    int bf16;
    int n_pages, page, max_pages;
    uint32_t pmul, pshr;                   // slot / page = (umulhi(slot, pmul) + slot) >> pshr
    int cap, ldw;                          // slots per sequence, row length of pos and of the weights
    int hu, nhb;                           // query heads of a unit (8 or 16), units per KV head
    long long ps, hs, rs;                  // page, head and row strides (elements)
    int U() const { return B * Hkv; }
    int esz() const { return bf16 ? 2 : 4; }
};

// What the kernels of the three operators read of a cache.
struct PagedView {
    const void* k;
    const void* v;
    const int32_t* table;
    const int32_t* lengths;
    const int32_t* pos;
    const int32_t* seen;
    int B, Hq, Hkv, G, hu, nhb;
    int n_pages, page, max_pages, cap, ldw;
    uint32_t pmul, pshr;
    long long ps, hs, rs;
};

inline PagedView paged_view(const PagedDims& d, const sa_paged_cache& c) {
    return PagedView{c.k, c.v, c.table, c.lengths, c.pos, c.seen, d.B, d.Hq, d.Hkv, d.G, d.hu, d.nhb,
                     d.n_pages, d.page, d.max_pages, d.cap, d.ldw, d.pmul, d.pshr, d.ps, d.hs, d.rs};
}

// Decode: the tiles of all units, in unit order, are split evenly over at
// most kPgSlots CTAs (on the device, from the lengths there), so a CTA ends
// at most two units it does not own alone: one record for the unit it
// continues, one for the unit it begins.
struct PagedDecodePlan {
    int grid;
    int rec;                               // floats per record: m[hu], l[hu], acc[hu][d]
    int ldx;                               // floats per row of logits
    int extra;                             // tiles a unit counts more than it has
    size_t off_cnt, off_rec, off_lse, off_x, bytes;
};

// What a CTA spends on a unit beside its tiles is about the time of 128 KB.  In
// us with 0 / 32 / 64 / 128 / 192 / 256 KB: 48 ragged windowed sequences, heads of
// 64: 65 / 58 / 53 / 52 / 52 / 54; 256 of 3..300 tokens: 104 / 82 / 77 / 75 / 75 /
// 77; 32 of 100..8K: 114 / 107 / 104 / 100 / 100 / 101; fp32, 64 of 20..4K: 299 /
// 300 / 285 / 273 / 274 / 277; 16 of 50..16K, 16 heads a group: 45 / 44 / 44 / 41 /
// 41 / 40; 1 x 32K: 38 / 38 / 37 / 36 / 34 / 34.
inline int paged_extra(const PagedDims& d) { return (1 << 17) / (2 * kPgTile * d.d * d.esz()); }

inline PagedDecodePlan paged_decode_plan(const PagedDims& d, bool weights) {
    PagedDecodePlan p;
    const long long tiles = (long long)d.U() * d.nhb * ((d.cap + kPgTile - 1) / kPgTile);
    p.grid = (int)(tiles < kPgSlots ? tiles : kPgSlots);
    p.rec = d.hu * (2 + d.d);
    p.extra = paged_extra(d);
    p.ldx = (d.cap + kPgTile - 1) / kPgTile * kPgTile;
    size_t off = 0;
    // a ticket per eight heads whatever the type's units hold, so that the bytes
    // to be zeroed, and where the records begin, follow from B, Hq and Hkv alone
    p.off_cnt = off; off = align256(off + sizeof(unsigned) * (size_t)d.U() * ((d.G + 7) / 8));
    p.off_rec = off; off = align256(off + sizeof(float) * 2 * (size_t)p.grid * p.rec);
    // with weights: log2 of every row's mass, and the logits (log2) of its slots
    p.off_lse = off; if (weights) off = align256(off + sizeof(float) * (size_t)d.B * d.Hq);
    p.off_x = off;   if (weights) off = align256(off + sizeof(float) * (size_t)d.B * d.Hq * p.ldx);
    p.bytes = off;
    return p;
}

struct PagedDecodeArgs {
    PagedView c;
    const void* q;
    long long q_stride;
    const float* slopes;
    const float* weight;
    float* weight_out;
    float* out;
    float* lse;
    float scale, softcap;
    int sink, local;
    char* ws;
};
cudaError_t launch_paged_decode(const PagedDims& d, const PagedDecodePlan& p, const PagedDecodeArgs& a,
                                cudaStream_t s);

struct PagedAppendArgs {
    PagedView c;
    const void* k_new;
    const void* v_new;
    long long token_stride, head_stride;
    const int32_t* start;
    int n_new;
    int32_t* pos;
    float* weight;
};
cudaError_t launch_paged_append(const PagedDims& d, const PagedAppendArgs& a, cudaStream_t s);

// Eviction: a cluster of CTAs per (sequence, KV head); scratch: the number of
// its moves, its freed slots and the late kept slots that move into them.
struct PagedEvictPlan {
    int cluster;                           // CTAs per unit
    int near_keys;                         // keys of a CTA in shared memory (0: in the workspace)
    int moves;                             // most moves of a unit
    size_t off_count, off_list, off_keys, bytes;
};

PagedEvictPlan paged_evict_plan(const PagedDims& d, int budget);

struct PagedEvictArgs {
    PagedView c;
    const float* weight;
    int budget, sink, local;
    int32_t* lengths_out;
    float* weight_out;
    int32_t* pos_out;
    char* ws;
};
cudaError_t launch_paged_evict(const PagedDims& d, const PagedEvictPlan& p, const PagedEvictArgs& a, cudaStream_t s);

}  // namespace sa
