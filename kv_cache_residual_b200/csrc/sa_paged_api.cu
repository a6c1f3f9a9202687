// C entry points of the paged cache (declared in include/sa_decode.h):
// argument checks, workspace sizing and dispatch.  Every check runs before
// anything is enqueued, so a rejected call leaves the stream untouched.
#include <float.h>

#include "sa_check.h"
#include "sa_paged.h"

using namespace sa;

namespace {

sa_status check_paged_shape(const sa_paged_shape* s, PagedDims* d) {
    if (s == nullptr) return SA_ERR_INVALID_ARG;
    if (s->B < 1 || s->Hq < 1 || s->Hkv < 1 || s->d < 1 || s->n_pages < 1 || s->page < 1 || s->max_pages < 1 ||
        s->ldw < 0)
        return SA_ERR_INVALID_ARG;
    if (s->Hq % s->Hkv != 0) return SA_ERR_INVALID_ARG;
    if (s->dtype != SA_F32 && s->dtype != SA_BF16) return SA_ERR_INVALID_ARG;
    if (s->d != 64 && s->d != 128) return SA_ERR_UNSUPPORTED;
    const long long cap = (long long)s->page * s->max_pages;
    if (cap > (1LL << 30)) return SA_ERR_UNSUPPORTED;
    if ((long long)s->B * s->Hkv >= 65536 || (long long)s->B * s->Hq >= (1LL << 24)) return SA_ERR_UNSUPPORTED;
    d->B = s->B; d->Hq = s->Hq; d->Hkv = s->Hkv; d->G = s->Hq / s->Hkv; d->d = s->d;
    d->bf16 = s->dtype == SA_BF16;
    d->n_pages = s->n_pages; d->page = s->page; d->max_pages = s->max_pages;
    // division of a slot (below 2^30) by the page size as a multiplication:
    // l = ceil(log2 page), pmul = floor(2^32 (2^l - page) / page) + 1
    d->pshr = 0;
    while ((1LL << d->pshr) < s->page) ++d->pshr;
    d->pmul = (uint32_t)((((1ULL << d->pshr) - (unsigned)s->page) << 32) / (unsigned)s->page + 1);
    d->cap = (int)cap;
    d->ldw = s->ldw == 0 ? d->cap : s->ldw;
    if (d->ldw < d->cap) return SA_ERR_INVALID_ARG;
    // the matrix instructions of the bf16 decode take sixteen rows of queries
    d->hu = d->bf16 && d->G > 8 ? 16 : 8;
    d->nhb = (d->G + d->hu - 1) / d->hu;
    d->ps = s->page_stride; d->hs = s->head_stride; d->rs = s->row_stride;
    if (d->ps == 0 && d->hs == 0 && d->rs == 0) {
        d->rs = s->d;
        d->hs = (long long)s->page * s->d;
        d->ps = (long long)s->Hkv * s->page * s->d;
    }
    const int chunk = 16 / d->esz();
    if (d->ps < 1 || d->hs < 1 || d->rs < 1 || d->ps % chunk != 0 || d->hs % chunk != 0 || d->rs % chunk != 0)
        return SA_ERR_INVALID_ARG;
    if ((long long)d->U() * d->nhb * ((d->cap + kPgTile - 1) / kPgTile + paged_extra(*d)) >= (1LL << 31))
        return SA_ERR_UNSUPPORTED;
    return SA_OK;
}

bool check_cache(const sa_paged_cache* c) {
    if (c == nullptr || !aligned16(c->k) || !aligned16(c->v) || !aligned4(c->table) || !aligned4(c->lengths))
        return false;
    if ((c->pos == nullptr) != (c->seen == nullptr)) return false;      // a pair, or neither
    return c->pos == nullptr || (aligned4(c->pos) && aligned4(c->seen));
}

// whether what a call writes lies apart from what it reads and from its other outputs
bool apart(const Span* out, int n_out, const Span* in, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return false;
        for (int j = 0; j < n_in; ++j)
            if (overlap(out[i], in[j])) return false;
    }
    return true;
}

Span table_span(const PagedDims& d, const sa_paged_cache& c) { return Span(c.table, 4LL * d.B * d.max_pages); }
Span per_slot(const PagedDims& d, const void* p) { return Span(p, 4LL * d.cap, d.U(), 4LL * d.ldw); }
Span per_sequence(const PagedDims& d, const void* p) { return Span(p, 4LL * d.B); }

bool strides_ok(long long x, const PagedDims& d) { return x >= 1 && x % (16 / d.esz()) == 0; }

}  // namespace

extern "C" {

size_t sa_paged_workspace_size(const sa_paged_shape* shape, int op, int arg) {
    PagedDims d;
    if (check_paged_shape(shape, &d) != SA_OK) return 0;
    if (op == SA_OP_PAGED_DECODE) return paged_decode_plan(d, arg != 0).bytes;
    if (op == SA_OP_PAGED_EVICT) return arg < 1 ? 0 : paged_evict_plan(d, arg).bytes;
    return 0;
}

sa_status sa_paged_append(const sa_paged_shape* shape, const sa_paged_cache* cache, const void* k_new,
                          const void* v_new, long long token_stride, long long head_stride, const int32_t* start,
                          int n_new, float* weight, void* stream) {
    NvtxRange r("sa_paged_append");
    PagedDims d;
    const sa_status e = check_paged_shape(shape, &d);
    if (e != SA_OK) return e;
    if (!check_cache(cache) || n_new < 0) return SA_ERR_INVALID_ARG;
    if (start == nullptr ? n_new != d.B : !aligned4(start)) return SA_ERR_INVALID_ARG;
    if (weight != nullptr && !aligned4(weight)) return SA_ERR_INVALID_ARG;
    if (n_new == 0) return SA_OK;
    if ((long long)n_new * d.Hkv >= (1LL << 31)) return SA_ERR_UNSUPPORTED;
    if (!aligned16(k_new) || !aligned16(v_new)) return SA_ERR_INVALID_ARG;
    if (token_stride == 0 && head_stride == 0) {
        head_stride = d.d;
        token_stride = (long long)d.Hkv * d.d;
    }
    if (!strides_ok(token_stride, d) || !strides_ok(head_stride, d)) return SA_ERR_INVALID_ARG;
    const Span out[] = {per_slot(d, cache->pos), per_slot(d, weight)};
    const Span in[] = {table_span(d, *cache), per_sequence(d, cache->lengths), per_sequence(d, cache->seen),
                       Span(start, 4LL * (d.B + 1))};
    if (!apart(out, 2, in, 4)) return SA_ERR_INVALID_ARG;
    const PagedAppendArgs a{paged_view(d, *cache), k_new, v_new, token_stride, head_stride, start, n_new,
                            cache->pos, weight};
    return launch_paged_append(d, a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

sa_status sa_paged_decode(const sa_paged_shape* shape, const sa_paged_cache* cache, const sa_paged_params* params,
                          const void* q, float* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    NvtxRange r("sa_paged_decode");
    PagedDims d;
    const sa_status e = check_paged_shape(shape, &d);
    if (e != SA_OK) return e;
    if (!check_cache(cache) || params == nullptr || !aligned16(q) || !aligned16(out)) return SA_ERR_INVALID_ARG;
    const sa_paged_params& p = *params;
    if (!(p.scale >= 0.f && p.scale < INFINITY) || !(p.softcap >= 0.f && p.softcap < INFINITY) || p.sink < 0 ||
        p.local < 0)
        return SA_ERR_INVALID_ARG;
    if ((lse != nullptr && !aligned4(lse)) || (p.slopes != nullptr && !aligned4(p.slopes)) ||
        (p.weight != nullptr && (!aligned4(p.weight) || p.weight_out == nullptr)) ||
        (p.weight_out != nullptr && !aligned4(p.weight_out)))
        return SA_ERR_INVALID_ARG;
    // what the kernel multiplies by has to be a number, and a quotient one of full precision
    const float scale = resolve_scale(p.scale, d.d), cap_in = p.softcap > 0.f ? scale / p.softcap : 1.f;
    if (!(scale * 1.5f < INFINITY) || !(p.softcap * 1.5f < INFINITY) || !(cap_in >= FLT_MIN && cap_in < INFINITY))
        return SA_ERR_INVALID_ARG;
    const long long qs = p.q_stride == 0 ? (long long)d.Hq * d.d : p.q_stride;
    if (!strides_ok(qs, d)) return SA_ERR_INVALID_ARG;
    const PagedDecodePlan plan = paged_decode_plan(d, p.weight_out != nullptr);
    if (ws == nullptr || ws_bytes < plan.bytes || !aligned16(ws)) return SA_ERR_WORKSPACE;
    // in place: weights at the very slots, and queries that are exactly the rows written
    const bool same_w = p.weight == p.weight_out, same_q = q == out && !d.bf16 && qs == (long long)d.Hq * d.d;
    const Span outs[] = {Span(out, 4LL * d.B * d.Hq * d.d), Span(lse, 4LL * d.B * d.Hq), per_slot(d, p.weight_out),
                         Span(ws, (long long)plan.bytes)};
    const Span ins[] = {Span(same_q ? nullptr : q, (long long)d.Hq * d.d * d.esz(), d.B, qs * d.esz()),
                        table_span(d, *cache), per_sequence(d, cache->lengths), per_sequence(d, cache->seen),
                        per_slot(d, cache->pos), Span(p.slopes, 4LL * d.Hq), per_slot(d, same_w ? nullptr : p.weight)};
    if (!apart(outs, 4, ins, 7)) return SA_ERR_INVALID_ARG;
    const PagedDecodeArgs a{paged_view(d, *cache), q, qs, p.slopes, p.weight, p.weight_out, out, lse,
                            scale, p.softcap, p.sink, p.local, static_cast<char*>(ws)};
    return launch_paged_decode(d, plan, a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

sa_status sa_paged_evict(const sa_paged_shape* shape, const sa_paged_cache* cache, const float* weight, int budget,
                         int sink, int local, int32_t* lengths_out, float* weight_out, int32_t* pos_out, void* ws,
                         size_t ws_bytes, void* stream) {
    NvtxRange r("sa_paged_evict");
    PagedDims d;
    const sa_status e = check_paged_shape(shape, &d);
    if (e != SA_OK) return e;
    if (!check_cache(cache) || !aligned4(weight) || !aligned4(lengths_out) || !aligned4(weight_out) ||
        !aligned4(pos_out))
        return SA_ERR_INVALID_ARG;
    if (budget < 1 || sink < 0 || local < 0 || (long long)sink + local > budget) return SA_ERR_INVALID_ARG;
    const PagedEvictPlan plan = paged_evict_plan(d, budget);
    if (ws == nullptr || ws_bytes < plan.bytes || !aligned16(ws)) return SA_ERR_WORKSPACE;
    const Span out[] = {per_sequence(d, lengths_out), per_slot(d, weight_out), per_slot(d, pos_out),
                        Span(ws, (long long)plan.bytes)};
    const Span in[] = {table_span(d, *cache), per_sequence(d, cache->lengths), per_sequence(d, cache->seen),
                       per_slot(d, cache->pos), per_slot(d, weight)};
    if (!apart(out, 4, in, 5)) return SA_ERR_INVALID_ARG;
    const PagedEvictArgs a{paged_view(d, *cache), weight, budget, sink, local, lengths_out, weight_out, pos_out,
                           static_cast<char*>(ws)};
    return launch_paged_evict(d, plan, a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // extern "C"
