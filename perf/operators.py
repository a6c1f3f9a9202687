"""Measured cases of the paged cache's operators: append, single-token decode
attention, and eviction by accumulated attention weight.

A cache holds pages of `page` tokens in pools k, v [n_pages, Hkv, page, d];
row b of `table` lists the pages of sequence b, and slot s of the sequence is
row s % page of page table[b, s / page].  A slot's `pos` is the position of
the token it holds (eviction moves tokens between slots); without `pos` the
two are the same.

  append   the tokens of this call, packed [N, Hkv, d], into the last slots of
           their sequences: slot lengths[b] - n_b + i takes token i of n_b,
           pos = seen[b] - n_b + i, accumulated weight 0
  decode   one query per sequence, out_h = sum_s p_hs v_s, p_h = softmax over
           the visible slots of x_hs = cap(scale q_h . k_s) - slope_h (newest - pos_s),
           cap(x) = c tanh(x / c), newest = seen[b] - 1; a slot is visible when
           pos < sink or pos > newest - local (every slot when local = 0); with
           weights, weight_out_gs = weight_gs + sum_{h in group g} p_hs
  evict    per sequence and KV head the `budget` slots that stay: the first
           `sink` and the last `local` positions, then the largest accumulated
           weights, ties to the lower slot; the kept slots past the new length
           move, in order, into the freed slots before it

The attention geometry is the repository's own (32 query / 8 KV heads of 128,
bf16, 32K and 128K caches; 4 / 1 heads of 64 in fp32) beside others of the kind.
"""
import math

import torch

own = False

F32 = torch.float32
I32 = torch.int32


# ---- cases ---------------------------------------------------------------------------

def _case(op, name=None, **kw):
    c = dict(op=op, B=1, Hq=32, Hkv=8, d=128, dtype="bf16", page=16, longest=1024, shortest=1024, rows_first=False,
             tracked=False)
    if op == "append":
        c.update(most_new=1)
    elif op == "decode":
        c.update(softcap=0.0, sink=0, local=0, alibi=False, weights=False)
    else:
        c.update(budget=512, sink=64, local=128)
    c.update(kw)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one token of each of 32 running sequences: what every layer of every decode step does first
        _case("append", "append one token, 32 seqs", B=32, longest=1024, shortest=17, tracked=True),
        # the ragged prompts of 8 requests written in one call, token-major pool, pages of 64
        _case("append", "append ragged prompts", B=8, longest=12000, shortest=501, page=64, rows_first=True, most_new=12000),
        # an fp32 cache of small heads with odd-sized pages, a few tokens each (a draft accepted in part)
        _case("append", "append fp32, odd pages", B=5, Hq=4, Hkv=2, d=64, dtype="f32", page=24, longest=777, shortest=9,
              tracked=True, most_new=9),
        # the smallest cache of the repository's own workloads, with a bias that grows with distance
        _case("decode", "decode 1 x 2K fp32, distance bias", Hq=4, Hkv=1, d=64, dtype="f32", longest=2048, shortest=2048,
              alibi=True),
        # one chat at 32K: few rows, so the length has to be split
        _case("decode", "decode 1 x 32K", longest=32768, shortest=32768),
        # a full batch at 32K: the most that is read in one step
        _case("decode", "decode 32 x 32K", B=32, longest=32768, shortest=32768),
        # four books at up to 128K, capped scores, large pages, token-major pool
        _case("decode", "decode 4 x 128K, capped", B=4, longest=131072, shortest=100001, page=64, rows_first=True,
              softcap=30.0),
        # a serving batch of all lengths, an empty row among them, sink and window, wide groups of small heads
        _case("decode", "decode 48 ragged, windowed", B=48, Hq=64, Hkv=8, d=64, longest=8191, shortest=0, sink=64, local=2000),
        # a step that also keeps the score by which the cache is thinned out later, after earlier evictions
        _case("decode", "decode 8 x 32K, weights", B=8, longest=32768, shortest=20000, tracked=True, weights=True),
        # a cache held at 4K: the sixteen tokens since the last eviction go
        _case("evict", "evict 16 of 4K, 32 seqs", B=32, longest=4112, shortest=4100, tracked=True, budget=4096),
        # eight prompts of 32K cut down to 8K
        _case("evict", "evict 8 x 32K to 8K", B=8, longest=32768, shortest=30001, budget=8192),
        # one 128K cache of large pages, token-major, cut to a quarter
        _case("evict", "evict 1 x 128K to 32K", longest=131071, shortest=131071, page=64, rows_first=True, tracked=True,
              budget=32768),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "evict"])
    Hkv, G, d = rng.choice([(8, 4, 128), (8, 4, 128), (8, 8, 64), (2, 7, 128), (4, 1, 128), (1, 4, 64), (4, 2, 64), (2, 16, 128)])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    B = _log(rng, 1, 64)
    # rows of a pool: at most a quarter of the largest listed case's
    longest = _log(rng, 40, max(64, min(131072, (1 << 21) // (B * Hkv))))
    shortest = rng.choice([longest, max(1, longest // 2), max(1, longest // 50)])
    c = dict(B=B, Hq=Hkv * G, Hkv=Hkv, d=d, dtype=dtype, page=rng.choice([16, 16, 32, 64, 24, 1, 128]), longest=longest,
             shortest=shortest, rows_first=rng.random() < 0.4, tracked=rng.random() < 0.5)
    if op == "append":
        c["most_new"] = rng.choice([1, _log(rng, 1, longest)])
    elif op == "decode":
        c["shortest"] = rng.choice([shortest, 0])
        c["softcap"] = rng.choice([0.0, 0.0, 30.0, 50.0])
        if rng.random() < 0.3:
            c["sink"], c["local"] = rng.choice([0, 4, 64]), _log(rng, 1, longest)
        c["alibi"] = rng.random() < 0.25
        c["weights"] = rng.random() < 0.3
    else:
        c["budget"] = _log(rng, max(8, longest // 16), longest)
        c["sink"] = min(c["budget"] // 4, rng.choice([0, 4, 64]))
        c["local"] = min(c["budget"] // 2, rng.choice([1, 32, 128]))
    return _case(op, **c)


def _capacity(case):
    """Table columns and slots per sequence."""
    cols = -(-case["longest"] // case["page"])
    return cols, cols * case["page"]


def _lengths(case, g):
    """Host lengths of the sequences: the longest first, an empty row last where the range allows one."""
    B, lo, hi = case["B"], case["shortest"], case["longest"]
    n = torch.randint(lo, hi + 1, (B,), generator=g)
    n[0] = hi
    if B > 1:
        n[-1] = lo
    return n


def _new_tokens(case, n, g):
    """Host token counts of an append: every sequence takes at least one, of those it holds."""
    most = torch.clamp(n, max=case["most_new"])
    return torch.clamp((most * torch.rand(case["B"], generator=g)).long() + 1, max=most) if case["most_new"] > 1 else most


# ---- inputs --------------------------------------------------------------------------

def _inputs(case, seed):
    dev = torch.device("cuda")
    host = torch.Generator().manual_seed(seed)
    g = torch.Generator(device=dev).manual_seed(seed + 1)
    B, Hq, Hkv, d, page = (case[n] for n in ("B", "Hq", "Hkv", "d", "page"))
    dt = torch.bfloat16 if case["dtype"] == "bf16" else F32
    cols, cap = _capacity(case)
    n_pages = B * cols + 3
    n = _lengths(case, host)

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    # pools: keys around a mean per head, a few of them along the queries' mean (the tokens that attention dwells on)
    mu_q, mu_k = normal(Hq, d, dtype=F32), normal(Hkv, d, dtype=F32)
    shape = (n_pages, page, Hkv, d) if case["rows_first"] else (n_pages, Hkv, page, d)
    k, v = normal(*shape), normal(*shape)
    if case["rows_first"]:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    k += mu_k.to(dt)[None, :, None, :]
    along = mu_q.view(Hkv, -1, d).sum(1)
    along = along / along.norm(dim=-1, keepdim=True)
    hot = torch.randint(0, n_pages * page, (max(1, n_pages * page // 500),), generator=g, device=dev).unique()
    k[hot // page, :, hot % page] += (4.0 * along).to(dt)
    # the sequences' pages, in no order, three of the pool left over
    table = torch.randperm(n_pages, generator=g, device=dev)[: B * cols].view(B, cols).to(I32)
    s = dict(case=case, k=k, v=v, table=table, lengths=n.to(dev, I32), pos=None, seen=None)
    slot = torch.arange(cap, device=dev)
    if case["tracked"]:
        # earlier evictions took a third of the tokens: slots hold rising positions in a shuffled neighbourhood
        seen = n + n // 3
        s["seen"] = seen.to(dev, I32)
        keep = torch.rand(B, Hkv, cap, generator=g, device=dev)
        base = (slot.double() * 4 / 3).floor().to(I32)
        keep = torch.where(slot < s["lengths"].view(B, 1, 1) - 25, keep, torch.zeros_like(keep))
        s["pos"] = base[torch.argsort(slot + 24 * keep, dim=-1, stable=True)]   # a permutation of the slots in use
    if case["op"] == "append":
        new = _new_tokens(case, n, host)
        start = torch.zeros(B + 1, dtype=torch.long)
        start[1:] = new.cumsum(0)
        s["start"] = None if case["most_new"] == 1 else start.to(dev, I32)
        N = int(start[-1])
        fused = normal(N, Hq + 2 * Hkv, d)                               # one projection gives queries, keys and values
        s["k_new"], s["v_new"] = fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
        s["weight"] = torch.rand(B, Hkv, cap, generator=g, device=dev) if case["tracked"] else None
    elif case["op"] == "decode":
        s["q"] = (mu_q + normal(B, Hq, d, dtype=F32)).to(dt)
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=dev, dtype=F32) / Hq) if case["alibi"] else None
        s["out"] = torch.zeros(B, Hq, d, device=dev)
        s["lse"] = torch.zeros(B, Hq, device=dev)
        if case["weights"]:
            s["weight"] = torch.rand(B, Hkv, cap, generator=g, device=dev).pow_(8)
            s["weight_out"] = torch.zeros(B, Hkv, cap, device=dev)
    else:
        # accumulated weights: most near nothing, a few large, some equal
        w = torch.rand(B, Hkv, cap, generator=g, device=dev).pow_(8)
        s["weight"] = torch.where(w < 1e-6, torch.zeros_like(w), w)
        s["lengths_out"] = torch.zeros(B, dtype=I32, device=dev)
        s["weight_out"] = torch.zeros(B, Hkv, cap, device=dev)
        s["pos_out"] = torch.full((B, Hkv, cap), -1, dtype=I32, device=dev)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        # the cache's handle: the arguments that stay the same from step to step
        import kv_cache_residual_b200 as sa
        s["cache"] = sa.PagedCache(s["k"], s["v"], s["table"], s["lengths"], pos=s["pos"], seen=s["seen"])
    return s


# ---- one pass --------------------------------------------------------------------------

def _own(s, c):
    import kv_cache_residual_b200 as sa
    if c["op"] == "append":
        sa.paged_append(s["cache"], s["k_new"], s["v_new"], start=s["start"], weight=s["weight"])
        return _appended(s)
    if c["op"] == "decode":
        sa.paged_decode(s["q"], s["cache"], softcap=c["softcap"], sink=c["sink"], local=c["local"], slopes=s["slopes"],
                        weight=s.get("weight"), weight_out=s.get("weight_out"), out=s["out"], lse=s["lse"])
        return _decoded(s)
    sa.paged_evict(s["cache"], s["weight"], c["budget"], sink=c["sink"], local=c["local"], lengths_out=s["lengths_out"],
                   weight_out=s["weight_out"], pos_out=s["pos_out"])
    return _evicted(s)


def _appended(s):
    r = {"k": s["k"], "v": s["v"]}
    if s["pos"] is not None:
        r["pos"] = s["pos"]
    if s["weight"] is not None:
        r["weight"] = s["weight"]
    return r


def _decoded(s):
    r = {"out": s["out"], "lse": s["lse"]}
    if "weight_out" in s:
        r["weight"] = s["weight_out"]
    return r


def _evicted(s):
    return {"k": s["k"], "v": s["v"], "lengths": s["lengths_out"], "weight": s["weight_out"], "pos": s["pos_out"]}


def _plain_append(s, c):
    N = s["k_new"].shape[0]
    tok = torch.arange(N, device=s["k"].device)
    if s["start"] is None:
        b, left = tok, torch.ones_like(tok)
    else:
        b = torch.searchsorted(s["start"][1:].long(), tok, right=True)
        left = s["start"].long()[b + 1] - tok                # tokens of the sequence from this one on
    slot = s["lengths"].long()[b] - left
    page, row = s["table"].long()[b, slot // c["page"]], slot % c["page"]
    s["k"][page, :, row] = s["k_new"]
    s["v"][page, :, row] = s["v_new"]
    if s["pos"] is not None:
        s["pos"][b, :, slot] = (s["seen"].long()[b] - left).to(I32)[:, None].expand(-1, c["Hkv"])
    if s["weight"] is not None:
        s["weight"][b, :, slot] = 0.0
    return _appended(s)


def _plain_decode(s, c):
    B, Hq, Hkv, d, page = (c[n] for n in ("B", "Hq", "Hkv", "d", "page"))
    cap = s["table"].shape[1] * page
    slot = torch.arange(cap, device=s["k"].device)
    pages, row = s["table"].long()[:, slot // page], (slot % page)[None, :].expand(B, -1)
    q = s["q"].float().view(B, Hkv, Hq // Hkv, d)
    x = torch.matmul(q, s["k"][pages, :, row].float().permute(0, 2, 3, 1)) * (1.0 / math.sqrt(d))    # [B, Hkv, G, cap]
    if c["softcap"] > 0:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    length = s["lengths"].long().view(B, 1, 1, 1)
    newest = (s["lengths"] if s["seen"] is None else s["seen"]).long().view(B, 1, 1, 1) - 1
    pos = slot.view(1, 1, 1, -1) if s["pos"] is None else s["pos"].long()[:, :, None, :]
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, Hkv, -1, 1) * (newest - pos).float()
    sees = slot.view(1, 1, 1, -1) < length
    if c["local"] > 0:
        sees = sees & ((pos < c["sink"]) | (pos > newest - c["local"]))
    x = torch.where(sees, x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True)
    e = torch.where(sees, torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m)), torch.zeros_like(x))
    z = e.sum(-1, keepdim=True)
    p = torch.where(z > 0, e / z, torch.zeros_like(e))
    s["out"].copy_(torch.matmul(p, s["v"][pages, :, row].float().transpose(1, 2)).view(B, Hq, d))
    s["lse"].copy_((m + torch.log(z)).view(B, Hq))
    if c["weights"]:
        here = slot < s["lengths"].long().view(B, 1, 1)
        s["weight_out"].copy_(torch.where(here, s["weight"] + p.sum(2), s["weight_out"]))
    return _decoded(s)


def _plain_evict(s, c):
    B, Hkv, page, budget = (c[n] for n in ("B", "Hkv", "page", "budget"))
    cap = s["table"].shape[1] * page
    slot = torch.arange(cap, device=s["k"].device).expand(B, Hkv, cap)
    length = s["lengths"].long().view(B, 1, 1)
    newest = (s["lengths"] if s["seen"] is None else s["seen"]).long().view(B, 1, 1) - 1
    pos = slot if s["pos"] is None else s["pos"].long()
    # rank of every slot: what always stays, then by weight, ties to the lower slot, then the slots past the end
    w = torch.where(torch.isnan(s["weight"]), torch.full_like(s["weight"], -math.inf), s["weight"])
    kind = torch.where(slot < length, torch.where((pos < c["sink"]) | (pos > newest - c["local"]), 2, 1), 0)
    by_weight = torch.sort(w, dim=-1, descending=True, stable=True).indices
    then = torch.sort(kind.gather(-1, by_weight), dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(slot).scatter_(-1, by_weight.gather(-1, then), slot)
    new = torch.clamp(length, max=budget)
    stays = rank < new
    # the i-th kept slot past the new length moves into the i-th freed slot before it
    late, hole = stays & (slot >= new), ~stays & (slot < new)
    nth = late.long().cumsum(-1) - 1
    spare = torch.zeros(B, Hkv, cap + 1, dtype=torch.long, device=slot.device)
    mover = spare.scatter_(-1, torch.where(late, nth, torch.full_like(nth, cap)), slot)
    src = torch.where(hole, mover.gather(-1, (hole.long().cumsum(-1) - 1).clamp(min=0)), slot)
    here = slot < new
    table = s["table"].long()[:, None, :].expand(B, Hkv, -1)
    head = torch.arange(Hkv, device=slot.device).view(1, Hkv, 1)
    # rows of the slots that can change: the first `budget`
    most = min(cap, budget)
    at = (table.gather(-1, slot[..., :most] // page), head, slot[..., :most] % page)
    frm = (table.gather(-1, src[..., :most] // page), head, src[..., :most] % page)
    s["k"][at] = s["k"][frm]
    s["v"][at] = s["v"][frm]
    s["lengths_out"].copy_(new.view(B))
    s["weight_out"].copy_(torch.where(here, s["weight"].gather(-1, src), s["weight_out"]))
    s["pos_out"].copy_(torch.where(here, pos.gather(-1, src).to(I32), s["pos_out"]))
    return _evicted(s)


def run(state):
    c = state["case"]
    if own:
        return _own(state, c)
    return {"append": _plain_append, "decode": _plain_decode, "evict": _plain_evict}[c["op"]](state, c)


# ---- what a pass cannot do without ------------------------------------------------------

def work(case):
    host = torch.Generator()
    B, Hq, Hkv, d, page = (case[n] for n in ("B", "Hq", "Hkv", "d", "page"))
    esz = 2 if case["dtype"] == "bf16" else 4
    n = _lengths(case, host.manual_seed(0))                   # the lengths' sum hardly depends on the seed
    per_slot = Hkv * (4 if case["tracked"] else 0)
    table = 4.0 * float((-(-n // page)).sum()) + 8.0 * B
    if case["op"] == "append":
        N = float(_new_tokens(case, n, host).sum())
        return {"bytes": N * (4.0 * Hkv * d * esz + (2 * per_slot)) + 8.0 * B + 4.0 * N, "flops": 0.0}
    if case["op"] == "decode":
        seen = n.double()
        if case["local"] > 0:
            total = (n + n // 3 if case["tracked"] else n).double().clamp(min=1)
            seen = torch.minimum(seen, (case["sink"] + case["local"]) * n.double() / total)
        rows = float(seen.sum())
        by = rows * 2 * Hkv * d * esz + B * Hq * d * (esz + 4.0) + 4.0 * B * Hq + table
        if case["tracked"] and (case["local"] > 0 or case["alibi"]):
            by += float(n.sum()) * per_slot
        if case["weights"]:
            by += float(n.sum()) * Hkv * 8
        return {"bytes": by, "flops": 4.0 * rows * Hq * d}
    new = torch.clamp(n, max=case["budget"]).double()
    gone = n.double() - new
    # tokens that stay lie anywhere: the share of the last `gone` slots that stays has to move
    moves = float((gone * new / n.double().clamp(min=1)).sum()) * Hkv
    scan = float(n.sum()) * (4 * Hkv + per_slot) + float(new.sum()) * Hkv * 8
    return {"bytes": moves * 4.0 * d * esz + scan + table, "flops": 0.0}


# ---- the definition, in 64 bits ----------------------------------------------------------

def exact(case, seed):
    """Sequence by sequence and head by head."""

    def rows(s, b, n, page):
        """(page, row) of slots [0, n) of sequence b."""
        i = torch.arange(n, device=s["k"].device)
        return s["table"][b].long()[torch.div(i, page, rounding_mode="floor")], i % page

    def exact_append(s, c):
        k, v = s["k"].double(), s["v"].double()
        pos = None if s["pos"] is None else s["pos"].clone()
        weight = None if s["weight"] is None else s["weight"].double()
        first = 0
        for b in range(c["B"]):
            n = 1 if s["start"] is None else int(s["start"][b + 1] - s["start"][b])
            length = int(s["lengths"][b])
            pg, row = rows(s, b, length, c["page"])
            pg, row = pg[length - n:], row[length - n:]
            k[pg, :, row] = s["k_new"][first:first + n].double()
            v[pg, :, row] = s["v_new"][first:first + n].double()
            if pos is not None:
                newest = int(s["seen"][b]) - 1
                pos[b, :, length - n:length] = torch.arange(newest - n + 1, newest + 1, device=pos.device, dtype=I32)
            if weight is not None:
                weight[b, :, length - n:length] = 0.0
            first += n
        r = {"k": k, "v": v}
        if pos is not None:
            r["pos"] = pos
        if weight is not None:
            r["weight"] = weight
        return r

    def exact_decode(s, c):
        B, Hq, Hkv, d = (c[n] for n in ("B", "Hq", "Hkv", "d"))
        G = Hq // Hkv
        out = torch.zeros(B, Hq, d, dtype=torch.float64, device=s["k"].device)
        lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=out.device)
        weight = s["weight_out"].double() if c["weights"] else None
        for b in range(B):
            n = int(s["lengths"][b])
            if n == 0:
                continue
            newest = (n if s["seen"] is None else int(s["seen"][b])) - 1
            pg, row = rows(s, b, n, c["page"])
            for h in range(Hkv):
                K, V = s["k"][pg, h, row].double(), s["v"][pg, h, row].double()
                x = s["q"][b, h * G:(h + 1) * G].double() @ K.T / math.sqrt(d)
                if c["softcap"] > 0:
                    x = torch.tanh(x / c["softcap"]) * c["softcap"]
                at = torch.arange(n, device=out.device) if s["pos"] is None else s["pos"][b, h, :n].long()
                away = newest - at
                if s["slopes"] is not None:
                    x = x - s["slopes"][h * G:(h + 1) * G].double()[:, None] * away.double()
                if c["local"] > 0:
                    x[:, ~((at < c["sink"]) | (away < c["local"]))] = -math.inf
                total = torch.logsumexp(x, dim=-1)
                p = torch.exp(x - total[:, None])
                p = torch.nan_to_num(p, nan=0.0)
                out[b, h * G:(h + 1) * G] = p @ V
                lse[b, h * G:(h + 1) * G] = total
                if weight is not None:
                    weight[b, h, :n] = s["weight"][b, h, :n].double() + p.sum(0)
        r = {"out": out, "lse": lse}
        if weight is not None:
            r["weight"] = weight
        return r

    def exact_evict(s, c):
        k, v = s["k"].double(), s["v"].double()
        lengths, weight, pos = s["lengths_out"].clone(), s["weight_out"].double(), s["pos_out"].clone()
        for b in range(c["B"]):
            n = int(s["lengths"][b])
            new = min(n, c["budget"])
            newest = (n if s["seen"] is None else int(s["seen"][b])) - 1
            lengths[b] = new
            pg, row = rows(s, b, n, c["page"])
            for h in range(c["Hkv"]):
                w = s["weight"][b, h, :n].double()
                at = torch.arange(n, device=w.device) if s["pos"] is None else s["pos"][b, h, :n].long()
                always = (at < c["sink"]) | (at > newest - c["local"])
                sure = always.nonzero()[:, 0]
                rest = (~always).nonzero()[:, 0]
                best = rest[torch.sort(-w[rest], stable=True).indices[: max(0, new - len(sure))]]
                stays = torch.zeros(n, dtype=torch.bool, device=w.device)
                stays[torch.cat([sure[:new], best])] = True
                holes = (~stays[:new]).nonzero()[:, 0]
                late = stays[new:].nonzero()[:, 0] + new
                src = torch.arange(new, device=w.device)
                src[holes] = late
                k[pg[holes], h, row[holes]] = s["k"][pg[late], h, row[late]].double()
                v[pg[holes], h, row[holes]] = s["v"][pg[late], h, row[late]].double()
                weight[b, h, :new] = w[src]
                pos[b, h, :new] = at[src].to(I32)
        return {"k": k, "v": v, "lengths": lengths, "weight": weight, "pos": pos}

    return {"append": exact_append, "decode": exact_decode, "evict": exact_evict}[case["op"]](_inputs(case, seed), case)
