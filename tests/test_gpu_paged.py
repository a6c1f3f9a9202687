"""GPU parity of the paged cache's operators (sa_paged_append, sa_paged_decode,
sa_paged_evict) against the fp64 oracle: cache forms, masks, sizes, strides and
streams, and a run of the three together.

Append and eviction move bits: they are compared exactly.  The decode's bound,
with u = 2^-24 (half a step of fp32):
  logit    d products summed in blocks of 16, each block off by at most 4 last
           places (8 u) whether by fused adds or by a matrix instruction, the
           blocks' sum likewise: 8 u (d/16 + 4) scale sum_e |q_e k_e|; then scaling,
           cap (tanhf: 2 places) and bias: 8 u of each term
  weight   relative: the logit's error, once for the weight and once for the sum;
           2^x off by 2^-22 at each of at most 24 rescalings and joins
  sum      one lane adds at most n/8 + 64 terms one after another: that many u
The capped, biased logit is bounded term by term, and every term relative to
sum p |v|, so no entry's own cancellation enters."""
import math

import numpy as np
import pytest
import torch

import kv_cache_residual_b200 as sa
from oracle import paged as opaged
from parity_util import f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _dev():
    return torch.device("cuda", torch.cuda.current_device())


class Case:
    """A paged cache on the GPU.  Everything in the pools that no live slot
    holds is NaN."""

    def __init__(self, lens, Hkv=2, G=4, d=128, page=16, dtype=BF, layout="heads", tracked=False, cols=None, seed=0,
                 scale_k=1.0):
        r = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        dev = _dev()
        self.B, self.Hkv, self.G, self.d, self.page, self.dtype = len(lens), Hkv, G, d, page, dtype
        self.Hq = Hkv * G
        self.lens = list(lens)
        self.cols = max(1, -(-max(lens) // page)) if cols is None else cols
        self.cap = self.cols * page
        self.n_pages = self.B * self.cols + 2
        nan = dict(fill_value=float("nan"), dtype=dtype, device=dev)
        n, H, p = self.n_pages, Hkv, page
        if layout == "heads":                      # [n_pages, Hkv, page, d]
            k, v = torch.full((n, H, p, d), **nan), torch.full((n, H, p, d), **nan)
        elif layout == "rows":                     # [n_pages, page, Hkv, d]
            k, v = (torch.full((n, p, H, d), **nan).transpose(1, 2) for _ in range(2))
        elif layout == "both":                     # [n_pages, 2, Hkv, page, d]
            kv = torch.full((n, 2, H, p, d), **nan)
            k, v = kv[:, 0], kv[:, 1]
        else:                                      # rows padded by 16 bytes, pages and heads by more
            pad = 16 // torch.tensor([], dtype=dtype).element_size()
            k, v = (torch.full((n, H + 1, p + 1, d + pad), **nan)[:, :H, :p, :d] for _ in range(2))
        self.k, self.v = k, v
        self.table_h = r.permutation(n)[:self.B * self.cols].reshape(self.B, self.cols).astype(np.int32)
        self.table = torch.from_numpy(self.table_h).to(dev)
        self.lengths = torch.tensor(lens, dtype=I32, device=dev)
        for b, L in enumerate(lens):
            pg, row, _ = opaged.slot_pages(self.table_h[b], L, page, n)
            pg, row = torch.from_numpy(pg).long().to(dev), torch.from_numpy(row).to(dev)
            for t, f in ((k, scale_k), (v, 1.0)):
                x = torch.randn(L, H, d, generator=g, device=dev) * f
                t[pg, :, row] = x.to(dtype)
        self.q = torch.randn(self.B, self.Hq, d, generator=g, device=dev).to(dtype)
        self.pos = self.seen = None
        if tracked:
            self.seen_h = [L + L // 2 + 1 for L in lens]
            pos = np.full((self.B, Hkv, self.cap), -7, dtype=np.int32)
            for b, L in enumerate(lens):
                for h in range(Hkv):
                    pos[b, h, :L] = r.permutation(self.seen_h[b])[:L]
                    if L:
                        pos[b, h, r.integers(L)] = self.seen_h[b] - 1
            self.pos = torch.from_numpy(pos).to(dev)
            self.seen = torch.tensor(self.seen_h, dtype=I32, device=dev)
        self.weight = torch.rand(self.B, Hkv, self.cap, generator=g, device=dev)

    def cache(self, **kw):
        a = dict(k=self.k, v=self.v, table=self.table, lengths=self.lengths, pos=self.pos, seen=self.seen)
        a.update(kw)
        return sa.PagedCache(*[a[n] for n in ("k", "v", "table", "lengths", "pos", "seen")])

    def unit(self, b, h):
        """Rows, positions, newest position and valid slots of a unit, on the host."""
        L = min(max(int(self.lengths[b]), 0), self.cap)
        pg, row, ok = opaged.slot_pages(self.table.cpu().numpy()[b], L, self.page, self.n_pages)
        at = np.where(ok, pg, 0)
        K, V = f64(self.k[at, h, row]), f64(self.v[at, h, row])
        pos = np.arange(L) if self.pos is None else self.pos[b, h, :L].cpu().numpy()
        newest = (L if self.seen is None else int(self.seen[b])) - 1
        return L, K, V, pos, newest, ok


def _check_decode(c, out, lse, weight_out=None, weight=None, before=None, scale=0.0, softcap=0.0, sink=0, local=0,
                  slopes=None):
    s = scale if scale > 0 else 1.0 / math.sqrt(c.d)
    q = f64(c.q)
    sl = None if slopes is None else f64(slopes)
    out, lse = f64(out), f64(lse)
    wo = None if weight_out is None else f64(weight_out)
    for b in range(c.B):
        for h in range(c.Hkv):
            L, K, V, pos, newest, ok = c.unit(b, h)
            sees = ok & opaged.visible(pos, newest, sink, local)
            at = slice(h * c.G, (h + 1) * c.G)
            slu = None if sl is None else sl[at]
            ro, rl, p = opaged.decode_unit(q[b, at], K, V, pos, newest, sees, s, softcap, slu)
            w = (b, h)
            if not sees.any():
                assert not out[b, at].any() and np.all(lse[b, at] == -np.inf), w
                dp = np.zeros((c.G, 1))
            else:
                Ks, Vs = K[sees], V[sees]
                mag = s * (np.abs(q[b, at]) @ np.abs(Ks).T)
                dx = 8 * U * (c.d / 16 + 4) * mag + 8 * U * mag
                if softcap > 0:
                    dx = dx + 8 * U * softcap
                if slu is not None:
                    dx = dx + 8 * U * slu[:, None] * (newest - pos[sees])
                    dx = dx + 8 * U * slu[:, None] * np.abs(newest - pos[sees])
                live = p[:, sees] > 1e-12                  # a weight below that does not show
                dx = np.where(live, dx, 0.0).max(axis=1)
                rel = np.expm1(dx) + 24 * 1.25 * 2.0 ** -22 + (L / 8 + 64) * U
                tol = (2 * rel + 1e-9)[:, None] * (p[:, sees] @ np.abs(Vs)) + 1e-9
                assert np.all(np.abs(out[b, at] - ro) <= tol), (w, np.max(np.abs(out[b, at] - ro) / tol))
                tl = rel + 4 * U * np.abs(rl) + dx
                assert np.all(np.abs(lse[b, at] - rl) <= tl), (w, lse[b, at], rl)
                dp = (2 * rel + 1e-9)[:, None]
            if wo is not None:
                w0 = np.zeros(c.cap) if weight is None else f64(weight[b, h])
                want = w0[:L] + p.sum(axis=0)
                tol = (dp * p).sum(axis=0) + 8 * U * (np.abs(w0[:L]) + p.sum(axis=0)) + 1e-12 * c.G
                assert np.all(np.abs(wo[b, h, :L] - want) <= tol), w
                assert np.array_equal(wo[b, h, L:], f64(before[b, h, L:])), w


def _decode(c, weights=False, cache=None, **kw):
    args = dict(kw)
    before = None
    if weights:
        before = torch.full((c.B, c.Hkv, c.cap), -3.0, device=_dev())
        args.update(weight=c.weight, weight_out=before.clone())
    out, lse = sa.paged_decode(c.q, cache or c.cache(), **args)
    torch.cuda.synchronize()
    _check_decode(c, out, lse, args.get("weight_out"), c.weight if weights else None, before, **kw)
    return out, lse


LENS = [[1], [0, 1, 15, 16, 17, 63], [64, 65, 0, 127, 128, 129], [1000, 3], [5003]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("dtype,d,G", [(BF, 128, 4), (BF, 64, 8), (F32, 128, 2), (F32, 64, 1)])
def test_decode_lengths(lens, dtype, d, G):
    c = Case(lens, G=G, d=d, dtype=dtype, seed=1)
    _decode(c)
    _decode(c, weights=True)


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8, 9, 12, 16, 17, 24])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
def test_decode_groups(G, dtype, d):
    c = Case([130, 0, 777], Hkv=3, G=G, d=d, dtype=dtype, seed=2)
    _decode(c, weights=True, softcap=3.0)


@pytest.mark.parametrize("page", [1, 3, 16, 24, 64, 100, 128])
@pytest.mark.parametrize("layout", ["heads", "rows", "both", "padded"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_pages_and_strides(page, layout, dtype):
    c = Case([333, 1, 64, 200], page=page, layout=layout, dtype=dtype, seed=3)
    _decode(c)
    _decode(c, sink=5, local=77)


@pytest.mark.parametrize("sink,local", [(0, 1), (0, 64), (64, 2000), (3, 100), (200, 1), (5000, 5000), (1, 63)])
@pytest.mark.parametrize("tracked", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_windows(sink, local, tracked, dtype):
    c = Case([2500, 64, 0, 1, 300], tracked=tracked, dtype=dtype, seed=4)
    slopes = torch.exp2(-torch.arange(1, c.Hq + 1, device=_dev(), dtype=F32))
    _decode(c, sink=sink, local=local)
    _decode(c, weights=True, sink=sink, local=local, slopes=slopes, softcap=20.0)


@pytest.mark.parametrize("softcap", [0.0, 0.5, 30.0])
@pytest.mark.parametrize("scale", [0.0, 0.7])
@pytest.mark.parametrize("biased", [False, True])
def test_decode_scores(softcap, scale, biased):
    for dtype in (BF, F32):
        c = Case([900, 31], dtype=dtype, seed=5, tracked=biased)
        slopes = torch.linspace(0.0, 0.5, c.Hq, device=_dev()) if biased else None
        _decode(c, weights=True, softcap=softcap, scale=scale, slopes=slopes)


def test_decode_rising_scores():
    """Logits that grow along the cache: the running maximum moves at every row."""
    for dtype in (BF, F32):
        c = Case([1500], dtype=dtype, seed=6)
        pg, row, _ = opaged.slot_pages(c.table_h[0], 1500, c.page, c.n_pages)
        ramp = torch.linspace(0, 3, 1500, device=_dev())[:, None, None]
        c.k[pg, :, row] = (c.q[0].float().view(c.Hkv, c.G, c.d).mean(1)[None] * ramp).to(dtype)
        _decode(c, weights=True)


@pytest.mark.parametrize("tracked", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_masked_slots_are_not_read(tracked, dtype):
    """Infinities and NaN in the keys and values of slots a query does not see."""
    c = Case([700, 90], tracked=tracked, dtype=dtype, seed=7)
    sink, local = 10, 120
    for b in range(c.B):
        for h in range(c.Hkv):
            L, K, V, pos, newest, ok = c.unit(b, h)
            out = np.nonzero(~opaged.visible(pos, newest, sink, local))[0]
            pg, row, _ = opaged.slot_pages(c.table_h[b], L, c.page, c.n_pages)
            for i, bad in enumerate((float("nan"), float("inf"), float("-inf"))):
                at = out[i::3]
                c.k[pg[at], h, row[at]] = bad
                c.v[pg[at], h, row[at]] = bad
    _decode(c, weights=True, sink=sink, local=local)


def test_decode_sees_nothing():
    c = Case([40, 5, 0], tracked=True, seed=8)
    c.seen += 10000                                     # every position lies before the window
    c.k.fill_(float("nan"))
    c.v.fill_(float("nan"))
    out, lse = _decode(c, weights=True, local=50)
    assert not out.any() and torch.all(lse == -math.inf)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_bad_pages_are_masked(dtype):
    c = Case([200, 64, 33], dtype=dtype, seed=9)
    c.table[0, 2], c.table[0, 12], c.table[2, 0] = -1, c.n_pages, 2 ** 31 - 1
    c.table[1, :] = -(2 ** 31)
    out, lse = _decode(c, weights=True)
    assert not out[1].any()


def test_decode_lengths_are_clamped():
    c = Case([64, 50], cols=4, seed=10)
    c.lengths.copy_(torch.tensor([1 << 30, -5]))
    _decode(c, weights=True)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_infinite_logits(dtype):
    """A key at -inf along a head's query has weight 0 there; NaN in a seen row
    stays within its unit."""
    c = Case([70, 70], dtype=dtype, seed=11)
    base, _ = sa.paged_decode(c.q, c.cache())
    pg, row, _ = opaged.slot_pages(c.table_h[0], 70, c.page, c.n_pages)
    c.q[0, 0] = 0.0
    c.q[0, 0, 0] = 1.0
    c.q[0, 1:c.G, 0] = 1.0
    for s in (0, 69):
        c.k[pg[s], 0, row[s]] = 0.0
        c.k[pg[s], 0, row[s], 0] = float("-inf")
    out, lse = sa.paged_decode(c.q, c.cache())
    L, K, V, pos, newest, _ = c.unit(0, 0)
    sees = np.ones(70, dtype=bool)
    sees[[0, 69]] = False
    ro, rl, _ = opaged.decode_unit(f64(c.q[0, :c.G]), K, V, pos, newest, sees, 1 / math.sqrt(c.d))
    assert np.allclose(f64(out[0, 0]), ro[0], rtol=0, atol=1e-4) and abs(float(lse[0, 0]) - rl[0]) < 1e-4
    c.k[pg[3], 1, row[3], 5] = float("nan")
    out, lse = sa.paged_decode(c.q, c.cache())
    assert torch.isnan(out[0, c.G:2 * c.G]).all() and torch.isnan(lse[0, c.G:2 * c.G]).all()
    assert torch.isfinite(out[0, 0]).all() and torch.equal(out[1], base[1])


def test_decode_query_strides_and_outputs():
    c = Case([100, 20, 7], seed=12)
    fused = torch.randn(c.B, c.Hq + 2 * c.Hkv, c.d, device=_dev()).to(BF)
    c.q = fused[:, :c.Hq]
    out, lse = torch.empty(c.B, c.Hq, c.d, device=_dev()), torch.empty(c.B, c.Hq, device=_dev())
    o, l = sa.paged_decode(c.q, c.cache(), out=out, lse=lse)
    assert o is out and l is lse
    _check_decode(c, out, lse)


def test_decode_weights_in_place_and_from_nothing():
    c = Case([300, 0, 17], seed=13)
    none = torch.full((c.B, c.Hkv, c.cap), 5.0, device=_dev())
    before = none.clone()
    out, lse = sa.paged_decode(c.q, c.cache(), weight_out=none)
    _check_decode(c, out, lse, none, None, before)
    acc, start = c.weight.clone(), c.weight.clone()
    sa.paged_decode(c.q, c.cache(), weight=acc, weight_out=acc)
    _check_decode(c, out, lse, acc, start, start)


def test_decode_many_sequences():
    """More sequences than threads of a CTA, most of them short or empty."""
    r = np.random.default_rng(14)
    c = Case([int(x) for x in r.integers(0, 40, 600)], Hkv=1, G=4, d=64, cols=3, seed=14)
    _decode(c)
    c = Case([0] * 300 + [900] + [0] * 50, Hkv=2, d=64, cols=57, seed=15)
    _decode(c, weights=True)


def test_decode_repeats_bit_for_bit():
    c = Case([9000, 100, 4000], seed=16)
    cache = c.cache()
    a = sa.paged_decode(c.q, cache)
    for _ in range(5):
        b = sa.paged_decode(c.q, cache)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_workspaces_of_one_size():
    """Shapes whose workspaces have one size but not the same tickets."""
    for B, Hkv in ((1, 2), (2, 4), (4, 8), (1, 16), (3, 2)):
        c = Case([5000] + [600] * (B - 1), Hkv=Hkv, d=64, seed=17)
        _decode(c)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_offsets_past_32_bits(dtype):
    """Pages whose rows start beyond 2^31 elements, in a token-major pool."""
    dev = _dev()
    H, d, page = 8, 128, 64
    n = 2 ** 31 // (H * d * page) + 40
    k = torch.empty(n, page, H, d, dtype=dtype, device=dev).transpose(1, 2)
    v = torch.empty(n, page, H, d, dtype=dtype, device=dev).transpose(1, 2)
    c = Case([500], Hkv=H, G=2, page=page, dtype=dtype, seed=18)
    c.table_h = c.table_h * 0 + np.arange(n - c.cols, n, dtype=np.int32)[None, ::-1]
    for i in range(c.cols):
        k[int(c.table_h[0, i])] = c.k[int(c.table[0, i])]
        v[int(c.table_h[0, i])] = c.v[int(c.table[0, i])]
    c.k, c.v, c.n_pages = k, v, n
    c.table.copy_(torch.from_numpy(c.table_h.copy()))
    _decode(c)
    new = torch.randn(1, H, d, device=dev).to(dtype)
    sa.paged_append(c.cache(), new, -new)
    assert torch.equal(k[int(c.table_h[0, 499 // page]), :, 499 % page], new[0])
    _decode(c)
    _evict(c, 200, 4, 30)


# ---- append ------------------------------------------------------------------

def _pools(c):
    return f64(c.k).copy(), f64(c.v).copy()


@pytest.mark.parametrize("page", [1, 16, 24])
@pytest.mark.parametrize("layout", ["heads", "rows", "both", "padded"])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("one", [True, False])
def test_append(page, layout, dtype, d, one):
    c = Case([40, 1, 77, 9], page=page, layout=layout, dtype=dtype, d=d, tracked=True, seed=20)
    n = [1] * 4 if one else [7, 0, 77, 2]
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    N = int(start[-1])
    dev = _dev()
    fused = torch.randn(N, 3 * c.Hkv, d, device=dev).to(dtype)
    kn, vn = fused[:, :c.Hkv], fused[:, c.Hkv:2 * c.Hkv]
    K, V = _pools(c)
    pos, w = c.pos.cpu().numpy().copy(), f64(c.weight).copy()
    for b in range(4):
        for j in range(n[b]):
            s = c.lens[b] - n[b] + j
            pg, row = c.table_h[b, s // page], s % page
            K[pg, :, row], V[pg, :, row] = f64(kn[start[b] + j]), f64(vn[start[b] + j])
            pos[b, :, s], w[b, :, s] = c.seen_h[b] - n[b] + j, 0.0
    sa.paged_append(c.cache(), kn, vn, start=None if one else torch.from_numpy(start).to(dev), weight=c.weight)
    torch.cuda.synchronize()
    for got, want in ((f64(c.k), K), (f64(c.v), V), (f64(c.weight), w)):
        assert np.array_equal(got, want, equal_nan=True)
    assert np.array_equal(c.pos.cpu().numpy(), pos)


def test_append_skips_what_has_no_place():
    """Tokens outside every sequence, more of them than the sequence is long,
    pages that are not the pool's, lengths past the capacity."""
    dev = _dev()
    c = Case([20, 3, 30, 64], cols=4, seed=21)
    c.lengths[3] = 1000                                             # clamped to 64
    c.table[2, 1], c.table[2, 0] = -1, c.n_pages
    new = torch.randn(30, c.Hkv, c.d, device=dev).to(BF)
    K, V = _pools(c)
    start = torch.tensor([2, 6, 12, 25, 28], dtype=I32, device=dev)     # 4, 6, 13 and 3 tokens
    for b, toks, first in ((0, range(2, 6), 16), (1, range(9, 12), 0), (3, range(25, 28), 61)):
        for j, t in enumerate(toks):
            pg, row = c.table_h[b, (first + j) // 16], (first + j) % 16
            K[pg, :, row], V[pg, :, row] = f64(new[t]), f64(-new[t])
    sa.paged_append(c.cache(), new, -new, start=start)
    assert np.array_equal(f64(c.k), K, equal_nan=True) and np.array_equal(f64(c.v), V, equal_nan=True)
    sa.paged_append(c.cache(), new[:0], new[:0], start=start * 0)
    assert np.array_equal(f64(c.k), K, equal_nan=True)


def test_append_many_tokens():
    c = Case([3000, 5000, 1], Hkv=4, layout="rows", page=64, seed=22)
    dev = _dev()
    new = torch.randn(8001, 4, c.d, device=dev).to(BF)
    start = torch.tensor([0, 3000, 8000, 8001], dtype=I32, device=dev)
    sa.paged_append(c.cache(), new, -new, start=start)
    for b in range(3):
        pg, row, _ = opaged.slot_pages(c.table_h[b], c.lens[b], 64, c.n_pages)
        assert torch.equal(c.k[pg, :, row], new[int(start[b]):int(start[b + 1])])
        assert torch.equal(c.v[pg, :, row], -new[int(start[b]):int(start[b + 1])])


# ---- eviction ----------------------------------------------------------------

def _evict(c, budget, sink, local, **kw):
    """Runs the eviction and compares everything it writes, and all it must not."""
    dev = _dev()
    K0, V0 = c.k.clone(), c.v.clone()
    units = [(b, h, c.unit(b, h)) for b in range(c.B) for h in range(c.Hkv)]
    wo = torch.full((c.B, c.Hkv, c.cap), -3.0, device=dev)
    po = torch.full((c.B, c.Hkv, c.cap), -9, dtype=I32, device=dev)
    lo, w2, p2 = sa.paged_evict(c.cache(), c.weight, budget, sink, local, weight_out=wo, pos_out=po, **kw)
    assert w2 is wo and p2 is po
    torch.cuda.synchronize()
    W, P = wo.cpu().numpy(), po.cpu().numpy()
    wt = c.weight.cpu().numpy()
    for b, h, (L, K, V, pos, newest, ok) in units:
        src = opaged.evict_unit(wt[b, h, :L], pos, newest, budget, sink, local)
        n = min(L, budget)
        assert int(lo[b]) == n and len(src) == n
        assert np.array_equal(W[b, h, :n], wt[b, h, src], equal_nan=True), (b, h)
        assert np.array_equal(P[b, h, :n], pos[src]), (b, h)
        assert np.all(W[b, h, n:] == -3.0) and np.all(P[b, h, n:] == -9)
        tb = c.table.cpu().numpy()[b]
        moved = np.nonzero(src != np.arange(n))[0]
        frm = src[moved]
        fine = ok[moved] & ok[frm]
        moved, frm = moved[fine], frm[fine]
        for now, old in ((c.k, K0), (c.v, V0)):
            x = old[tb[frm // c.page], h, frm % c.page]
            old[tb[moved // c.page], h, moved % c.page] = x
    bits = torch.int16 if c.dtype == BF else torch.int32
    assert torch.equal(c.k.view(bits), K0.view(bits)) and torch.equal(c.v.view(bits), V0.view(bits))
    return lo, wo, po


@pytest.mark.parametrize("budget,sink,local", [(1, 0, 0), (1, 0, 1), (16, 4, 4), (100, 0, 100), (100, 30, 10), (299, 4, 32),
                                               (300, 4, 32), (5000, 64, 128)])
@pytest.mark.parametrize("tracked", [False, True])
@pytest.mark.parametrize("dtype,d,layout", [(BF, 128, "heads"), (F32, 64, "rows"), (F32, 128, "both"), (BF, 64, "padded")])
def test_evict(budget, sink, local, tracked, dtype, d, layout):
    c = Case([300, 0, 1, 299, 17, 2000], d=d, dtype=dtype, layout=layout, tracked=tracked, page=24, seed=30)
    _evict(c, budget, sink, local)


def test_evict_odd_weights():
    """Ties, both zeros, infinities, NaN, negative and subnormal weights."""
    inf, nan = math.inf, math.nan
    pool = torch.tensor([0.0, -0.0, 1.0, 1.0, 1.0, inf, -inf, nan, -1.0, 1e-40, 2e-40, 3.4e38, -nan], device=_dev())
    for budget in (5, 64, 150, 333):
        c = Case([400, 334, 20], seed=31)
        c.weight = pool[torch.randint(0, 13, c.weight.shape, device=_dev(),
                                      generator=torch.Generator(device="cuda").manual_seed(budget))]
        _evict(c, budget, 2, 3)
        c.weight = torch.ones_like(c.weight)
        _evict(c, budget, 0, 0)
        c.weight = torch.full_like(c.weight, nan)
        _evict(c, budget, 1, 0)


def test_evict_bad_pages_and_lengths():
    c = Case([200, 100, 64], cols=13, seed=32)
    c.table[0, 0], c.table[0, 10], c.table[1, 3] = -1, c.n_pages, 2 ** 31 - 1
    c.lengths[2] = 1 << 30
    _evict(c, 60, 4, 8)


def test_evict_long_units():
    """Slices too long for the keys in shared memory, one unit and several."""
    c = Case([420001], Hkv=1, G=1, d=64, page=64, seed=33)
    _evict(c, 100000, 64, 128)
    c = Case([60000, 70003], Hkv=2, G=1, d=64, page=16, layout="rows", tracked=True, seed=34)
    c.weight = (c.weight * 50).floor()                  # many ties
    _evict(c, 20000, 64, 128)


def test_evict_many_units():
    r = np.random.default_rng(35)
    c = Case([int(x) for x in r.integers(0, 90, 200)], Hkv=4, G=1, d=64, cols=6, seed=35)
    _evict(c, 33, 4, 8)


# ---- together, graphs, streams -------------------------------------------------

def test_a_run_of_all_three():
    """Prompts, then steps of append, decode with weights and, now and then, an
    eviction: against an fp64 cache of plain lists that does the same."""
    dev = _dev()
    B, Hkv, G, d, page, budget, sink, local = 3, 2, 4, 64, 16, 48, 4, 16
    Hq, cols, n_pages = Hkv * G, 6, 3 * 6
    g = torch.Generator(device="cuda").manual_seed(40)
    k = torch.zeros(n_pages, Hkv, page, d, device=dev)
    v = torch.zeros_like(k)
    table = torch.randperm(n_pages, generator=g, device=dev).view(B, cols).to(I32)
    prompts = [50, 1, 31]
    lengths = torch.tensor(prompts, dtype=I32, device=dev)
    seen = lengths.clone()
    pos = torch.zeros(B, Hkv, cols * page, dtype=I32, device=dev)
    weight = torch.zeros(B, Hkv, cols * page, device=dev)
    start = torch.tensor([0, 50, 51, 82], dtype=I32, device=dev)
    kn, vn = (torch.randn(82, Hkv, d, generator=g, device=dev) for _ in range(2))
    sa.paged_append(sa.PagedCache(k, v, table, lengths, pos, seen), kn, vn, start=start, weight=weight)
    rows = [[[(f64(kn[i, h]), f64(vn[i, h]), i - int(start[b]), 0.0) for i in range(int(start[b]), int(start[b + 1]))]
             for h in range(Hkv)] for b in range(B)]
    evictions = 0
    for step in range(40):
        lengths = lengths + 1
        seen = seen + 1
        kn, vn = (torch.randn(B, Hkv, d, generator=g, device=dev) for _ in range(2))
        q = torch.randn(B, Hq, d, generator=g, device=dev) * 2
        cache = sa.PagedCache(k, v, table, lengths, pos, seen)
        sa.paged_append(cache, kn, vn, weight=weight)
        out, lse = sa.paged_decode(q, cache, softcap=15.0, weight=weight, weight_out=weight)
        evict = step % 9 == 8
        if evict:
            lengths, weight, pos = sa.paged_evict(cache, weight, budget, sink, local)
        torch.cuda.synchronize()
        for b in range(B):
            newest = int(seen[b]) - 1
            for h in range(Hkv):
                u = rows[b][h]
                u.append((f64(kn[b, h]), f64(vn[b, h]), newest, 0.0))
                K, V, P, W = (np.array([t[i] for t in u]) for i in range(4))
                o, l, p = opaged.decode_unit(f64(q[b, h * G:(h + 1) * G]), K, V, P, newest, np.ones(len(u), dtype=bool),
                                             1 / math.sqrt(d), 15.0)
                # the bound of the module's head with |x| < 15: well below 1e-4 of sums of unit normals
                assert np.abs(f64(out[b, h * G:(h + 1) * G]) - o).max() < 1e-4
                assert np.abs(f64(lse[b, h * G:(h + 1) * G]) - l).max() < 1e-4
                W = W + p.sum(axis=0)
                if evict and len(u) > budget:
                    evictions += 1
                    src = opaged.evict_unit(W, P, newest, budget, sink, local)
                    K, V, P, W = K[src], V[src], P[src], W[src]
                rows[b][h] = [(K[i], V[i], int(P[i]), W[i]) for i in range(len(P))]
                n = int(lengths[b])
                assert n == len(P) and pos[b, h, :n].tolist() == P.tolist()
                assert np.abs(f64(weight[b, h, :n]) - W).max() < 1e-4 * (step + 2)
    assert evictions >= 8


def test_graphs_follow_lengths_and_do_not_share():
    """Two captured graphs, replayed in turn and at the same time, with lengths,
    tables and queries that change between replays."""
    dev = _dev()
    cs = [Case([3000, 700], cols=200, seed=50), Case([100, 2500], cols=200, seed=51)]
    runs = []
    for c in cs:
        cache = c.cache()
        new = torch.randn(c.B, c.Hkv, c.d, device=dev).to(BF)
        wo = torch.zeros_like(c.weight)
        out, lse = torch.empty(c.B, c.Hq, c.d, device=dev), torch.empty(c.B, c.Hq, device=dev)

        def step(c=c, cache=cache, new=new, wo=wo, out=out, lse=lse):
            sa.paged_append(cache, new, new)
            sa.paged_decode(c.q, cache, weight=c.weight, weight_out=wo, out=out, lse=lse)

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        runs.append((c, graph, step, wo, out, lse))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, lens in enumerate(([3000, 700], [1, 64], [3200, 0], [17, 2999])):
        for c, *_ in runs:
            c.lengths.copy_(torch.tensor(lens))
            c.q.copy_(torch.randn(c.q.shape, device=dev).to(BF))
            # slots never written hold NaN: fill them
            c.k.nan_to_num_(nan=0.25)
            c.v.nan_to_num_(nan=0.5)
        torch.cuda.synchronize()
        for (c, graph, *_), s in zip(runs, streams):
            with torch.cuda.stream(s):
                for _ in range(3):
                    graph.replay()
        torch.cuda.synchronize()
        for c, graph, step, wo, out, lse in runs:
            got = [t.clone() for t in (wo, out, lse)]
            step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, (wo, out, lse))), i
            _check_decode(c, out, lse)


def test_evict_captured():
    c = Case([500, 90], seed=52)
    cache = c.cache()
    out = sa.paged_evict(cache, c.weight, 64, 4, 8)
    torch.cuda.synchronize()
    c = Case([500, 90], seed=52)
    cache = c.cache()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sa.paged_evict(cache, c.weight, 64, 4, 8)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, got))


def test_streams_side_by_side():
    """One cache read on several streams at once: no shared scratch."""
    c = Case([6000, 800, 40], seed=53)
    cache = c.cache()
    want = sa.paged_decode(c.q, cache)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for _ in range(8):
        for s in streams:
            got.append(sa.paged_decode(c.q, cache, stream=s))
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


# ---- refusals ------------------------------------------------------------------

def test_python_refusals():
    dev = _dev()
    c = Case([40, 9], tracked=True, seed=60)
    cache = c.cache()
    long_k = c.k.clone().unsqueeze(0)
    for kw in (dict(pos=None), dict(seen=None), dict(table=c.table.long()), dict(lengths=c.lengths[:1]),
               dict(lengths=c.lengths.cpu()), dict(k=c.k.float()), dict(k=long_k), dict(v=c.v[:, :1]),
               dict(pos=c.pos[..., :-1]), dict(k=c.k.half(), v=c.v.half()),
               dict(k=c.k[..., ::2], v=c.v[..., ::2]), dict(k=c.k[:1].expand_as(c.k), v=c.v[:1].expand_as(c.v)),
               dict(k=c.k.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises((ValueError, TypeError)):
            c.cache(**kw)
    q = c.q
    for bad in (q.float(), q[:1], q[..., :64], q[:, :c.Hkv + 1], q.cpu(), q.transpose(0, 1).contiguous().transpose(0, 1)):
        with pytest.raises((ValueError, sa.SAError)):
            sa.paged_decode(bad, cache)
    w = torch.zeros(c.B, c.Hkv, c.cap, device=dev)
    for kw in (dict(weight=w), dict(weight_out=w[..., :-1]), dict(weight_out=w.double()), dict(slopes=w[0, 0, :3]),
               dict(out=w), dict(lse=w), dict(scale=-1.0), dict(softcap=-1.0), dict(sink=-1), dict(local=-1),
               dict(softcap=math.nan)):
        with pytest.raises((ValueError, sa.SAError)):
            sa.paged_decode(q, cache, **kw)
    new = torch.randn(2, c.Hkv, c.d, device=dev).to(BF)
    for a in ((new.float(), new.float()), (new, new[:1]), (new[:1], new[:1]), (new[..., :64], new[..., :64]),
              (new, new.transpose(0, 1).contiguous().transpose(0, 1)), (new.cpu(), new.cpu()),
              (new[:1].expand(2, -1, -1), new[:1].expand(2, -1, -1))):
        with pytest.raises((ValueError, sa.SAError)):
            sa.paged_append(cache, *a)
    with pytest.raises(ValueError):
        sa.paged_append(cache, new, new, start=torch.zeros(2, dtype=I32, device=dev))
    for a, kw in (((w, 0), {}), ((w, 8, 5, 4), {}), ((w[..., :-1], 8), {}), ((w, 8), dict(weight_out=w)),
                  ((w, 8), dict(pos_out=c.pos)), ((w, 8), dict(lengths_out=c.lengths))):
        with pytest.raises((ValueError, sa.SAError)):
            sa.paged_evict(cache, *a, **kw)
    d96 = torch.zeros(4, 2, 16, 96, dtype=BF, device=dev)
    with pytest.raises(sa.SAError):
        sa.paged_decode(torch.zeros(2, 2, 96, dtype=BF, device=dev),
                        sa.PagedCache(d96, d96.clone(), c.table[:, :2].contiguous(), c.lengths))


@pytest.mark.parametrize("lens", [[900, 40], [9000, 5000, 8000]])
def test_evict_threshold_among_zeros(lens):
    """The last one kept has the weight 0, with and without subnormals beside the zeros."""
    for tiny in (0.0, 1e-40, -1e-40):
        for budget in (lens[0] // 2, lens[0] - 3):
            c = Case(lens, Hkv=1, G=1, d=64, seed=36)
            c.weight = torch.where(c.weight < 0.8, torch.zeros_like(c.weight), c.weight)
            c.weight[..., 7::50] = tiny
            _evict(c, budget, 2, 5)


@pytest.mark.parametrize("lens,Hkv,dtype", [
    ([int(x) for x in np.random.default_rng(70).integers(2000, 4000, 40)], 8, BF),      # several units a CTA
    ([910001], 1, BF),                                                                  # one unit over all CTAs
    ([int(x) for x in np.random.default_rng(71).integers(0, 41, 1000)], 4, F32),        # many units of one tile
], ids=["several", "one", "short"])
def test_decode_much_work(lens, Hkv, dtype):
    c = Case(lens, Hkv=Hkv, G=2, d=64, dtype=dtype, cols=-(-max(lens) // 16), seed=72)
    out, lse = _decode(c, weights=len(lens) < 100)
    for _ in range(3):
        again = sa.paged_decode(c.q, c.cache())
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_a_cache_keeps_its_tensors():
    c = Case([20], seed=80)
    cache = c.cache()
    with pytest.raises(AttributeError):
        cache.lengths = c.lengths.clone()
    assert cache.lengths is c.lengths and cache.k is c.k


def test_threads_on_one_stream():
    """Calls of two threads on one stream share its scratch one after another."""
    import threading
    cs = [Case([3000, 40], seed=81), Case([3000, 40], seed=82)]
    want = []
    for c in cs:
        wo = torch.zeros_like(c.weight)
        want.append((*sa.paged_decode(c.q, c.cache(), weight=c.weight, weight_out=wo), wo))
    torch.cuda.synchronize()
    bad = []

    def work(c, w):
        for _ in range(40):
            wo = torch.zeros_like(c.weight)
            got = (*sa.paged_decode(c.q, c.cache(), weight=c.weight, weight_out=wo), wo)
            torch.cuda.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, w)):
                bad.append(c)

    threads = [threading.Thread(target=work, args=x) for x in zip(cs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("G", [1, 4, 7, 8, 12, 20])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
def test_decode_many_short_units(G, dtype, d):
    """More short units than there are SMs."""
    r = np.random.default_rng(90)
    c = Case([int(x) for x in r.integers(0, 260, 110)], Hkv=4, G=G, d=d, dtype=dtype, page=24, seed=90)
    _decode(c, weights=True, softcap=5.0)
    out, lse = _decode(c)
    again = sa.paged_decode(c.q, c.cache())
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("tracked", [False, True])
def test_decode_many_short_units_masked(tracked):
    r = np.random.default_rng(91)
    c = Case([int(x) for x in r.integers(0, 200, 200)], Hkv=2, G=4, d=128, tracked=tracked, seed=91)
    c.table[3, 0], c.table[5, 1] = -1, c.n_pages
    slopes = torch.exp2(-torch.arange(1, c.Hq + 1, device=_dev(), dtype=F32))
    _decode(c, weights=True, sink=5, local=40, slopes=slopes)


def test_decode_scratch_of_two_types():
    """Wide groups in bf16, then in fp32, on one stream: as many bytes of scratch
    and tickets, not as many heads in a record."""
    r = np.random.default_rng(100)
    cases = [Case([3000] * 16 + [1] * 576, Hkv=8, G=16, d=64, seed=101),          # long units: records of the first CTAs
             Case([int(x) for x in r.integers(1, 193, 592)], Hkv=8, G=16, dtype=F32, cols=12, seed=102)]
    for _ in range(2):
        for c in cases:
            out = torch.full((c.B, c.Hq, c.d), 7.0, device=_dev())
            lse = torch.full((c.B, c.Hq), 7.0, device=_dev())
            sa.paged_decode(c.q, c.cache(), out=out, lse=lse)
            torch.cuda.synchronize()
            _check_decode(c, out, lse)


def test_scratch_is_kept_by_stream_not_by_shape():
    """A table that grows and a batch that grows, with weights: what stays
    allocated is the scratch of the largest call, not of all."""
    dev = _dev()
    stream = torch.cuda.Stream()
    c = Case([40, 9, 300, 7, 64, 1, 200, 90], G=8, d=64, cols=64, seed=110)
    k, v = c.k, c.v

    def call(B, cols):
        table = torch.from_numpy(c.table_h[:B, :cols].copy()).to(dev)
        cache = sa.PagedCache(k, v, table, c.lengths[:B])
        wo = torch.zeros(cache.slots, device=dev)
        sa.paged_decode(c.q[:B], cache, weight_out=wo, stream=stream)
        sa.paged_evict(cache, wo, 16, 2, 2, stream=stream)
        torch.cuda.synchronize()

    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    call(8, 64)
    most = torch.cuda.memory_allocated() - before
    for B in range(1, 9):
        for cols in range(1, 65, 3):
            call(B, cols)
    assert torch.cuda.memory_allocated() - before <= most
    assert most < 2 ** 22


def test_outputs_beside_inputs():
    """Arrays that touch one another in one buffer, and fp32 queries that become
    the output; one element further in is refused."""
    dev = _dev()
    c = Case([300, 0, 17, 64], dtype=F32, tracked=True, seed=120)
    n = c.weight.numel()
    buf = torch.zeros(3 * n + 8, device=dev)
    w, wo = buf[:n].view(c.weight.shape), buf[n:2 * n].view(c.weight.shape)
    w.copy_(c.weight)
    cache = c.cache()
    out, lse = sa.paged_decode(c.q, cache, weight=w, weight_out=wo)
    _check_decode(c, out, lse, wo, c.weight, wo)
    with pytest.raises(sa.SAError):
        sa.paged_decode(c.q, cache, weight=w, weight_out=buf[n - 1:2 * n - 1].view(c.weight.shape))
    mine = c.q.clone()
    o, l = sa.paged_decode(mine, cache, out=mine)
    assert o is mine and torch.equal(o, out) and torch.equal(l, lse)
    fused = torch.randn(c.B, c.Hq + 2, c.d, device=dev)
    fused[:, :c.Hq] = c.q
    rows = fused.view(-1)[:c.B * c.Hq * c.d].view(c.B, c.Hq, c.d)
    with pytest.raises(sa.SAError):
        sa.paged_decode(fused[:, :c.Hq], cache, out=rows)
    # a sum row of every sequence between its queries and the next one's
    lse2 = fused.view(c.B, -1)[1, c.Hq * c.d:][:c.B * c.Hq].view(c.B, c.Hq)
    o, l = sa.paged_decode(fused[:, :c.Hq], cache, lse=lse2)
    assert torch.equal(o, out) and torch.equal(l, lse)
    with pytest.raises(sa.SAError):
        sa.paged_evict(cache, w, 32, 2, 2, weight_out=buf[1:n + 1].view(c.weight.shape))
    ints = torch.zeros(n + 4, dtype=I32, device=dev)
    with pytest.raises(sa.SAError):
        sa.paged_evict(cache, w, 32, 2, 2, pos_out=ints[:n].view(c.weight.shape), lengths_out=ints[n - 4:n])
    c.weight.copy_(w)
    kept, w2, p2 = sa.paged_evict(cache, w, 32, 2, 2, weight_out=buf[n:2 * n].view(c.weight.shape),
                                  pos_out=ints[:n].view(c.weight.shape), lengths_out=ints[n:])
    assert kept.tolist() == [min(x, 32) for x in c.lens]


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_caps_that_do_not_bind(dtype):
    """A cap at the largest that is taken is no cap.  Logits here stay below 8, off
    by 2^-150 of the cap (the quotient's subnormals: 5e-9) and 8 u of their own on
    either side; weights are off by twice that, and values lie below 6."""
    c = Case([700, 3], dtype=dtype, seed=130)
    out, lse = sa.paged_decode(c.q, c.cache())
    capped, l = sa.paged_decode(c.q, c.cache(), softcap=7.5e36)
    off = 2 * 8 * U * 8 + 2.0 ** -150 * 7.5e36
    assert (l - lse).abs().max() <= off + 4 * U * 16
    assert (out - capped).abs().max() <= 2 * off * 6 + 1e-6


@pytest.mark.parametrize("dtype,d,G", [(BF, 128, 4), (BF, 64, 8), (BF, 128, 12), (F32, 128, 4), (F32, 64, 8)])
@pytest.mark.parametrize("lens", [[200, 40], [9000, 30], [40] * 200], ids=["short", "long", "many"])
def test_decode_queries_that_are_not_numbers(lens, dtype, d, G):
    """A head's query with a NaN gives a row of NaN, and leaves the other heads as they are."""
    c = Case(lens, G=G, d=d, dtype=dtype, seed=150)
    base, lse0 = sa.paged_decode(c.q, c.cache())
    rows = [(0, 0), (0, G), (1, 2 * G - 1), (len(lens) - 1, 1)]
    want, wl = base.clone(), lse0.clone()
    for b, h in rows:
        c.q[b, h, 5] = float("nan")
        want[b, h], wl[b, h] = float("nan"), float("nan")
    wo = torch.zeros_like(c.weight)
    out, lse = sa.paged_decode(c.q, c.cache(), weight_out=wo)
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(torch.isnan(lse), torch.isnan(wl))
    # the other heads' maxima move at other steps: both runs are within the bound of
    # the module's head, for logits of sum |q k| / sqrt(d) < 16 and sums of p |v| < 4
    rel = 8 * U * (d / 16 + 5) * 16
    rel = 4 * rel + 2 * (24 * 1.25 * 2.0 ** -22 + (max(lens) / 8 + 64) * U)
    assert (out - want).nan_to_num(nan=0.0).abs().max() <= 2 * rel * 4
    assert (lse - wl).nan_to_num(nan=0.0).abs().max() <= 2 * rel
    live = torch.arange(c.cap, device=_dev()) < c.lengths[:, None]
    for b in range(c.B):
        for g in range(c.Hkv):
            bad = any(x == b and h // G == g for x, h in rows)
            assert torch.equal(torch.isnan(wo[b, g]), live[b] & bad)


@pytest.mark.parametrize("dtype,d,G", [(BF, 128, 4), (BF, 64, 8), (BF, 128, 12), (F32, 128, 4), (F32, 64, 8), (F32, 64, 12)])
@pytest.mark.parametrize("lens", [[200, 1, 64], [9000, 30], [40] * 200], ids=["short", "long", "many"])
def test_decode_values_that_are_not_finite(lens, dtype, d, G):
    """An infinity among the values of seen slots goes where the formula has it;
    opposite ones, NaN, and a weight of zero times an infinity give NaN; no other
    dim or unit changes.  Weights here are at least e^-40 of the largest."""
    c = Case(lens, G=G, d=d, dtype=dtype, seed=140)
    inf = float("inf")
    base, _ = sa.paged_decode(c.q, c.cache())
    want = base.clone()
    r = np.random.default_rng(141)

    def put(b, h, s, e, x, y, heads=slice(None)):
        pg, row, _ = opaged.slot_pages(c.table_h[b], c.lens[b], c.page, c.n_pages)
        c.v[int(pg[s]), h, int(row[s]), e] = x
        want[b, h * G:(h + 1) * G][heads, e] = y

    for b in range(0, len(lens), 1 if len(lens) < 10 else 17):
        at = r.integers(0, c.lens[b], 8)
        put(b, 0, at[0], 3, inf, inf)
        put(b, 0, at[1], 4, -inf, -inf)
        put(b, 1, at[2], d - 1, inf, inf)
        put(b, 1, c.lens[b] - 1, 0, -inf, -inf)
        put(b, 1, at[3], 9, float("nan"), float("nan"))
        if c.lens[b] > 1:
            put(b, 0, 0, 7, inf, inf)
            put(b, 0, c.lens[b] - 1, 7, -inf, float("nan"))
    out, lse = sa.paged_decode(c.q, c.cache())
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out.nan_to_num(nan=5.0, posinf=inf, neginf=-inf), want.nan_to_num(nan=5.0, posinf=inf, neginf=-inf))
    # the first head's logit of slot 2 is -inf: its weight is 0, and 0 times an infinity NaN
    if lens[0] > 2:
        c.q[0, 0], c.q[0, 1:G] = 0.0, 0.0
        c.q[0, 0, 0] = 1.0
        c.q[0, 1:G, 1] = 1.0
        pg, row, _ = opaged.slot_pages(c.table_h[0], c.lens[0], c.page, c.n_pages)
        c.k[int(pg[2]), 0, int(row[2])] = 1.0
        c.k[int(pg[2]), 0, int(row[2]), 0] = -3e38
        c.v[int(pg[2]), 0, int(row[2]), 11] = inf
        out, lse = sa.paged_decode(c.q, c.cache(), scale=1e4)
        assert torch.isnan(out[0, 0, 11]) and torch.isfinite(lse[0, :G]).all()
        # a query that is not a number keeps its whole row
        c.q[0, 0, 0] = float("nan")
        out, lse = sa.paged_decode(c.q, c.cache())
        assert torch.isnan(out[0, 0]).all() and not torch.isnan(out[0, 1, 0])


@pytest.mark.parametrize("B,tracked", [(16, False), (3, True)])
def test_evict_keys_of_long_slices(B, tracked):
    """Tables of 256K slots: the keys in the workspace, and in shared memory."""
    r = np.random.default_rng(160)
    lens = [int(x) for x in r.integers(100, 3000, B)]
    lens[0], lens[-1] = 262144, 90001
    c = Case(lens, Hkv=1, G=1, d=64, page=64, tracked=tracked, seed=161)
    c.weight = (c.weight * 2000).floor()                # ties
    _evict(c, 70000, 64, 128)
    c.lengths[0] = 200003
    _evict(c, 60001, 5, 2)


@pytest.mark.parametrize("page,cols", [(1, 301), (3, 101), (5, 67), (7, 43)])
@pytest.mark.parametrize("tracked", [False, True])
def test_odd_capacities(page, cols, tracked):
    """Rows of pos and of the weights that do not begin on 16 bytes."""
    c = Case([301, 1, 150, 0, 299], page=page, cols=cols, d=64, tracked=tracked, seed=170)
    slopes = torch.exp2(-torch.arange(1, c.Hq + 1, device=_dev(), dtype=F32))
    _decode(c, weights=True, softcap=9.0)
    _decode(c, weights=True, sink=3, local=50, slopes=slopes)
    for budget in (1, 50, 149, 298):
        c = Case([301, 1, 150, 0, 299], page=page, cols=cols, d=64, tracked=tracked, seed=171)
        _evict(c, budget, 1 if budget > 1 else 0, 0 if budget < 9 else 7)


@pytest.mark.parametrize("off", [1, 2, 3])
def test_arrays_that_begin_anywhere(off):
    """Weights, positions and lse on 4 bytes but not on 16."""
    dev = _dev()
    c = Case([320, 100, 3], tracked=True, cols=20, seed=172)
    n = c.weight.numel()

    def at(t, dtype=F32):
        x = torch.zeros(t.numel() + 8, dtype=dtype, device=dev)[off:off + t.numel()].view(t.shape)
        return x.copy_(t)

    c.weight, c.pos = at(c.weight), at(c.pos, I32)
    c.lengths, c.seen = at(c.lengths, I32), at(c.seen, I32)
    c.table = at(c.table, I32)
    assert c.weight.data_ptr() % 16 == 4 * off and n % 4 == 0
    before = torch.full(c.weight.shape, -3.0, device=dev)
    wo, lse = at(before), at(torch.zeros(c.B, c.Hq, device=dev))
    out, _ = sa.paged_decode(c.q, c.cache(), weight=c.weight, weight_out=wo, lse=lse, sink=2, local=200)
    _check_decode(c, out, lse, wo, c.weight, before, sink=2, local=200)
    _evict(c, 64, 4, 8)
    lo, w2, p2 = sa.paged_evict(c.cache(), c.weight, 64, 4, 8, weight_out=at(before), pos_out=at(c.pos, I32),
                                lengths_out=at(c.lengths, I32))
    # the rows have moved once already, the weights and positions are as they were: the same choice again
    again = sa.paged_evict(c.cache(), c.weight, 64, 4, 8)
    live = torch.arange(c.cap, device=dev) < lo[:, None, None]
    assert torch.equal(lo, again[0]) and torch.equal(torch.where(live, p2, 0), again[2])
    assert torch.equal(torch.where(live, w2, torch.zeros_like(w2)), again[1])


@pytest.mark.parametrize("ldw", [320, 321, 324, 333])
@pytest.mark.parametrize("tracked", [False, True])
def test_longer_rows_of_slots(ldw, tracked):
    """pos and the weights as parts of wider arrays (ldw), through the C calls; what
    lies past the capacity is left as it was."""
    import ctypes
    dev, lib = _dev(), sa._lib()
    c = Case([320, 0, 17, 319], cols=20, tracked=tracked, seed=173)
    wide = lambda t, fill, dtype: torch.full((c.B, c.Hkv, ldw), fill, dtype=dtype, device=dev).index_copy_(
        2, torch.arange(c.cap, device=dev), t)
    w, wo = wide(c.weight, -5.0, F32), torch.full((c.B, c.Hkv, ldw), -3.0, device=dev)
    pos = wide(c.pos, -8, I32) if tracked else None
    cache = c.cache()
    shape = sa.sa_paged_shape.from_buffer_copy(cache._for_heads(c.Hq))
    shape.ldw = ldw
    raw = sa.sa_paged_cache.from_buffer_copy(cache._c)
    raw.pos = None if pos is None else pos.data_ptr()
    sh, rc = ctypes.byref(shape), ctypes.byref(raw)
    stream = torch.cuda.current_stream().cuda_stream
    out, lse = torch.empty(c.B, c.Hq, c.d, device=dev), torch.empty(c.B, c.Hq, device=dev)
    n = lib.sa_paged_workspace_size(sh, sa.OP_PAGED_DECODE, 1)
    ws = torch.zeros(n, dtype=torch.uint8, device=dev)
    p = sa.sa_paged_params(0.0, 0.0, 3, 100, None, w.data_ptr(), wo.data_ptr(), 0)
    assert lib.sa_paged_decode(sh, rc, ctypes.byref(p), c.q.data_ptr(), out.data_ptr(), lse.data_ptr(), ws.data_ptr(), n,
                               stream) == sa.SA_OK
    torch.cuda.synchronize()
    before = torch.full((c.B, c.Hkv, c.cap), -3.0, device=dev)
    _check_decode(c, out, lse, wo[..., :c.cap], c.weight, before, sink=3, local=100)
    assert torch.all(wo[..., c.cap:] == -3.0) and torch.all(w[..., c.cap:] == -5.0)

    lo = torch.zeros(c.B, dtype=I32, device=dev)
    po = torch.full((c.B, c.Hkv, ldw), -9, dtype=I32, device=dev)
    wo.fill_(-3.0)
    n = lib.sa_paged_workspace_size(sh, sa.OP_PAGED_EVICT, 40)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    assert lib.sa_paged_evict(sh, rc, w.data_ptr(), 40, 2, 5, lo.data_ptr(), wo.data_ptr(), po.data_ptr(), ws.data_ptr(), n,
                              stream) == sa.SA_OK
    torch.cuda.synchronize()
    for b in range(c.B):
        for h in range(c.Hkv):
            L = c.lens[b]
            at = np.arange(L) if pos is None else pos[b, h, :L].cpu().numpy()
            newest = (L if c.seen is None else int(c.seen[b])) - 1
            src = opaged.evict_unit(f64(w[b, h, :L]), at, newest, 40, 2, 5)
            m = min(L, 40)
            assert int(lo[b]) == m and po[b, h, :m].tolist() == at[src].tolist()
            assert torch.equal(wo[b, h, :m], w[b, h, torch.from_numpy(src).to(dev)])
            assert torch.all(po[b, h, m:] == -9) and torch.all(wo[b, h, m:] == -3.0)
    new = torch.randn(c.B, c.Hkv, c.d, device=dev).to(BF)
    c.lengths.clamp_(min=1)
    w2 = w.clone()
    assert lib.sa_paged_append(sh, rc, new.data_ptr(), new.data_ptr(), 0, 0, None, c.B, w2.data_ptr(), stream) == sa.SA_OK
    torch.cuda.synchronize()
    last = torch.zeros_like(w, dtype=torch.bool)
    for b in range(c.B):
        last[b, :, int(c.lengths[b]) - 1] = True
    assert torch.equal(w2, torch.where(last, torch.zeros_like(w), w))


@pytest.mark.parametrize("n", [700, 9000])
def test_evict_more_protected_than_may_stay(n):
    """Every slot claims the newest position: the largest weights stay, with ties,
    with weights that are not numbers, and in place where none moves."""
    for weights in ("rand", "ties", "nan"):
        c = Case([n, 20, n // 2], Hkv=2, G=1, d=64, tracked=True, seed=174)
        c.pos.copy_((c.seen - 1)[:, None, None].expand_as(c.pos))
        if weights == "ties":
            c.weight = (c.weight * 3).floor()
        if weights == "nan":
            c.weight[..., ::3] = float("nan")
        for b in range(c.B):                            # a few are not protected, with the largest weights
            c.pos[b, :, 3:n:97] = 0
            c.weight[b, :, 3:n:97] = 100.0
        _evict(c, 64, 0, 8)


def test_scratch_grows_under_calls_in_flight():
    """Calls that need ever more scratch, enqueued behind one another with no wait,
    a captured one among them."""
    dev = _dev()
    cs = [Case([L, 37, L // 3], G=G, d=64, dtype=dt, seed=180 + i)
          for i, (L, G, dt) in enumerate([(40, 1, BF), (900, 4, F32), (2000, 12, BF), (5000, 20, F32), (9000, 4, BF)])]
    want = []
    for c in cs:
        wo = torch.zeros_like(c.weight)
        want.append((*sa.paged_decode(c.q, c.cache(), weight=c.weight, weight_out=wo), wo))
    stream = torch.cuda.Stream()
    caches, wos = [c.cache() for c in cs], [torch.zeros_like(c.weight) for c in cs]
    graph = torch.cuda.CUDAGraph()
    wg = torch.zeros_like(cs[2].weight)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        og, lg = sa.paged_decode(cs[2].q, caches[2], weight=cs[2].weight, weight_out=wg)
    torch.cuda.synchronize()
    sa._PAGED_WS.pop((dev.index, stream.cuda_stream), None)
    got = []
    with torch.cuda.stream(stream):
        for c, cache, wo in zip(cs, caches, wos):
            got.append((*sa.paged_decode(c.q, cache, weight=c.weight, weight_out=wo), wo))
            graph.replay()
            out, _, _ = sa.paged_evict(caches[0], cs[0].weight, 16, 1, 1)
        for c, cache, wo in zip(cs, caches, wos):
            sa.paged_decode(c.q, cache, weight=c.weight, weight_out=torch.zeros_like(wo))
    torch.cuda.synchronize()
    for a, b in zip(got[1:] + [(og, lg, wg)], want[1:] + [want[2]]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_threads_on_streams_of_their_own():
    import threading
    c = Case([4000, 77, 900], G=8, d=64, seed=190)
    cache = c.cache()
    want = sa.paged_decode(c.q, cache, softcap=20.0)
    torch.cuda.synchronize()
    bad = []

    def work():
        stream = torch.cuda.Stream()
        for _ in range(30):
            o, l = sa.paged_decode(c.q, cache, softcap=20.0, stream=stream)
            stream.synchronize()
            if not (torch.equal(o, want[0]) and torch.equal(l, want[1])):
                bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n_pages,Hkv,page", [(1, 1, 1), (1, 1, 48), (40, 1, 1), (1, 3, 48), (40, 3, 1), (3, 1, 16)])
def test_dims_of_one(n_pages, Hkv, page, dtype):
    """A pool's, a batch's and a call's dims of size one, whose strides mean nothing."""
    dev, d, G = _dev(), 64, 2
    n = min(n_pages, 40) * page
    st = [7 if n_pages == 1 else Hkv * page * d + 64, 3 if Hkv == 1 else page * d, 5 if page == 1 else d, 1]
    size = (n_pages, Hkv, page, d)
    store = [torch.full((2 ** 16 * 4,), float("nan"), dtype=dtype, device=dev) for _ in range(2)]
    k, v = (torch.as_strided(t, size, st) for t in store)
    table = torch.arange(n_pages, dtype=I32, device=dev).flip(0)[None].contiguous()
    lengths = torch.tensor([n], dtype=I32, device=dev)
    cache = sa.PagedCache(k, v, table, lengths)
    g = torch.Generator(device="cuda").manual_seed(200)
    kn, vn = (torch.randn(n, Hkv, d, generator=g, device=dev).to(dtype) for _ in range(2))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    sa.paged_append(cache, kn[:n - 1], vn[:n - 1], start=torch.tensor([1, n], dtype=I32, device=dev)) if n > 1 else None
    lengths.fill_(n - 1)
    torch.cuda.synchronize()
    # n - 1 tokens one place on: the first was skipped; write all in their places, the last one alone
    if n > 1:
        sa.paged_append(cache, kn[:n - 1], vn[:n - 1], start=torch.tensor([0, n - 1], dtype=I32, device=dev), stream=stream)
    stream.synchronize()
    lengths.fill_(n)
    torch.cuda.synchronize()
    last = [torch.as_strided(t[n - 1:].contiguous(), (1, Hkv, d), (9, 11 if Hkv == 1 else d, 1)) for t in (kn, vn)]
    sa.paged_append(cache, *last, stream=stream)
    stream.synchronize()
    q = torch.randn(1, Hkv * G, d, generator=g, device=dev).to(dtype)
    q1 = torch.as_strided(q, q.shape, (13, d, 1))
    out, lse = sa.paged_decode(q1, cache)
    for h in range(Hkv):
        ro, rl, _ = opaged.decode_unit(f64(q[0, h * G:(h + 1) * G]), f64(kn[:, h]), f64(vn[:, h]), np.arange(n), n - 1,
                                       np.ones(n, dtype=bool), d ** -0.5)
        # logits below 8 and values below 6, the bound of the module's head: well below 1e-4
        assert np.abs(f64(out[0, h * G:(h + 1) * G]) - ro).max() < 1e-4
        assert np.abs(f64(lse[0, h * G:(h + 1) * G]) - rl).max() < 1e-4
    w = torch.rand(cache.slots, generator=g, device=dev)
    budget = max(1, n // 3)
    torch.cuda.synchronize()
    kept, w2, p2 = sa.paged_evict(cache, w, budget, stream=stream)
    stream.synchronize()
    assert kept.tolist() == [budget]
    for h in range(Hkv):
        src = opaged.evict_unit(f64(w[0, h]), np.arange(n), n - 1, budget, 0, 0)
        assert p2[0, h, :budget].tolist() == src.tolist()
        pg, row, _ = opaged.slot_pages(table.cpu().numpy()[0], budget, page, n_pages)
        assert torch.equal(k[pg, h, row], kn[torch.from_numpy(src).to(dev), h])
        assert torch.equal(v[pg, h, row], vn[torch.from_numpy(src).to(dev), h])
