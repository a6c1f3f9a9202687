"""The paged cache's fp64 definitions against brute force, and the refusals of
its entry points (no GPU: every call fails its checks, nothing is enqueued)."""
import ctypes
import math

import numpy as np
import pytest

import kv_cache_residual_b200 as sa
from oracle import paged

GOOD, ODD = 0x10000, 0x10004


@pytest.mark.parametrize("softcap", [0.0, 5.0])
@pytest.mark.parametrize("sink,local", [(0, 0), (3, 4), (0, 1), (2, 100)])
def test_decode_unit_is_the_formula(softcap, sink, local):
    r = np.random.default_rng(3)
    n, d = 23, 8
    q, K, V = r.normal(size=(2, d)), r.normal(size=(n, d)), r.normal(size=(n, d))
    pos, newest, slopes = np.sort(r.permutation(40)[:n]), 39, np.array([0.1, 0.0])
    out, lse, p = paged.decode_unit(q, K, V, pos, newest, paged.visible(pos, newest, sink, local), 0.3, softcap, slopes)
    for h in range(2):
        z, num, total = 0.0, np.zeros(d), 0.0
        for s in range(n):
            if local > 0 and not (pos[s] < sink or newest - pos[s] < local):
                assert p[h, s] == 0.0
                continue
            x = 0.3 * sum(q[h, e] * K[s, e] for e in range(d))
            x = softcap * math.tanh(x / softcap) if softcap > 0 else x
            w = math.exp(x - slopes[h] * (newest - pos[s]))
            z, num, total = z + w, num + w * V[s], total + p[h, s]
        if z == 0.0:
            assert lse[h] == -np.inf and not out[h].any()
            continue
        np.testing.assert_allclose(out[h], num / z, rtol=1e-12)
        assert lse[h] == pytest.approx(math.log(z), rel=1e-12) and total == pytest.approx(1.0)


def test_nothing_seen_gives_zero():
    out, lse, p = paged.decode_unit(np.ones((2, 4)), np.ones((3, 4)), np.full((3, 4), np.nan), [0, 1, 2], 2,
                                    np.zeros(3, dtype=bool), 1.0)
    assert not out.any() and (lse == -np.inf).all() and not p.any()


def test_evict_unit_keeps_the_best_and_moves_the_late():
    inf, nan = np.inf, np.nan
    #          0    1    2    3    4    5    6    7
    w = [0.5, 0.1, 0.3, nan, 0.3, inf, 0.3, 0.0]
    pos = np.arange(8)
    # newest position 7 always stays; then inf (5), 0.5 (0), and of the three 0.3 the lowest slots
    assert paged.evict_unit(w, pos, 7, 4, 0, 1).tolist() == [0, 5, 2, 7]
    assert paged.evict_unit(w, pos, 7, 8, 0, 1).tolist() == list(range(8))
    assert paged.evict_unit(w, pos, 7, 7, 0, 1).tolist() == [0, 1, 2, 7, 4, 5, 6]
    # positions, not slots, are protected
    assert paged.evict_unit(w, pos[::-1].copy(), 7, 2, 1, 1).tolist() == [0, 7]
    assert paged.evict_unit([], [], -1, 3, 0, 0).tolist() == []


def _shape(**kw):
    base = dict(B=2, Hq=8, Hkv=2, d=128, dtype=sa.SA_BF16, n_pages=40, page=16, max_pages=20, ldw=0, page_stride=0,
                head_stride=0, row_stride=0)
    base.update(kw)
    return sa.sa_paged_shape(*[base[n] for n, _ in sa.sa_paged_shape._fields_])


def _cache(**kw):
    base = dict(k=GOOD, v=GOOD, table=GOOD, lengths=GOOD, pos=None, seen=None)
    base.update(kw)
    return sa.sa_paged_cache(*[base[n] for n, _ in sa.sa_paged_cache._fields_])


def _params(**kw):
    base = dict(scale=0.0, softcap=0.0, sink=0, local=0, slopes=None, weight=None, weight_out=None, q_stride=0)
    base.update(kw)
    return sa.sa_paged_params(*[base[n] for n, _ in sa.sa_paged_params._fields_])


def _append(shape=None, cache=None, k=GOOD, v=GOOD, ts=0, hs=0, start=None, n=2, weight=None):
    return sa._lib().sa_paged_append(ctypes.byref(shape or _shape()), ctypes.byref(cache or _cache()), k, v, ts, hs,
                                     start, n, weight, None)


def _decode(shape=None, cache=None, params=None, q=GOOD, out=GOOD, lse=GOOD, ws=GOOD, n=1 << 40):
    return sa._lib().sa_paged_decode(ctypes.byref(shape or _shape()), ctypes.byref(cache or _cache()),
                                     ctypes.byref(params or _params()), q, out, lse, ws, n, None)


def _evict(shape=None, cache=None, weight=GOOD, budget=64, sink=4, local=8, lengths_out=0x20000, weight_out=0x20000,
           pos_out=0x20000, ws=GOOD, n=1 << 40):
    return sa._lib().sa_paged_evict(ctypes.byref(shape or _shape()), ctypes.byref(cache or _cache()), weight, budget,
                                    sink, local, lengths_out, weight_out, pos_out, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), sa.SA_ERR_INVALID_ARG),
    (dict(Hq=0), sa.SA_ERR_INVALID_ARG),
    (dict(Hkv=0), sa.SA_ERR_INVALID_ARG),
    (dict(Hq=9), sa.SA_ERR_INVALID_ARG),
    (dict(d=96), sa.SA_ERR_UNSUPPORTED),
    (dict(dtype=2), sa.SA_ERR_INVALID_ARG),
    (dict(page=0), sa.SA_ERR_INVALID_ARG),
    (dict(n_pages=0), sa.SA_ERR_INVALID_ARG),
    (dict(max_pages=0), sa.SA_ERR_INVALID_ARG),
    (dict(ldw=319), sa.SA_ERR_INVALID_ARG),                       # shorter than the capacity of 320
    (dict(page=1 << 20, max_pages=1 << 11), sa.SA_ERR_UNSUPPORTED),
    (dict(B=8192, Hq=64, Hkv=8), sa.SA_ERR_UNSUPPORTED),
    (dict(page_stride=4096, head_stride=2048, row_stride=0), sa.SA_ERR_INVALID_ARG),
    (dict(page_stride=4096, head_stride=-2048, row_stride=128), sa.SA_ERR_INVALID_ARG),
    (dict(page_stride=4096, head_stride=2048, row_stride=132), sa.SA_ERR_INVALID_ARG),   # not 16 bytes
])
def test_bad_shapes_are_refused_by_all(kw, status):
    sh = _shape(**kw)
    assert _append(shape=sh, n=max(sh.B, 0)) == status
    assert _decode(shape=sh) == status
    assert _evict(shape=sh) == status
    assert sa._lib().sa_paged_workspace_size(ctypes.byref(sh), sa.OP_PAGED_DECODE, 0) == 0


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=ODD), dict(table=None), dict(lengths=0x10002), dict(pos=GOOD),
                                dict(seen=GOOD), dict(pos=0x10001, seen=GOOD)])
def test_bad_caches_are_refused_by_all(kw):
    c = _cache(**kw)
    assert _append(cache=c) == _decode(cache=c) == _evict(cache=c) == sa.SA_ERR_INVALID_ARG


def test_append_refusals():
    bad = sa.SA_ERR_INVALID_ARG
    assert _append(n=3) == bad                                   # one token each, and B = 2
    assert _append(n=-1, start=GOOD) == bad
    assert _append(k=None) == _append(v=ODD) == _append(weight=0x10002) == _append(start=0x10001, n=5) == bad
    assert _append(ts=1024, hs=0) == _append(ts=1020, hs=128) == _append(ts=-1024, hs=128) == bad
    assert _append(n=(1 << 31) - 1, start=GOOD) == sa.SA_ERR_UNSUPPORTED
    assert _append(n=0, start=GOOD, k=None, v=None) == sa.SA_OK   # nothing to do


def test_decode_refusals():
    bad, inf, nan = sa.SA_ERR_INVALID_ARG, float("inf"), float("nan")
    assert _decode(q=None) == _decode(q=ODD) == _decode(out=None) == _decode(lse=0x10002) == bad
    for kw in (dict(scale=-1.0), dict(scale=nan), dict(scale=inf), dict(softcap=-2.0), dict(softcap=nan), dict(softcap=inf),
               dict(sink=-1), dict(local=-1), dict(slopes=0x10001), dict(weight=GOOD), dict(weight_out=0x10001),
               dict(weight=0x10001, weight_out=GOOD), dict(q_stride=-1024), dict(q_stride=1028)):
        assert _decode(params=_params(**kw)) == bad, kw
    need = sa._lib().sa_paged_workspace_size(ctypes.byref(_shape()), sa.OP_PAGED_DECODE, 0)
    more = sa._lib().sa_paged_workspace_size(ctypes.byref(_shape()), sa.OP_PAGED_DECODE, 1)
    assert 0 < need < more
    assert _decode(ws=None) == _decode(n=need - 1) == _decode(ws=ODD) == sa.SA_ERR_WORKSPACE
    assert _decode(params=_params(weight_out=GOOD), n=need) == sa.SA_ERR_WORKSPACE


def test_evict_refusals():
    bad = sa.SA_ERR_INVALID_ARG
    assert _evict(weight=None) == _evict(budget=0) == _evict(sink=-1) == _evict(local=-1) == bad
    assert _evict(budget=11, sink=4, local=8) == bad             # more protected than may stay
    assert _evict(lengths_out=None) == _evict(weight_out=None) == _evict(pos_out=None) == bad
    # outputs are other arrays than the inputs
    assert _evict(lengths_out=GOOD) == _evict(weight_out=GOOD) == bad
    assert _evict(cache=_cache(pos=0x20000, seen=GOOD)) == bad
    need = sa._lib().sa_paged_workspace_size(ctypes.byref(_shape()), sa.OP_PAGED_EVICT, 64)
    assert need > 0 and _evict(ws=None) == _evict(n=need - 1) == sa.SA_ERR_WORKSPACE
    assert sa._lib().sa_paged_workspace_size(ctypes.byref(_shape()), sa.OP_PAGED_EVICT, 0) == 0
    assert sa._lib().sa_paged_workspace_size(ctypes.byref(_shape()), 99, 1) == 0


def test_python_refuses_host_tensors():
    import torch
    k = torch.zeros(4, 2, 16, 64)
    with pytest.raises(ValueError):
        sa.PagedCache(k, k.clone(), torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_factors_that_overflow_are_refused():
    bad = sa.SA_ERR_INVALID_ARG
    for kw in (dict(scale=3.3e38), dict(softcap=1e-45), dict(softcap=3.3e38), dict(scale=1e30, softcap=1e-20)):
        assert _decode(params=_params(**kw)) == bad, kw


def test_evict_refuses_to_write_over_seen():
    assert _evict(cache=_cache(pos=0x30000, seen=0x20000)) == sa.SA_ERR_INVALID_ARG


@pytest.mark.parametrize("G", [1, 8, 9, 10, 16, 17, 32])
@pytest.mark.parametrize("dtype,d", [(sa.SA_BF16, 64), (sa.SA_BF16, 128), (sa.SA_F32, 64), (sa.SA_F32, 128)])
def test_decode_scratch_has_the_tickets_before_the_records(G, dtype, d):
    """The tickets of every type take the bytes the header names, so that two
    shapes with as many of them have no record where the other has a ticket."""
    for B in (1, 148, 592):
        sh = _shape(B=B, Hq=8 * G, Hkv=8, d=d, dtype=dtype)
        hu = 16 if dtype == sa.SA_BF16 and G > 8 else 8                # heads of a record
        units = B * 8 * -(-G // hu)
        records = 4 * 2 * min(148, units * 5) * hu * (2 + d)           # 320 slots are 5 tiles
        tickets = 4 * B * 8 * -(-G // 8)
        n = sa._lib().sa_paged_workspace_size(ctypes.byref(sh), sa.OP_PAGED_DECODE, 0)
        assert n == -(-tickets // 256) * 256 + -(-records // 256) * 256


def test_scratch_of_a_stream_is_its_largest_calls(monkeypatch):
    """Calls of many sizes on one stream keep one buffer, with zeros before the
    place where every call writes."""
    import torch
    monkeypatch.setattr(sa, "_PAGED_WS", {})
    r = np.random.default_rng(5)
    cpu, most = torch.device("cpu"), [0, 0]
    for _ in range(200):
        tickets, rest = 256 * int(r.integers(0, 40)), 256 * int(r.integers(1, 4000))
        most = [max(most[0], tickets), max(most[1], rest)]
        at = sa._stream_scratch(cpu, 7, tickets, rest)
        assert sa._stream_scratch(cpu, 7, tickets, rest) == at          # kept
        assert list(sa._PAGED_WS) == [(None, 7)]
        t = sa._PAGED_WS[(None, 7)][0]
        assert t.numel() == sum(most)
        first = at - t.data_ptr()
        assert first >= 0 and not t[first:first + tickets].any() and first + tickets + rest <= t.numel()
        t[first + tickets:first + tickets + rest] = 1                   # as a call leaves it
    other = sa._stream_scratch(cpu, 8, 0, 256)
    assert len(sa._PAGED_WS) == 2 and other == sa._PAGED_WS[(None, 8)][0].data_ptr()


FAR = [0x1000000 * i for i in range(1, 12)]           # addresses apart from one another


def test_outputs_that_overlap_are_refused():
    """The shape's per-slot arrays take 5120 bytes, out 8192, lse 64, queries 4096."""
    bad = sa.SA_ERR_INVALID_ARG
    k, v, table, lengths, pos, seen, a, b, c, d, ws = FAR
    cache = _cache(k=k, v=v, table=table, lengths=lengths, pos=pos, seen=seen)
    for kw in (dict(weight_out=a + 5116), dict(weight_out=a - 5116), dict(pos_out=a + 4), dict(pos_out=pos + 5116),
               dict(weight_out=pos - 5116), dict(lengths_out=a + 5116), dict(lengths_out=lengths + 4),
               dict(lengths_out=seen - 4), dict(lengths_out=table + 156), dict(weight_out=table - 4000),
               dict(pos_out=b + 64), dict(lengths_out=b + 5116), dict(lengths_out=c), dict(ws=a + 4096), dict(ws=b - 16)):
        args = dict(weight=a, weight_out=b, pos_out=c, lengths_out=d, ws=ws)
        args.update(kw)
        assert _evict(cache=cache, **args) == bad, kw
    for kw in (dict(weight_out=a + 5116), dict(weight_out=a + 4), dict(weight_out=pos + 16), dict(weight_out=b + 8188),
               dict(weight_out=b - 5116), dict(weight_out=c + 60), dict(weight_out=lengths - 5116), dict(slopes=b + 4),
               dict(weight_out=d + 4092), dict(slopes=c + 60)):
        args = dict(weight=a, weight_out=FAR[10] + 0x1000000)
        args.update(kw)
        assert _decode(cache=cache, params=_params(**args), q=d, out=b, lse=c, ws=ws) == bad, kw
    for kw in (dict(out=d), dict(out=d + 4080), dict(lse=d + 4092), dict(lse=b + 8188), dict(ws=b + 16), dict(ws=d + 16),
               dict(out=table - 16), dict(lse=lengths), dict(lse=seen + 4)):
        args = dict(q=d, out=b, lse=c, ws=ws)
        args.update(kw)
        assert _decode(cache=cache, **args) == bad, kw
    # fp32 queries in the place of the output, but not its rows
    f32 = _shape(dtype=sa.SA_F32)
    assert _decode(shape=f32, cache=cache, q=b + 16, out=b, lse=c, ws=ws) == bad
    assert _decode(shape=f32, cache=cache, q=b, out=b, lse=c, ws=ws, params=_params(q_stride=2048)) == bad
    for kw in (dict(weight=pos + 4), dict(weight=table), dict(weight=lengths - 4), dict(weight=seen - 5116),
               dict(weight=a, start=a + 5116, n=5)):
        assert _append(cache=cache, **kw) == bad, kw
    assert _append(cache=cache, start=pos + 8, n=5) == bad


def test_factors_that_underflow_are_refused():
    """scale / softcap below the least normal number has too few bits to multiply by."""
    bad = sa.SA_ERR_INVALID_ARG
    k, v, table, lengths, pos, seen, a, b, c, d, ws = FAR
    cache = _cache(k=k, v=v, table=table, lengths=lengths)
    for kw in (dict(softcap=1e37), dict(scale=1e-6, softcap=1e38), dict(scale=1e-20, softcap=1e20)):
        assert _decode(cache=cache, params=_params(**kw), q=a, out=b, lse=c, ws=ws) == bad, kw


@pytest.mark.parametrize("B,pages,keys", [(4, 4096, True), (2, 4096, True), (1, 4096, False), (4, 2048, False),
                                          (32, 512, False), (16, 1024, True), (1, 8192, True)])
def test_evict_clusters_are_resident(B, pages, keys):
    """Clusters are as large as fit at once with two CTAs on an SM: slices with
    more keys than half an SM's memory have them in the workspace, but where
    there are few CTAs or one a unit.  Pages of 64, eight KV heads."""
    sh = _shape(B=B, Hq=8, Hkv=8, page=64, max_pages=pages, n_pages=B * pages)
    cap, budget = 64 * pages, 1000
    n = sa._lib().sa_paged_workspace_size(ctypes.byref(sh), sa.OP_PAGED_EVICT, budget)
    lists = 4 * 2 * 8 * B * min(budget, cap - budget)
    least = -(-4 * 8 * B // 256) * 256 + -(-lists // 256) * 256
    assert n == least + (4 * 8 * B * cap if keys else 0)
