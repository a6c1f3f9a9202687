"""fp64 restatement of the paged cache's operators (definitions of
sa_paged_append, sa_paged_decode and sa_paged_evict in sa_decode.h), unit by
unit over dense rows: which slots a query sees, its attention, and the slots
that stay when a cache is thinned out."""
import numpy as np


def slot_pages(table_row, n, page, n_pages):
    """(page [n], row [n], valid [n]) of slots [0, n) of a sequence."""
    s = np.arange(n)
    pg = np.asarray(table_row)[s // page]
    return pg, s % page, (pg >= 0) & (pg < n_pages)


def visible(pos, newest, sink, local):
    """Slots whose position a query at `newest` sees."""
    pos = np.asarray(pos, dtype=np.int64)
    if local <= 0:
        return np.ones(len(pos), dtype=bool)
    return (pos < sink) | (pos > newest - local)


def decode_unit(q, K, V, pos, newest, sees, scale, softcap=0.0, slopes=None):
    """Attention of queries q [G, d] over rows K, V [n, d] where sees [n]:
    (out [G, d], lse [G], p [G, n]); nothing seen: 0, -inf, 0."""
    q, K, V = (np.asarray(x, dtype=np.float64) for x in (q, K, V))
    G, n = q.shape[0], K.shape[0]
    out, lse, p = np.zeros((G, V.shape[1])), np.full(G, -np.inf), np.zeros((G, n))
    at = np.nonzero(sees)[0]
    if len(at) == 0:
        return out, lse, p
    x = scale * (q @ K[at].T)
    if softcap > 0:
        x = softcap * np.tanh(x / softcap)
    if slopes is not None:
        x = x - np.asarray(slopes, dtype=np.float64)[:, None] * (newest - np.asarray(pos, dtype=np.int64)[at])
    m = x.max(axis=1)
    e = np.exp(x - m[:, None])
    z = e.sum(axis=1)
    p[:, at] = e / z[:, None]
    out = p[:, at] @ V[at]
    lse = m + np.log(z)
    return out, lse, p


def evict_unit(weight, pos, newest, budget, sink, local):
    """Sources of the slots that are left: src[s] is the slot whose token is in
    slot s afterwards (weight, pos [n])."""
    w = np.asarray(weight, dtype=np.float64)
    n = len(w)
    if n <= budget:
        return np.arange(n)
    pos = np.asarray(pos, dtype=np.int64)
    w = np.where(np.isnan(w), -np.inf, w)
    always = (pos < sink) | (pos > newest - local)
    order = sorted(range(n), key=lambda s: (not always[s], -w[s], s))
    stays = np.zeros(n, dtype=bool)
    stays[order[:budget]] = True
    src = np.arange(budget)
    src[~stays[:budget]] = np.nonzero(stays[budget:])[0] + budget
    return src
