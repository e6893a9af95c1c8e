"""Paged latent cache, fp64 (test infrastructure only): append, attention of new
rows over the cache, and eviction by accumulated attention weight, user by user
and from the definitions.

The cache keeps the latent K = V rows c_t of the absorbed form of MLA (LLaTTE
notes, huaxiaozhuan.com, appendix A.3) between requests; the visibility rules
are the forward pass's (a history row at position p sees keys t <= p, a query
token sees every key), plus a window with leading events that stay visible.
"""
from __future__ import annotations

from typing import Optional

import numpy as np


def slots(table_row, length: int, page: int):
    """(page ids, rows in the page) of a user's events 0 .. length - 1."""
    t = np.arange(length)
    return np.asarray(table_row)[t // page], t % page


def append(pool, mass, x, offsets, table, lengths, gain=None, eps: float = 1e-6):
    """Writes the rows (normalised when gain is given) in place, masses to 0."""
    for u in range(len(lengths)):
        rows = np.asarray(x[offsets[u]:offsets[u + 1]], np.float64)
        if gain is not None:
            rows = rows / np.sqrt((rows ** 2).mean(-1, keepdims=True) + eps) * gain
        pg, rw = slots(table[u], lengths[u], pool.shape[1])
        m = len(rows)
        pool[pg[len(pg) - m:], rw[len(rw) - m:]] = rows
        if mass is not None:
            mass[pg[len(pg) - m:], rw[len(rw) - m:]] = 0.0


def visible(n_new: int, n_cand: int, length: int, window: int, n_sink: int) -> np.ndarray:
    """bool [n_new + n_cand, length]."""
    pos = np.concatenate([np.arange(length - n_new, length),
                          np.full(n_cand, length - 1)])[:, None]
    t = np.arange(length)[None]
    see = t <= pos
    if window > 0:
        see &= (t > pos - window) | (t < n_sink)
    return see


def attend(pool, mass, q, offsets, table, lengths, n_cand: int = 0, scale: float = 1.0,
           window: int = 0, n_sink: int = 0, spread: Optional[dict] = None):
    """(out [rows, h, r], lse [rows, h]); adds the weights to `mass` in place when
    it is given.  `spread` receives per-element quantities that error bounds are
    made of: `abs` = sum_t p_t |c_t|, `dot` = max_t scale sum |q| |c_t|, and per
    event `got` (the weight added) and `hits` (rows and heads that see it)."""
    rows, h, r = q.shape
    out, lse = np.zeros((rows, h, r)), np.full((rows, h), -np.inf)
    if spread is not None:
        spread["abs"], spread["dot"] = np.zeros((rows, h, r)), np.zeros((rows, h))
        spread["got"], spread["hits"] = np.zeros(pool.shape[:2]), np.zeros(pool.shape[:2])
        spread["maxdot"] = np.zeros(pool.shape[:2])
    for u in range(len(lengths)):
        a, b = offsets[u], offsets[u + 1]
        cand = min(n_cand, b - a)
        see = visible(b - a - cand, cand, lengths[u], window, n_sink)
        at = slots(table[u], lengths[u], pool.shape[1])
        c = pool[at].astype(np.float64)
        for i in range(a, b):
            k = np.flatnonzero(see[i - a])
            if len(k) == 0:
                continue
            ck = c[k]
            s = scale * (q[i].astype(np.float64) @ ck.T)              # [h, k]
            m = s.max(-1, keepdims=True)
            e = np.exp(s - m)
            l = e.sum(-1, keepdims=True)
            p = e / l
            out[i], lse[i] = p @ ck, (m + np.log(l))[:, 0]
            where = at[0][k], at[1][k]
            if mass is not None:
                mass[where] += p.sum(0)
            if spread is not None:
                spread["abs"][i] = p @ np.abs(ck)
                d = abs(scale) * (np.abs(q[i].astype(np.float64)) @ np.abs(ck).T)
                spread["dot"][i] = d.max(-1)
                spread["got"][where] += p.sum(0)
                spread["hits"][where] += h
                spread["maxdot"][where] = np.maximum(spread["maxdot"][where], d.max())
    return out, lse


def evict(pool, mass, table, lengths, budget: int, n_sink: int = 0, n_recent: int = 0,
          dst_table=None):
    """Packs the kept rows in place; returns (new lengths, list of kept slots)."""
    P = pool.shape[1]
    dst_table = table if dst_table is None else dst_table
    new, kept = [], []
    for u in range(len(lengths)):
        T = int(lengths[u])
        at = slots(table[u], T, P)
        w = np.where(np.isnan(mass[at]), -np.inf, mass[at])
        if T <= budget:
            keep = list(range(T))
        else:
            stay = set(range(n_sink)) | set(range(T - n_recent, T))
            rest = sorted((t for t in range(T) if t not in stay),
                          key=lambda t: (not np.isnan(mass[at][t]), w[t], -t), reverse=True)
            keep = sorted(stay | set(rest[:budget - n_sink - n_recent]))
        rows, ws = pool[at][keep].copy(), mass[at][keep].copy()
        to = slots(dst_table[u], len(keep), P)
        pool[to], mass[to] = rows, ws
        new.append(len(keep))
        kept.append(keep)
    return np.array(new, np.int32), kept
