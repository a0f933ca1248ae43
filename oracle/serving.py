"""Float64 definitions of the serving operators around the paged decode, in numpy.

TEST INFRASTRUCTURE ONLY, as the rest of this package: nothing here is shared
with the CUDA path.  Written per sequence and over explicit token sets, straight
from the formulas of include/paged_attn.h:

* ``attend``        -- decode and multi-token attention with capped scores, a
                       distance bias, a window, a prefix and documents;
* ``attend_shared`` -- decode of groups that share a prefix;
* ``assign``        -- block tables, offsets and slots from request lengths.

The attention functions return a ``Result``: the output and, per element, a
bound on how far a computation may be off it that rounds the weights to
``eps_p`` and the output to bf16 and keeps everything else in float32.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

BF16_STEP = 2.0 ** -8   # half a step, relative
F16_STEP = 2.0 ** -11


def bf16_to_f64(t) -> np.ndarray:
    """A bf16 tensor's values."""
    return t.detach().cpu().float().numpy().astype(np.float64)


@dataclass
class Result:
    out: np.ndarray   # [rows, H_q, D]
    tol: np.ndarray   # [rows, H_q, D]


def rows_of(cache, table, n):
    """Rows [n, H_kv, D] of the first n tokens of one sequence; cache [NB, H_kv, BS, D]."""
    BS = cache.shape[2]
    pages = cache[np.asarray(table[:-(-n // BS)], dtype=np.int64)] if n else cache[:0]
    return pages.transpose(0, 2, 1, 3).reshape(-1, cache.shape[1], cache.shape[3])[:n]


def _sequence(q, K, V, pos, seen, scale, softcap, slopes, eps_p, f16):
    """One sequence: q [r, H_q, D], K, V [n, H_kv, D], pos [r], seen [r, n]."""
    r, H, D = q.shape
    G = H // K.shape[1]
    out, tol = np.zeros((r, H, D)), np.zeros((r, H, D))
    some = seen.any(axis=0)  # rows nobody sees may hold anything: they take no part
    K, V, seen, t = K[some], V[some], seen[:, some], np.nonzero(some)[0]
    dist = np.abs(pos[:, None] - t[None, :])
    for h in range(H):
        k, v = K[:, h // G], V[:, h // G]
        with np.errstate(invalid="ignore"):
            x = (q[:, h] @ k.T) * scale
            reach = (np.abs(q[:, h]) @ np.abs(k).T) * abs(scale)
        if softcap > 0:
            x = softcap * np.tanh(x / softcap)
        bias = np.zeros_like(x) if slopes is None else slopes[h] * dist
        for i in range(r):
            m = seen[i]
            if not m.any():
                continue
            xi = x[i, m] - bias[i, m]
            w = np.exp(xi - xi.max())
            l = w.sum()
            out[i, h] = (w @ v[m]) / l
            mean_abs = (w @ np.abs(v[m])) / l
            # float32 dot products of D terms, the cap's and the bias's rounding
            err = D * 2.0 ** -24 * reach[i, m].max() + 4e-6 * np.abs(x[i, m]).max() + \
                2.0 ** -22 * np.abs(bias[i, m]).max()
            tol[i, h] = mean_abs * (2 * eps_p + 2 * err) + BF16_STEP * np.abs(out[i, h]) + 1e-30
            if f16:  # weights below f16's normal range: half its smallest step each
                tol[i, h] += m.sum() * 448 * 2.0 ** -25 / l
    return out, tol


def visible(pos, n, causal, window, prefix, doc_start):
    """[rows, n]: what each query position sees."""
    t = np.arange(n)[None, :]
    lo = np.zeros(len(pos), dtype=np.int64)
    if window:
        lo = np.maximum(lo, pos - window + 1)
    if doc_start is not None:
        lo = np.maximum(lo, np.clip(doc_start, 0, n))
    seen = t >= lo[:, None]
    if causal:
        seen = seen & (t <= pos[:, None])
    return seen | (t < min(max(prefix, 0), n))


def attend(q, k, v, qo, bt, lens, scale, causal=True, softcap=0.0, slopes=None, window=0,
           prefix_lens=None, doc_starts=None, eps_p=BF16_STEP, f16=False) -> Result:
    """Rows qo[s] .. qo[s+1] - 1 of q [rows, H_q, D] are the last tokens of sequence s
    (qo None: one row each); k, v [NB, H_kv, BS, D] float64; arrays as paged_attn.h."""
    if qo is None:
        qo = np.arange(len(lens) + 1)
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    cap = bt.shape[1] * k.shape[2]
    for s, n in enumerate(np.clip(np.asarray(lens, dtype=np.int64), 0, cap)):
        a, b = int(qo[s]), int(qo[s + 1])
        if a == b:
            continue
        pos = n - (b - a) + np.arange(b - a)
        seen = visible(pos, n, causal, window, 0 if prefix_lens is None else int(prefix_lens[s]),
                       None if doc_starts is None else np.asarray(doc_starts[a:b], dtype=np.int64))
        out[a:b], tol[a:b] = _sequence(q[a:b], rows_of(k, bt[s], int(n)), rows_of(v, bt[s], int(n)),
                                       pos, seen, scale, softcap, slopes, eps_p, f16)
    return Result(out, tol)


def attend_shared(q, k, v, group_indptr, prefix_tables, prefix_lens, bt, lens, scale, softcap=0.0,
                  slopes=None) -> Result:
    """Sequence s of group g sees the group's prefix, then its own lens[s] tokens."""
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for g in range(len(prefix_lens)):
        P = int(np.clip(prefix_lens[g], 0, prefix_tables.shape[1] * k.shape[2]))
        for s in range(int(group_indptr[g]), int(group_indptr[g + 1])):
            n = int(np.clip(lens[s], 0, bt.shape[1] * k.shape[2]))
            K = np.concatenate([rows_of(k, prefix_tables[g], P), rows_of(k, bt[s], n)])
            V = np.concatenate([rows_of(v, prefix_tables[g], P), rows_of(v, bt[s], n)])
            pos = np.array([P + n - 1])
            out[s:s + 1], tol[s:s + 1] = _sequence(q[s:s + 1], K, V, pos,
                                                   np.ones((1, P + n), dtype=bool), scale, softcap,
                                                   slopes, BF16_STEP, False)
    return Result(out, tol)


def assign(lens, new, table, free, free_count, BS, max_new):
    """(lens_out, qo_indptr, slot_map, free_count_out, refused, table) as paged_kv_assign."""
    table = np.array(table)
    n, maxb = table.shape
    count = min(max(int(free_count), 0), len(free))
    qo, lens_out = np.zeros(n + 1, dtype=np.int64), np.array(lens, dtype=np.int64)
    slots = np.full(max_new, -1, dtype=np.int64)
    asked = taken = refused = row = 0
    for s in range(n):
        L, m = int(lens[s]), int(new[s])
        rows = max(m, 0)
        fits = L >= 0 and m >= 0 and L + m <= maxb * BS
        need = -(-(L + m) // BS) - -(-L // BS) if fits else 0
        ok = fits and (need == 0 or asked + need <= count) and row + rows <= max_new
        if ok:
            for i in range(need):
                table[s, -(-L // BS) + i] = free[count - 1 - (asked + i)]
            for i in range(m):
                t = L + i
                slots[row + i] = int(table[s, t // BS]) * BS + t % BS
            lens_out[s] = L + m
            taken += need
        else:
            refused += 1
        asked += need
        row += rows
        qo[s + 1] = row
    return lens_out, np.minimum(qo, 2 ** 31 - 1), slots, count - taken, refused, table
