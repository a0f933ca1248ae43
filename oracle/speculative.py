"""Float64 definitions of the operators of speculative and parallel decoding, in numpy.

TEST INFRASTRUCTURE ONLY, as the rest of this package: nothing here is shared with the
CUDA path.  Written per sequence and per entry, straight from the formulas of
include/paged_attn.h:

* ``attend_tree`` -- attention of drafted trees;
* ``turn``        -- norm and rotation of heads, with a bound on float32's error;
* ``compact``, ``fork``, ``release`` -- the rows and pages of a cache.
"""
from __future__ import annotations

from collections import Counter

import numpy as np

from oracle.serving import BF16_STEP, Result, _sequence, rows_of

F32_STEP = 2.0 ** -24
E4M3_STEP = 2.0 ** -4


def mask_bits(words, q_len):
    """[rows, words] int32 -> bool [rows, q_len]: the drafted tokens that each row sees."""
    w = np.asarray(words).astype(np.int64) & 0xffffffff
    out = np.zeros((w.shape[0], q_len), dtype=bool)
    for j in range(min(q_len, 32 * w.shape[1])):
        out[:, j] = w[:, j // 32] >> (j % 32) & 1
    return out


def mask_words(bits, words):
    """bool [rows, n] -> int32 [rows, words]."""
    out = np.zeros((bits.shape[0], words), dtype=np.uint32)
    for j in range(min(bits.shape[1], 32 * words)):
        out[:, j // 32] |= bits[:, j].astype(np.uint32) << np.uint32(j % 32)
    return out.view(np.int32)


def attend_tree(q, k, v, qo, words, bt, lens, scale, softcap=0.0, slopes=None, window=0,
                prefix_lens=None, eps_p=BF16_STEP) -> Result:
    """Rows qo[s] .. qo[s+1] - 1 of q [rows, H_q, D] are the drafted tokens of sequence s, its
    last ones; k, v [NB, H_kv, BS, D] float64."""
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    cap = bt.shape[1] * k.shape[2]
    for s, n in enumerate(np.clip(np.asarray(lens, dtype=np.int64), 0, cap)):
        a, b = int(qo[s]), int(qo[s + 1])
        if a == b:
            continue
        n, m = int(n), b - a
        ctx = n - m
        bits = mask_bits(words[a:b], m)
        for j in range(m):  # a drafted token before the sequence's first is none
            if ctx + j < 0:
                bits[:, j] = False
        pos = ctx + bits.sum(1) - 1
        seen = np.zeros((m, n), dtype=bool)
        at = np.arange(n)
        for i in range(m):
            for t in range(max(ctx, 0)):
                inside = window == 0 or t > pos[i] - window
                first = prefix_lens is not None and t < int(prefix_lens[s])
                seen[i, t] = inside or first
            for j in range(m):
                if ctx + j >= 0 and bits[i, j]:
                    seen[i, ctx + j] = True
        for j in range(m):
            if ctx + j >= 0:
                at[ctx + j] = pos[j]
        out[a:b], tol[a:b] = _sequence(q[a:b], rows_of(k, bt[s], n), rows_of(v, bt[s], n), pos, seen,
                                       scale, softcap, slopes, eps_p, False, at)
    return Result(out, tol)


def turn(x, norm, eps, positions, axis, cos_sin, interleaved):
    """Norm and rotation of x [rows, heads, D] (float64; norm None: none) and, per element, a
    bound on float32's error: the sum of D squares, its root and three products are off by
    less than 16 half steps (the sum over 8 terms a thread and a tree of 5 more has 13
    roundings, halved by the root; then the root, the division by D, the sum with eps
    and two products), the two products and the sum of the rotation by three more."""
    x = np.asarray(x, dtype=np.float64)
    rows, heads, D = x.shape
    y = x
    if norm is not None:
        y = x / np.sqrt((x * x).sum(-1, keepdims=True) / D + eps) * np.asarray(norm, dtype=np.float64)
    z, reach = y.copy(), np.abs(y)
    most, R = cos_sin.shape
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        p = np.clip(positions[min(max(int(axis[i]), 0), len(positions) - 1)], 0, most - 1)
        c, s = (cos_sin[p, j].astype(np.float64)[:, None] for j in (i, R // 2 + i))
        z[..., a] = y[..., a] * c - y[..., b] * s
        z[..., b] = y[..., b] * c + y[..., a] * s
        reach[..., a] = np.abs(y[..., a] * c) + np.abs(y[..., b] * s)
        reach[..., b] = np.abs(y[..., b] * c) + np.abs(y[..., a] * s)
    return z, 19 * F32_STEP * reach


def compact(cache, qo, accepted, bt, lens):
    """Moves the rows of one cache array [NB, H_kv, BS, ...] (a copy is returned) and gives the
    new lengths."""
    cache = cache.copy()
    BS, out = cache.shape[2], []
    for s, L in enumerate(lens):
        L = min(max(int(L), 0), bt.shape[1] * BS)
        m = int(qo[s + 1]) - int(qo[s])
        ctx, last, kept = L - m, -1, []
        for x in accepted[s]:
            if x <= last or x >= m:
                break
            last = int(x)
            kept.append(last)
        rows = {}
        for j in kept:
            if ctx + j >= 0:
                rows[j] = cache[bt[s, (ctx + j) // BS], :, (ctx + j) % BS].copy()
        for i, j in enumerate(kept):
            if ctx + i >= 0:
                cache[bt[s, (ctx + i) // BS], :, (ctx + i) % BS] = rows[j]
        out.append(max(ctx + len(kept), 0))
    return cache, np.array(out, dtype=np.int64)


def fork(caches, bt, lens, parents, children, refs, free, free_count):
    """(caches, bt, lens, refs, free_count_out, refused); caches: arrays [NB, H_kv, BS, ...]."""
    caches = [c.copy() for c in caches]
    bt, lens, refs = bt.copy(), np.array(lens, dtype=np.int64), np.array(refs, dtype=np.int64)
    BS = caches[0].shape[2]
    count = min(max(int(free_count), 0), len(free))
    used = refused = 0
    for p, c in zip((int(x) for x in parents), (int(x) for x in children)):
        rows = range(len(bt))
        if p not in rows or c not in rows or p == c:
            refused += 1
            if c in rows and c != p:
                lens[c] = 0
            continue
        L = min(max(int(lens[p]), 0), bt.shape[1] * BS)
        full, tail = divmod(L, BS)
        if tail and used >= count:
            refused += 1
            lens[c] = 0
            continue
        for j in range(full):
            bt[c, j] = bt[p, j]
            if 0 <= bt[p, j] < len(refs):
                refs[bt[p, j]] += 1
        if tail:
            fresh = int(free[count - 1 - used])
            used += 1
            bt[c, full] = fresh
            last = int(bt[p, full])
            if 0 <= last < len(refs) and 0 <= fresh < len(refs):
                for x in caches:
                    x[fresh, :, :tail] = x[last, :, :tail]
        lens[c] = L
    return caches, bt, lens, refs, count - used, refused


def release(bt, lens, keep, refs, free, free_count, BS):
    """(lens_out, refs, free, free_count_out); refs None: no block is shared."""
    free = np.array(free)
    refs = None if refs is None else np.array(refs, dtype=np.int64)
    count = min(max(int(free_count), 0), len(free))
    gone, lens_out = [], []
    for s, L in enumerate(lens):
        L = min(max(int(L), 0), bt.shape[1] * BS)
        n = min(max(int(keep[s]), 0), L)
        lens_out.append(n)
        gone += [int(b) for b in bt[s, -(-n // BS):-(-L // BS)]
                 if b >= 0 and (refs is None or b < len(refs))]
    held, done = Counter(gone), set()
    for b in gone:
        if refs is None or (b not in done and refs[b] < held[b]):
            if count < len(free):
                free[count] = b
                count += 1
        done.add(b)
    if refs is not None:
        for b in done:
            refs[b] = max(refs[b] - held[b], 0)
    return np.array(lens_out, dtype=np.int64), refs, free, count
