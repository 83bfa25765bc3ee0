"""Block-scaled one-byte caches, accumulated attention weights and eviction (oracle; test infrastructure only).

Sources: "KV-Cache——为什么AI回复越来越快" section 08 (KV-Cache quantisation; keeping part of the rows) and the closing
section of "KV缓存原理与显存估算" (state that leaves the cache). The pages fix no scale granularity and no rule for what
leaves; the readings:

* one scale per (block, kv head), the largest magnitude the block was given over the largest code; it grows while the
  block fills, and the earlier rows are then rounded to the new scale; writing row 0 starts the block afresh;
* the weight of a cached row is the sum of its softmax weights over the queries of its kv head; a call adds it to the
  row's score, and the call's own rows start at it;
* eviction keeps, per kv head, the newest rows and those with the largest scores, in their order.
"""

from __future__ import annotations

import numpy as np

from . import quant as Q

F = np.float32
TINY = F(2.0 ** -126)


def _encode(x, code):
    x = np.asarray(x, dtype=F)
    if code == "int8":
        y = np.where(np.isnan(x), F(0), np.clip(x, F(-127), F(127)))
        return np.rint(y).astype(np.int8)
    flat, inverse = np.unique(x.view(np.uint32).reshape(-1), return_inverse=True)  # each value once: encode is a loop
    return Q.encode_e4m3(flat.view(F))[inverse].reshape(x.shape)


def code_values(codes):
    """Values of codes in units of their scale (float64)."""
    return codes.astype(np.float64) if codes.dtype == np.int8 else Q.decode_e4m3(codes)


def append_block8(x, slots, codes, scale, code):
    """Append of one of K and V: x [T, Hkv, D] float32, codes [nb, Hkv, bs, D], scale float32 [nb, Hkv]; returns new
    arrays. The tokens of one block are taken together."""
    codes, scale = codes.copy(), scale.copy()
    bs, top = codes.shape[2], F(127 if code == "int8" else 448)
    x = np.asarray(x, dtype=F)
    runs = {}
    for t, slot in enumerate(np.asarray(slots).reshape(-1).tolist()):
        if slot >= 0:
            runs.setdefault(slot // bs, []).append((t, slot % bs))
    with np.errstate(invalid="ignore", over="ignore", under="ignore", divide="ignore"):
        for b, run in runs.items():
            first = min(r for _, r in run)
            for h in range(codes.shape[1]):
                rows = x[[t for t, _ in run], h]
                finite = np.where(np.isfinite(rows), np.abs(rows), F(0))
                old = F(0) if first == 0 else scale[b, h]
                s = max(old, F(finite.max() * F(F(1) / top)))
                if not s >= TINY:
                    s = F(0)
                if first > 0 and s != old:
                    f = F(old / s) if s > 0 else F(0)
                    codes[b, h, :first] = _encode(code_values(codes[b, h, :first]).astype(F) * f, code)
                inv = F(F(1) / s) if s > 0 else F(0)
                for (_, r), row in zip(run, rows):
                    codes[b, h, r] = _encode(row * inv if s > 0 else np.zeros_like(row), code)
                scale[b, h] = s
    return codes, scale


def dequantized(codes, scale):
    return code_values(codes) * scale.astype(np.float64)[:, :, None, None]


def decode_scored(q, K, V, tables, lens, sm_scale, scores=None):
    """q [B, T, Hq, D], pools K, V [nb, Hkv, bs, D] (float64); returns (out [B, T, Hq, D], new scores or None).
    Sequences of invalid length give zeros and keep their scores; rows of blocks outside the pool get no weight."""
    B, T, Hq, D = q.shape
    nb, H, bs, _ = K.shape
    G, R = Hq // H, tables.shape[1] * bs
    out = np.zeros(q.shape)
    new = None if scores is None else scores.astype(np.float64).copy()
    for i in range(B):
        n = int(lens[i])
        if n < T or n > R:
            continue
        blocks = tables[i, :-(-n // bs)]
        good = (blocks >= 0) & (blocks < nb)
        safe = np.where(good, blocks, 0)
        there = np.repeat(good, bs)[:n]
        if new is not None:
            new[i, :, n - T:n] = 0
        for h in range(H):
            k = K[safe, h].reshape(-1, D)[:n]
            v = np.where(there[:, None], V[safe, h].reshape(-1, D)[:n], 0)
            for t in range(T):
                seen = there & (np.arange(n) <= n - T + t)
                if not seen.any():
                    continue
                x = np.where(seen, (q[i, t, h * G:(h + 1) * G] @ k.T) * sm_scale, -np.inf)
                p = np.exp(x - x.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                out[i, t, h * G:(h + 1) * G] = p @ np.where(seen[:, None], v, 0)
                if new is not None:
                    new[i, h, :n] += p.sum(0)
    return out, new


def evict(scores, lens, budget, recent):
    """Kept rows [B, H, budget] (-1 past the end) and new lengths."""
    B, H, R = scores.shape
    kept = np.full((B, H, budget), -1, dtype=np.int32)
    new_lens = np.zeros(B, dtype=np.int32)
    for i in range(B):
        n = int(lens[i])
        if n < 0 or n > R:
            n = 0
        m = min(n, budget)
        last = min(recent, m)
        new_lens[i] = m
        for h in range(H):
            rows = list(range(n - last))
            # largest first, ties by the lower row, NaN behind everything
            rows.sort(key=lambda r: (np.isnan(scores[i, h, r]), 0.0 if np.isnan(scores[i, h, r]) else -scores[i, h, r],
                                     r))
            kept[i, h, :m] = sorted(rows[:m - last]) + list(range(n - last, n))
    return kept, new_lens


def move_rows(pool, kept, new_lens, tables, new_tables, scale=None, code=None):
    """The pool (and its scales) after the kept rows were copied to the new blocks."""
    pool = pool.copy()
    src = pool.copy()
    old = None if scale is None else scale.copy()
    scale = None if scale is None else scale.copy()
    nb, H, bs, _ = pool.shape
    for i, m in enumerate(new_lens.tolist()):
        for h in range(H):
            for j0 in range(0, m, bs):
                to = int(new_tables[i, j0 // bs])
                js = [j for j in range(j0, min(m, j0 + bs)) if 0 <= tables[i, kept[i, h, j] // bs] < nb]
                froms = [int(tables[i, kept[i, h, j] // bs]) for j in js]
                if not 0 <= to < nb:
                    continue
                if scale is not None:
                    s = max([old[b, h] for b in froms], default=F(0))
                    scale[to, h] = s
                for j, b in zip(js, froms):
                    row = src[b, h, kept[i, h, j] % bs]
                    if scale is not None and old[b, h] != s:
                        row = _encode(code_values(row).astype(F) * F(old[b, h] / s), code)
                    pool[to, h, j % bs] = row
    return pool if scale is None else (pool, scale)
