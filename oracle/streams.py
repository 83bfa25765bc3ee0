"""Windows with sinks, prompts over the paged cache and four-bit rows (oracle; test infrastructure only).

Sources: the chunk mask of "单请求 KV Cache" (query row i of a chunk sees columns up to past_len + i), Window Attention and
KV-Cache quantisation of "KV-Cache——为什么AI回复越来越快" section 08. The pages fix neither which early rows stay nor a
four-bit format; the readings:

* the token at position pos sees row r if r <= pos and (r > pos - window or r < sinks);
* a group of 16 elements of a row with largest finite magnitude A has the scale e4m3(A / 6) and the codes e2m1(x / scale),
  both nearest, ties to even, saturating; infinities saturate, NaN is 0.
"""

from __future__ import annotations

from fractions import Fraction

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m if e == 0 else 8 + m) * 2.0 ** (max(e, 1) - 10) for e in range(16) for m in range(8)][:127])

SCALES = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])  # of every code; the append writes the first 127


def nearest(x, table):
    """Index of the table's entry nearest to x >= 0 (a Fraction); ties to the even index, the last one beyond it."""
    i = int(np.searchsorted(table, float(x)))
    best = None
    for j in range(max(0, i - 2), min(len(table), i + 2)):
        d = abs(Fraction(float(table[j])) - x)
        if best is None or d < best[0] or (d == best[0] and j % 2 == 0):
            best = (d, j)
    return best[1]


def encode_fp4(x):
    """x [..., D]: codes uint8 [..., D] (bit 3 the sign) and scale codes uint8 [..., D / 16], from exact quotients."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(-1, 16)
    codes, scales = np.zeros(g.shape, np.uint8), np.zeros(len(g), np.uint8)
    for i, row in enumerate(g):
        fine = row[np.isfinite(row)]
        top = np.abs(fine).max() if len(fine) else 0.0
        scales[i] = nearest(Fraction(float(top)) / 6, E4M3)
        s = Fraction(float(E4M3[scales[i]]))
        for j, y in enumerate(row):
            if np.isnan(y) or s == 0:
                continue
            codes[i, j] = (7 if np.isinf(y) else nearest(abs(Fraction(float(y))) / s, E2M1)) + (8 if y < 0 else 0)
    return codes.reshape(x.shape), scales.reshape(*x.shape[:-1], -1)


def pack(codes):
    return (codes[..., ::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    return np.stack((packed & 15, packed >> 4), -1).reshape(*packed.shape[:-1], -1)


def values_fp4(packed, scales):
    """The values that packed codes [..., D / 2] with scale codes [..., D / 16] stand for."""
    c = unpack(packed)
    x = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
    return x * np.repeat(SCALES[scales], 16, -1)


def visible(pos, rows, window, sinks):
    """[len(pos), rows]: which rows the tokens at these positions see (window None: all up to their own)."""
    pos, r = np.asarray(pos)[:, None], np.arange(rows)[None]
    seen = r <= pos
    if window is not None:
        seen = seen & ((r > pos - window) | (r < sinks))
    return seen


def attend(q, K, V, table, n, scale, window=None, sinks=0):
    """q [m, Hq, D] of the m newest of a sequence's n rows, pools K, V [nb, H, bs, D] in 64 bits, its block table.
    Returns (out, sum of p |v|, largest sum |q k| of a seen row) per output, the last per query. Rows of blocks outside
    the pool get no weight."""
    m, Hq, D = q.shape
    nb, H, bs, _ = K.shape
    G = Hq // H
    blocks = np.asarray(table[:-(-n // bs)])
    good = (blocks >= 0) & (blocks < nb)
    seen = visible(np.arange(n - m, n), n, window, sinks) & np.repeat(good, bs)[None, :n]
    blocks = np.where(good, blocks, 0)
    use = seen.any(0)  # rows that nobody sees may hold anything
    out, mass, size = np.zeros(q.shape), np.zeros(q.shape), np.zeros((m, Hq))
    for h in range(H):
        k = np.where(use[:, None], K[blocks, h].reshape(-1, D)[:n], 0)
        v = np.where(use[:, None], V[blocks, h].reshape(-1, D)[:n], 0)
        odd = ~np.isfinite(v)
        for j in range(h * G, (h + 1) * G):
            x = np.where(seen, (q[:, j] @ np.where(np.isfinite(k), k, 0).T) * scale, -np.inf)
            top = x.max(1, keepdims=True)
            p = np.exp(x - np.where(np.isfinite(top), top, 0))
            p /= np.maximum(p.sum(1, keepdims=True), 1e-300)
            out[:, j] = p @ np.where(odd, 0, v)
            mass[:, j] = p @ np.abs(np.where(odd, 0, v))
            size[:, j] = np.where(seen, np.abs(q[:, j]) @ np.abs(np.where(np.isfinite(k), k, 0)).T, 0).max(1)
            for r, d in zip(*np.nonzero(odd)):  # an infinity or NaN is the output of those who see it
                out[seen[:, r], j, d] += v[r, d]
    return out, mass, size
