"""Inputs on which the scored decode's arithmetic can be followed weight by weight, and error bounds for them.

Queries and keys are small whole numbers (times a power of two per block for one-byte caches): every product and every
sum of a score is exact in fp32, in any order. The value of row r is a small whole number in dim r mod D and 0 elsewhere:
an output adds up the weights of the few rows of its dim, so a row that is left out, a weight in too few bits or a score
that is off by a percent shows at its own size, not beside the largest value of the pool.

What is left, per weight p = 2^(x - m) / l with x = S * (scale * log2 e) in fp32:
* x: the factor and the product are rounded, 2^-24 of |x| each; x - m and the sums with lse are rounded, 2^-24 of what
  they give; ex2.approx and lg2.approx 2^-22 each;
* the same for the denominator, a mean of such errors, and its sum of positive terms: a chain of two additions per 16
  rows, and of the joins, 2^-24 each;
* outputs: the parts of a weight 2^-21, and at most 3 products per row whose two addends are cut at 2^-23; f16 parts (all
  but bf16 caches) also 2^-47 of the query's largest weight. One-byte caches have the V scale in the weight: what is cut
  into parts is p * v_scale, to 2^-47 of its largest value over the rows, and meets the row's code, so a row whose scale
  is small beside that row's is off by more than 2^-47 of p times its value; references
  move at most once for every 4 binary places that the scores span, with a factor (2^-22) and a rounding each;
* the merge of records: a factor (2^-22 and the difference of the maxima, 2^-24) and two roundings for each of at most
  64 of them, and the division.
"""

import numpy as np
import torch

from oracle import long_context as O

from long_context_helpers import TORCH, make_tables

U = 2.0 ** -24

# (lens, T, Hq, H, D, block size, scale): lengths around the tile, several tokens, odd groups, every head size; the
# last ones with scores of some hundreds
CASES = [
    ([1, 15, 16, 17, 100, 303], 1, 8, 2, 128, 16, 2.0 ** -5),
    ([64, 130, 47], 1, 3, 3, 64, 32, 2.0 ** -4),
    ([200, 1000], 1, 20, 1, 256, 48, 2.0 ** -6),
    ([9, 150, 400], 5, 6, 2, 128, 16, 2.0 ** -5),
    ([40, 260], 33, 4, 2, 64, 80, 2.0 ** -4),
    ([2100], 1, 4, 1, 128, 16, 2.0 ** -5),
    ([700, 31], 1, 8, 2, 128, 16, 2.0 ** -3),
    ([120, 300], 3, 3, 1, 256, 16, 2.0 ** -4),
    ([700, 31], 1, 8, 2, 128, 16, 1.0),
    ([120, 300], 3, 3, 1, 256, 16, 0.5),
]
PEAKED = 0.5  # from this scale on most weights vanish beside the largest: faults in one row or a permille do not show


def inputs(kind, case, seed=0):
    """q (numpy), [(cache as a CPU tensor, scales or None, float64 pool)] for K and V, tables, old scores."""
    lens, T, Hq, H, D, bs, _ = case
    rng = np.random.default_rng(seed + 1)
    tables, nb, _ = make_tables(lens, bs, 2, rng)
    q = rng.integers(-4, 5, (len(lens), T, Hq, D)).astype(np.float64)
    k = rng.integers(-4, 5, (nb, H, bs, D)).astype(np.float64)
    v = np.zeros((nb, H, bs, D))
    for i, n in enumerate(lens):
        for r in range(n):
            v[tables[i, r // bs], :, r % bs, r % D] = rng.integers(1, 8, H) * rng.choice([-1, 1], H)
    scores = (rng.random((len(lens), H, tables.shape[1] * bs)) * 3).astype(np.float32)
    pools = []
    for x, spread in ((k, [0.5, 1.0]), (v, [0.25, 1.0, 3.0])):
        if kind in TORCH:
            pools.append((torch.from_numpy(x).to(TORCH[kind]), None, x))
        else:
            t = torch.from_numpy(x)
            t = t.to(torch.int8) if kind == "int8" else t.float().to(torch.float8_e4m3fn).view(torch.uint8)
            s = rng.choice(spread, (nb, H)).astype(np.float32)
            pools.append((t, torch.from_numpy(s), O.dequantized(t.numpy(), s)))
    return q, pools, tables, scores


def scaled(q, K, tables, i, h, G, n, scale):
    """Scores of sequence i's queries of kv head h in log2 units, [T, G, n]."""
    bs = K.shape[2]
    k = K[tables[i, :-(-n // bs)], h].reshape(-1, K.shape[3])[:n]
    return (q[i, :, h * G:(h + 1) * G] @ k.T) * scale * np.log2(np.e)


def bounds(kind, q, K, V, vs, tables, lens, scale, out_dtype, ref, old):
    """Error bounds of the outputs and of the new scores, for every entry. vs: V's scales, None for 16-bit caches."""
    B, T, Hq, D = q.shape
    H = K.shape[1]
    G = Hq // H
    mass, _ = O.decode_scored(q, K, np.abs(V), tables, lens, scale)
    tol, tol_scores = np.zeros(ref.shape), np.zeros(old.shape)
    for i, n in enumerate(lens):
        for h in range(H):
            x = scaled(q, K, tables, i, h, G, n, scale)
            hidden = np.arange(n)[None, None] > (n - T + np.arange(T))[:, None, None]
            x = np.where(hidden, -np.inf, x)
            top = x.max(-1, keepdims=True)
            p = np.exp2(x - top)
            p /= p.sum(-1, keepdims=True)
            big = np.abs(np.where(hidden, 0, x)).max(-1)  # per query
            span = big + np.abs(top[..., 0])
            # a weight against the exact one, its exponent's errors times ln 2: those of its own x and of the mean
            # over the denominator
            weight = 2 * (0.7 * (2 * big + span + 20) * U + 4 * U) + (n / 8 + 64) * U
            moves = (span / 4 + 1) * 2 * 5 * U
            merge = 64 * (0.7 * span * U + 6 * U)
            adds = (6 * (n // D + 1) + 4) * 2 * U
            tol[i, :, h * G:(h + 1) * G] = ((weight + 8 * U + moves + merge + adds)[..., None]
                                            * mass[i, :, h * G:(h + 1) * G])
            if kind != "bf16":
                blocks = tables[i, :-(-n // V.shape[2])]
                vscale = np.ones(len(blocks)) if vs is None else vs[blocks, h].astype(np.float64)
                code = np.abs(V[blocks, h] / vscale[:, None, None]).reshape(-1, D)[:n].sum(0)
                largest = (p * np.repeat(vscale, V.shape[2])[:n]).max(-1)
                tol[i, :, h * G:(h + 1) * G] += 2.0 ** -46 * largest[..., None] * code
            w = (p * (weight + moves + merge)[..., None]).sum((0, 1)) + p.sum((0, 1)) * T * G * U
            tol_scores[i, h, :n] = w + 2 * U * (old[i, h, :n] + p.sum((0, 1)))
    if out_dtype != torch.float32:
        tol += torch.finfo(out_dtype).eps / 2 * np.abs(ref) * (1 + 2 ** -8)
        tol += float(torch.finfo(out_dtype).tiny) * torch.finfo(out_dtype).eps
    return tol + 2.0 ** -120, tol_scores + 2.0 ** -120


def wrong(kind, q, K, V, tables, lens, scale, old, fault):
    """Outputs and scores of a decode with a fault planted, in float64 but for it."""
    B, T, Hq, D = q.shape
    H, bs = K.shape[1], K.shape[2]
    G = Hq // H
    out, new = np.zeros(q.shape), old.astype(np.float64).copy()
    f16 = kind != "bf16"
    for i, n in enumerate(lens):
        new[i, :, n - T:n] = 0
        for h in range(H):
            x = scaled(q * (1.01 if fault == "query" else 1.0), K, tables, i, h, G, n, scale)
            x = np.where(np.arange(n)[None, None] > (n - T + np.arange(T))[:, None, None], -np.inf, x)
            if fault == "tile" and n >= 48:
                x[..., 32:48] = -np.inf
            if fault == "mask" and T > 1:  # every token sees what the last one sees
                x = scaled(q, K, tables, i, h, G, n, scale)
            p = np.exp2(x - x.max(-1, keepdims=True))
            total = p.sum(-1, keepdims=True)
            if fault == "parts":  # one 16-bit part per weight
                p = torch.from_numpy(p).to(torch.float16 if f16 else torch.bfloat16).double().numpy()
            if fault == "last":  # the newest row is left out of the sum of outputs
                p[..., -1] = 0
            v = V[tables[i, :-(-n // bs)], h].reshape(-1, D)[:n]
            out[i, :, h * G:(h + 1) * G] = (p @ v) / total
            new[i, h, :n] += (p / total).sum((0, 1)) * (0.999 if fault == "scores" else 1.0)
    return out, new
