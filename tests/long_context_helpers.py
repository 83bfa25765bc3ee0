"""Inputs, library calls and error bounds shared by the tests of the block-scaled caches, the scored decode and the
eviction."""

import math

import numpy as np
import torch

from oracle import long_context as O

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def f64(t):
    return t.detach().cpu().double().numpy()


def make_tables(lens, bs, spare, rng, width=None):
    """Block tables over a shuffled pool; unused entries hold an id outside the pool (never read)."""
    need = [min(width or 1 << 30, -(-max(0, n) // bs)) for n in lens]
    ids = rng.permutation(sum(need) + spare)
    table = np.full((len(lens), width or max(1, max(need))), 1 << 28, dtype=np.int32)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = ids[at:at + k]
        at += k
    return table, len(ids), ids[at:]


def make_pools(nb, H, bs, D, kind, rng):
    """K, V (and scales) of one kind: "f16"/"bf16" rows, or "e4m3"/"int8" codes. Returns device tensors and the
    float64 pools they stand for."""
    res = []
    for _ in range(2):
        x = rng.standard_normal((nb, H, bs, D)) * np.exp(0.7 * rng.standard_normal((nb, H, 1, 1)))
        if kind in TORCH:
            t = torch.from_numpy(x).to(TORCH[kind])
            res.append((t.cuda(), None, f64(t)))
        else:
            top = 127.0 if kind == "int8" else 448.0
            scale = (np.abs(x).max((2, 3)) / top).astype(np.float32)
            y = torch.from_numpy(np.clip(x / scale[:, :, None, None], -top, top))
            t = torch.round(y).to(torch.int8) if kind == "int8" else y.float().to(torch.float8_e4m3fn).view(torch.uint8)
            res.append((t.cuda(), torch.from_numpy(scale).cuda(), O.dequantized(t.numpy(), scale)))
    return res


def workspace_for(kvc, q, k_cache, tables, scored):
    B, T, hq, d = q.shape
    return kvc.new_scored_workspace(B, T, hq, k_cache.shape[1], d, k_cache.shape[2], tables.shape[1], scored=scored)


def call_decode(kvc, kind, q, pools, tables, lens, scale, out, scores, ws, stream=None):
    (k, ks, _), (v, vs, _) = pools
    if ks is None:
        kvc.decode_attention_scored(q, k, v, tables, lens, scale, out, scores, ws, stream=stream)
    else:
        kvc.decode_attention_block8(q, k, v, ks, vs, tables, lens, scale, out, ws, scores=scores, stream=stream)


def bounds(q, K, V, tables, lens, scale, out_dtype, ref_out, ref_scores):
    """Error bounds of the outputs and of the scores, from the arithmetic:
    a scaled score x is a sum of D products in fp32, each addition off by at most 2^-23 of what is summed (the tensor
    cores cut, where rounding would give 2^-24), so |dx| <= (D + 4) 2^-23 scale max sum |q k|; exp2 and log2 add 2^-21
    relative to a weight; the sums run over chains of at most 3 additions per 16 rows (the parts of a weight) plus 64
    for the joins, each off by 2^-23 of sum p |v| <= max |v|; the last rounding is half a step of the output type."""
    nb = K.shape[0]
    used = np.unique(np.clip(tables, 0, nb - 1))
    D = q.shape[-1]
    qk = float(np.abs(q).max() * np.abs(K[used]).sum(-1).max())
    dx = (D + 4) * 2.0 ** -23 * scale * qk
    chain = (3 * (int(max(lens)) / 16 + 1) + 64) * 2.0 ** -23
    weight = 2 * dx + 2.0 ** -21 + chain
    vmax = float(np.abs(V[used]).max())
    half = 0.0 if out_dtype == torch.float32 else torch.finfo(out_dtype).eps / 2
    tiny = float(torch.finfo(out_dtype).tiny) * half  # below the normal numbers the step no longer shrinks
    out = weight * vmax * 2 + half * np.abs(ref_out) * (1 + 2 ** -8) + tiny
    sc = None if ref_scores is None else (weight * 2 + q.shape[1] * q.shape[2] * 2.0 ** -23) * (1 + np.abs(ref_scores))
    return out, sc
