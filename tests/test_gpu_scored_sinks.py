"""Attention sinks: one row takes nearly all the weight and brings nothing (its value is zero), so that the outputs are
made of weights far below the largest one."""

import numpy as np
import pytest
import torch

from oracle import long_context as O

from long_context_helpers import TORCH, call_decode, f64, workspace_for

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "f16", "e4m3", "int8"]


def sink_case(kind, n, sinks, depth, H, G, D, bs, seed, same):
    """Keys whose first entry is the score itself (scale 1, queries of 1 there and 0 elsewhere): 0 for the sinks,
    -depth (or 2 less) for the other rows. Values of the sinks are 0, the others' positive."""
    rng = np.random.default_rng(seed)
    nb = -(-n // bs)
    tables = rng.permutation(nb).astype(np.int32)[None]
    k = np.zeros((nb, H, bs, D))
    v = np.zeros((nb, H, bs, D))
    row = -depth - (np.zeros(n) if same else 2 * rng.integers(0, 2, n))
    row[sinks] = 0
    val = rng.integers(1, 8, (n, H, D)).astype(np.float64)
    val[sinks] = 0
    for r in range(n):
        b = tables[0, r // bs]
        k[b, :, r % bs, 0] = row[r]
        v[b, :, r % bs] = val[r]
    q = np.zeros((1, 1, H * G, D))
    q[..., 0] = 1
    pools = []
    for x in (k, v):
        if kind in TORCH:
            pools.append((torch.from_numpy(x).to(TORCH[kind]).cuda(), None, x))
        else:  # small whole numbers are codes of scale 1
            t = torch.from_numpy(x)
            t = t.to(torch.int8) if kind == "int8" else t.float().to(torch.float8_e4m3fn).view(torch.uint8)
            pools.append((t.cuda(), torch.ones((nb, H), device="cuda"), x))
    q = torch.from_numpy(q).to(TORCH.get(kind, torch.bfloat16)).cuda()
    return q, pools, tables


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("depth", [4, 8, 12, 16, 18])  # e^-18: 2^-26 of the sink's weight
@pytest.mark.parametrize("n,sinks,per", [(864, [0], 0), (864, [0], 1000), (4100, [1, 2000], 1000), (16, [3], 0),
                                         (300, [299], 1000)])
def test_small_weights_keep_their_precision(kvc, kind, depth, n, sinks, per):
    # Scaled scores are small whole numbers: exact but for the product with log2(e), off by 2^-24 of at most 29
    # (twice: the factor itself and the product), which moves a weight by 29 * 2^-23 * ln 2; exp2 adds 2^-22, and the
    # parts of a weight that reach 2^-26 of the largest one give it at 2^-21. Nothing cancels (every value is
    # positive), so the errors of the sums stay relative to the output: at most 3 products per 16 rows, of 17 terms
    # each with the sum so far, every term off by at most 2^-23 of the largest, and 64 for the joins.
    rel = 29 * 2.0 ** -23 * 0.7 * 2 + 2.0 ** -21 + 2.0 ** -21 + (3 * 17 * (n / 16 + 1) + 64) * 2.0 ** -23
    kvc.set_option(kvc.OPT_BLOCKS_PER_CTA, per)  # 1000: one warp has the whole sequence
    try:
        for same in (True, False):
            q, pools, tables = sink_case(kind, n, sinks, depth, 2, 4, 128, 16, 5 + depth, same)
            scores = torch.zeros((1, 2, tables.shape[1] * 16), device="cuda")
            ref, ref_scores = O.decode_scored(f64(q), pools[0][2], pools[1][2], tables, [n], 1.0, f64(scores))
            out = torch.empty(q.shape, device="cuda")
            call_decode(kvc, kind, q, pools, torch.from_numpy(tables).cuda(),
                        torch.tensor([n], dtype=torch.int32, device="cuda"), 1.0, out, scores,
                        workspace_for(kvc, q, pools[0][0], tables, True))
            torch.cuda.synchronize()
            err = np.abs(f64(out) - ref) / ref
            assert err.max() <= rel, f"relative error {err.max():.2e} (bound {rel:.2e})"
            err = (np.abs(f64(scores) - ref_scores) / np.where(ref_scores > 0, ref_scores, 1))
            assert err.max() <= rel
    finally:
        kvc.set_option(kvc.OPT_BLOCKS_PER_CTA, 0)


@pytest.mark.parametrize("kind", KINDS)
def test_the_largest_weights_stay_in_range(kvc, kind):
    # scores that climb slowly, so that the running reference is exceeded as far as it may be before it moves
    H, G, D, bs, n = 1, 4, 64, 16, 480
    q, pools, tables = sink_case(kind, n, [0], 4, H, G, D, bs, 3, True)
    steps = np.floor(np.arange(n) / 16 * 0.75) if kind != "e4m3" else np.floor(np.arange(n) / 16 * 0.5)
    k = np.zeros((tables.shape[1], H, bs, D))
    v = np.zeros_like(k)
    rng = np.random.default_rng(4)
    for r in range(n):
        b = tables[0, r // bs]
        k[b, :, r % bs, 0] = steps[r] - 10
        v[b, :, r % bs] = rng.integers(1, 8, D)
    for i, x in enumerate((k, v)):
        t = torch.from_numpy(x)
        t = (t.to(TORCH[kind]) if kind in TORCH else t.to(torch.int8) if kind == "int8" else
             t.float().to(torch.float8_e4m3fn).view(torch.uint8))
        pools[i] = (t.cuda(), pools[i][1], x)
    assert kind != "e4m3" or set(np.unique(k[..., 0])) <= set(O.code_values(pools[0][0].cpu().numpy()).ravel())
    ref, _ = O.decode_scored(f64(q), pools[0][2], pools[1][2], tables, [n], 1.0)
    scores = torch.zeros((1, H, tables.shape[1] * bs), device="cuda")
    out = torch.empty(q.shape, device="cuda")
    call_decode(kvc, kind, q, pools, torch.from_numpy(tables).cuda(),
                torch.tensor([n], dtype=torch.int32, device="cuda"), 1.0, out, scores,
                workspace_for(kvc, q, pools[0][0], tables, True))
    torch.cuda.synchronize()
    rel = 20 * 2.0 ** -23 * 0.7 * 2 + 2.0 ** -20 + (3 * 17 * n / 16 + 64) * 2.0 ** -23
    err = np.abs(f64(out) - ref) / ref
    assert err.max() <= rel, f"relative error {err.max():.2e} (bound {rel:.2e})"
