"""GPU parity: prompt attention over the ends of its ranges: many sequences, many tokens, long rows, small weights."""

import numpy as np
import pytest
import torch

from oracle import streams as O

from long_context_helpers import TORCH, f64
from stream_helpers import Prompt, int32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,tokens,long", [
    (1500, 3, []),             # more sequences than the plan has threads, more tiles too
    (1300, 2, [3000, 2500]),   # the same where units may be split, and a few long ones among them
    (4096, 2, []),
    (300, 0, [40, 9, 130]),    # nearly all without new tokens
])
def test_many_sequences(kvc, batch, tokens, long):
    rng = np.random.default_rng(batch)
    new = [int(x) for x in rng.integers(0, tokens + 1, batch)]
    rows = [int(m + x) for m, x in zip(new, rng.integers(0, 180, batch))]
    for at, n in zip(rng.permutation(batch), long):
        new[at], rows[at] = 20, max(20, n)
    p = Prompt(new, rows, 4, 2, 64, 16, "bf16", seed=batch, garbage=False)
    p.run(kvc)
    p.check()
    assert kvc.get_error_flags() == 0


@pytest.mark.parametrize("sizes,window,sinks", [
    (([2000, 1100], [2000, 4000], 4, 2, 128, 16), None, 0),
    (([5000], [5000], 2, 1, 64, 32), 700, 5),
    (([3001], [3001], 3, 1, 128, 64), 1, 1),
])
def test_many_tokens(kvc, sizes, window, sinks):
    p = Prompt(*sizes, "f16", window, sinks, seed=41)
    p.run(kvc)
    p.check()
    assert kvc.get_error_flags() == 0


@pytest.mark.parametrize("per_sm", [0.1, 1, 4.2])
@pytest.mark.parametrize("window,sinks", [(None, 0), (135000, 300)])
def test_rows_beyond_1024_tiles(kvc, per_sm, window, sinks):
    """140,000 rows (classes of more than one cost), few, some and many units, beside short sequences. Values are alike
    within a sequence: its outputs are that value, and every token was served."""
    D, G = 64, 128  # two tokens per unit
    units = int(per_sm * torch.cuda.get_device_properties(0).multi_processor_count)
    new = [2 * units, 3, 40, 0, 1]
    rows = [140000, 3, 5000, 77, 133000]
    need = [-(-n // 128) for n in rows]
    gen = torch.Generator(device="cuda").manual_seed(3)
    k = torch.randn((sum(need), 1, 128, D), generator=gen, device="cuda").to(torch.bfloat16)
    v = torch.zeros_like(k)
    tables = torch.zeros((len(rows), max(need)), dtype=torch.int32, device="cuda")
    for i, m in enumerate(need):
        at = torch.arange(sum(need[:i]), sum(need[:i]) + m, device="cuda")
        tables[i, :m] = at
        v[at] = i + 1.0
    starts = [0]
    for m in new:
        starts.append(starts[-1] + m)
    q = torch.randn((starts[-1], G, D), generator=gen, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 7.0)
    ws = kvc.new_prompt_workspace(len(rows), len(q), G, 1, D, 128, tables.shape[1])
    kvc.prompt_attention(q, k, v, tables, int32(starts), int32(rows), D ** -0.5, out, ws, window=window, sinks=sinks)
    assert kvc.get_error_flags() == 0
    for i in range(len(rows)):
        # weights of half a bf16 step, their sum unrounded, and the output's own rounding
        assert ((out[starts[i]:starts[i + 1]].float() / (i + 1) - 1).abs() <= 2.0 ** -7).all(), i


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("depth", [5, 10, 14])
@pytest.mark.parametrize("n,new,window", [(300, 3, None), (2100, 140, None), (2100, 2, 100), (5000, 2, None)])
def test_small_weights_beside_a_sink_keep_their_precision(kvc, dtype, depth, n, new, window):
    """The first row takes nearly all the weight and brings nothing; the outputs are made of the others' weights, which
    are 2^-20 of it at the least."""
    H, G, D, bs = 2, 4, 128, 16
    rng = np.random.default_rng(depth)
    p = Prompt([new], [n], H * G, H, D, bs, dtype, window, 1, garbage=False)
    at = p.tables[0, np.arange(n) // bs], np.arange(n) % bs
    k, v = (np.zeros(p.pools[0][1].shape) for _ in range(2))
    k[at[0], :, at[1], 0] = -depth
    v[at[0], :, at[1]] = rng.choice([1.0, 2.0, 3.0, 4.0, 6.0], (n, H, D))
    k[p.tables[0, 0], :, 0] = v[p.tables[0, 0], :, 0] = 0
    p.pools = [[torch.from_numpy(x).to(TORCH[dtype]).cuda(), x] for x in (k, v)]
    p.scale = 1.0
    p.q.zero_()
    p.q[..., 0] = 1
    p.run(kvc)
    ref, _, _ = O.attend(f64(p.q[:new]), k, v, p.tables[0], n, 1.0, window, 1)
    # all values are positive, so errors stay relative to the output: scores are whole numbers but for the factor log2(e)
    # and its product, 2^-24 of at most 24 each, which moves a weight by 24 * 2^-23 * ln 2; exp2 2^-22; sums of 5000 rows
    # over 8 at a time 2^-13 at most; half a step for a weight and half a step for the output
    half = torch.finfo(TORCH[dtype]).eps / 2
    assert np.abs(f64(p.out[:new]) / ref - 1).max() <= 2 * half * (1 + half) + 2.0 ** -13 + 2.0 ** -18
    assert kvc.get_error_flags() == 0
