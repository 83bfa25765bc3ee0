"""Scored decode: an infinity or NaN in a cached value reaches exactly the outputs of the queries that see its row, as
itself, whatever the row's weight, the number of new tokens and the split of the work."""

import numpy as np
import pytest
import torch

from long_context_helpers import call_decode, f64, workspace_for
from test_gpu_scored import make

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True)
def _options(kvc):
    yield
    kvc.set_option(kvc.OPT_BLOCKS_PER_CTA, 0)
    kvc.set_option(kvc.OPT_MAX_CTAS, 0)


def run(kvc, kind, q, pools, tables, lens, scale, scores, out_dtype=torch.float32):
    out = torch.empty(q.shape, dtype=out_dtype, device="cuda")
    sc = scores.clone()
    call_decode(kvc, kind, q, pools, torch.from_numpy(tables).cuda(),
                torch.tensor(lens, dtype=torch.int32, device="cuda"), scale, out, sc,
                workspace_for(kvc, q, pools[0][0], tables, True))
    torch.cuda.synchronize()
    return out, sc


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("T,per,ctas,lens", [(1, 0, 0, [41, 130]), (1, 1, 0, [41, 700]), (1, 1000, 0, [41, 130]),
                                             (1, 1, 3, [2000, 5]), (1, 0, 0, [12000]), (5, 0, 0, [41, 130]),
                                             (5, 1, 0, [41, 700]), (20, 3, 0, [64, 200])])
@pytest.mark.parametrize("D,out_dtype", [(64, torch.float32), (128, torch.bfloat16), (256, torch.float16),
                                         (128, torch.float32)])
def test_infinities_reach_those_that_see_them(kvc, kind, T, per, ctas, lens, D, out_dtype):
    H, G, bs = 2, 3, 16
    kvc.set_option(kvc.OPT_BLOCKS_PER_CTA, per)
    kvc.set_option(kvc.OPT_MAX_CTAS, ctas)
    q, pools, tables, scores = make(kind, lens, T, H * G, H, D, bs, seed=81)
    clean, clean_scores = run(kvc, kind, q, pools, tables, lens, 0.1, scores, out_dtype)
    assert torch.isfinite(clean).all()
    want = clean.clone().view(len(lens), T, H, G, D)
    for i, n in enumerate(lens):
        # (row, head, dim, value): a row all see, both signs in one dim, the newest row, the first row
        for r, h, d, x in ((n // 2, 0, 3, INF), (n // 3, 0, 7, -INF), (n // 2 + 1, 0, D - 1, INF),
                           (n // 3, 0, D - 1, -INF), (n - 1, 1, 9, INF), (0, 1, 20, -INF), (n // 2, 1, 21, NAN)):
            pools[1][0][int(tables[i, r // bs]), h, r % bs, d] = x
            for t in range(T):
                if r <= n - T + t:
                    want[i, t, h, :, d] = x if torch.isfinite(want[i, t, h, 0, d]) else NAN
    got, got_scores = run(kvc, kind, q, pools, tables, lens, 0.1, scores, out_dtype)
    got = got.view_as(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    fine = ~torch.isnan(want)
    # rows that some new tokens see and others do not may be summed apart: the finite rest within the roundings of
    # 200 rows, 2^-22 each of at most the largest value, and half a step of the output
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf])
    both = fine & ~inf
    spread = (got[both].double() - want[both].double()).abs().max().item()
    big = max(1.0, float(np.abs(pools[1][2]).max()))
    assert spread <= 200 * 2.0 ** -22 * big + (0 if out_dtype == torch.float32 else torch.finfo(out_dtype).eps * big)
    assert torch.equal(got_scores, clean_scores)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("per", [0, 1, 1000])
def test_infinities_of_vanishing_weight(kvc, kind, per):
    # the weight of the row, e^-150, is not 0, although no fp32 number is that small beside the others
    H, G, D, bs, n = 1, 4, 128, 16, 200
    kvc.set_option(kvc.OPT_BLOCKS_PER_CTA, per)
    q, pools, tables, scores = make(kind, [n], 1, H * G, H, D, bs, seed=82)
    q.zero_()
    q[..., 0] = 1
    k = pools[0][0]
    k[..., 0] = 0
    for r in (0, 100, 199):  # each far below the others
        k[int(tables[0, r // bs]), 0, r % bs, 0] = -150
    for b in range(5, 7):  # a whole stretch of such rows
        k[int(tables[0, b]), 0, :, 0] = -150
    clean, _ = run(kvc, kind, q, pools, tables, [n], 1.0, scores)
    for r, d in ((0, 1), (100, 2), (199, 3), (83, 4)):
        pools[1][0][int(tables[0, r // bs]), 0, r % bs, d] = INF
    got, got_scores = run(kvc, kind, q, pools, tables, [n], 1.0, scores)
    assert (got[..., 1:5] == INF).all()
    assert torch.equal(got[..., 5:], clean[..., 5:]) and torch.equal(got[..., 0], clean[..., 0])
    assert torch.isfinite(got_scores).all()


def test_overflow_of_the_output_type_is_left_alone(kvc):
    # finite sums that f16 cannot hold round to infinity; nothing in the cache is one
    q, pools, tables, scores = make("bf16", [50], 1, 4, 1, 64, 16, seed=83)
    pools[1][0].fill_(1e6)
    out, _ = run(kvc, "bf16", q, pools, tables, [50], 0.1, scores, torch.float16)
    assert (out == INF).all()
    out, _ = run(kvc, "bf16", q, pools, tables, [50], 0.1, scores, torch.float32)
    v = float(torch.tensor(1e6).bfloat16())
    assert np.abs(f64(out) - v).max() <= 200 * 2.0 ** -22 * v
