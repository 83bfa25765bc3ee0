"""GPU parity of the scored and block-scaled decode weight by weight: inputs whose scores are exact, values that keep the
rows apart, and bounds for every entry from its own weights (scored_exact_helpers; what they catch:
test_scored_exact_bounds)."""

import numpy as np
import pytest
import torch

from oracle import long_context as O

import scored_exact_helpers as X
from long_context_helpers import call_decode, f64, workspace_for

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "f16", "e4m3", "int8"]


@pytest.fixture(autouse=True)
def _options(kvc):
    yield
    kvc.set_option(kvc.OPT_BLOCKS_PER_CTA, 0)
    kvc.set_option(kvc.OPT_MAX_CTAS, 0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", X.CASES, ids=lambda c: f"D{c[4]}-T{c[1]}-{len(c[0])}x{max(c[0])}-{c[6]:g}")
@pytest.mark.parametrize("per,ctas", [(0, 0), (1, 0), (1000, 0), (2, 3)])
def test_every_weight(kvc, kind, case, per, ctas):
    lens, T, Hq, H, D, bs, scale = case
    kvc.set_option(kvc.OPT_BLOCKS_PER_CTA, per)
    kvc.set_option(kvc.OPT_MAX_CTAS, ctas)
    qn, host, tables, old = X.inputs(kind, case)
    K, V = host[0][2], host[1][2]
    ref, ref_scores = O.decode_scored(qn, K, V, tables, lens, scale, old)
    pools = [(t.cuda(), None if s is None else s.cuda(), x) for t, s, x in host]
    q = torch.from_numpy(qn).to(torch.float16 if kind == "f16" else torch.bfloat16).cuda()
    out_dtype = torch.float32 if per != 2 else torch.float16
    out = torch.full(q.shape, float("nan"), dtype=out_dtype, device="cuda")
    scores = torch.from_numpy(old).cuda()
    ws = workspace_for(kvc, q, pools[0][0], tables, True)
    ws.fill_(0xff)
    call_decode(kvc, kind, q, pools, torch.from_numpy(tables).cuda(),
                torch.tensor(lens, dtype=torch.int32, device="cuda"), scale, out, scores, ws)
    torch.cuda.synchronize()
    assert kvc.get_error_flags() == 0
    vs = None if host[1][1] is None else host[1][1].numpy()
    tol, tol_scores = X.bounds(kind, qn, K, V, vs, tables, lens, scale, out_dtype, ref, old)
    worst = (np.abs(f64(out) - ref) / tol).max()
    assert worst <= 1, f"out: {worst:.2f} of the bound"
    worst = (np.abs(f64(scores) - ref_scores) / tol_scores).max()
    assert worst <= 1, f"scores: {worst:.2f} of the bound"
    # all the weight of a call: one per query, each within the bound of a weight
    G = Hq // H
    for i, n in enumerate(lens):
        base = np.where(np.arange(n) < n - T, old[i, :, :n], 0)
        total = (f64(scores)[i, :, :n] - base).sum(-1)
        assert np.all(np.abs(total - T * G) <= tol_scores[i, :, :n].sum(-1))


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("q_dtype", [torch.bfloat16, torch.float16])
def test_far_apart_block_scales_that_contribute_alike(kvc, code, q_dtype):
    # V scales from 1 down to e^-27 (2^-39), and weights the other way round: every block brings about as much, so
    # that each has to keep its precision
    H, G, D, bs, n = 2, 4, 128, 16, 16 * 28
    rng = np.random.default_rng(17)
    tables = rng.permutation(28).astype(np.int32)[None]
    k, v = np.zeros((28, H, bs, D)), np.zeros((28, H, bs, D))
    vs = np.zeros((28, H), dtype=np.float32)
    order = rng.permutation(28)
    for j in range(28):
        b = tables[0, j]
        k[b, :, :, 0], k[b, :, :, 1] = order[j] // 2, order[j] - order[j] // 2  # codes up to 14: exact in e4m3
        v[b] = rng.integers(1, 8, (H, bs, D))
        vs[b] = np.exp(-float(order[j]))
    qn = np.zeros((1, 1, H * G, D))
    qn[..., :2] = 1
    codes = []
    for x in (k, v):
        t = torch.from_numpy(x)
        codes.append(t.to(torch.int8) if code == "int8" else t.float().to(torch.float8_e4m3fn).view(torch.uint8))
    ones = np.ones((28, H), dtype=np.float32)
    K, V = O.dequantized(codes[0].numpy(), ones), O.dequantized(codes[1].numpy(), vs)
    assert np.array_equal(K, k) and np.array_equal(V, v * vs.astype(np.float64)[:, :, None, None])
    ref, _ = O.decode_scored(qn, K, V, tables, [n], 1.0)
    q = torch.from_numpy(qn).to(q_dtype).cuda()
    for per in (0, 1000):
        kvc.set_option(kvc.OPT_BLOCKS_PER_CTA, per)
        out = torch.empty(q.shape, device="cuda")
        kvc.decode_attention_block8(q, codes[0].cuda(), codes[1].cuda(), torch.from_numpy(ones).cuda(),
                                    torch.from_numpy(vs).cuda(), torch.from_numpy(tables).cuda(),
                                    torch.tensor([n], dtype=torch.int32, device="cuda"), 1.0, out,
                                    workspace_for(kvc, q, codes[0].cuda(), tables, False))
        # Every value is positive, so errors stay relative to the output. A weight: x of up to 39 with 2^-24 of it
        # three times over, the logarithm of the scale 2^-22 and 2^-24 of 40 twice, exp2 2^-22, its parts 2^-21, and
        # the same for the denominator. The sums: 2 products per 16 rows of 17 terms, each cut at 2^-23.
        rel = 2 * (0.7 * (3 * 39 + 4 + 2 * 40) * X.U + 4 * X.U + 8 * X.U) + (2 * 17 * n / 16 + 128) * 2 * X.U
        err = (np.abs(f64(out) - ref) / ref).max()
        assert err <= rel <= 2e-4, f"{err:.2e} (bound {rel:.2e})"
