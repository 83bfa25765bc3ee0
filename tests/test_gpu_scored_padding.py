"""Scored decode with an odd number of queries per kv head: the column that pads it takes no part in the scores, also
where a cached key is not finite."""

import numpy as np
import pytest
import torch

from oracle import long_context as O

from long_context_helpers import bounds, call_decode, f64, workspace_for
from test_gpu_scored import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("T,Hq,H", [(1, 2, 2), (1, 3, 1), (3, 2, 2), (1, 8, 2)])
def test_rows_of_weight_zero_add_nothing(kvc, kind, T, Hq, H):
    # keys of -inf in a dim where every query is positive: the rows' scaled scores are -inf, their weights 0
    lens, D, bs, scale = [70, 33], 64, 16, 0.1
    q, pools, tables, scores = make(kind, lens, T, Hq, H, D, bs, seed=71)
    q[..., 5] = q[..., 5].abs() + 0.5
    K = pools[0][2].copy()
    for i, rows in enumerate(([4, 40, 41], [0, 17])):
        for r in rows:
            b = int(tables[i, r // bs])
            pools[0][0][b, :, r % bs, 5] = float("-inf")
            K[b, :, r % bs, 5] = -np.inf
    before = f64(scores)
    with np.errstate(invalid="ignore"):
        ref, ref_scores = O.decode_scored(f64(q), K, pools[1][2], tables, lens, scale, before)
    assert np.isfinite(ref).all() and np.isfinite(ref_scores).all()
    out = torch.empty(q.shape, device="cuda")
    call_decode(kvc, kind, q, pools, torch.from_numpy(tables).cuda(),
                torch.tensor(lens, dtype=torch.int32, device="cuda"), scale, out, scores,
                workspace_for(kvc, q, pools[0][0], tables, True))
    torch.cuda.synchronize()
    tol, tol_scores = bounds(f64(q), pools[0][2], pools[1][2], tables, lens, scale, out.dtype, ref, ref_scores)
    assert np.all(np.abs(f64(out) - ref) <= tol)
    assert np.all(np.abs(f64(scores) - ref_scores) <= tol_scores)
    for i, rows in enumerate(([4, 40, 41], [0, 17])):
        for r in rows:  # exactly: the old score, or 0 for the call's own rows
            want = before[i, :, r] if r < lens[i] - T else 0
            assert np.array_equal(f64(scores)[i, :, r], want + 0 * before[i, :, r])
