"""A scored decode in pieces, as a caller with little scratch memory makes it: the sequences of a batch over several calls,
or the tokens of a window, with one workspace of a piece's size. Scores and outputs are those of the whole."""

import numpy as np
import pytest
import torch

from oracle import long_context as O

import scored_exact_helpers as X
from long_context_helpers import call_decode, f64, workspace_for

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3", "int8"])
def test_sequences_and_tokens_in_pieces(kvc, kind):
    case = ([200, 33, 500, 78, 64], 24, 6, 2, 128, 16, 2.0 ** -5)
    lens, T, Hq, H, D, bs, scale = case
    qn, host, tables, old = X.inputs(kind, case)
    ref, ref_scores = O.decode_scored(qn, host[0][2], host[1][2], tables, lens, scale, old)
    vs = None if host[1][1] is None else host[1][1].numpy()
    tol, tol_scores = X.bounds(kind, qn, host[0][2], host[1][2], vs, tables, lens, scale, torch.float32, ref, old)
    pools = [(t.cuda(), None if s is None else s.cuda(), x) for t, s, x in host]
    q = torch.from_numpy(qn).to(torch.float16 if kind == "f16" else torch.bfloat16).cuda()
    t = torch.from_numpy(tables).cuda()
    out, scores = torch.empty(q.shape, device="cuda"), torch.from_numpy(old).cuda()
    step = 7
    sizes = [kvc.scored_workspace_size(2, step, Hq, H, D, bs, t.shape[1]),
             kvc.scored_workspace_size(len(lens), T, Hq, H, D, bs, t.shape[1])]
    ws = workspace_for(kvc, q[:2, :step], pools[0][0], t, True)
    for a in range(0, len(lens), 2):
        b = min(len(lens), a + 2)
        for t0 in range(0, T, step):
            t1 = min(T, t0 + step)
            # the tokens t0 .. t1 - 1 are the newest rows of the sequences' first n - T + t1
            n = torch.tensor([m - T + t1 for m in lens[a:b]], dtype=torch.int32, device="cuda")
            part = torch.empty((b - a, t1 - t0, Hq, D), device="cuda")
            call_decode(kvc, kind, q[a:b, t0:t1].contiguous(), pools, t[a:b], n, scale, part, scores[a:b], ws)
            out[a:b, t0:t1] = part
    torch.cuda.synchronize()
    assert kvc.get_error_flags() == 0
    assert np.all(np.abs(f64(out) - ref) <= tol)
    # every piece rounds the sum once more
    assert np.all(np.abs(f64(scores) - ref_scores) <= tol_scores + 8 * X.U * np.abs(ref_scores))
    assert sizes[0] < sizes[1]
