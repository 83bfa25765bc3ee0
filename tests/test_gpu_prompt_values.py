"""GPU parity: what values at the ends of their type, infinities and NaN give in prompt attention."""

import pytest
import torch

from stream_helpers import int32

pytestmark = pytest.mark.gpu


def call(kvc, q, k, v, starts, rows, scale=1.0, window=None, sinks=0, tables=None):
    """Attention of the tokens q over pools whose blocks lie in order, from sequence to sequence."""
    nb, H, bs, D = k.shape
    if tables is None:
        need = [-(-n // bs) for n in rows]
        tables = torch.zeros((len(rows), max(need)), dtype=torch.int32)
        for i, n in enumerate(need):
            tables[i, :n] = torch.arange(sum(need[:i]), sum(need[:i]) + n)
    tables = tables.cuda()
    out = torch.full_like(q, 7.0)
    ws = kvc.new_prompt_workspace(len(rows), len(q), q.shape[1], H, D, bs, tables.shape[1])
    kvc.prompt_attention(q, k, v, tables, int32(starts), int32(rows), scale, out, ws, window=window, sinks=sinks)
    torch.cuda.synchronize()
    return out.float()


@pytest.mark.parametrize("rows", [20, 3000])
@pytest.mark.parametrize("later", [False, True])
def test_finite_dims_do_not_change_beside_an_infinity(kvc, rows, later):
    """A row of weight 2^-202 holds 1e38 in one dim, which is nothing; its weight is small from the start, or becomes so
    when later rows' scores are larger. All else is 1, and so are the outputs; an infinity in another dim changes
    that dim alone."""
    D = 64
    k, v = (torch.zeros((-(-rows // 16), 1, 16, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros((1, 1, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    if later:
        k[..., 0] = 140.0
        k[0, 0, :5, 0] = 0.0
    else:
        k[0, 0, 0, 0] = -140.0
    v[...] = 1.0
    v[0, 0, 0, 5] = 1e38
    for odd in (None, float("inf"), float("nan")):
        if odd is not None:
            v[0, 0, 3, 9] = odd
        out = call(kvc, q, k, v, [0, 1], [rows])[0, 0]
        assert (out[:9] == 1.0).all() and (out[10:] == 1.0).all()
        assert out[9].isnan() if odd != odd else out[9] == (1.0 if odd is None else odd)
