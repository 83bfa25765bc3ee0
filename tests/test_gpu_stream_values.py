"""GPU parity: what values and scores at the ends of their types give in decode with a window and sinks and in its
relatives."""

import pytest
import torch

from stream_helpers import int32

pytestmark = pytest.mark.gpu


def one_sequence(n, Hq, H, D, dtype=torch.bfloat16):
    """Empty pools of n rows in order, their table, and queries that read the keys' first dim."""
    k, v = (torch.zeros((-(-n // 16), H, 16, D), dtype=dtype, device="cuda") for _ in range(2))
    q = torch.zeros((1, Hq, D), dtype=dtype, device="cuda")
    q[..., 0] = 1
    return q, k, v, torch.arange(len(k), dtype=torch.int32, device="cuda")[None].contiguous(), int32([n])


@pytest.fixture(params=[0, 1, 40])
def split(kvc, request):
    """Ways of splitting the work: as the library does, a warp per block, a warp for 40 blocks."""
    kvc.set_option(kvc.OPT_BLOCKS_PER_CTA, request.param)
    yield
    kvc.set_option(kvc.OPT_BLOCKS_PER_CTA, 0)


@pytest.mark.parametrize("odd", [None, float("inf"), float("nan")])
@pytest.mark.parametrize("op", ["sinks", "scored"])
def test_a_large_value_without_weight_adds_nothing(kvc, op, odd, split):
    """The first 640 rows' weights, of whole parts of the work, are 2^-202 of the others'; one row holds 1e38 in a dim, and
    an infinity in another."""
    q, k, v, tables, lens = one_sequence(3000, 8, 2, 64)
    k[..., 0] = 140.0
    k[:40, ..., 0] = 0.0
    v[...] = 1.0
    v[0, :, 0, 5] = 1e38
    if odd is not None:
        v[0, :, 3, 9] = odd
    out = torch.full((1, 8, 64), 7.0, device="cuda")
    ws = kvc.new_scored_workspace(1, 1, 8, 2, 64, 16, tables.shape[1], scored=op == "scored")
    if op == "sinks":
        kvc.decode_attention_sinks(q, k, v, tables, lens, 1.0, None, 0, out, ws)
    else:
        scores = torch.zeros((1, 2, 16 * tables.shape[1]), device="cuda")
        kvc.decode_attention_scored(q, k, v, tables, lens, 1.0, out, scores, ws)
    assert kvc.get_error_flags() == 0
    if odd is not None:
        x = out[..., 9].clone()
        assert x.isnan().all() if odd != odd else (x == odd).all()
        out[..., 9] = 1.0
    # 2360 equal weights over their sum: an fp32 division, products and sums of whole numbers
    assert (out - 1).abs().max() <= 2.0 ** -20
