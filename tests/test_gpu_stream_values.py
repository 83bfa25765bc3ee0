"""GPU parity: what values and scores at the ends of their types give in decode with a window and sinks and in its
relatives."""

import pytest
import torch

from stream_helpers import Decode, int32

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


@pytest.mark.parametrize("score", [-1e10, 1e12, -1e29, -1e31, -3e38, 3e38])
@pytest.mark.parametrize("op", ["sinks", "fp4", "prompt"])
def test_scores_of_any_size(kvc, op, score, split):
    """All scores alike and far from 0, none of them exact in fp32 once scaled: equal weights, also where a sequence is done
    in parts."""
    q, k, v, tables, lens = one_sequence(3000, 8, 2, 64)
    q[..., 0] = abs(score) / 2 ** 10  # (the product of 3e38 is rounded to within bf16's range)
    k[..., 0] = 1.0 if score > 0 else -1.0
    v[...] = 2.0
    v[:, :, ::2] = 1.0
    out = torch.full((1, 8, 64), 7.0, device="cuda")
    args = (tables, lens, 2.0 ** 10 / 1.4426950408889634 * 0.9837)  # scores in log2 units within fp32
    if op == "prompt":
        out = torch.full((1, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        ws = kvc.new_prompt_workspace(1, 1, 8, 2, 64, 16, tables.shape[1])
        kvc.prompt_attention(q, k, v, tables, int32([0, 1]), *args[1:], out, ws, window=2000, sinks=40)
    else:
        ws = kvc.new_scored_workspace(1, 1, 8, 2, 64, 16, tables.shape[1], scored=False)
        if op == "sinks":
            kvc.decode_attention_sinks(q, k, v, *args, 2000, 40, out, ws)
        else:
            codes = [torch.zeros((*k.shape[:3], 32), dtype=torch.uint8, device="cuda") for _ in range(2)]
            scales = [torch.zeros((*k.shape[:3], 4), dtype=torch.uint8, device="cuda") for _ in range(2)]
            slots = torch.arange(k.shape[0] * 16, device="cuda")
            kvc.append_fp4(*(x.transpose(1, 2).reshape(-1, 2, 64).contiguous() for x in (k, v)), slots, *codes, *scales)
            kvc.decode_attention_fp4(q, *codes, *scales, *args, out, ws, window=2000, sinks=40)
    assert kvc.get_error_flags() == 0
    # half of the 2040 rows hold 1 (a step of 0.125 in e4m3 x 6: 1.03), half 2: within 2^-4 of 1.5, the scales' rounding
    assert (out.float() / 1.5 - 1).abs().max() <= (2.0 ** -4 if op == "fp4" else 2.0 ** -8)


@pytest.mark.parametrize("kind", ["bf16", "f16", "fp4"])
@pytest.mark.parametrize("out", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T", [2, 3, 17])
def test_types_and_splits_of_several_tokens(kvc, kind, out, T, split):
    """A 16-bit output, several new tokens and a sequence that has no others, in every way of splitting the work."""
    d = Decode([700, 90, T], T, 8, 2, 128, 16, kind, 300, 20, seed=50 + T, q_dtype="f16", out_dtype=out)
    d.run(kvc)
    d.check()
    assert kvc.get_error_flags() == 0
