"""GPU parity: decode with a window and sinks over 16-bit caches (kvc_decode_attention_sinks) and over four-bit ones
(kvc_decode_attention_fp4)."""

import numpy as np
import pytest
import torch

from stream_helpers import Decode, int32

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "f16", "fp4"]

# rows, new tokens, query heads, kv heads, D, block size, window, sinks
CASES = [
    ([1, 2, 15, 16, 17, 33], 1, 4, 1, 128, 16, None, 0),
    ([1, 100, 303], 1, 8, 2, 128, 16, 1, 0),
    ([1, 5, 6, 7, 100, 303], 1, 8, 2, 128, 16, 5, 1),
    ([40, 700, 64, 255, 256, 257], 1, 16, 4, 64, 16, 255, 4),
    ([700, 31], 1, 3, 3, 64, 32, 64, 16),
    ([1000, 130], 1, 20, 1, 256, 48, 200, 33),
    ([900, 57], 1, 4, 1, 256, 16, None, 0),
    ([9, 150, 400], 5, 6, 2, 128, 16, 20, 3),
    ([9, 150, 400], 5, 6, 2, 128, 16, 3, 7),
    ([40, 260], 33, 4, 2, 64, 80, 16, 100),
    ([120, 300], 3, 3, 1, 256, 16, 50, 1),
    ([300, 5000, 1100], 4, 28, 4, 128, 32, 1000, 21),
    ([260, 256], 256, 2, 1, 64, 16, 100, 9),
    ([2100], 1, 4, 1, 128, 16, None, 7),
    ([500] * 40, 1, 4, 2, 128, 128, 77, 4),
    ([64, 33], 2, 4, 1, 128, 64, 1, 64),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_decode_matches_the_oracle(kvc, case, kind):
    *sizes, window, sinks = case
    d = Decode(*sizes, kind, window, sinks, seed=sizes[0][0])
    d.run(kvc)
    d.check()
    assert kvc.get_error_flags() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("out", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("per", [0, 1, 1000])
def test_types_and_splits(kvc, kind, out, per):
    """Every split of the work, from a warp per block to one for all."""
    kvc.set_option(kvc.OPT_BLOCKS_PER_CTA, per)
    try:
        for T in (1, 2):
            d = Decode([700, 90, 1], T if T == 1 else 1, 8, 2, 128, 16, kind, 300, 20, seed=5, q_dtype="f16", out_dtype=out)
            d.run(kvc)
            d.check()
    finally:
        kvc.set_option(kvc.OPT_BLOCKS_PER_CTA, 0)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_a_window_without_sinks_is_the_window_decode(kvc, kind):
    d = Decode([700, 90, 30], 1, 8, 2, 128, 16, kind, 100, 0, seed=6, garbage=False)
    d.run(kvc)
    d.check()
    out = torch.zeros((3, 8, 128), device="cuda")
    kvc.decode_attention_window(d.q[:, 0].contiguous(), d.pools[0][0], d.pools[1][0],
                                torch.from_numpy(d.tables).cuda(), int32(d.lens), d.scale, 100, out,
                                kvc.new_decode_workspace(3, 8, 2, 128, 16, d.tables.shape[1]))
    # two results of one value: the other decode keeps its weights to 2^-17
    assert (out - d.out[:, 0]).abs().max() <= 5 * 2.0 ** -16


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("T,window,sinks", [(1, 40, 3), (5, 40, 3), (5, 2, 0), (5, None, 0)])
@pytest.mark.parametrize("per", [0, 1000])
def test_values_that_are_not_finite_stay_with_those_who_see_them(kvc, kind, value, T, window, sinks, per):
    kvc.set_option(kvc.OPT_BLOCKS_PER_CTA, per)
    try:
        d = Decode([140, 200], T, 4, 2, 128, 16, kind, window, sinks, seed=6)
        # around the sinks' end, the window's start and the newest rows
        for i, r, dim in ((0, 2, 5), (0, 99, 7), (0, 102, 9), (0, 137, 64), (0, 139, 65), (1, 158, 1), (1, 198, 100)):
            b, o = int(d.tables[i, r // 16]), r % 16
            if b >= len(d.pools[1][1]) or np.isnan(d.pools[1][1][b, 0, o, 0]):
                continue
            d.pools[1][0][b, :, o, dim] = value
            d.pools[1][1][b, :, o, dim] = value
        d.run(kvc)
        d.check()
    finally:
        kvc.set_option(kvc.OPT_BLOCKS_PER_CTA, 0)


@pytest.mark.parametrize("kind", KINDS)
def test_invalid_lengths_and_bad_blocks(kvc, kind):
    d = Decode([40, 3, 90], 4, 8, 2, 128, 16, kind, 20, 3, seed=7, garbage=False)
    d.run(kvc)
    assert kvc.get_error_flags() == kvc.FLAG_BAD_LEN
    assert (d.out[1] == 0).all()
    d.check(skip=[1])
    d.lens = [40, 20, 97]
    d.tables[1, 0], d.tables[2, 0] = -1, 1 << 27
    d.run(kvc)
    assert kvc.get_error_flags() & kvc.FLAG_BAD_BLOCK
    d.lens[2] = 96
    d.run(kvc)
    kvc.get_error_flags()
    d.check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("garbage", [0, 255])
def test_a_workspace_holds_nothing_between_calls(kvc, kind, garbage):
    a = Decode([3000, 40], 1, 8, 2, 128, 16, kind, 1000, 4, seed=8)
    b = Decode([90, 500], 3, 8, 2, 128, 16, kind, None, 0, seed=9)
    ws = torch.full((max(a.workspace(kvc).numel(), b.workspace(kvc).numel()),), garbage, dtype=torch.uint8, device="cuda")
    first = [a.run(kvc, ws).clone(), b.run(kvc, ws).clone()]
    for _ in range(3):
        assert torch.equal(a.run(kvc, ws), first[0]) and torch.equal(b.run(kvc, ws), first[1])
    a.check()
    b.check()


@pytest.mark.parametrize("kind", KINDS)
def test_captured_and_on_other_streams(kvc, kind):
    d = Decode([140, 700], 1, 8, 2, 128, 16, kind, None, 5, seed=10)
    tables, lens, ws = torch.from_numpy(d.tables).cuda(), int32(d.lens), d.workspace(kvc)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    d.call(kvc, tables, lens, ws, side)
    side.synchronize()
    d.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.call(kvc, tables, lens, ws)
    for n in ([140, 700], [3, 699], [77, 1]):
        d.lens = n
        lens.copy_(int32(n))
        graph.replay()
        torch.cuda.synchronize()
        d.check()


@pytest.mark.parametrize("kind", KINDS)
def test_lengths_written_by_the_kernel_before(kvc, kind):
    d = Decode([140, 700, 33], 1, 8, 2, 128, 16, kind, 90, 5, seed=11)
    tables, lens, ws = torch.from_numpy(d.tables).cuda(), int32(d.lens), d.workspace(kvc)
    torch.cuda.synchronize()
    for _ in range(3):
        lens.sub_(1)
        lens.add_(1)
        d.call(kvc, tables, lens, ws)
    torch.cuda.synchronize()
    d.check()


def test_the_freed_middle_of_a_stream(kvc):
    """Blocks between the sinks and the window go back to the pool and are used by another sequence."""
    window, sinks, bs = 64, 4, 16
    d = Decode([400], 1, 4, 1, 128, bs, "bf16", window, sinks, seed=12, garbage=False)
    first = -(-sinks // bs)
    last = (400 - window) // bs
    for b in d.tables[0, first:last]:
        for t, _ in d.pools:
            t[int(b)] = float("nan")
    d.tables[0, first:last] = -1
    d.run(kvc)
    assert kvc.get_error_flags() == 0
    d.check()
