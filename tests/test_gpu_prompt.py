"""GPU parity: prompt attention over the paged cache (kvc_prompt_attention)."""

import numpy as np
import pytest
import torch

from oracle import streams as O

from long_context_helpers import f64
from stream_helpers import Prompt, int32

pytestmark = pytest.mark.gpu

# new tokens, rows, query heads, kv heads, D, block size, window, sinks
CASES = [
    ([1], [1], 4, 1, 128, 16, None, 0),
    ([5, 16, 37, 0, 129], [5, 40, 100, 30, 300], 8, 2, 128, 16, None, 0),
    ([64, 65, 63, 256], [64, 65, 127, 257], 4, 1, 128, 16, None, 0),
    ([300], [300], 1, 1, 128, 16, None, 0),
    ([257, 130], [257, 400], 2, 2, 64, 32, None, 0),
    ([100, 1, 33], [400, 700, 129], 6, 2, 128, 48, None, 0),
    ([90, 41], [90, 1041], 7, 1, 64, 80, None, 0),
    ([40, 17], [200, 1500], 16, 2, 128, 128, None, 0),
    ([3, 2], [131, 260], 128, 1, 64, 16, None, 0),
    ([7], [300], 65, 1, 128, 16, None, 0),
    ([200, 50], [200, 333], 4, 1, 128, 16, 1, 0),
    ([200, 50], [200, 333], 4, 1, 128, 16, 5, 1),
    ([500, 77], [500, 900], 4, 2, 128, 16, 100, 4),
    ([300, 129], [700, 2000], 8, 2, 64, 64, 129, 130),
    ([130, 64], [1300, 500], 3, 1, 128, 32, 128, 256),
    ([520], [3000], 4, 1, 128, 96, 700, 21),
    ([260, 1], [260, 1000], 5, 1, 64, 112, 1000, 300),
    # many units: dealt out whole, sorted by cost
    ([200, 57, 0, 60], [200, 300, 7, 190], 512, 8, 64, 16, None, 0),
    ([9] * 50 + [1] * 30, [9] * 50 + [40] * 30, 64, 8, 128, 32, 20, 3),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_prompt_matches_the_oracle(kvc, case, dtype):
    *sizes, window, sinks = case
    p = Prompt(*sizes, dtype, window, sinks, seed=len(sizes[0]) + sizes[1][0])
    p.run(kvc)
    p.check()
    assert kvc.get_error_flags() == 0


def test_a_chunk_is_the_rest_of_its_prompt(kvc):
    """One call for the whole prompt and one for each chunk give the same rows, up to the rounding of each."""
    p = Prompt([700], [700], 8, 2, 128, 16, "f16", 200, 4, seed=3, garbage=False)
    p.run(kvc)
    whole = p.out.clone()
    tables = torch.from_numpy(p.tables).cuda()
    for a, b in ((0, 1), (1, 130), (130, 131), (131, 600), (600, 700)):
        out = torch.zeros((b - a, 8, 128), dtype=p.dtype, device="cuda")
        kvc.prompt_attention(p.q[a:b].contiguous(), p.pools[0][0], p.pools[1][0], tables, int32([0, b - a]),
                             int32([b]), p.scale, out, p.workspace(kvc), window=200, sinks=4)
        # two results of one value, each within 2^-11 of its weights' sum (p |v| below 4.5) and its own rounding
        assert (out.float() - whole[a:b].float()).abs().max() <= 2 * (2.0 ** -11 * 4.5 * 2)
    p.check()


@pytest.mark.parametrize("scale", [0.0, -0.09, 1e-9, 3.0])
def test_scales(kvc, scale):
    p = Prompt([150, 20], [150, 300], 4, 1, 128, 16, "bf16", None, 0, seed=9)
    p.scale = scale
    p.run(kvc)
    p.check()


def test_scores_that_grow_move_the_reference(kvc):
    """Keys of one sequence grow along it, so that the running maximum rises in every tile."""
    p = Prompt([400], [1600], 4, 1, 128, 16, "bf16", None, 0, seed=4, garbage=False)
    for r in range(1600):
        b, o = int(p.tables[0, r // 16]), r % 16
        for t, host in p.pools[:1]:
            t[b, :, o] *= 0.02 + 0.002 * r
            host[b, :, o] = f64(t[b, :, o])
    p.run(kvc)
    p.check()


@pytest.mark.parametrize("kind", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("window,sinks", [(None, 0), (40, 3)])
def test_values_that_are_not_finite_stay_with_those_who_see_them(kvc, kind, window, sinks):
    p = Prompt([140, 30], [140, 200], 4, 2, 128, 16, "bf16", window, sinks, seed=6)
    for i, r, d in ((0, 1, 5), (0, 77, 9), (0, 139, 64), (1, 180, 100), (1, 180, 7)):
        b, o = int(p.tables[i, r // 16]), r % 16
        if b >= len(p.pools[1][1]):
            continue
        p.pools[1][0][b, :, o, d] = kind
        p.pools[1][1][b, :, o, d] = kind
    p.run(kvc)
    p.check()


@pytest.mark.parametrize("sizes", [([300, 40], [300, 40], 512, 8, 64, 16), ([70], [9000], 8, 1, 128, 16),
                                   ([5, 9], [50, 90], 8, 2, 128, 16)])
def test_a_sequence_that_is_not_finite_throughout(kvc, sizes):
    """One value of a first row: every output of that dim, in whole units, split ones and a call without a plan."""
    p = Prompt(*sizes, "bf16", seed=16)
    b = int(p.tables[0, 0])
    p.pools[1][0][b, :, 0, 3] = float("inf")
    p.pools[1][1][b, :, 0, 3] = np.inf
    p.run(kvc)
    p.check()
    assert np.isinf(f64(p.out)[:p.new[0], :, 3]).all() and kvc.get_error_flags() == 0


def test_keys_that_are_not_finite_in_hidden_rows(kvc):
    p = Prompt([100], [100], 4, 1, 128, 16, "bf16", None, 0, seed=7)
    b, o = int(p.tables[0, 5]), 3  # row 83
    p.pools[0][0][b, :, o] = float("nan")
    p.run(kvc)
    out = f64(p.out)
    assert np.isfinite(out[:83]).all() and np.isnan(out[83:100]).all()


@pytest.mark.parametrize("sizes", [([70], [9000], 8, 1, 128, 16), ([100], [100], 4, 1, 128, 16)])
def test_queries_that_are_not_finite(kvc, sizes):
    p = Prompt(*sizes, "bf16", seed=21)
    p.q[5, 3, 7] = float("nan")
    p.q[9, 1, 0] = float("inf")
    p.run(kvc)
    out = f64(p.out)
    bad = np.zeros(out.shape[:2], bool)
    bad[5, 3] = bad[9, 1] = True
    assert np.isnan(out[bad]).all() and np.isfinite(out[~bad]).all() and kvc.get_error_flags() == 0


def test_invalid_lengths_and_starts(kvc):
    p = Prompt([20, 30, 10, 5], [20, 60, 10, 5], 4, 1, 128, 16, "bf16", seed=8, garbage=False)
    tables, _, _ = p.device()
    for rows, starts, zero, left in (
            ([20, 29, 10, 5], [0, 20, 50, 60, 65], [(20, 50)], []),  # fewer rows than new tokens
            ([20, 60, 4096, 5], [0, 20, 50, 60, 65], [(50, 60)], []),  # more than the table holds
            ([20, 60, 10, 5], [0, 20, 50, 60, 1000], [], [(60, 68)]),  # beyond q
            ([20, 60, 10, 5], [-4, 20, 50, 60, 65], [], [(0, 20)])):
        p.out.fill_(7.0)
        kvc.prompt_attention(p.q, p.pools[0][0], p.pools[1][0], tables, int32(starts), int32(rows), p.scale, p.out,
                             p.workspace(kvc))
        assert kvc.get_error_flags() & kvc.FLAG_BAD_LEN
        out = f64(p.out)
        for a, b in zero:
            assert (out[a:b] == 0).all()
        for a, b in left:
            assert (out[a:b] == 7.0).all()
        skip = [i for i in range(4) if any(a <= p.starts[i] < b for a, b in zero + left)]
        p.check(skip)


def test_blocks_outside_the_pool_get_no_weight(kvc):
    p = Prompt([200], [300], 4, 1, 128, 16, "bf16", seed=10, garbage=False)
    p.tables[0, [3, 18]] = [-1, 1 << 27]  # 18: rows 288 .. 299, of the last tokens themselves
    p.run(kvc)
    p.check()
    assert kvc.get_error_flags() & kvc.FLAG_BAD_BLOCK


def test_rows_of_bad_blocks_only_give_zeros(kvc):
    p = Prompt([16], [16], 4, 1, 128, 16, "bf16", seed=10, garbage=False)
    p.tables[0, 0] = -1
    p.run(kvc)
    assert (p.out[:16] == 0).all() and kvc.get_error_flags() & kvc.FLAG_BAD_BLOCK


def test_no_tokens(kvc):
    p = Prompt([0, 0], [5, 0], 4, 1, 128, 16, "bf16", pad=0)
    p.run(kvc)
    assert kvc.get_error_flags() == 0
    p = Prompt([0, 3, 0], [0, 3, 9], 4, 1, 128, 16, "bf16", pad=2, garbage=False)
    p.run(kvc)
    p.check()


@pytest.mark.parametrize("garbage", [0, 255])
def test_a_workspace_holds_nothing_between_calls(kvc, garbage):
    """Filled with anything, shared by calls of different shapes one behind the other, and the same bits each time."""
    a = Prompt([300, 40], [900, 2500], 8, 2, 128, 16, "bf16", seed=11)
    b = Prompt([600], [600], 8, 2, 128, 16, "bf16", 90, 5, seed=12)
    ws = torch.full((max(a.workspace(kvc).numel(), b.workspace(kvc).numel()),), garbage, dtype=torch.uint8, device="cuda")
    first = [a.run(kvc, ws).clone(), b.run(kvc, ws).clone()]
    for _ in range(3):
        assert torch.equal(a.run(kvc, ws), first[0]) and torch.equal(b.run(kvc, ws), first[1])
    a.check()
    b.check()


def test_captured_and_on_other_streams(kvc):
    p = Prompt([130, 9], [200, 700], 8, 2, 128, 16, "bf16", seed=13)
    tables, starts, rows = p.device()
    ws = p.workspace(kvc)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def call(stream=None):
        kvc.prompt_attention(p.q, p.pools[0][0], p.pools[1][0], tables, starts, rows, p.scale, p.out, ws,
                             stream=stream)

    call(side)
    side.synchronize()
    p.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new in ([130, 9], [30, 109], [0, 139]):  # lengths are read when the graph runs
        p.new, p.starts = new, [0, new[0], 139]
        starts.copy_(int32(p.starts))
        p.out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        p.check()


def test_inputs_written_by_the_kernel_before(kvc):
    p = Prompt([70, 300], [70, 400], 8, 2, 128, 16, "bf16", seed=14)
    tables, starts, rows = p.device()
    ws = p.workspace(kvc)
    late, q, t0 = rows - 3, torch.zeros_like(p.q), torch.zeros_like(tables)
    torch.cuda.synchronize()
    for last in range(3):
        late.copy_(rows - 3)
        q.zero_()
        t0.zero_()
        writes = [lambda: late.add_(3), lambda: q.add_(p.q), lambda: t0.add_(tables)]
        for w in writes[last + 1:] + writes[:last + 1]:
            w()
        kvc.prompt_attention(q, p.pools[0][0], p.pools[1][0], t0, starts, late, p.scale, p.out, ws)
    torch.cuda.synchronize()
    p.check()


def test_checked_mode_reports(kvc):
    p = Prompt([4], [4], 4, 1, 64, 16, "f16", garbage=False)
    kvc.set_option(kvc.OPT_CHECKED, 1)
    try:
        p.run(kvc)
        p.rows = [3]
        with pytest.raises(kvc.KvcError) as e:
            p.run(kvc)
        assert e.value.status == kvc.ERR_OUT_OF_RANGE
    finally:
        kvc.set_option(kvc.OPT_CHECKED, 0)


def test_blocks_far_up_a_large_pool(kvc):
    """Byte offsets beyond 32 bits."""
    p = Prompt([90, 20], [300, 20], 8, 8, 128, 16, "bf16", seed=17, garbage=False)
    nb = 150000
    small = [x[0] for x in p.pools]
    for x in p.pools:
        large = torch.empty((nb, *x[0].shape[1:]), dtype=x[0].dtype, device="cuda")
        large[nb - len(x[0]):] = x[0].flip(0)
        x[0] = large
    tables = p.tables
    p.tables = np.where(tables < (1 << 28), nb - 1 - tables, tables).astype(np.int32)
    p.run(kvc)
    p.tables = tables
    for x, t in zip(p.pools, small):
        x[0] = t
    p.check()
    assert kvc.get_error_flags() == 0


def test_two_streams_at_once(kvc):
    a = Prompt([300, 40], [900, 2500], 8, 2, 128, 16, "bf16", seed=18)
    b = Prompt([60], [300], 8, 2, 128, 16, "f16", 90, 5, seed=19)
    args = [(p, p.device(), p.workspace(kvc), torch.cuda.Stream()) for p in (a, b)]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, (tables, starts, rows), ws, stream in args:
            kvc.prompt_attention(p.q, p.pools[0][0], p.pools[1][0], tables, starts, rows, p.scale, p.out, ws,
                                 window=p.window, sinks=p.sinks, stream=stream)
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_fewer_ctas(kvc):
    """Any number of CTAs gives the same outputs up to the order of the sums, in every way of handing out units."""
    for sizes in (([300, 40], [300, 2500], 8, 2, 128, 16), ([200, 57], [200, 300], 512, 8, 64, 16),
                  ([5, 9], [50, 90], 8, 2, 128, 16)):
        p = Prompt(*sizes, "bf16", seed=20)
        for ctas in (1, 2, 7, 100):
            kvc.set_option(kvc.OPT_MAX_CTAS, ctas)
            try:
                p.run(kvc)
            finally:
                kvc.set_option(kvc.OPT_MAX_CTAS, 0)
            p.check()
