"""GPU parity: decode with a window and sinks over 16-bit caches (kvc_decode_attention_sinks) and over four-bit ones
(kvc_decode_attention_fp4)."""

import numpy as np
import pytest
import torch

from oracle import streams as O

from long_context_helpers import f64
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


@pytest.mark.parametrize("kind", KINDS)
def test_blocks_far_up_a_large_pool(kvc, kind):
    """Byte offsets beyond 32 bits, in the codes, the scales and the rows."""
    d = Decode([200, 33], 1, 8, 8, 128, 16, kind, 60, 4, seed=13, garbage=False)
    nb = 700000 if kind == "fp4" else 150000
    move = torch.from_numpy(np.unique(d.tables[d.tables < len(d.pools[0][1])]).astype(np.int64)).cuda()
    far = nb - 1 - move
    before = [p[0] for p in d.pools]
    for i, p in enumerate(d.pools):
        parts = p[0] if kind == "fp4" else (p[0],)
        large = [torch.empty((nb, *t.shape[1:]), dtype=t.dtype, device="cuda") for t in parts]
        for t, x in zip(parts, large):
            x[far] = t[move]
        p[0] = tuple(large) if kind == "fp4" else large[0]
    tables = torch.from_numpy(np.where(d.tables < (1 << 28), nb - 1 - d.tables, d.tables).astype(np.int32)).cuda()
    d.call(kvc, tables, int32(d.lens), d.workspace(kvc))
    torch.cuda.synchronize()
    for p, t in zip(d.pools, before):
        p[0] = t
    d.check()
    assert kvc.get_error_flags() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_two_streams_at_once(kvc, kind):
    a = Decode([700, 300], 1, 8, 2, 128, 16, kind, 200, 4, seed=14)
    b = Decode([90, 1500], 1, 8, 2, 128, 16, kind, None, 0, seed=15)
    args = [(d, torch.from_numpy(d.tables).cuda(), int32(d.lens), d.workspace(kvc), torch.cuda.Stream()) for d in (a, b)]
    torch.cuda.synchronize()
    for _ in range(20):
        for d, tables, lens, ws, stream in args:
            d.call(kvc, tables, lens, ws, stream)
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_many_sequences(kvc):
    """Prefix sums in shared memory, up to the largest batch of a four-bit cache."""
    for kind, n in (("bf16", 4096), ("fp4", 2048)):
        lens = [1 + (7 * i) % 37 for i in range(n)]
        d = Decode(lens, 1, 1, 1, 64, 16, kind, 20, 2, seed=16, garbage=False)
        d.run(kvc)
        d.check(skip=set(range(n)) - set(range(0, n, 41)))
        assert torch.isfinite(d.out).all() and (d.out != 7.0).any(-1).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("depth", [3, 6, 12, 16.5])  # e^-16.5: 2^-24 of the sink's weight
@pytest.mark.parametrize("n,window,per", [(864, None, 0), (864, 300, 1000), (2100, 2000, 1000), (300, 17, 0)])
def test_small_weights_beside_a_sink_keep_their_precision(kvc, kind, depth, n, window, per):
    """The first row takes nearly all the weight and brings nothing; the outputs are made of the others' weights."""
    H, G, D, bs = 2, 4, 128, 16
    rng = np.random.default_rng(int(depth))
    nb = -(-n // bs)
    tables = rng.permutation(nb).astype(np.int32)[None]
    k, v = np.zeros((nb, H, bs, D)), np.zeros((nb, H, bs, D))
    at = tables[0, np.arange(n) // bs], np.arange(n) % bs
    k[at[0], :, at[1], 0] = -depth
    v[at[0], :, at[1]] = rng.choice([1.0, 2.0, 3.0, 4.0, 6.0], (n, H, D))
    v[at[0], :, at[1], ::16] = 6.0  # a group's scale is then 1
    k[tables[0, 0], :, 0] = v[tables[0, 0], :, 0] = 0
    d = Decode([n], 1, H * G, H, D, bs, kind, window, 1, garbage=False)
    if kind == "fp4":
        caches = []
        for x in (k, v):
            c, s = O.encode_fp4(x)  # exact: -6 * (depth / 6), and codes of scale 1
            assert np.array_equal(O.values_fp4(O.pack(c), s), x)
            caches.append([(torch.from_numpy(O.pack(c)).cuda(), torch.from_numpy(s).cuda()), x])
        d.pools = caches
    else:
        d.pools = [[torch.from_numpy(x).to(d.q.dtype).cuda(), x] for x in (k, v)]
    d.tables, d.scale = tables, 1.0
    d.q.zero_()
    d.q[..., 0] = 1
    kvc.set_option(kvc.OPT_BLOCKS_PER_CTA, per)
    try:
        d.run(kvc)
    finally:
        kvc.set_option(kvc.OPT_BLOCKS_PER_CTA, 0)
    ref, _, _ = O.attend(f64(d.q[0]), k, v, tables[0], n, 1.0, window, 1)
    # scores are whole numbers but for the factor log2(e) and its product, 2^-24 of at most 24 each, which moves a weight
    # by 24 * 2^-23 * ln 2; exp2 2^-22; the parts 2^-21; all values are positive, so errors stay relative to the output:
    # 3 products of 17 terms per 16 rows, each off by 2^-23 of the sum, and 64 joins
    rel = 24 * 2.0 ** -23 * 0.7 * 2 + 2.0 ** -20 + (3 * 17 * (n / 16 + 1) + 64) * 2.0 ** -23
    assert (np.abs(f64(d.out[0]) - ref) / ref).max() <= rel
