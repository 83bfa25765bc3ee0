"""GPU parity: what values at the ends of their type, infinities and NaN give in prompt attention."""

import numpy as np
import pytest
import torch

from stream_helpers import Prompt, int32

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


def plant(p, i, r, h, d, x):
    """x into dim d of row r of sequence i's values, unless the row's block is one that nobody sees."""
    b, o = int(p.tables[i, r // p.bs]), r % p.bs
    if 0 <= b < len(p.pools[1][1]):
        p.pools[1][0][b, h, o, d] = x
        p.pools[1][1][b, h, o, d] = x


# new tokens, rows, query heads, kv heads, D, block size, window, sinks
CASES = [
    ([300], [300], 1, 1, 64, 16, None, 0),            # 256 tokens per unit
    ([256, 129], [700, 129], 2, 2, 128, 48, None, 0),
    ([256, 100], [300, 600], 1, 1, 128, 16, 1, 0),    # windows shorter than a unit
    ([256, 200], [512, 900], 1, 1, 64, 32, 30, 5),
    ([200, 77], [500, 900], 4, 2, 128, 16, 100, 140),
    ([130, 64], [1300, 500], 3, 1, 128, 32, 128, 256),
    ([70], [5000], 8, 1, 128, 16, None, 0),           # units in parts
    ([40, 100], [3000, 4000], 8, 2, 64, 16, 2500, 30),
    ([200, 57, 0, 60], [200, 300, 7, 190], 512, 8, 64, 16, None, 0),  # many units, dealt out whole
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("ctas", [0, 1, 7])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_infinities_and_nan_anywhere(kvc, case, ctas, dtype):
    """In rows that all see, on the causal border, in those that leave the window and in hidden ones; several in one dim."""
    *sizes, window, sinks = case
    p = Prompt(*sizes, dtype, window, sinks, seed=30, garbage=case != CASES[-1])
    rng = np.random.default_rng(31)
    kinds = [np.inf, -np.inf, np.nan]
    for i, (m, n) in enumerate(zip(p.new, p.rows)):
        if m == 0:
            continue
        low = max(0, n - m + 1 - (window or n))
        at = list(rng.integers(max(0, n - m - 3), n, 12)) + list(rng.integers(low, min(n, low + 40), 8))
        for r in at + list(rng.integers(0, n, 12)) + list(rng.integers(0, min(n, sinks + 2), 2)):
            plant(p, i, int(r), int(rng.integers(p.H)), int(rng.integers(p.D)), kinds[rng.integers(3)])
        for r, x in ((n - 1, np.inf), (n - m, -np.inf), (max(0, n - m - 1), np.inf)):  # both signs in one dim
            plant(p, i, r, 0, 11, x)
    kvc.set_option(kvc.OPT_MAX_CTAS, ctas)
    try:
        p.run(kvc)
    finally:
        kvc.set_option(kvc.OPT_MAX_CTAS, 0)
    p.check()
    assert kvc.get_error_flags() == 0


@pytest.mark.parametrize("sizes", [([300, 40], [300, 900], 4, 2, 128, 16), ([70], [5000], 8, 1, 64, 16)])
@pytest.mark.parametrize("window,sinks", [(None, 0), (37, 3)])
def test_every_value_nan(kvc, sizes, window, sinks):
    p = Prompt(*sizes, "bf16", window, sinks, seed=32)
    p.pools[1][0].fill_(float("nan"))
    p.run(kvc)
    out, n = p.out.float(), p.starts[-1]
    assert out[:n].isnan().all() and (out[n:] == 7.0).all() and kvc.get_error_flags() == 0


@pytest.mark.parametrize("rows", [300, 5000])
def test_values_near_the_end_of_bf16(kvc, rows):
    """Scores that rise by 2^7 along the sequence: weights against an early reference, times 2e38, leave fp32; the
    output, 2e38 to a part in 2^7 (the first row's weight), does not."""
    D = 128
    k, v = (torch.zeros((-(-rows // 16), 1, 16, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros((3, 2, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    k[..., 0] = -1000.0
    k[0, 0, 0, 0] = 0.0
    k[200 // 16, 0, 200 % 16, 0] = 7.0  # (scale log 2)
    v[200 // 16, 0, 200 % 16] = 2e38
    v[0, 0, 0] = -1e38
    out = call(kvc, q, k, v, [0, 3], [rows], scale=float(np.log(2)))
    want = (128 * float(v[200 // 16, 0, 200 % 16, 0]) + float(v[0, 0, 0, 0])) / 129
    assert (out / want - 1).abs().max() <= 2.0 ** -7 and kvc.get_error_flags() == 0


def test_a_single_cta_with_long_rows_finishes(kvc):
    """Every output row of three units with 120,000 rows behind them is infinite in one dim: nobody waits so long for
    another warp that its bounded wait runs out."""
    n, G, D = 120000, 32, 128
    gen = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn((3 * n // 16, 1, 16, D), generator=gen, device="cuda").to(torch.bfloat16)
    v = torch.ones_like(k)
    q = torch.randn((12, G, D), generator=gen, device="cuda").to(torch.bfloat16)
    for i in range(3):
        v[i * n // 16, 0, 0, 3] = float("inf")
    kvc.set_option(kvc.OPT_MAX_CTAS, 1)
    try:
        out = call(kvc, q, k, v, [0, 4, 8, 12], [n] * 3, scale=D ** -0.5)
    finally:
        kvc.set_option(kvc.OPT_MAX_CTAS, 0)
    assert kvc.get_error_flags() == 0
    assert (out[..., 3] == float("inf")).all()
    out[..., 3] = 1.0
    # weights of half a bf16 step, their sum unrounded, and the output's own rounding
    assert (out - 1).abs().max() <= 2.0 ** -7


@pytest.mark.parametrize("new,rows,Hq,H", [(2048, 2048, 32, 8), (70, 9000, 8, 1)])
def test_an_infinity_costs_a_second_pass(kvc, new, rows, Hq, H):
    """One infinity in the first row: all outputs of its kv head are done again. That is a second pass over the same
    tiles with their values looked through (about 3 times the finite call), not one warp per output row (700 times)."""
    D = 128
    gen = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((-(-rows // 16), H, 16, D), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((new, Hq, D), generator=gen, device="cuda").to(torch.bfloat16)
    out = torch.zeros_like(q)
    tables = torch.arange(len(k), dtype=torch.int32, device="cuda")[None].contiguous()
    ws = kvc.new_prompt_workspace(1, new, Hq, H, D, 16, len(k))
    starts, lens = int32([0, new]), int32([rows])

    def time(n):
        events = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        for e in events:
            e.record()
            for _ in range(n if e is events[0] else 0):
                kvc.prompt_attention(q, k, v, tables, starts, lens, D ** -0.5, out, ws)
        torch.cuda.synchronize()
        return events[0].elapsed_time(events[1]) / n

    time(3)
    finite = time(20)
    v[0, :, 0, 3] = float("inf")
    assert min(time(3), time(3)) < 20 * finite
    assert (out[..., 3].float() == float("inf")).all() and kvc.get_error_flags() == 0
    out[..., 3] = 0
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("sizes", [([300, 40], [300, 900], 4, 2, 128, 16), ([70, 9], [5000, 30], 8, 1, 64, 16),
                                   ([5, 9], [50, 90], 8, 2, 128, 16)])
@pytest.mark.parametrize("garbage", [0, 255])
def test_infinities_that_come_and_go_between_replays(kvc, sizes, garbage):
    """One captured call, its workspace full of anything: whether a row is done again is decided when the graph runs."""
    p = Prompt(*sizes, "bf16", 90, 5, seed=34)
    tables, starts, rows = p.device()
    ws = torch.full_like(p.workspace(kvc), garbage)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvc.prompt_attention(p.q, p.pools[0][0], p.pools[1][0], tables, starts, rows, p.scale, p.out, ws, window=90,
                             sinks=5)
    dev, host = p.pools[1][0].clone(), p.pools[1][1].copy()
    for r in (None, 0, sizes[1][0] - 3, None, sizes[1][0] - 40):
        p.pools[1][0].copy_(dev)
        p.pools[1][1] = host.copy()
        if r is not None:
            plant(p, 0, r, 0, 17, np.inf)
        p.out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        p.check()
    assert kvc.get_error_flags() == 0


def test_two_streams_with_infinities(kvc):
    """Calls that are done again, side by side, give the same bits every time."""
    a = Prompt([300, 40], [900, 2500], 8, 2, 128, 16, "bf16", seed=35)
    b = Prompt([60], [300], 8, 2, 128, 16, "f16", 90, 5, seed=36)
    for p in (a, b):
        for r, x in ((1, np.inf), (p.rows[0] - 20, np.nan), (p.rows[0] - 70, -np.inf)):
            plant(p, 0, r, 1, r % 128, x)
    args = [(p, p.device(), p.workspace(kvc), torch.cuda.Stream()) for p in (a, b)]
    torch.cuda.synchronize()
    first = None
    for _ in range(20):
        for p, (tables, starts, rows), ws, stream in args:
            kvc.prompt_attention(p.q, p.pools[0][0], p.pools[1][0], tables, starts, rows, p.scale, p.out, ws,
                                 window=p.window, sinks=p.sinks, stream=stream)
        torch.cuda.synchronize()
        bits = [p.out.view(torch.int16).clone() for p in (a, b)]
        first = first or bits
        assert all(torch.equal(x, y) for x, y in zip(first, bits))
    a.check()
    b.check()
    assert kvc.get_error_flags() == 0
