"""GPU parity: eviction by accumulated weight (kvc_evict_rows, kvc_evict_rows_block8): kept rows, moved rows and scores
bit for bit."""

import numpy as np
import pytest
import torch

from oracle import long_context as O

from long_context_helpers import TORCH, make_pools, make_tables

pytestmark = pytest.mark.gpu


def setup(kind, lens, H, D, bs, budget, seed, width=None, new_width=None):
    rng = np.random.default_rng(seed)
    m = [min(max(0, n), budget) for n in lens]
    need = [-(-x // bs) for x in m]
    tables, nb, spare = make_tables(lens, bs, sum(need) + 2, rng, width)
    new_width = new_width or max(1, -(-budget // bs))
    new_tables = np.full((len(lens), new_width), 1 << 28, dtype=np.int32)
    at = 0
    for i, k in enumerate(need):
        new_tables[i, :k] = spare[at:at + k]
        at += k
    if kind == "f32":
        pools = []
        for _ in range(2):
            t = torch.from_numpy(rng.standard_normal((nb, H, bs, D))).float().cuda()
            pools.append((t, None, None))
    else:
        pools = make_pools(nb, H, bs, D, kind, rng)
    scores = np.exp(2 * rng.standard_normal((len(lens), H, tables.shape[1] * bs))).astype(np.float32)
    return tables, new_tables, pools, scores


def bits(t):
    a = t.detach().cpu()
    return a.view(torch.int16).numpy() if a.dtype in (torch.bfloat16, torch.float16) else a.numpy()


def run(kvc, kind, tables, new_tables, pools, scores, lens, budget, recent, stream=None, bufs=None):
    B, H, _ = scores.shape
    bs = pools[0][0].shape[2]
    if bufs is None:
        bufs = (torch.full((B, H, budget), 7, dtype=torch.int32, device="cuda"),
                torch.full((B,), 7, dtype=torch.int32, device="cuda"),
                torch.full((B, H, new_tables.shape[1] * bs), 7.0, device="cuda"))
    kvc.evict_rows(torch.from_numpy(scores).cuda(), pools[0][0], pools[1][0], torch.from_numpy(tables).cuda(),
                   torch.tensor(lens, dtype=torch.int32, device="cuda"), budget, recent,
                   torch.from_numpy(new_tables).cuda(), *bufs, k_scale=pools[0][1], v_scale=pools[1][1], stream=stream)
    return bufs


def check(kvc, kind, lens, H, D, bs, budget, recent, seed=0, scores=None, width=None, new_width=None, flags=0):
    tables, new_tables, pools, sc = setup(kind, lens, H, D, bs, budget, seed, width, new_width)
    if scores is not None:
        sc = scores(sc)
    kept_ref, lens_ref = O.evict(sc, lens, budget, recent)
    before = [(bits(t), None if s is None else s.cpu().numpy()) for t, s, _ in pools]
    kept, new_lens, new_scores = run(kvc, kind, tables, new_tables, pools, sc, lens, budget, recent)
    torch.cuda.synchronize()
    assert kvc.get_error_flags() == flags
    assert np.array_equal(new_lens.cpu().numpy(), lens_ref)
    assert np.array_equal(kept.cpu().numpy(), kept_ref)
    for (b, s), (t, dev_s, _) in zip(before, pools):
        if s is None:
            assert np.array_equal(bits(t), O.move_rows(b, kept_ref, lens_ref, tables, new_tables))
        else:
            codes, scale = O.move_rows(b, kept_ref, lens_ref, tables, new_tables, s, kind)
            assert np.array_equal(dev_s.cpu().numpy(), scale)
            assert np.array_equal(bits(t), codes)
    want = np.full(new_scores.shape, 7, dtype=np.float32)
    for i, m in enumerate(lens_ref):
        for h in range(H):
            want[i, h, :m] = sc[i, h, kept_ref[i, h, :m]]
    assert np.array_equal(new_scores.cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16", "e4m3", "int8"])
@pytest.mark.parametrize("bs", [16, 48, 128])
def test_ragged_batches(kvc, kind, bs):
    check(kvc, kind, [1, 50, 49, 51, 400, 0, 777], 2, 64, bs, 50, 13, seed=bs)


@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (33, 0), (33, 33), (160, 7), (500, 499), (2000, 100)])
def test_budgets(kvc, budget, recent):
    check(kvc, "bf16", [600, 33, 161, 1], 3, 128, 16, budget, recent, seed=budget + recent)
    check(kvc, "e4m3", [600, 33, 161, 1], 2, 128, 16, budget, recent, seed=budget + recent)


@pytest.mark.parametrize("n", [4097, 20000, 140001])
def test_long_rows_split_over_a_cluster(kvc, n):
    check(kvc, "f16", [n, n - 999], 1, 64, 32, n // 7, n // 50, seed=n)


def test_many_units(kvc):
    check(kvc, "bf16", [100 + i for i in range(90)], 4, 64, 16, 64, 16)


def test_ties_go_to_the_lower_row(kvc):
    def few(s):
        return np.round(np.log(s)).astype(np.float32)  # a handful of values, negative ones and both zeros
    check(kvc, "bf16", [5000, 700, 90], 2, 64, 16, 60, 5, scores=few)
    check(kvc, "bf16", [9000], 2, 64, 16, 4000, 5, scores=few, seed=1)
    check(kvc, "bf16", [5000, 700, 90], 2, 64, 16, 60, 5, scores=np.zeros_like)
    check(kvc, "int8", [300], 2, 64, 16, 60, 5, scores=lambda s: np.where(s > 1, -0.0, 0.0).astype(np.float32))


def test_scores_that_are_not_finite(kvc):
    def odd(s):
        s = s.copy()
        s[..., ::3] = np.nan
        s[..., 1::7] = np.inf
        s[..., 2::5] = -np.inf
        return s
    for budget in (10, 60, 250):
        check(kvc, "bf16", [300, 257], 2, 64, 16, budget, 4, scores=odd)


def test_wide_tables(kvc):
    check(kvc, "bf16", [100, 40], 2, 64, 16, 30, 3, width=64, new_width=9)


def test_invalid_lengths_keep_nothing(kvc):
    check(kvc, "bf16", [-1, 100, 129], 2, 64, 16, 30, 3, width=8, flags=kvc.FLAG_BAD_LEN)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_blocks_outside_the_pool_are_not_moved(kvc, kind):
    lens, budget = [100, 64], 40
    tables, new_tables, pools, sc = setup(kind, lens, 2, 64, 16, budget, 3)
    nb = pools[0][0].shape[0]
    tables[0, 1], tables[1, 3], new_tables[1, 0] = -4, nb, nb + 9
    kept_ref, lens_ref = O.evict(sc, lens, budget, 8)
    before = [(bits(t), None if s is None else s.cpu().numpy()) for t, s, _ in pools]
    kept, _, _ = run(kvc, kind, tables, new_tables, pools, sc, lens, budget, 8)
    torch.cuda.synchronize()
    assert kvc.get_error_flags() == kvc.FLAG_BAD_BLOCK
    assert np.array_equal(kept.cpu().numpy(), kept_ref)
    for (b, s), (t, dev_s, _) in zip(before, pools):
        got = O.move_rows(b, kept_ref, lens_ref, tables, new_tables, s, kind if s is not None else None)
        assert np.array_equal(bits(t), got if s is None else got[0])
        if s is not None:
            assert np.array_equal(dev_s.cpu().numpy(), got[1])


def test_on_a_stream_and_in_a_graph(kvc):
    lens, budget = [300, 500], 64
    tables, new_tables, pools, sc = setup("bf16", lens, 2, 64, 16, budget, 4)
    kept_ref, _ = O.evict(sc, lens, budget, 9)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        kept, _, _ = run(kvc, "bf16", tables, new_tables, pools, sc, lens, budget, 9)
    torch.cuda.synchronize()
    assert np.array_equal(kept.cpu().numpy(), kept_ref)
    dev = [torch.from_numpy(x).cuda() for x in (sc, tables, new_tables)]
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    new_lens, new_scores = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros((2, 2, 64), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvc.evict_rows(dev[0], pools[0][0], pools[1][0], dev[1], n, budget, 9, dev[2], kept, new_lens, new_scores)
    for seed in (1, 2):
        sc2 = np.random.default_rng(seed).random(sc.shape).astype(np.float32)
        dev[0].copy_(torch.from_numpy(sc2))
        lens2 = [290 + seed, 40 + seed]
        n.copy_(torch.tensor(lens2, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        ref, ref_lens = O.evict(sc2, lens2, budget, 9)
        assert np.array_equal(kept.cpu().numpy(), ref) and np.array_equal(new_lens.cpu().numpy(), ref_lens)


def test_offsets_past_32_bits(kvc):
    H, D, bs, nb = 8, 256, 128, 16500  # 4.3e9 elements per pool
    assert nb * H * bs * D > 2 ** 32
    lens, budget = [300], 140
    tables, new_tables, pools, sc = setup("bf16", lens, H, D, bs, budget, 5)
    used = pools[0][0].shape[0]
    far = np.array([nb - 1 - i for i in range(used)])
    at = torch.from_numpy(far).cuda()
    big = []
    for t, _, _ in pools:
        b = torch.empty((nb, H, bs, D), dtype=t.dtype, device="cuda")
        b[at] = t
        big.append((b, None, None))
    run(kvc, "bf16", tables, new_tables, pools, sc, lens, budget, 20)
    run(kvc, "bf16", far[np.minimum(tables, used - 1)].astype(np.int32),
        far[np.minimum(new_tables, used - 1)].astype(np.int32), big, sc, lens, budget, 20)
    torch.cuda.synchronize()
    for (t, _, _), (b, _, _) in zip(pools, big):
        assert np.array_equal(bits(t), bits(b[at]))  # the small pool's result is checked by test_ragged_batches
