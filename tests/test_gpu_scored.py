"""GPU parity: decode that adds up the weights of the cached rows (kvc_decode_attention_scored), and decode over
block-scaled one-byte caches (kvc_decode_attention_block8), against float64."""

import math

import numpy as np
import pytest
import torch

from oracle import long_context as O

from long_context_helpers import TORCH, bounds, call_decode, f64, make_pools, make_tables, workspace_for

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "f16", "e4m3", "int8"]


@pytest.fixture(autouse=True)
def _options(kvc):
    opts = (kvc.OPT_BLOCKS_PER_CTA, kvc.OPT_MAX_CTAS, kvc.OPT_CHECKED, kvc.OPT_WAIT_POLLS)
    for o in opts:
        kvc.set_option(o, 0)
    yield
    for o in opts:
        kvc.set_option(o, 0)


def make(kind, lens, T, Hq, H, D, bs, seed, q_dtype=None, width=None, gain=1.0):
    rng = np.random.default_rng(seed)
    tables, nb, _ = make_tables(lens, bs, 3, rng, width)
    pools = make_pools(nb, H, bs, D, kind, rng)
    q = torch.from_numpy(gain * rng.standard_normal((len(lens), T, Hq, D)))
    q = q.to(TORCH[q_dtype or (kind if kind in TORCH else "bf16")]).cuda()
    scores = torch.from_numpy(rng.random((len(lens), H, tables.shape[1] * bs)) * 3).float().cuda()
    return q, pools, tables, scores


def check(kvc, kind, lens, T, Hq, H, D, bs, seed=0, out_dtype=torch.float32, scored=True, q_dtype=None, width=None,
          gain=1.0, flags=0):
    q, pools, tables, scores = make(kind, lens, T, Hq, H, D, bs, seed, q_dtype, width, gain)
    scale = 1 / math.sqrt(D)
    before = f64(scores)
    ref, ref_scores = O.decode_scored(f64(q), pools[0][2], pools[1][2], tables, lens, scale,
                                      before if scored else None)
    t, n = torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, float("nan"), dtype=out_dtype, device="cuda")
    ws = workspace_for(kvc, q, pools[0][0], tables, scored)
    ws.fill_(0xff)  # the workspace needs no particular contents
    call_decode(kvc, kind, q, pools, t, n, scale, out, scores if scored else None, ws)
    torch.cuda.synchronize()
    assert kvc.get_error_flags() == flags
    tol, tol_scores = bounds(f64(q), pools[0][2], pools[1][2], tables, lens, scale, out_dtype, ref, ref_scores)
    err = np.abs(f64(out) - ref)
    assert np.all(err <= tol), f"out: {err.max():.3e} (bound {np.min(tol):.3e})"
    if scored:
        got = f64(scores)
        err = np.abs(got - ref_scores)
        assert np.all(err <= tol_scores), f"scores: {err.max():.3e}"
        for i, m in enumerate(lens):  # rows behind the last one are left as they were
            keep = max(0, m) if T <= m <= got.shape[2] else 0
            assert np.array_equal(got[i, :, keep:], before[i, :, keep:])
    return out, scores


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,H", [(8, 8), (8, 2), (3, 1), (14, 2), (32, 2), (20, 1)])
def test_head_layouts(kvc, kind, D, Hq, H):
    check(kvc, kind, [1, 15, 16, 17, 100, 303], 1, Hq, H, D, 16, seed=D + Hq)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bs", [16, 32, 48, 80, 128])
def test_block_sizes_and_output_types(kvc, kind, bs):
    dt = {16: torch.float32, 32: torch.bfloat16, 48: torch.float16, 80: torch.float32, 128: torch.bfloat16}[bs]
    check(kvc, kind, [5, bs, bs + 1, 3 * bs - 1, 700], 1, 8, 2, 128, bs, seed=bs, out_dtype=dt, width=60)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [2, 7, 16, 33])
def test_several_new_tokens(kvc, kind, T):
    check(kvc, kind, [T, T + 1, T + 15, 64 + T, 250], T, 8, 2, 128, 16, seed=T)
    check(kvc, kind, [T, 40 + T], T, 3, 1, 64, 32, seed=T + 100)
    check(kvc, kind, [T, 40 + T], T, 4, 2, 256, 16, seed=T + 200)


def test_the_most_new_tokens(kvc):
    check(kvc, "bf16", [256, 300], 256, 16, 1, 64, 16, seed=5)  # 4096 queries of one kv head


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_plain_decode_of_block_scaled_codes(kvc, kind):
    for q_dtype in ("bf16", "f16"):
        check(kvc, kind, [1, 130, 999], 1, 8, 2, 128, 16, seed=3, scored=False, q_dtype=q_dtype)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("per,ctas", [(1, 0), (3, 0), (1, 2), (7, 1), (1000, 0)])
def test_work_splits_give_the_same(kvc, kind, per, ctas):
    kvc.set_option(kvc.OPT_BLOCKS_PER_CTA, per)
    kvc.set_option(kvc.OPT_MAX_CTAS, ctas)
    check(kvc, kind, [1, 900, 16, 333, 2000], 1, 8, 2, 64, 16, seed=per)
    check(kvc, kind, [9, 500], 9, 4, 2, 128, 32, seed=per)


@pytest.mark.parametrize("kind", KINDS)
def test_one_long_sequence_with_many_records(kvc, kind):
    check(kvc, kind, [20001], 1, 4, 1, 64, 16, seed=8)


def test_large_batch(kvc):
    rng = np.random.default_rng(1)
    check(kvc, "bf16", rng.integers(1, 40, 1500).tolist(), 1, 2, 1, 64, 16, seed=9)


@pytest.mark.parametrize("kind", KINDS)
def test_peaked_and_wide_scores(kvc, kind):
    # scores of some hundreds: one row takes all the weight, and the references move often
    check(kvc, kind, [700, 31], 1, 8, 2, 128, 16, seed=4, gain=30.0)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_block_scales_far_apart(kvc, code):
    # neighbouring blocks whose V scales differ by 2^40, weights that favour the small ones, and blocks of scale 0
    lens, H, D, bs = [300], 2, 128, 16
    q, pools, tables, scores = make(code, lens, 1, 8, H, D, bs, seed=11)
    (k, ks, _), (v, vs, _) = pools
    factor = torch.tensor([2.0 ** (-40 if i % 3 == 0 else 0 if i % 3 == 1 else -20) for i in range(vs.shape[0])])
    vs *= factor.cuda()[:, None]
    vs[int(tables[0, 4])] = 0
    ks[int(tables[0, 5])] = 0
    # the first block's keys are loud: nearly all weight goes to the block with the smallest V scale
    ks[int(tables[0, 0])] *= 12
    vs[int(tables[0, 0])] *= 2.0 ** -30
    K, V = O.dequantized(k.cpu().numpy(), ks.cpu().numpy()), O.dequantized(v.cpu().numpy(), vs.cpu().numpy())
    scale = 1 / math.sqrt(D)
    before = f64(scores)
    ref, ref_scores = O.decode_scored(f64(q), K, V, tables, lens, scale, before)
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    kvc.decode_attention_block8(q, k, v, ks, vs, torch.from_numpy(tables).cuda(),
                                torch.tensor(lens, dtype=torch.int32, device="cuda"), scale, out,
                                workspace_for(kvc, q, k, tables, True), scores=scores)
    # the bound counts each row's own contribution, p |v|, instead of the largest |v|
    _, tol_scores = bounds(f64(q), K, V, tables, lens, scale, torch.float32, ref, ref_scores)
    mass, _ = O.decode_scored(f64(q), K, np.abs(V), tables, lens, scale)
    rel = (tol_scores / (1 + np.abs(ref_scores))).max()
    # a weight's f16 parts reach 2^-25 of the largest contribution of a segment: 300 rows of 448 or 127 codes
    # relative to a largest contribution of one code, at most
    big = np.abs(V[np.unique(tables[0])]).max((0, 2, 3))  # per kv head
    assert np.all(np.abs(f64(out) - ref) <= rel * mass * 2 + 300 * 2.0 ** -24 * mass.max(-1, keepdims=True) * 448)
    assert np.all(np.abs(f64(scores) - ref_scores) <= tol_scores)
    assert big.shape == (H,)


@pytest.mark.parametrize("kind", KINDS)
def test_rows_behind_the_end_may_hold_anything(kvc, kind):
    lens, H, D, bs = [1, 17, 40, 100], 2, 128, 32
    q, pools, tables, scores = make(kind, lens, 1, 8, H, D, bs, seed=21)
    other = scores.clone()
    t, n = torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = workspace_for(kvc, q, pools[0][0], tables, True)
    res = []
    for fill in (False, True):
        if fill:
            for i, m in enumerate(lens):
                b = int(tables[i, (m - 1) // bs])
                for p in pools:
                    p[0][b, :, (m - 1) % bs + 1:] = float("nan") if kind in TORCH else 0x7f if kind == "e4m3" else -128
        out = torch.empty(q.shape, device="cuda")
        call_decode(kvc, kind, q, pools, t, n, 0.1, out, other if fill else scores, ws)
        res.append(out)
    assert torch.equal(res[0], res[1])
    assert torch.equal(scores, other)


@pytest.mark.parametrize("kind", KINDS)
def test_invalid_lengths_and_blocks(kvc, kind):
    # lengths below the new tokens, negative, and beyond the table: zeros, flagged, scores left
    check(kvc, kind, [3, 0, 2, -5, 97, 64], 3, 8, 2, 64, 16, seed=31, width=6, flags=kvc.FLAG_BAD_LEN)
    check(kvc, kind, [0, -1, 49], 1, 8, 2, 64, 16, seed=33, width=3, flags=kvc.FLAG_BAD_LEN)  # none is valid
    # entries outside the pool: their rows get no weight; a sequence with no other rows gives zeros
    lens, H, D, bs = [100, 16, 33], 2, 128, 16
    q, pools, tables, scores = make(kind, lens, 1, 8, H, D, bs, seed=32)
    nb = pools[0][0].shape[0]
    tables[0, 2], tables[0, 6], tables[1, 0], tables[2, 1] = -1, nb, 2 ** 31 - 1, -2 ** 31
    before = f64(scores)
    ref, ref_scores = O.decode_scored(f64(q), pools[0][2], pools[1][2], tables, lens, 0.1, before)
    out = torch.full(q.shape, float("nan"), device="cuda")
    call_decode(kvc, kind, q, pools, torch.from_numpy(tables).cuda(),
                torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.1, out, scores,
                workspace_for(kvc, q, pools[0][0], tables, True))
    torch.cuda.synchronize()
    assert kvc.get_error_flags() == kvc.FLAG_BAD_BLOCK
    tol, tol_scores = bounds(f64(q), pools[0][2], pools[1][2], tables, lens, 0.1, torch.float32, ref, ref_scores)
    assert np.all(np.abs(f64(out) - ref) <= tol)
    assert np.all(f64(out)[1] == 0)
    assert np.all(np.abs(f64(scores) - ref_scores) <= tol_scores)


def test_checked_mode_reports(kvc):
    lens = [100]
    q, pools, tables, scores = make("bf16", lens, 1, 8, 2, 64, 16, seed=33)
    out = torch.empty(q.shape, device="cuda")
    args = (q, pools, torch.from_numpy(tables).cuda(), torch.tensor([200], dtype=torch.int32, device="cuda"), 0.1, out,
            scores, workspace_for(kvc, q, pools[0][0], tables, True))
    kvc.set_option(kvc.OPT_CHECKED, 1)
    with pytest.raises(kvc.KvcError) as e:
        call_decode(kvc, "bf16", *args)
    assert e.value.status == kvc.ERR_OUT_OF_RANGE


def test_giving_up_on_a_copy(kvc):
    # 0.5 GB of cache, several times L2 and read by every SM: the copies run at HBM's pace, behind the
    # products, so that a single poll for their data fails
    B, H, D, bs, n = 32, 8, 128, 16, 4096
    nb = B * n // bs
    gen = torch.Generator(device="cuda").manual_seed(34)
    tables = torch.randperm(nb, generator=gen, device="cuda").to(torch.int32).view(B, n // bs)
    pools = [(torch.randn((nb, H, bs, D), generator=gen, device="cuda", dtype=torch.bfloat16), None, None)
             for _ in range(2)]
    q = torch.randn((B, 1, 32, D), generator=gen, device="cuda").to(torch.bfloat16)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    scores = [torch.zeros((B, H, n), device="cuda") for _ in range(3)]
    outs = [torch.empty(q.shape, device="cuda") for _ in range(3)]
    ws = [workspace_for(kvc, q, pools[0][0], tables, True) for _ in range(2)]
    call_decode(kvc, "bf16", q, pools, tables, lens, 0.1, outs[0], scores[0], ws[0])
    kvc.set_option(kvc.OPT_WAIT_POLLS, 1)
    call_decode(kvc, "bf16", q, pools, tables, lens, 0.1, outs[1], scores[1], ws[1])
    torch.cuda.synchronize()
    assert kvc.get_error_flags() == kvc.FLAG_TIMEOUT
    kvc.set_option(kvc.OPT_WAIT_POLLS, 0)
    call_decode(kvc, "bf16", q, pools, tables, lens, 0.1, outs[2], scores[2], ws[1])  # the same workspace serves on
    torch.cuda.synchronize()
    assert kvc.get_error_flags() == 0
    assert torch.equal(outs[0], outs[2]) and torch.equal(scores[0], scores[2])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_same_bits_on_streams_and_in_graphs(kvc, kind):
    lens = [800, 3, 250]
    q, pools, tables, scores = make(kind, lens, 1, 8, 2, 128, 16, seed=41)
    t, n = torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    first, second, third = scores.clone(), scores.clone(), scores.clone()
    o1, o2, o3 = (torch.empty(q.shape, device="cuda") for _ in range(3))
    ws = workspace_for(kvc, q, pools[0][0], tables, True)
    call_decode(kvc, kind, q, pools, t, n, 0.1, o1, first, ws)
    torch.cuda.synchronize()
    # two calls at once, on two streams, with a workspace each
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    ws2 = workspace_for(kvc, q, pools[0][0], tables, True)
    call_decode(kvc, kind, q, pools, t, n, 0.1, o2, second, ws, stream=a)
    call_decode(kvc, kind, q, pools, t, n, 0.1, o3, third, ws2, stream=b)
    torch.cuda.synchronize()
    assert torch.equal(o1, o2) and torch.equal(o1, o3)
    assert torch.equal(first, second) and torch.equal(first, third)
    # captured once, replayed twice with other inputs in the same buffers
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call_decode(kvc, kind, q, pools, t, n, 0.1, o2, second, ws)
    q.mul_(-0.5)
    n.copy_(torch.tensor([500, 4, 251], dtype=torch.int32))
    for _ in range(2):
        g.replay()
        call_decode(kvc, kind, q, pools, t, n, 0.1, o1, first, ws2)
        torch.cuda.synchronize()
        assert torch.equal(o1, o2) and torch.equal(first, second)


def test_shared_blocks_keep_separate_scores(kvc):
    lens = [100, 100, 70]
    q, pools, tables, scores = make("bf16", lens, 1, 8, 2, 64, 16, seed=51)
    tables[1] = tables[0]
    tables[2, :4] = tables[0, :4]
    before = f64(scores)
    ref, ref_scores = O.decode_scored(f64(q), pools[0][2], pools[1][2], tables, lens, 0.1, before)
    out = torch.empty(q.shape, device="cuda")
    call_decode(kvc, "bf16", q, pools, torch.from_numpy(tables).cuda(),
                torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.1, out, scores,
                workspace_for(kvc, q, pools[0][0], tables, True))
    tol, tol_scores = bounds(f64(q), pools[0][2], pools[1][2], tables, lens, 0.1, torch.float32, ref, ref_scores)
    assert np.all(np.abs(f64(out) - ref) <= tol) and np.all(np.abs(f64(scores) - ref_scores) <= tol_scores)


def test_non_finite_values_stay_in_their_sequence(kvc):
    lens = [60, 60]
    q, pools, tables, scores = make("bf16", lens, 1, 8, 2, 64, 16, seed=52)
    pools[1][0][int(tables[0, 1]), 0, 3, 5] = float("nan")
    out = torch.empty(q.shape, device="cuda")
    call_decode(kvc, "bf16", q, pools, torch.from_numpy(tables).cuda(),
                torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.1, out, scores,
                workspace_for(kvc, q, pools[0][0], tables, True))
    bad = torch.isnan(out)
    assert bad[0, 0, :4, 5].all() and int(bad.sum()) == 4
    assert torch.isfinite(scores).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", KINDS[:3])  # every int8 code is finite
def test_tokens_do_not_see_non_finite_rows_behind_them(kvc, kind, D):
    # the rows of the last tokens hold infinities and NaN: the tokens before give the same bits as without them, a
    # token that sees one gives what fp64 gives, in the dims where it stands
    lens, H, bs, T = [41, 16, 9, 64, 130], 2, 16, 7
    q, pools, tables, scores = make(kind, lens, T, 6, H, D, bs, seed=61)
    n, t = torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.from_numpy(tables).cuda()
    ws = workspace_for(kvc, q, pools[0][0], tables, True)
    res = []
    for odd in (False, True):
        if odd:
            for i, m in enumerate(lens):
                for back, dim in ((1, D - 3), (3, 0), (3, D // 2 + 9)):  # rows n - 1 and n - 3
                    b, r = int(tables[i, (m - back) // bs]), (m - back) % bs
                    pools[1][0][b, 0, r, dim] = 0x7f if kind == "e4m3" else float("inf") if dim == 0 else float("nan")
        out = torch.empty(q.shape, device="cuda")
        call_decode(kvc, kind, q, pools, t, n, 0.1, out, scores.clone(), ws)
        res.append(out.view(len(lens), T, H, 3, D))
    clean, got = res
    assert torch.isfinite(clean).all()
    seen = torch.zeros_like(clean, dtype=torch.bool)  # token T - 1 sees row n - 1, T - 3 and later see n - 3
    seen[:, T - 1:, 0, :, D - 3] = True
    seen[:, T - 3:, 0, :, 0] = True
    seen[:, T - 3:, 0, :, D // 2 + 9] = True
    assert torch.equal(torch.isfinite(got), ~seen)
    assert torch.equal(got[:, :T - 3], clean[:, :T - 3])
    assert torch.equal(got[:, :, 1], clean[:, :, 1])
    if kind != "e4m3":
        assert (got[:, T - 3:, 0, :, 0] == float("inf")).all()
    # the other dims of a row that is taken by itself: within a few roundings of the weights' parts and the sums
    spread = (got - clean)[~seen].abs().max().item()
    assert spread <= 130 * 2.0 ** -22 * max(1.0, float(np.abs(pools[1][2]).max()))


@pytest.mark.parametrize("kind", KINDS)
def test_more_sequences_than_lanes_with_several_tokens(kvc, kind):
    rng = np.random.default_rng(3)
    for B in (31, 32, 33, 50):
        lens = rng.integers(3, 120, B).tolist()
        lens[B // 2], lens[B - 1] = 0, 2  # invalid ones inside and at the end
        check(kvc, kind, lens, 3, 6, 2, 64, 16, seed=B, width=9, flags=kvc.FLAG_BAD_LEN)


def test_the_largest_batch(kvc):
    rng = np.random.default_rng(2)
    lens = rng.integers(1, 20, 4096).tolist()
    lens[0], lens[100], lens[4095] = 150, 33, 64
    check(kvc, "int8", lens, 1, 2, 1, 64, 16, seed=61)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_offsets_past_32_bits(kvc, kind):
    H, D, bs, nb = 8, 256, 128, 16500  # 4.3e9 elements per pool, of which a few blocks at both ends are used
    assert nb * H * bs * D > 2 ** 32
    lens = [300, 129]
    q, pools, tables, scores = make(kind, lens, 1, 16, H, D, bs, seed=62)
    used = pools[0][0].shape[0]
    far = np.array([nb - 1 - i if i % 2 else i for i in range(used)])  # where the small pool's blocks go
    at = torch.from_numpy(far).cuda()
    big = []
    for t, s, _ in pools:
        b = torch.empty((nb, H, bs, D), dtype=t.dtype, device="cuda")
        b[at] = t
        bs_ = None
        if s is not None:
            bs_ = torch.zeros((nb, H), device="cuda")
            bs_[at] = s
        big.append((b, bs_, None))
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    far_tables = np.where(tables < used, far[np.minimum(tables, used - 1)], tables).astype(np.int32)
    other = scores.clone()
    out, far_out = torch.empty(q.shape, device="cuda"), torch.empty(q.shape, device="cuda")
    ws = workspace_for(kvc, q, pools[0][0], tables, True)
    call_decode(kvc, kind, q, pools, torch.from_numpy(tables).cuda(), n, 0.1, out, scores, ws)
    call_decode(kvc, kind, q, big, torch.from_numpy(far_tables).cuda(), n, 0.1, far_out, other, ws)
    torch.cuda.synchronize()
    assert kvc.get_error_flags() == 0
    assert torch.equal(out, far_out) and torch.equal(scores, other)  # and out is what test_head_layouts checks


def test_two_graphs_share_a_workspace(kvc):
    lens = [800, 3]
    q, pools, tables, scores = make("bf16", lens, 1, 8, 2, 128, 16, seed=63)
    t, n = torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = workspace_for(kvc, q, pools[0][0], tables, True)
    qs = [q, -q]
    want = []
    for x in qs:
        o, sc = torch.empty(q.shape, device="cuda"), scores.clone()
        call_decode(kvc, "bf16", x, pools, t, n, 0.1, o, sc, workspace_for(kvc, q, pools[0][0], tables, True))
        want.append((o, sc))
    graphs, got = [], []
    for x in qs:
        o, sc = torch.empty(q.shape, device="cuda"), scores.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call_decode(kvc, "bf16", x, pools, t, n, 0.1, o, sc, ws)
        graphs.append(g)
        got.append((o, sc))
    for g in graphs:  # one after the other on one stream
        g.replay()
    torch.cuda.synchronize()
    for (o, sc), (wo, wsc) in zip(got, want):
        assert torch.equal(o, wo) and torch.equal(sc, wsc)
