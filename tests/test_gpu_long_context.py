"""A conversation kept within a budget: prompt, scored prompt window, decode steps, eviction, more steps, with forks and
copy-on-write, on 16-bit and on block-scaled caches. Every call is checked against the oracle on the state it met."""

import numpy as np
import pytest
import torch

from oracle import long_context as O

from long_context_helpers import TORCH, bounds, f64

pytestmark = pytest.mark.gpu

H, HQ, D, BS, BLOCKS, WIDTH = 2, 8, 128, 16, 96, 20
SCALE = D ** -0.5


class Serving:
    """Block pool, device pools and per-sequence scores of a few sequences, with the oracle's copies."""

    def __init__(self, kvc, kind):
        self.kvc, self.kind, self.one = kvc, kind, kind not in TORCH
        self.pool = kvc.BlockPool(BLOCKS, BS)
        self.gen = torch.Generator().manual_seed(7)
        shape = (BLOCKS, H, BS, D)
        if self.one:
            dt = torch.int8 if kind == "int8" else torch.uint8
            self.k, self.v = (torch.zeros(shape, dtype=dt, device="cuda") for _ in range(2))
            self.ks, self.vs = (torch.zeros((BLOCKS, H), device="cuda") for _ in range(2))
        else:
            self.k, self.v = (torch.zeros(shape, dtype=TORCH[kind], device="cuda") for _ in range(2))
            self.ks = self.vs = None
        self.dtype = torch.bfloat16 if self.one else TORCH[kind]
        self.scores = {}  # sequence -> [H, WIDTH * BS] on the device

    def rows(self, T, heads, spread=0.5):
        x = torch.randn((T, heads, D), generator=self.gen) * torch.exp(spread * torch.randn((T, heads, 1), generator=self.gen))
        return x.to(self.dtype)

    def append(self, slots):
        k, v = self.rows(len(slots), H), self.rows(len(slots), H)
        t = torch.tensor(slots, dtype=torch.int64, device="cuda")
        if self.one:
            want = [O.append_block8(x.float().numpy(), slots, c.cpu().numpy(), s.cpu().numpy(), self.kind)
                    for x, c, s in ((k, self.k, self.ks), (v, self.v, self.vs))]
            self.kvc.append_block8(k.cuda(), v.cuda(), t, self.k, self.v, self.ks, self.vs)
            for (c, s), (wc, ws) in zip(((self.k, self.ks), (self.v, self.vs)), want):
                assert np.array_equal(c.cpu().numpy(), wc) and np.array_equal(s.cpu().numpy(), ws)
        else:
            self.kvc.append(k.cuda(), v.cuda(), t, self.k, self.v)

    def tables(self, seqs, width=WIDTH):
        rows, lens = self.pool.tables(seqs, width)
        return (torch.tensor(rows, dtype=torch.int32, device="cuda"),
                torch.tensor(lens, dtype=torch.int32, device="cuda"))

    def decode(self, seqs, T):
        tables, lens = self.tables(seqs)
        q = torch.stack([self.rows(T, HQ, 0.0) for _ in seqs]).cuda()
        scores = torch.stack([self.scores[s] for s in seqs])
        K, V = ((O.dequantized(c.cpu().numpy(), s.cpu().numpy()) if self.one else f64(c))
                for c, s in ((self.k, self.ks), (self.v, self.vs)))
        ref, ref_scores = O.decode_scored(f64(q), K, V, tables.cpu().numpy(), lens.tolist(), SCALE, f64(scores))
        out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
        ws = self.kvc.new_scored_workspace(len(seqs), T, HQ, H, D, BS, WIDTH)
        if self.one:
            self.kvc.decode_attention_block8(q, self.k, self.v, self.ks, self.vs, tables, lens, SCALE, out, ws,
                                             scores=scores)
        else:
            self.kvc.decode_attention_scored(q, self.k, self.v, tables, lens, SCALE, out, scores, ws)
        tol, tol_scores = bounds(f64(q), K, V, tables.cpu().numpy(), lens.tolist(), SCALE, out.dtype, ref, ref_scores)
        assert np.all(np.abs(f64(out) - ref) <= tol)
        assert np.all(np.abs(f64(scores) - ref_scores) <= tol_scores)
        for i, s in enumerate(seqs):
            self.scores[s] = scores[i]

    def evict(self, seqs, budget, recent):
        tables, lens = self.tables(seqs)
        scores = torch.stack([self.scores[s] for s in seqs])
        kept_ref, lens_ref = O.evict(scores.cpu().numpy(), lens.tolist(), budget, recent)
        self.pool.evict_batch(seqs, [min(n, budget) for n in lens.tolist()])
        new_tables, new_n = self.tables(seqs)
        view = (lambda t: t.cpu().view(torch.int16).numpy()) if not self.one else (lambda t: t.cpu().numpy())
        want = []
        for c, s in ((self.k, self.ks), (self.v, self.vs)):
            want.append(O.move_rows(view(c), kept_ref, lens_ref, tables.cpu().numpy(), new_tables.cpu().numpy(),
                                    None if s is None else s.cpu().numpy(), self.kind if self.one else None))
        kept = torch.zeros((len(seqs), H, budget), dtype=torch.int32, device="cuda")
        new_lens = torch.zeros(len(seqs), dtype=torch.int32, device="cuda")
        new_scores = torch.zeros_like(scores)
        self.kvc.evict_rows(scores, self.k, self.v, tables, lens, budget, recent, new_tables, kept, new_lens,
                            new_scores, k_scale=self.ks, v_scale=self.vs)
        assert np.array_equal(kept.cpu().numpy(), kept_ref)
        assert torch.equal(new_lens, new_n) and np.array_equal(new_n.cpu().numpy(), lens_ref)
        for (c, s), w in zip(((self.k, self.ks), (self.v, self.vs)), want):
            if self.one:
                assert np.array_equal(c.cpu().numpy(), w[0]) and np.array_equal(s.cpu().numpy(), w[1])
            else:
                assert np.array_equal(view(c), w)
        for i, s in enumerate(seqs):
            self.scores[s] = new_scores[i]


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3", "int8"])
def test_conversations_within_a_budget(kvc, kind):
    sv = Serving(kvc, kind)
    seqs = [sv.pool.add() for _ in range(3)]
    for s in seqs:
        sv.scores[s] = torch.zeros((H, WIDTH * BS), device="cuda")
    # ragged prompts, in one append; the last 5 tokens of each are scored against all of it
    sv.append(sum((sv.pool.reserve(s, n) for s, n in zip(seqs, (150, 33, 97))), []))
    sv.decode(seqs, 5)
    for _ in range(3):
        sv.append(sum(sv.pool.reserve_batch(seqs, 1), []))
        sv.decode(seqs, 1)
    # the long ones are cut back; the short one keeps everything but moves too
    sv.evict(seqs, 64, 12)
    assert [sv.pool.length(s) for s in seqs] == [64, 36, 64]
    for _ in range(2):
        sv.append(sum(sv.pool.reserve_batch(seqs, 1), []))
        sv.decode(seqs, 1)
    # a fork shares the blocks, then one of the two writes: copy-on-write takes the block's scales along
    fork = sv.pool.fork(seqs[0])
    sv.scores[fork] = sv.scores[seqs[0]].clone()
    slots, pair = sv.pool.reserve_cow(fork, 1)
    assert pair is not None
    pairs = torch.tensor([pair], dtype=torch.int64, device="cuda")
    kvc.copy_blocks(sv.k, pairs)
    kvc.copy_blocks(sv.v, pairs)
    if sv.one:
        for s in (sv.ks, sv.vs):
            s[pair[1]] = s[pair[0]]
    sv.append(slots)
    sv.decode([fork, seqs[1]], 1)
    # evicting the fork leaves its parent's rows, and the parent decodes on
    sv.evict([fork], 40, 8)
    sv.append(sv.pool.reserve(seqs[0], 2))
    sv.decode([seqs[0], fork], 2)
    for s in (*seqs, fork):
        sv.pool.free(s)
    assert sv.pool.stats()["free_blocks"] == BLOCKS
    assert kvc.get_error_flags() == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_captured_step_replays(kvc, kind):
    """Append and scored decode in one CUDA graph, the lengths and slots fed through the same buffers."""
    sv = Serving(kvc, kind)
    seqs = [sv.pool.add() for _ in range(2)]
    for s in seqs:
        sv.scores[s] = torch.zeros((H, WIDTH * BS), device="cuda")
    sv.append(sum((sv.pool.reserve(s, n) for s, n in zip(seqs, (40, 71))), []))
    sv.decode(seqs, 3)
    tables, lens = sv.tables(seqs)
    k, v = (torch.zeros((2, H, D), dtype=sv.dtype, device="cuda") for _ in range(2))
    q = torch.zeros((2, HQ, D), dtype=sv.dtype, device="cuda")
    slots = torch.full((2,), -1, dtype=torch.int64, device="cuda")
    out = torch.empty(q.shape, device="cuda")
    scores = torch.stack([sv.scores[s] for s in seqs])
    ws = kvc.new_scored_workspace(2, 1, HQ, H, D, BS, WIDTH)

    def step():
        if sv.one:
            kvc.append_block8(k, v, slots, sv.k, sv.v, sv.ks, sv.vs)
            kvc.decode_attention_block8(q, sv.k, sv.v, sv.ks, sv.vs, tables, lens, SCALE, out, ws, scores=scores)
        else:
            kvc.append(k, v, slots, sv.k, sv.v)
            kvc.decode_attention_scored(q, sv.k, sv.v, tables, lens, SCALE, out, scores, ws)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(20):  # past the ends of both sequences' last blocks
        new = sum(sv.pool.reserve_batch(seqs, 1), [])
        t, n = sv.tables(seqs)
        tables.copy_(t), lens.copy_(n)
        slots.copy_(torch.tensor(new))
        k.copy_(sv.rows(2, H)), v.copy_(sv.rows(2, H)), q.copy_(sv.rows(2, HQ, 0.0))
        before = f64(scores)
        g.replay()
        torch.cuda.synchronize()
        K, V = ((O.dequantized(c.cpu().numpy(), s.cpu().numpy()) if sv.one else f64(c))
                for c, s in ((sv.k, sv.ks), (sv.v, sv.vs)))
        ref, ref_scores = O.decode_scored(f64(q)[:, None], K, V, t.cpu().numpy(), n.tolist(), SCALE, before)
        tol, tol_scores = bounds(f64(q)[:, None], K, V, t.cpu().numpy(), n.tolist(), SCALE, out.dtype, ref, ref_scores)
        assert np.all(np.abs(f64(out)[:, None] - ref) <= tol)
        assert np.all(np.abs(f64(scores) - ref_scores) <= tol_scores)
    assert kvc.get_error_flags() == 0


def test_refusals_on_the_device(kvc):
    B, mb = 2, 4
    k = torch.zeros((9, H, BS, D), dtype=torch.bfloat16, device="cuda")
    codes = torch.zeros((9, H, BS, D), dtype=torch.uint8, device="cuda")
    s = torch.zeros((9, H), device="cuda")
    q = torch.zeros((B, HQ, D), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    tables = torch.zeros((B, mb), dtype=torch.int32, device="cuda")
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    scores = torch.zeros((B, H, mb * BS), device="cuda")
    ws = kvc.new_scored_workspace(B, 1, HQ, H, D, BS, mb)

    def scored(**kw):
        a = dict(q=q, k_cache=k, v_cache=k, block_tables=tables, context_lens=lens, scale=0.1, out=out, scores=scores,
                 workspace=ws)
        a.update(kw)
        kvc.decode_attention_scored(**a)

    with pytest.raises(kvc.KvcError) as e:
        scored(workspace=ws[:-300])
    assert e.value.status == kvc.ERR_WORKSPACE
    with pytest.raises(kvc.KvcError) as e:
        scored(workspace=torch.empty(ws.numel() + 16, dtype=torch.uint8, device="cuda")[16:])
    assert e.value.status == kvc.ERR_INVALID_ARG
    small = kvc.new_scored_workspace(B, 1, HQ, H, D, BS, mb, scored=False)
    with pytest.raises(kvc.KvcError) as e:  # sized for calls without scores
        scored(workspace=small)
    assert e.value.status == kvc.ERR_WORKSPACE
    for kw, err in ((dict(q=q.half()), TypeError), (dict(q=q[:, :, :64].contiguous()), ValueError),
                    (dict(out=out[:1]), ValueError), (dict(v_cache=k[:8]), ValueError),
                    (dict(block_tables=tables.long()), TypeError), (dict(block_tables=tables[:1]), ValueError),
                    (dict(context_lens=lens[:1]), ValueError), (dict(scores=scores[:, :, 1:].contiguous()), ValueError),
                    (dict(scores=scores.half()), TypeError), (dict(scores=None), TypeError),
                    (dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), ValueError),
                    (dict(q=q.cpu()), ValueError), (dict(workspace=None), TypeError)):
        with pytest.raises(err):
            scored(**kw)
    f32 = torch.zeros((9, H, BS, D), device="cuda")
    with pytest.raises(kvc.KvcError) as e:
        scored(k_cache=f32, v_cache=f32, q=q.float())
    assert e.value.status == kvc.ERR_UNSUPPORTED

    def block8(**kw):
        a = dict(q=q, k_cache=codes, v_cache=codes, k_scale=s, v_scale=s, block_tables=tables, context_lens=lens,
                 scale=0.1, out=out, workspace=ws, scores=scores)
        a.update(kw)
        kvc.decode_attention_block8(**a)

    for kw, err in ((dict(k_cache=k, v_cache=k), TypeError), (dict(k_scale=s[:8]), ValueError),
                    (dict(v_scale=s.half()), TypeError), (dict(v_cache=codes.to(torch.int8)), TypeError),
                    (dict(q=q.float()), kvc.KvcError)):
        with pytest.raises(err):
            block8(**kw)

    x = torch.zeros((3, H, D), dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([0, 1, 2], device="cuda")
    for a in ((x, x, slots[:2], codes, codes, s, s), (x, x.half(), slots, codes, codes, s, s),
              (x, x, slots.int(), codes, codes, s, s), (x, x, slots, codes, codes, s, s[:5]),
              (x, x, slots, k, k, s, s), (x[:, :1], x[:, :1], slots, codes, codes, s, s)):
        with pytest.raises((TypeError, ValueError)):
            kvc.append_block8(*a)

    new_tables = torch.zeros((B, 2), dtype=torch.int32, device="cuda")
    kept = torch.zeros((B, H, 32), dtype=torch.int32, device="cuda")
    new_lens, new_scores = torch.zeros_like(lens), torch.zeros((B, H, 32), device="cuda")

    def evict(**kw):
        a = dict(scores=scores, k_cache=k, v_cache=k, block_tables=tables, context_lens=lens, budget=32, recent=4,
                 new_block_tables=new_tables, kept=kept, new_lens=new_lens, new_scores=new_scores)
        a.update(kw)
        kvc.evict_rows(**a)

    for kw, err in ((dict(kept=kept[:, :, :8].contiguous()), ValueError), (dict(k_scale=s), ValueError),
                    (dict(new_scores=scores), ValueError), (dict(new_lens=lens), kvc.KvcError),
                    (dict(recent=40), kvc.KvcError), (dict(scores=scores.double()), TypeError),
                    (dict(new_block_tables=new_tables[:1]), ValueError), (dict(k_scale=s, v_scale=s), TypeError)):
        with pytest.raises(err):
            evict(**kw)
    torch.cuda.synchronize()
    assert kvc.get_error_flags() == 0
