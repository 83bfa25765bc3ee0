"""GPU parity: append into block-scaled one-byte caches (kvc_append_block8): codes and scales bit for bit."""

import numpy as np
import pytest
import torch

from oracle import long_context as O

from long_context_helpers import TORCH

pytestmark = pytest.mark.gpu
CODES = ["e4m3", "int8"]


class Pools:
    def __init__(self, nb, H, bs, D, code, seed=0):
        rng = np.random.default_rng(seed)
        self.code, self.H, self.D, self.bs = code, H, D, bs
        if code == "int8":
            c = rng.integers(-127, 128, (2, nb, H, bs, D)).astype(np.int8)
        else:
            c = rng.integers(0, 256, (2, nb, H, bs, D)).astype(np.uint8)  # NaN codes among them: stale rows
        s = (rng.random((2, nb, H)) * 0.02).astype(np.float32)
        self.host = [(c[i], s[i]) for i in range(2)]
        self.dev = [(torch.from_numpy(a).cuda(), torch.from_numpy(b).cuda()) for a, b in self.host]

    def append(self, kvc, k, v, slots, stream=None):
        t = torch.tensor(slots, dtype=torch.int64, device="cuda")
        (kc, ks), (vc, vs) = self.dev
        kvc.append_block8(k.cuda(), v.cuda(), t, kc, vc, ks, vs, stream=stream)
        self.host = [O.append_block8(x.float().numpy(), slots, c, s, self.code) for x, (c, s) in zip((k, v), self.host)]

    def same(self):
        torch.cuda.synchronize()
        for (c, s), (hc, hs) in zip(self.dev, self.host):
            assert np.array_equal(s.cpu().numpy().view(np.uint32), hs.view(np.uint32))
            assert np.array_equal(c.cpu().numpy(), hc)


def rows(T, H, D, dtype, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((2, T, H, D)) * np.exp(spread * rng.standard_normal((2, T, H, 1)))
    return [torch.from_numpy(a).to(TORCH[dtype]) for a in x]


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,bs,H", [(64, 16, 3), (128, 32, 2), (256, 48, 1), (128, 128, 2)])
def test_prompts_then_steps(kvc, code, dtype, D, bs, H):
    """A ragged prefill, then single tokens that grow the scales of partly filled blocks."""
    p = Pools(40, H, bs, D, code, seed=D)
    pool = kvc.BlockPool(40, bs)
    seqs = [pool.add() for _ in range(4)]
    slots = sum((pool.reserve(s, n) for s, n in zip(seqs, (1, bs - 1, bs, 2 * bs + 5))), [])
    p.append(kvc, *rows(len(slots), H, D, dtype, 1), slots)
    p.same()
    for step in range(5):
        slots = sum(pool.reserve_batch(seqs, 1), [])
        p.append(kvc, *rows(len(slots), H, D, dtype, 2 + step, spread=2.0), slots)
    p.same()
    slots = sum(pool.reserve_batch(seqs, bs + 3), [])
    p.append(kvc, *rows(len(slots), H, D, dtype, 9), slots)
    p.same()


@pytest.mark.parametrize("code", CODES)
def test_long_prompts_share_warps(kvc, code):
    # enough tokens that a warp looks at many of them, with runs that begin and end anywhere
    rng = np.random.default_rng(3)
    H, D, bs, nb = 8, 64, 16, 700
    slots = []
    for b in rng.permutation(nb):
        first = int(rng.integers(0, bs))
        slots += [int(b) * bs + r for r in range(first, int(rng.integers(first + 1, bs + 1)))]
        slots += [-1] * int(rng.integers(0, 3))
    p = Pools(nb, H, bs, D, code, seed=5)
    p.append(kvc, *rows(len(slots), H, D, "bf16", 4), slots)
    p.same()


@pytest.mark.parametrize("code", CODES)
def test_skipped_and_bad_slots(kvc, code):
    H, D, bs, nb = 2, 128, 16, 6
    p = Pools(nb, H, bs, D, code)
    slots = [-1, 16, 17, -7, 40, nb * bs, 2 ** 40, -1]
    k, v = rows(len(slots), H, D, "bf16", 6)
    t = torch.tensor(slots, dtype=torch.int64, device="cuda")
    kvc.append_block8(k.cuda(), v.cuda(), t, p.dev[0][0], p.dev[1][0], p.dev[0][1], p.dev[1][1])
    torch.cuda.synchronize()
    assert kvc.get_error_flags() == kvc.FLAG_BAD_SLOT
    good = [s if s < nb * bs else -1 for s in slots]
    p.host = [O.append_block8(x.float().numpy(), good, c, s, code) for x, (c, s) in zip((k, v), p.host)]
    p.same()
    none = torch.empty((0, H, D), dtype=torch.bfloat16, device="cuda")
    kvc.append_block8(none, none, t[:0], p.dev[0][0], p.dev[1][0], p.dev[0][1], p.dev[1][1])
    p.same()


@pytest.mark.parametrize("code", CODES)
def test_zeros_infinities_nan_and_the_ends_of_the_range(kvc, code):
    H, D, bs = 1, 64, 16
    p = Pools(8, H, bs, D, code)
    k, v = rows(8, H, D, "f32", 7)
    k[0] = 0
    k[1, 0, 3], k[1, 0, 4], k[1, 0, 5] = float("inf"), float("-inf"), float("nan")
    k[2] = 0
    k[2, 0, 1] = float("inf")  # no finite entry but 0
    k[3] *= 1e-44  # denormal values: a scale below the smallest normal number
    k[4] *= 3e-38
    k[5] *= 1e38 / k[5].abs().max()
    k[6, 0, 0] = 3.4028234663852886e38
    v[7] = -0.0
    slots = [i * bs for i in range(8)]
    p.append(kvc, k, v, slots)
    p.same()
    # after an all-zero (or too small) row the next one sets the scale; a louder one rounds the codes again
    p.append(kvc, *rows(8, H, D, "f32", 8), [s + 1 for s in slots])
    p.same()


def test_rewriting_rows(kvc):
    """Rejected speculative tokens: the rows are written again; row 0 starts a block afresh."""
    for code in CODES:
        p = Pools(3, 2, 16, 128, code)
        p.append(kvc, *rows(12, 2, 128, "bf16", 1), list(range(16, 28)))
        p.append(kvc, *rows(4, 2, 128, "bf16", 2, spread=3.0), list(range(20, 24)))
        p.append(kvc, *rows(2, 2, 128, "bf16", 3), [22, 23])
        p.same()
        p.append(kvc, *rows(1, 2, 128, "bf16", 4), [16])
        p.same()


@pytest.mark.parametrize("code", CODES)
def test_on_a_stream_and_in_a_graph(kvc, code):
    p = Pools(4, 2, 16, 64, code)
    s = torch.cuda.Stream()
    p.append(kvc, *rows(5, 2, 64, "f16", 1), list(range(5)), stream=s)
    p.same()
    k, v = (x.cuda() for x in rows(3, 2, 64, "f16", 2, spread=2.0))
    t = torch.tensor([5, 6, 7], dtype=torch.int64, device="cuda")
    (kc, ks), (vc, vs) = p.dev
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvc.append_block8(k, v, t, kc, vc, ks, vs)
    for step in range(3):
        k2, v2 = rows(3, 2, 64, "f16", 20 + step, spread=2.0)
        slots = [5 + 3 * step, 6 + 3 * step, 7 + 3 * step]
        k.copy_(k2), v.copy_(v2), t.copy_(torch.tensor(slots))
        g.replay()
        p.host = [O.append_block8(x.float().numpy(), slots, c, sc, code) for x, (c, sc) in zip((k2, v2), p.host)]
        p.same()


def test_unwritten_blocks_are_left_alone(kvc):
    p = Pools(5, 2, 32, 128, "e4m3")
    p.append(kvc, *rows(3, 2, 128, "bf16", 1), [64, 65, 66])
    p.same()  # compares every block


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("T", [40, 300, 700])
def test_one_slot_named_many_times(kvc, code, T):
    """Tokens of one slot race; with equal rows the result is theirs. The runs are longer than any block."""
    H, D, bs = 2, 64, 16
    p = Pools(6, H, bs, D, code, seed=T)
    k, v = (x[:1].expand(T, H, D).contiguous() for x in rows(1, H, D, "bf16", 3))
    p.append(kvc, k, v, [2 * bs + 5] * T)
    p.same()
    p.append(kvc, k, v, [3 * bs] * (T - 3) + [3 * bs + 1, 4 * bs + 7, -1])
    p.same()


def test_offsets_past_32_bits(kvc):
    H, D, bs, nb = 8, 256, 128, 16500  # 4.3e9 codes per pool
    assert nb * H * bs * D > 2 ** 32
    codes = [torch.empty((nb, H, bs, D), dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.zeros((nb, H), device="cuda") for _ in range(2)]
    slots = [(nb - 1) * bs + r for r in range(100)] + [(nb - 2) * bs + 3, 5]
    k, v = rows(len(slots), H, D, "bf16", 1)
    before = [c[torch.tensor([nb - 1, nb - 2, 0], device="cuda")].cpu().numpy() for c in codes]
    kvc.append_block8(k.cuda(), v.cuda(), torch.tensor(slots, device="cuda"), *codes, *scales)
    small = [r for r in range(100)] + [bs + 3, 2 * bs + 5]  # the same in a pool of the three blocks
    for x, c, s, b in zip((k, v), codes, scales, before):
        want, ws = O.append_block8(x.float().numpy(), small, b, np.zeros((3, H), dtype=np.float32), "int8")
        at = torch.tensor([nb - 1, nb - 2, 0], device="cuda")
        assert np.array_equal(c[at].cpu().numpy(), want) and np.array_equal(s[at].cpu().numpy(), ws)
