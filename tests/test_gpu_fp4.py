"""GPU parity: four-bit caches: append, reading back, and both with the attentions that use them."""

import numpy as np
import pytest
import torch

from oracle import streams as O

from long_context_helpers import TORCH, f64
from stream_helpers import close, int32, tolerance

pytestmark = pytest.mark.gpu


class Cache:
    def __init__(self, nb, H, bs, D, seed=0):
        rng = np.random.default_rng(seed)
        self.host = [rng.integers(0, 256, (nb, H, bs, D // n)).astype(np.uint8) for n in (2, 2, 16, 16)]
        self.dev = [torch.from_numpy(x).cuda() for x in self.host]  # k, v, k_scale, v_scale
        self.bs = bs

    def append(self, kvc, k, v, slots, stream=None):
        kvc.append_fp4(k, v, torch.tensor(slots, dtype=torch.int64, device="cuda"), *self.dev, stream=stream)
        for j, x in enumerate((f64(k), f64(v))):
            codes, scales = O.encode_fp4(x)
            for t, s in enumerate(slots):
                if s >= 0:
                    self.host[j][s // self.bs, :, s % self.bs] = O.pack(codes[t])
                    self.host[j + 2][s // self.bs, :, s % self.bs] = scales[t]

    def same(self):
        torch.cuda.synchronize()
        got = [x.cpu().numpy() for x in self.dev]
        for j in range(2):
            assert np.array_equal(got[j + 2], self.host[j + 2])
            a, b = O.unpack(got[j]), O.unpack(self.host[j])
            # a zero may have either sign
            assert np.array_equal(np.where(a == 8, 0, a), np.where(b == 8, 0, b))


def rows(T, H, D, dtype, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((2, T, H, D)) * np.exp(1.5 * rng.standard_normal((2, T, H, 1)))
    return [torch.from_numpy(a).to(TORCH[dtype]).cuda() for a in x]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,bs,H", [(64, 16, 3), (128, 48, 2), (256, 128, 1)])
def test_append_and_read_back(kvc, dtype, D, bs, H):
    c = Cache(6, H, bs, D, seed=D)
    slots = list(np.random.default_rng(1).permutation(6 * bs)[:37])
    slots[5] = slots[20] = -1
    k, v = rows(37, H, D, dtype, 2)
    c.append(kvc, k, v, slots)
    c.same()
    for out in ("f32", "f16", "bf16"):
        a, b = (torch.full((37, H, D), 7.0, dtype=TORCH[out], device="cuda") for _ in range(2))
        kvc.read_fp4(torch.tensor(slots, dtype=torch.int64, device="cuda"), *c.dev, a, b)
        for j, x in enumerate((a, b)):
            want = O.values_fp4(c.host[j], c.host[j + 2])
            for t, s in enumerate(slots):
                assert np.array_equal(f64(x[t]), want[s // bs, :, s % bs] if s >= 0 else np.full((H, D), 7.0))
    assert kvc.get_error_flags() == 0


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_values_beside_every_border(kvc, dtype):
    """Quotients on every midpoint of codes and of scales, and the nearest inputs on either side."""
    mids = (O.E2M1[1:] + O.E2M1[:-1]) / 2
    groups = []
    for s in list(O.E4M3[8:127:7]) + [O.E4M3[1], O.E4M3[5], O.E4M3[8], O.E4M3[126]]:
        groups.append([6 * s] + [m * s for m in mids] + [-m * s for m in mids] + [0.0])
    for a, b in zip(O.E4M3[:-1], O.E4M3[1:]):  # scales halfway between two
        groups.append([3 * (a + b)] + [0.25 * a, 5 * b, -2.5 * a, a] + [0.0] * 11)
    x = torch.tensor(np.array(groups)).to(TORCH[dtype])
    up, down = (torch.nextafter(x, torch.full_like(x, w)) for w in (float("inf"), float("-inf")))
    x = torch.cat([x, up, down])
    x = torch.cat([x, torch.zeros((-len(x)) % 4, 16, dtype=x.dtype)]).reshape(-1, 1, 64).cuda()
    x = x[torch.isfinite(x).all(-1)[:, 0]]
    c = Cache(-(-len(x) // 16), 1, 16, 64)
    c.append(kvc, x, x.flip(0).contiguous(), list(range(len(x))))
    c.same()


def test_what_is_not_finite_and_extreme(kvc):
    inf, nan = float("inf"), float("nan")
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).tiny
        x = torch.zeros((8, 1, 64), dtype=dtype)
        x[0, 0, :4] = torch.tensor([inf, -inf, nan, 3.0])
        x[1] = nan
        x[2] = inf
        x[3, 0, ::3] = big
        x[4, 0, ::5] = -tiny
        x[5, 0, :] = 6 * 2.0 ** -10  # halfway between the scales 0 and 2^-9: 0
        x[6, 0, :] = -0.0
        x[7, 0, 1] = 2.0 ** -6
        c = Cache(1, 1, 16, 64)
        c.append(kvc, x.cuda(), x.flip(0).contiguous().cuda(), list(range(8)))
        c.same()


def test_slots_outside_the_pool(kvc):
    c = Cache(2, 2, 16, 64)
    k, v = rows(4, 2, 64, "bf16", 3)
    kvc.append_fp4(k, v, torch.tensor([5, 32, -7, 1 << 40], device="cuda"), *c.dev)
    assert kvc.get_error_flags() == kvc.FLAG_BAD_SLOT
    c.append(kvc, k[:1], v[:1], [5])
    c.same()
    a, b = (torch.full((3, 2, 64), 7.0, device="cuda") for _ in range(2))
    kvc.read_fp4(torch.tensor([32, 5, -1], device="cuda"), *c.dev, a, b)
    assert kvc.get_error_flags() == kvc.FLAG_BAD_SLOT
    assert (a[[0, 2]] == 7).all() and (b[[0, 2]] == 7).all()
    assert np.array_equal(f64(a[1]), O.values_fp4(c.host[0], c.host[2])[0, :, 5])
    empty = torch.zeros((0, 2, 64), device="cuda")
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    kvc.append_fp4(empty, empty, none, *c.dev)
    kvc.read_fp4(none, *c.dev, empty, empty)


def test_copied_blocks_keep_their_values(kvc):
    c = Cache(4, 2, 16, 128)
    pairs = torch.tensor([[1, 3], [0, 2]], device="cuda")
    for x, h in zip(c.dev, c.host):
        kvc.copy_blocks(x, pairs)
        h[3], h[2] = h[1], h[0]
        assert np.array_equal(x.cpu().numpy(), h)


def test_a_stream_served_in_four_bits(kvc):
    """Together as they are used, captured steps among them: a prompt's 16-bit rows go into a four-bit cache; its next
    chunk reads the history back and attends to what is cached; single tokens follow through the window with sinks."""
    H, G, D, bs, window, sinks = 2, 4, 128, 16, 100, 4
    rng = np.random.default_rng(5)
    nb = 40
    pool = kvc.BlockPool(nb, bs)
    seqs = [pool.add(), pool.add()]
    c = Cache(nb, H, bs, D, seed=1)
    wide = [torch.zeros((nb, H, bs, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = kvc.new_prompt_workspace(2, 512, H * G, H, D, bs, 16)
    wd = kvc.new_scored_workspace(2, 1, H * G, H, D, bs, 16, scored=False)

    def draw(*shape):
        return torch.from_numpy(1.2 * rng.standard_normal(shape)).to(torch.bfloat16).cuda()

    def check(out, q, i, n):
        K, V = O.values_fp4(c.host[0], c.host[2]), O.values_fp4(c.host[1], c.host[3])
        ref, mass, size = O.attend(f64(q), K, V, pool.tables([seqs[i]], 16)[0][0], n, D ** -0.5, window, sinks)
        close(f64(out), ref, tolerance(ref, mass, size, D, n, D ** -0.5, torch.bfloat16 if out.dtype == torch.bfloat16 else None,
                                       out.dtype))

    history = []  # slots of every cached row, in the pool of 16-bit rows too
    for new in ((70, 130), (90, 1), (33, 60)):
        slots = [pool.reserve(s, m) for s, m in zip(seqs, new)]
        flat = sum(slots, [])
        history += flat
        c.append(kvc, draw(len(flat), H, D), draw(len(flat), H, D), flat)
        k, v = (torch.empty((len(history), H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        t = torch.tensor(history, dtype=torch.int64, device="cuda")
        kvc.read_fp4(t, *c.dev, k, v)
        kvc.append(k, v, t, *wide)
        rows_, lens = pool.tables(seqs, 16)
        q = draw(len(flat), H * G, D)
        out = torch.empty_like(q)
        kvc.prompt_attention(q, *wide, int32(rows_), int32([0, new[0], sum(new)]), int32(lens), D ** -0.5, out, ws,
                             window=window, sinks=sinks)
        torch.cuda.synchronize()
        check(out[:new[0]], q[:new[0]], 0, lens[0])
        check(out[new[0]:], q[new[0]:], 1, lens[1])
    k, v, q = draw(2, H, D), draw(2, H, D), draw(2, H * G, D)
    out = torch.empty((2, H * G, D), device="cuda")
    slots, tables, lens = torch.zeros(2, dtype=torch.int64, device="cuda"), int32([[0] * 16] * 2), int32([1, 1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvc.append_fp4(k, v, slots, *c.dev)
        kvc.decode_attention_fp4(q, c.dev[0], c.dev[1], c.dev[2], c.dev[3], tables, lens, D ** -0.5, out, wd,
                                 window=window, sinks=sinks)
    for _ in range(3):
        new = sum(pool.reserve_batch(seqs, 1), [])
        rows_, n = pool.tables(seqs, 16)
        for dst, src in ((k, draw(2, H, D)), (v, draw(2, H, D)), (q, draw(2, H * G, D)), (tables, int32(rows_)),
                         (lens, int32(n)), (slots, torch.tensor(new, device="cuda"))):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        for j, x in enumerate((k, v)):
            codes, scales = O.encode_fp4(f64(x))
            for i, s in enumerate(new):
                c.host[j][s // bs, :, s % bs], c.host[j + 2][s // bs, :, s % bs] = O.pack(codes[i]), scales[i]
        c.same()
        for i in range(2):
            check(out[i:i + 1], q[i:i + 1], i, n[i])
    assert kvc.get_error_flags() == 0


def test_rows_far_up_a_large_pool(kvc):
    """Byte offsets beyond 32 bits, and rows on both sides of them."""
    nb, H, bs, D = 700000, 8, 16, 128
    dev = [torch.zeros((nb, H, bs, D // n), dtype=torch.uint8, device="cuda") for n in (2, 2, 16, 16)]
    slots = [0, 5, nb * bs - 1, (nb - 3) * bs + 7, 524287 * bs + 15, 524288 * bs]
    k, v = rows(len(slots), H, D, "bf16", 9)
    t = torch.tensor(slots, dtype=torch.int64, device="cuda")
    kvc.append_fp4(k, v, t, *dev)
    a, b = torch.zeros_like(k), torch.zeros_like(v)
    kvc.read_fp4(t, *dev, a, b)
    for j, (x, back) in enumerate(((k, a), (v, b))):
        codes, scales = O.encode_fp4(f64(x))
        want = O.values_fp4(O.pack(codes), scales)
        assert np.array_equal(f64(back), want)
        for i, s in enumerate(slots):
            assert np.array_equal(dev[j + 2][s // bs, :, s % bs].cpu().numpy(), scales[i])
        assert int((dev[j + 2] != 0).sum()) == int((scales != 0).sum())  # nothing else was written
    assert kvc.get_error_flags() == 0
