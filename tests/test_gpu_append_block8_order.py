"""Block-scaled append: a slot mapping whose tokens of one block are not adjacent is flagged, whatever lies between them,
and one that keeps them together never is. In the flagged mappings here the blocks' scales are large enough already, so
that the runs of a block write the same scale and rows of their own: the result is that of the sorted mapping."""

import numpy as np
import pytest
import torch

from oracle import long_context as O

from test_gpu_append_block8 import Pools, rows

pytestmark = pytest.mark.gpu
CODES = ["e4m3", "int8"]


@pytest.fixture(autouse=True)
def _checked(kvc):
    kvc.get_error_flags()
    yield
    kvc.set_option(kvc.OPT_CHECKED, 0)
    kvc.get_error_flags()


def filled(nb, H, bs, D, code):
    """Pools whose scales no test row exceeds."""
    p = Pools(nb, H, bs, D, code)
    for i, (c, s) in enumerate(p.host):
        s[:] = 8.0
        p.dev[i][1].fill_(8.0)
    return p


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("B,T", [(2, 2), (7, 3), (64, 4), (300, 5)])
def test_token_major_mappings_are_flagged(kvc, code, B, T):
    H, D, bs = 2, 64, 16
    p = filled(B, H, bs, D, code)
    order = np.random.default_rng(B).permutation(B)
    slots = [int(b) * bs + 4 + t for t in range(T) for b in order]
    p.append(kvc, *rows(len(slots), H, D, "bf16", 1), slots)
    p.same()
    assert kvc.get_error_flags() == kvc.FLAG_BAD_SLOT
    slots = [int(b) * bs + 9 + t for b in order for t in range(T)]
    p.append(kvc, *rows(len(slots), H, D, "bf16", 2), slots)
    p.same()
    assert kvc.get_error_flags() == 0


@pytest.mark.parametrize("slots", [[3, -1, 4], [1, 20, 2], [40, 41, 7, 42], [5, 16 * 9, 6], [5, -7, -7, -7, 5]])
def test_a_block_left_and_met_again(kvc, slots):
    H, D, bs, nb = 1, 128, 16, 9
    p = filled(nb, H, bs, D, "e4m3")
    k, v = rows(len(slots), H, D, "f16", 3)
    if slots[0] == slots[-1]:  # one slot twice: equal rows
        k[-1], v[-1] = k[0], v[0]
    t = torch.tensor(slots, dtype=torch.int64, device="cuda")
    kvc.append_block8(k.cuda(), v.cuda(), t, p.dev[0][0], p.dev[1][0], p.dev[0][1], p.dev[1][1])
    torch.cuda.synchronize()
    assert kvc.get_error_flags() == kvc.FLAG_BAD_SLOT
    good = [s if s < nb * bs else -1 for s in slots]
    p.host = [O.append_block8(x.float().numpy(), good, c, s, "e4m3") for x, (c, s) in zip((k, v), p.host)]
    p.same()


@pytest.mark.parametrize("T,gap,H", [(641, 640, 1), (2560, 2559, 1), (2000, 2, 3), (2561, 1280, 1), (20000, 1280, 1),
                                     (20000, 1, 2), (20000, 700, 5), (70000, 1200, 1), (1920, 1919, 40)])
def test_among_many_blocks(kvc, T, gap, H):
    # every token in a block of its own but for two, `gap` tokens apart, at the beginning, the end and in between
    D, bs = 64, 16
    rng = np.random.default_rng(T)
    blocks = rng.permutation(T)
    slots = blocks * bs + rng.integers(1, bs, T)
    codes = [torch.zeros((T, H, bs, D), dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.ones((T, H), device="cuda") for _ in range(2)]
    x = torch.randn((T, H, D), device="cuda", dtype=torch.bfloat16)

    def flags():
        kvc.append_block8(x, x, torch.from_numpy(slots).cuda(), *codes, *scales)
        return kvc.get_error_flags()

    assert flags() == 0
    for a in sorted({min(a, T - gap - 1) for a in (0, 1, (T - gap) // 3, (T - gap) // 2, T)}):
        old = slots[a + gap]
        slots[a + gap] = slots[a] // bs * bs + (slots[a] % bs % (bs - 1)) + 1
        assert flags() == (kvc.FLAG_BAD_SLOT if gap > 1 else 0)  # neighbours make one run
        slots[a + gap] = old
    assert flags() == 0


def test_long_mappings_in_order_are_not_flagged(kvc):
    rng = np.random.default_rng(7)
    H, D, bs, nb = 1, 64, 32, 6000
    slots = []
    for b in rng.permutation(nb):
        first = int(rng.integers(0, bs))
        run = [int(b) * bs + r for r in range(first, int(rng.integers(first + 1, bs + 1)))]
        slots += run[::-1] if rng.random() < 0.2 else run
        slots += [-1] * int(rng.integers(0, 3))
    p = Pools(nb, H, bs, D, "int8")
    p.append(kvc, *rows(len(slots), H, D, "bf16", 4), slots)
    p.same()
    assert kvc.get_error_flags() == 0


def test_checked_mode_and_replays_report(kvc):
    H, D, bs = 2, 64, 16
    p = filled(3, H, bs, D, "int8")
    k, v = (x.cuda() for x in rows(3, H, D, "f16", 5))
    t = torch.tensor([4, 5, 6], dtype=torch.int64, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvc.append_block8(k, v, t, p.dev[0][0], p.dev[1][0], p.dev[0][1], p.dev[1][1])
    g.replay()
    assert kvc.get_error_flags() == 0
    t.copy_(torch.tensor([7, 17, 8]))
    g.replay()
    assert kvc.get_error_flags() == kvc.FLAG_BAD_SLOT
    kvc.set_option(kvc.OPT_CHECKED, 1)
    with pytest.raises(kvc.KvcError) as e:
        kvc.append_block8(k, v, t, p.dev[0][0], p.dev[1][0], p.dev[0][1], p.dev[1][1])
    assert e.value.status == kvc.ERR_OUT_OF_RANGE
    t.copy_(torch.tensor([7, 8, 17]))
    kvc.append_block8(k, v, t, p.dev[0][0], p.dev[1][0], p.dev[0][1], p.dev[1][1])
