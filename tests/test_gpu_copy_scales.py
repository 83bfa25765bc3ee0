"""Copy-on-write of the scales of one-byte caches: kvc_copy_blocks on pools whose blocks are no multiple of 16 bytes."""

import ctypes

import numpy as np
import pytest
import torch

from test_gpu_append_block8 import Pools, rows

P, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1002)


def test_what_copy_blocks_refuses(kvc):
    def call(cache, block_bytes, n=1):
        return kvc.raw().kvc_copy_blocks(cache, 4, block_bytes, P, n, ctypes.c_void_p(0))

    for block_bytes in (-4, 0, 2, 6, 17):
        assert call(P, block_bytes) == kvc.ERR_INVALID_ARG
    assert call(ODD, 4) == kvc.ERR_INVALID_ARG
    assert call(ctypes.c_void_p(0x1004), 32) == kvc.ERR_INVALID_ARG
    assert call(ctypes.c_void_p(0), 8) == kvc.ERR_INVALID_ARG
    assert call(P, 8, n=-1) == kvc.ERR_INVALID_ARG
    assert call(P, 8, n=0) == kvc.OK


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [1, 2, 3, 4, 5, 7, 8])
def test_scales_of_any_number_of_heads(kvc, heads):
    gen = torch.Generator(device="cuda").manual_seed(heads)
    s = torch.rand((40, heads), generator=gen, device="cuda")
    want = s.clone()
    pairs = torch.tensor([[3, 39], [7, 0], [3, 12], [5, 5]], dtype=torch.int64, device="cuda")
    for a, b in pairs.tolist():
        want[b] = s[a]
    kvc.copy_blocks(s, pairs)
    assert torch.equal(s, want) and kvc.get_error_flags() == 0
    bad = torch.tensor([[1, 2], [40, 4], [6, -1]], dtype=torch.int64, device="cuda")
    want[2] = want[1]
    kvc.copy_blocks(s, bad)
    assert torch.equal(s, want) and kvc.get_error_flags() == kvc.FLAG_BAD_BLOCK
    view = torch.rand(40 * heads + 1, generator=gen, device="cuda")[1:].view(40, heads)  # 4-byte aligned
    if heads % 4:
        want = view.clone()
        want[9] = view[8]
        kvc.copy_blocks(view, torch.tensor([[8, 9]], device="cuda"))
        assert torch.equal(view, want)


@pytest.mark.gpu
@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_a_fork_writes_its_own_copy(kvc, code):
    H, D, bs = 3, 64, 16
    p = Pools(6, H, bs, D, code)
    pool = kvc.BlockPool(6, bs)
    parent = pool.add()
    p.append(kvc, *rows(20, H, D, "bf16", 1), pool.reserve(parent, 20))
    child = pool.fork(parent)
    slots, pair = pool.reserve_cow(child, 2)
    pairs = torch.tensor([pair], dtype=torch.int64, device="cuda")
    for i, (c, s) in enumerate(p.dev):
        kvc.copy_blocks(c, pairs)
        kvc.copy_blocks(s, pairs)
        p.host[i][0][pair[1]] = p.host[i][0][pair[0]]
        p.host[i][1][pair[1]] = p.host[i][1][pair[0]]
    p.append(kvc, *rows(2, H, D, "bf16", 2, spread=2.0), slots)
    p.append(kvc, *rows(1, H, D, "bf16", 3), pool.reserve(parent, 1))
    p.same()
    assert not np.array_equal(p.host[0][1][pair[0]], p.host[0][1][pair[1]])  # the child's rows were louder
