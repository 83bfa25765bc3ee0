"""What the block-scaled caches, the scored decode and the eviction refuse, before any device work (no GPU), and the
host pool's side of an eviction."""

import ctypes

import pytest
import torch

Z = ctypes.c_void_p(0)
P = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails before any device work
ODD = ctypes.c_void_p(0x1008)


def append(kvc, **kw):
    a = dict(k=P, v=P, slots=P, T=4, kc=P, vc=P, ks=P, vs=P, code=0, nb=10, bs=16, H=2, D=128, dtype=2)
    a.update(kw)
    return kvc.raw().kvc_append_block8(*a.values(), Z)


@pytest.mark.parametrize("kw,status", [
    (dict(code=2), "INVALID_ARG"), (dict(code=-1), "INVALID_ARG"), (dict(dtype=3), "INVALID_ARG"),
    (dict(T=-1), "INVALID_ARG"), (dict(nb=0), "INVALID_ARG"), (dict(H=0), "INVALID_ARG"),
    (dict(D=96), "UNSUPPORTED"), (dict(D=32), "UNSUPPORTED"), (dict(bs=8), "UNSUPPORTED"),
    (dict(bs=144), "UNSUPPORTED"), (dict(k=Z), "INVALID_ARG"), (dict(ks=Z), "INVALID_ARG"),
    (dict(slots=Z), "INVALID_ARG"), (dict(k=ODD), "INVALID_ARG"), (dict(vc=ODD), "INVALID_ARG"),
])
def test_append_block8_refuses(kvc, kw, status):
    assert append(kvc, **kw) == getattr(kvc, "ERR_" + status)
    assert kvc.raw().kvc_last_error_message() != b""


def test_append_block8_of_nothing(kvc):
    assert append(kvc, T=0, k=Z, v=Z, slots=Z, kc=Z, vc=Z, ks=Z, vs=Z) == kvc.OK


def scored(kvc, **kw):
    a = dict(q=P, k=P, v=P, tables=P, mb=4, lens=P, B=2, T=1, scale=0.1, hq=8, h=2, D=128, bs=16, nb=10, dtype=2, out=P,
             odt=0, scores=P, ws=Z, wsb=0)
    a.update(kw)
    return kvc.raw().kvc_decode_attention_scored(*a.values(), Z)


def block8(kvc, **kw):
    a = dict(q=P, k=P, v=P, ks=P, vs=P, code=0, tables=P, mb=4, lens=P, B=2, T=1, scale=0.1, hq=8, h=2, D=128, bs=16,
             nb=10, dtype=2, out=P, odt=0, scores=Z, ws=Z, wsb=0)
    a.update(kw)
    return kvc.raw().kvc_decode_attention_block8(*a.values(), Z)


DECODE = [
    (dict(B=0), "INVALID_ARG"), (dict(T=0), "INVALID_ARG"), (dict(mb=0), "INVALID_ARG"), (dict(hq=7), "INVALID_ARG"),
    (dict(D=32), "UNSUPPORTED"), (dict(D=100), "UNSUPPORTED"), (dict(bs=24), "UNSUPPORTED"),
    (dict(bs=256), "UNSUPPORTED"), (dict(B=4097), "UNSUPPORTED"), (dict(T=257), "UNSUPPORTED"),
    (dict(T=256, hq=34), "UNSUPPORTED"), (dict(mb=1 << 27), "UNSUPPORTED"), (dict(B=4096, mb=1 << 20), "UNSUPPORTED"),
    (dict(odt=5), "INVALID_ARG"), (dict(dtype=9), "INVALID_ARG"), (dict(dtype=0), "UNSUPPORTED"),
    (dict(nb=0), "INVALID_ARG"), (dict(nb=1 << 40), "UNSUPPORTED"), (dict(q=Z), "INVALID_ARG"),
    (dict(lens=Z), "INVALID_ARG"), (dict(out=Z), "INVALID_ARG"), (dict(q=ODD), "INVALID_ARG"),
    (dict(k=ODD), "INVALID_ARG"),
]


@pytest.mark.parametrize("kw,status", DECODE + [(dict(scores=Z), "INVALID_ARG")])
def test_decode_scored_refuses(kvc, kw, status):
    assert scored(kvc, **kw) == getattr(kvc, "ERR_" + status)


@pytest.mark.parametrize("kw,status", DECODE + [(dict(code=2), "INVALID_ARG"), (dict(ks=Z), "INVALID_ARG"),
                                                (dict(vs=Z), "INVALID_ARG")])
def test_decode_block8_refuses(kvc, kw, status):
    assert block8(kvc, **kw) == getattr(kvc, "ERR_" + status)


def test_workspace_query_refuses(kvc):
    n = ctypes.c_size_t()
    fn = kvc.raw().kvc_decode_scored_workspace_size
    assert fn(2, 1, 7, 2, 128, 16, 4, 1, ctypes.byref(n)) == kvc.ERR_INVALID_ARG
    assert fn(2, 1, 8, 2, 96, 16, 4, 1, ctypes.byref(n)) == kvc.ERR_UNSUPPORTED
    assert fn(2, 1, 8, 2, 128, 16, 4, 1, None) == kvc.ERR_INVALID_ARG


def evict(kvc, **kw):
    a = dict(scores=P, k=P, v=P, tables=P, mb=8, lens=P, B=2, budget=32, recent=8, new=ctypes.c_void_p(0x2000), nmb=2,
             nb=10, bs=16, H=2, D=128, dtype=2, kept=P, nl=ctypes.c_void_p(0x2000), ns=ctypes.c_void_p(0x2000))
    a.update(kw)
    return kvc.raw().kvc_evict_rows(*a.values(), Z)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), "INVALID_ARG"), (dict(H=0), "INVALID_ARG"), (dict(bs=0), "INVALID_ARG"), (dict(nb=0), "INVALID_ARG"),
    (dict(budget=0), "INVALID_ARG"), (dict(recent=-1), "INVALID_ARG"), (dict(recent=33), "INVALID_ARG"),
    (dict(budget=33), "INVALID_ARG"), (dict(D=0), "INVALID_ARG"), (dict(D=4), "UNSUPPORTED"),
    (dict(D=1 << 30), "UNSUPPORTED"), (dict(dtype=3), "INVALID_ARG"), (dict(mb=1 << 27), "UNSUPPORTED"), (dict(scores=Z), "INVALID_ARG"),
    (dict(kept=Z), "INVALID_ARG"), (dict(k=ODD), "INVALID_ARG"), (dict(ns=P), "INVALID_ARG"),
    (dict(nl=P), "INVALID_ARG"), (dict(new=P), "INVALID_ARG"),
])
def test_evict_refuses(kvc, kw, status):
    assert evict(kvc, **kw) == getattr(kvc, "ERR_" + status)


def test_evict_block8_refuses(kvc):
    fn = kvc.raw().kvc_evict_rows_block8
    q = ctypes.c_void_p(0x2000)

    def call(ks=P, vs=P, code=0, D=128):
        return fn(P, P, P, ks, vs, code, P, 8, P, 2, 32, 8, q, 2, 10, 16, 2, D, P, q, q, Z)

    assert call(ks=Z) == kvc.ERR_INVALID_ARG
    assert call(vs=Z) == kvc.ERR_INVALID_ARG
    assert call(code=7) == kvc.ERR_INVALID_ARG
    assert call(D=24) == kvc.ERR_UNSUPPORTED


def test_the_binding_refuses_host_tensors_and_wrong_shapes(kvc):
    x = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.decode_attention_scored(x, x, x, x, x, 0.1, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.append_block8(x, x, x, x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.evict_rows(x, x, x, x, x, 1, 0, x, x, x, x)
    with pytest.raises(TypeError):
        kvc.decode_attention_block8(None, None, None, None, None, None, None, 0.1, None, None)


def test_pool_evict(kvc):
    pool = kvc.BlockPool(12, 16)
    a, b = pool.add(), pool.add()
    pool.reserve(a, 70)  # blocks 0 .. 4
    pool.reserve(b, 16)  # block 5
    c = pool.fork(a)
    assert pool.tables([a], 5) == ([[0, 1, 2, 3, 4]], [70])
    pool.evict_batch([a], [33])
    assert pool.tables([a], 3) == ([[6, 7, 8]], [33])
    assert pool.tables([c], 5) == ([[0, 1, 2, 3, 4]], [70])  # the fork keeps the old blocks
    assert [pool.refcount(i) for i in range(9)] == [1] * 9
    with pytest.raises(kvc.KvcError):
        pool.evict_batch([c], [70])  # needs 5 of the 3 free blocks
    pool.free(c)
    assert pool.stats()["free_blocks"] == 8


def test_pool_evict_needs_blocks(kvc):
    pool = kvc.BlockPool(8, 16)
    a = pool.add()
    pool.reserve(a, 80)
    with pytest.raises(kvc.KvcError) as e:
        pool.evict_batch([a], [64])  # 4 fresh blocks, 3 free: the old ones still hold the rows
    assert e.value.status == kvc.ERR_NO_BLOCKS
    assert pool.length(a) == 80 and pool.tables([a], 5)[0] == [[0, 1, 2, 3, 4]]
    for n in (-1, 81):
        with pytest.raises(kvc.KvcError) as e:
            pool.evict_batch([a], [n])
        assert e.value.status == kvc.ERR_INVALID_ARG
    with pytest.raises(kvc.KvcError):
        pool.evict_batch([99], [0])
    pool.evict_batch([a], [48])
    assert pool.tables([a], 3) == ([[5, 6, 7]], [48])
    assert pool.reserve(a, 1) == [0]  # the old blocks are free again
    pool.evict_batch([a], [0])
    assert pool.length(a) == 0 and pool.stats()["free_blocks"] == 8
    pool.evict_batch([], [])


def test_pool_evict_batch_keeps_old_and_new_blocks_apart(kvc):
    pool = kvc.BlockPool(20, 16)
    seqs = [pool.add() for _ in range(3)]
    pool.reserve_batch(seqs, 64)  # blocks 0 .. 11
    old = {b for row in pool.tables(seqs, 4)[0] for b in row}
    for bad in ([seqs[0], seqs[0]], [seqs[0], 77, seqs[1]]):
        with pytest.raises(kvc.KvcError) as e:
            pool.evict_batch(bad, [16] * len(bad))
        assert e.value.status == kvc.ERR_INVALID_ARG
    with pytest.raises(kvc.KvcError) as e:
        pool.evict_batch(seqs, [48, 48, 48])  # 9 fresh blocks, 8 free: nothing changes
    assert e.value.status == kvc.ERR_NO_BLOCKS
    with pytest.raises(ValueError):
        pool.evict_batch(seqs, [1, 2])
    assert {b for row in pool.tables(seqs, 4)[0] for b in row} == old
    pool.evict_batch(seqs, [33, 17, 0])
    rows, lens = pool.tables(seqs, 3)
    assert rows == [[12, 13, 14], [15, 16, 0], [0, 0, 0]] and lens == [33, 17, 0]
    assert pool.stats()["free_blocks"] == 15
