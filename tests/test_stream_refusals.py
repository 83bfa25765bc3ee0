"""What prompts, windows with sinks and four-bit caches refuse, before any device work (no GPU)."""

import ctypes

import pytest
import torch

Z = ctypes.c_void_p(0)
P = ctypes.c_void_p(0x1000)  # never dereferenced: every call below fails before any device work
ODD = ctypes.c_void_p(0x1008)


def cache4(kvc, **kw):
    a = dict(k=P, v=P, slots=P, T=4, kc=P, vc=P, ks=P, vs=P, nb=10, bs=16, H=2, D=128, dtype=2)
    a.update(kw)
    lib = kvc.raw()
    first = lib.kvc_append_fp4(*a.values(), Z)
    second = lib.kvc_read_fp4(*[a[n] for n in ("slots", "T", "kc", "vc", "ks", "vs", "nb", "bs", "H", "D", "k", "v",
                                               "dtype")], Z)
    assert first == second
    return first


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), "INVALID_ARG"), (dict(T=-1), "INVALID_ARG"), (dict(nb=0), "INVALID_ARG"),
    (dict(H=0), "INVALID_ARG"), (dict(bs=0), "INVALID_ARG"), (dict(D=96), "UNSUPPORTED"), (dict(D=32), "UNSUPPORTED"),
    (dict(bs=8), "UNSUPPORTED"), (dict(bs=144), "UNSUPPORTED"), (dict(T=1 << 60), "UNSUPPORTED"),
    (dict(nb=1 << 60), "UNSUPPORTED"), (dict(k=Z), "INVALID_ARG"), (dict(vs=Z), "INVALID_ARG"),
    (dict(slots=Z), "INVALID_ARG"), (dict(v=ODD), "INVALID_ARG"), (dict(kc=ODD), "INVALID_ARG"),
    (dict(ks=ODD), "INVALID_ARG"),
])
def test_four_bit_rows_refuse(kvc, kw, status):
    assert cache4(kvc, **kw) == getattr(kvc, "ERR_" + status)
    assert kvc.raw().kvc_last_error_message() != b""


def test_four_bit_rows_of_nothing(kvc):
    assert cache4(kvc, T=0, k=Z, v=Z, slots=Z, kc=Z, vc=Z, ks=Z, vs=Z) == kvc.OK


def sinks(kvc, **kw):
    a = dict(q=P, k=P, v=P, tables=P, mb=4, lens=P, B=2, T=1, scale=0.1, hq=8, h=2, D=128, bs=16, nb=10, window=8,
             sinks=4, dtype=2, out=P, odt=0, ws=Z, wsb=0)
    a.update(kw)
    return kvc.raw().kvc_decode_attention_sinks(*a.values(), Z)


def fp4(kvc, **kw):
    a = dict(q=P, k=P, v=P, ks=P, vs=P, tables=P, mb=4, lens=P, B=2, T=1, scale=0.1, hq=8, h=2, D=128, bs=16, nb=10,
             window=8, sinks=4, dtype=2, out=P, odt=0, ws=Z, wsb=0)
    a.update(kw)
    return kvc.raw().kvc_decode_attention_fp4(*a.values(), Z)


DECODE = [
    (dict(B=0), "INVALID_ARG"), (dict(T=0), "INVALID_ARG"), (dict(mb=0), "INVALID_ARG"), (dict(hq=7), "INVALID_ARG"),
    (dict(D=32), "UNSUPPORTED"), (dict(D=100), "UNSUPPORTED"), (dict(bs=24), "UNSUPPORTED"),
    (dict(bs=256), "UNSUPPORTED"), (dict(B=4097), "UNSUPPORTED"), (dict(T=257), "UNSUPPORTED"),
    (dict(T=256, hq=34), "UNSUPPORTED"), (dict(mb=1 << 27), "UNSUPPORTED"), (dict(B=4096, mb=1 << 20), "UNSUPPORTED"),
    (dict(odt=5), "INVALID_ARG"), (dict(dtype=9), "INVALID_ARG"), (dict(dtype=0), "UNSUPPORTED"),
    (dict(nb=0), "INVALID_ARG"), (dict(nb=1 << 40), "UNSUPPORTED"), (dict(q=Z), "INVALID_ARG"),
    (dict(lens=Z), "INVALID_ARG"), (dict(out=Z), "INVALID_ARG"), (dict(q=ODD), "INVALID_ARG"),
    (dict(k=ODD), "INVALID_ARG"), (dict(window=0), "INVALID_ARG"), (dict(window=-5), "INVALID_ARG"),
    (dict(sinks=-1), "INVALID_ARG"),
]


@pytest.mark.parametrize("kw,status", DECODE)
def test_decode_with_sinks_refuses(kvc, kw, status):
    assert sinks(kvc, **kw) == getattr(kvc, "ERR_" + status)


@pytest.mark.parametrize("kw,status", DECODE + [(dict(ks=Z), "INVALID_ARG"), (dict(vs=Z), "INVALID_ARG"),
                                                (dict(ks=ODD), "INVALID_ARG"), (dict(B=2049), "UNSUPPORTED")])
def test_decode_fp4_refuses(kvc, kw, status):
    assert fp4(kvc, **kw) == getattr(kvc, "ERR_" + status)


def prompt(kvc, **kw):
    a = dict(q=P, k=P, v=P, tables=P, mb=4, starts=P, lens=P, B=2, T=9, scale=0.1, hq=8, h=2, D=128, bs=16, nb=10,
             window=8, sinks=4, dtype=2, out=P, ws=Z, wsb=0)
    a.update(kw)
    return kvc.raw().kvc_prompt_attention(*a.values(), Z)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), "INVALID_ARG"), (dict(T=-1), "INVALID_ARG"), (dict(mb=0), "INVALID_ARG"), (dict(hq=7), "INVALID_ARG"),
    (dict(h=0), "INVALID_ARG"), (dict(D=32), "UNSUPPORTED"), (dict(D=256), "UNSUPPORTED"),
    (dict(bs=24), "UNSUPPORTED"), (dict(bs=256), "UNSUPPORTED"), (dict(B=4097), "UNSUPPORTED"),
    (dict(hq=258), "UNSUPPORTED"), (dict(mb=1 << 27), "UNSUPPORTED"), (dict(T=1 << 29), "UNSUPPORTED"),
    (dict(dtype=9), "INVALID_ARG"), (dict(dtype=0), "UNSUPPORTED"), (dict(nb=0), "INVALID_ARG"),
    (dict(nb=1 << 40), "UNSUPPORTED"), (dict(q=Z), "INVALID_ARG"), (dict(starts=Z), "INVALID_ARG"),
    (dict(lens=Z), "INVALID_ARG"), (dict(out=Z), "INVALID_ARG"), (dict(q=ODD), "INVALID_ARG"),
    (dict(out=ODD), "INVALID_ARG"), (dict(window=0), "INVALID_ARG"), (dict(sinks=-1), "INVALID_ARG"),
])
def test_prompt_refuses(kvc, kw, status):
    assert prompt(kvc, **kw) == getattr(kvc, "ERR_" + status)
    assert kvc.raw().kvc_last_error_message() != b""


def test_prompt_of_nothing(kvc):
    assert prompt(kvc, T=0, q=Z, out=Z, starts=Z) == kvc.OK


def test_prompt_workspace_query_refuses(kvc):
    n = ctypes.c_size_t()
    fn = kvc.raw().kvc_prompt_workspace_size
    assert fn(2, 9, 7, 2, 128, 16, 4, ctypes.byref(n)) == kvc.ERR_INVALID_ARG
    assert fn(2, 9, 8, 2, 96, 16, 4, ctypes.byref(n)) == kvc.ERR_UNSUPPORTED
    assert fn(2, 9, 8, 2, 128, 16, 4, None) == kvc.ERR_INVALID_ARG


def test_the_binding_refuses_host_tensors_and_wrong_windows(kvc):
    x = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.append_fp4(x.float(), x.float(), x.long(), x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.read_fp4(x.long(), x, x, x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.decode_attention_fp4(x, x, x, x, x, x.int(), x.int(), 0.1, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.decode_attention_sinks(x, x, x, x.int(), x.int(), 0.1, None, 0, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.prompt_attention(x, x, x, x.int(), x.int(), x.int(), 0.1, x, x)
    for window, n in ((0, 0), (-1, 0), (1 << 31, 0), (5, -1), (5, 1 << 31)):
        with pytest.raises(ValueError, match="window"):
            kvc.decode_attention_sinks(x, x, x, x, x, 0.1, window, n, x, x)
        with pytest.raises(ValueError, match="window"):
            kvc.prompt_attention(x, x, x, x, x, x, 0.1, x, x, window=window, sinks=n)
