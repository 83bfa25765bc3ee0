"""The oracle of windows with sinks and four-bit rows, against direct statements and exhaustive tables (no GPU)."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import streams as O


def test_tables():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert np.array_equal(O.E4M3, codes.float().numpy())
    for c in range(8):  # sign, two exponent bits, one mantissa bit
        e, m = c >> 1, c & 1
        assert O.E2M1[c] == (m * 0.5 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1))


def test_nearest_is_nearest_even():
    for table in (O.E2M1, O.E4M3):
        for i in range(len(table) - 1):
            mid = (Fraction(float(table[i])) + Fraction(float(table[i + 1]))) / 2
            assert O.nearest(mid, table) == (i if i % 2 == 0 else i + 1)
            assert O.nearest(mid * Fraction(2 ** 40 - 1, 2 ** 40), table) == i
            assert O.nearest(mid * Fraction(2 ** 40 + 1, 2 ** 40), table) == i + 1
        assert O.nearest(Fraction(10 ** 9), table) == len(table) - 1


def test_rows_of_representable_values_come_back():
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 16, (6, 64)).astype(np.uint8)
    codes[:, ::16] = 7  # the largest code in every group: the scale is then exact
    scales = rng.integers(1, 127, (6, 4)).astype(np.uint8)
    x = O.values_fp4(O.pack(codes), scales)
    c, s = O.encode_fp4(x)
    assert np.array_equal(s, scales) and np.array_equal(O.values_fp4(O.pack(c), s), x)


def test_what_is_not_finite():
    x = np.zeros(16)
    x[:4] = [np.inf, -np.inf, np.nan, 3.0]
    c, s = O.encode_fp4(x)
    assert list(c[:4]) == [7, 15, 0, 7] and O.E4M3[s[0]] == 0.5


@pytest.mark.parametrize("window,sinks", [(None, 0), (1, 0), (3, 2), (100, 4), (2, 50)])
def test_visible_is_the_rule(window, sinks):
    seen = O.visible(range(5, 9), 9, window, sinks)
    for t, pos in enumerate(range(5, 9)):
        for r in range(9):
            assert seen[t, r] == (r <= pos and (window is None or r > pos - window or r < sinks))


def test_attend_is_softmax():
    rng = np.random.default_rng(1)
    K, V = rng.standard_normal((2, 3, 2, 16, 64))
    q = rng.standard_normal((4, 6, 64))
    table = [2, 0, 1]
    out, mass, _ = O.attend(q, K, V, table, 40, 0.3, 10, 3)
    k, v = (torch.from_numpy(x[table].transpose(1, 0, 2, 3).reshape(2, 48, 64)[:, :40]) for x in (K, V))
    mask = torch.from_numpy(O.visible(range(36, 40), 40, 10, 3))
    ref = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q).transpose(0, 1), k.repeat_interleave(3, 0), v.repeat_interleave(3, 0), mask, scale=0.3)
    assert np.allclose(out, ref.transpose(0, 1).numpy(), atol=1e-12) and (mass >= np.abs(out) - 1e-12).all()
