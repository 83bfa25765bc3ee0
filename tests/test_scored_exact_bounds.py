"""The bounds of tests/test_gpu_scored_exact.py catch errors: faults planted in a float64 decode exceed them, and the same
decode without one does not."""

import numpy as np
import pytest
import torch

from oracle import long_context as O

import scored_exact_helpers as X

KINDS = ["bf16", "f16", "e4m3", "int8"]


def setup(kind, case):
    q, pools, tables, old = X.inputs(kind, case)
    K, V = pools[0][2], pools[1][2]
    ref, ref_scores = O.decode_scored(q, K, V, tables, case[0], case[6], old)
    vs = None if pools[1][1] is None else pools[1][1].numpy()
    return q, K, V, vs, tables, old, ref, ref_scores


def faults(case):
    """Those that show on a case: one new token has no mask; in peaked cases the weights of single rows vanish."""
    yield from ("none", "query", "parts")
    if case[6] < X.PEAKED:
        yield from ("tile", "last", "scores")
        if case[1] > 1:
            yield "mask"


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case,fault", [
    pytest.param(c, f, id=f"{f}-D{c[4]}-T{c[1]}-{len(c[0])}x{max(c[0])}-{c[6]:g}") for c in X.CASES for f in faults(c)])
def test_a_planted_fault_exceeds_the_bounds(kind, case, fault):
    q, K, V, vs, tables, old, ref, ref_scores = setup(kind, case)
    tol, tol_scores = X.bounds(kind, q, K, V, vs, tables, case[0], case[6], torch.float32, ref, old)
    out, new = X.wrong(kind, q, K, V, tables, case[0], case[6], old, fault)
    worst, worst_scores = (np.abs(out - ref) / tol).max(), (np.abs(new - ref_scores) / np.maximum(tol_scores, 1e-300)).max()
    if fault == "none":
        assert worst < 0.01 and worst_scores < 0.01
    elif fault == "scores":
        assert worst_scores > 2
    else:
        assert worst > 2
        if fault in ("query", "tile", "mask"):
            assert worst_scores > 2


@pytest.mark.parametrize("kind", KINDS)
def test_the_scores_of_these_inputs_are_exact_in_fp32(kind):
    for case in X.CASES:
        q, pools, tables, _ = X.inputs(kind, case)
        assert np.abs(q).sum(-1).max() * np.abs(pools[0][2]).max() < 2 ** 23  # and every term a multiple of 1/2
        assert np.array_equal(pools[0][2] * 2, np.round(pools[0][2] * 2))
