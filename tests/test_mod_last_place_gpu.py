"""Scores so large that neighbouring floats are further apart than the lag that
the running maximum is allowed."""
import numpy as np
import pytest
import torch

import oracle

from mod_ref import LOG2E, Case, Mod, bits, run_decode, run_prefill

pytestmark = pytest.mark.gpu

UNIT = 128  # tokens of one score: a unit of the decode kernel, two tiles of the chunks'


@pytest.mark.parametrize("power", [20, 23, 24, 25, 26, 27, 28, 30])
@pytest.mark.parametrize("c", [(8, 2, 128, 1), (24, 4, 256, 1), (24, 4, 256, 4), (16, 2, 128, 10), (24, 4, 256, 16),
                               (8, 2, 256, 0), (24, 4, 128, 0)], ids=lambda c: f"{c[0]}_{c[1]}_{c[2]}_T{c[3]}")
def test_scores_that_rise_by_their_last_place(c, power):
    """Nine runs of keys whose base-2 scores 1.3125 * 2^power go up by one float
    each.  Scores are good to some 2^-20 of their size, so any weighing of the
    runs is right: the output lies between the values, and is a number."""
    Hq, Hkv, D, T = c
    n = T or 40
    L = 9 * UNIT + n - 1
    case = Case(Hq, Hkv, D, [L], [n], seed=97)
    run = np.minimum(np.arange(L) // UNIT, 8)
    code = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, 6.0])[run]
    k, v = np.zeros((L, Hkv, D)), np.zeros((L, Hkv, D))
    k[:, :, 0] = 2688.0                                # group 0: scale 448
    k[:, :, 16] = code[:, None] * 2.0 ** -9            # group 1: scale 2^-9, by its
    k[:, :, 17] = 6.0 * 2.0 ** -9                      # element 17, which no query has
    v[:] = np.array([1.0, 1.5, 2.0, 3.0, 6.0, 4.0, 2.0, 1.0, 3.0])[run][:, None, None]
    kb, vb = bits(k), bits(v)
    oracle.append(case.pool, Hkv, D, case.pt, np.array([L], np.int32), kb, vb, np.array([0, L], np.int32))
    assert (oracle.qdq_rows(kb)[:, 0, :18] == k[:, 0, :18]).all()
    vhat = oracle.qdq_rows(vb)[:, 0, 0]
    q = np.zeros((n, Hq, D))
    q[:, :, 0], q[:, :, 16] = 1.0, 0.25  # 2688 + code * 2^-11: steps of 2^-12, the last place of 2688
    case.q = bits(q)
    case.device()
    scale = 2.0 ** (power - 11) / LOG2E
    for splits in (0, 1, 2):
        out = run_decode(case, Mod(), T, scale, splits) if T else run_prefill(case, Mod(), scale, splits)
        assert torch.isfinite(out).all(), f"S{splits}"
        assert out.min() >= vhat.min() * (1 - 2.0 ** -8) and out.max() <= vhat.max() * (1 + 2.0 ** -8), f"S{splits}"
    assert int(case.err.item()) == 0
