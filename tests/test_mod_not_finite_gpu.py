"""Queries of the masked attention that are not finite."""
import numpy as np
import pytest
import torch

from mod_ref import Case, Mod, run_decode, run_prefill

pytestmark = pytest.mark.gpu


def slopes(h):
    return [2.0 ** (-8 * (i + 1) / h) for i in range(h)]


BAD = [  # Hq, Hkv, D, T (0: a chunk of 70 rows, -1: a chunk of few rows), K8V4 cache
    (24, 4, 256, 1, False), (8, 2, 128, 1, False), (8, 4, 256, 3, False), (24, 4, 256, 4, False),
    (16, 2, 128, 6, False), (24, 4, 256, 0, False), (8, 2, 128, 0, False), (24, 4, 256, -1, False),
    (8, 2, 256, 1, True), (8, 2, 256, 4, True), (8, 2, 128, 1, True), (8, 2, 128, 0, True),
]


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("kernel", ["default", "simt"])
@pytest.mark.parametrize("c", BAD, ids=[f"{c[0]}_{c[1]}_{c[2]}_T{c[3]}{'_k8v4' if c[4] else ''}" for c in BAD])
def test_a_query_that_is_not_finite_gives_nan_and_stays_alone(c, kernel, value, monkeypatch):
    """Its row is NaN in every kernel and at every split count, zero where it
    sees no key; the other rows keep their bits."""
    if kernel != "default":
        monkeypatch.setenv("NVKV_DECODE_KERNEL", kernel)
    Hq, Hkv, D, T, k8 = c
    n = {0: 70, -1: 3}.get(T, T)
    decode = T > 0
    case = Case(Hq, Hkv, D, [260, 140, 300], [n] * 3, seed=81, k8=k8).device()
    rows = 3 * n
    # the third sequence sees nothing at all
    starts = [0, 7, 300] if decode else [0] * n + [7] * n + [300] * n
    for m in (Mod(starts=starts), Mod(cap=20.0, window=150, starts=starts), Mod(slopes=slopes(Hq), starts=starts)):
        for splits in (0, 1, 3):
            run = (lambda: run_decode(case, m, T, D ** -0.5, splits)) if decode else (
                lambda: run_prefill(case, m, D ** -0.5, splits))
            case.q_dev.copy_(torch.from_numpy(case.q.view(np.int16)).view(torch.bfloat16))
            good = run()
            assert torch.isfinite(good).all()
            hit = torch.zeros(rows, Hq, dtype=torch.bool, device="cuda")
            for r, h, e in ((0, 0, 3), (n - 1, Hq - 1, D - 1), (n, 1, D // 2), (2 * n - 1, Hq // 2, 17), (2 * n, 2, 0)):
                case.q_dev[r, h, e] = value
                hit[r, h] = r < 2 * n
            out = run()
            assert torch.isnan(out[hit]).all(), f"{m}/S{splits}"
            assert torch.equal(out[~hit], good[~hit]), f"{m}/S{splits}"
    assert int(case.err.item()) == 0
