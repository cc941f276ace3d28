"""The query's side of the masked attention: as many bits of it as the plain
calls take, at any size."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_kv_b200 as nv

from mod_ref import Case, Mod, assert_within, run_decode, run_prefill

pytestmark = pytest.mark.gpu


def slopes(h):
    return [2.0 ** (-8 * (i + 1) / h) for i in range(h)]


# The reference's "f16 weights" bound has no rounding of the query: exact
# products of codes and scales and fp32 sums.
MANY = [  # Hq, Hkv, D, lens, T: more than 6 rows a pair, in tiles of 32, 64, 128
    (24, 4, 256, [300, 77], 4),
    (12, 1, 256, [190], 1),
    (24, 4, 256, [260, 130, 12], 10),
    (16, 1, 256, [150], 8),
    (16, 2, 128, [300, 64], 2),
    (12, 2, 128, [333, 20], 9),
    (8, 1, 128, [140], 16),
]
IDS = [f"{c[0]}_{c[1]}_{c[2]}_T{c[4]}" for c in MANY]


@pytest.mark.parametrize("gain", [1e-30, 1e-4, 1.0, 30.0, 1e4, 1e8])
@pytest.mark.parametrize("c", MANY, ids=IDS)
def test_decode_of_many_rows_at_any_size_of_query(c, gain):
    Hq, Hkv, D, lens, T = c
    case = Case(Hq, Hkv, D, lens, [T] * len(lens), seed=71, q_gain=gain).device()
    for m in (Mod(), Mod(window=90), Mod(slopes=slopes(Hq)), Mod(cap=30.0)):
        ref, tol = case.reference(m, D ** -0.5, True, "f16 weights")
        for splits in (0, 1):
            assert_within(run_decode(case, m, T, D ** -0.5, splits), ref, tol, f"{m}/S{splits}")
    assert int(case.err.item()) == 0


@pytest.mark.parametrize("gain", [1e-30, 1e-4, 1.0, 30.0, 1e4, 1e8])
@pytest.mark.parametrize("D,Hq,Hkv,n", [(256, 24, 4, 70), (128, 8, 2, 100), (256, 24, 4, 3), (128, 16, 2, 7)])
def test_chunks_at_any_size_of_query(D, Hq, Hkv, n, gain):
    case = Case(Hq, Hkv, D, [230], [n], seed=72, q_gain=gain).device()
    for m in (Mod(), Mod(slopes=slopes(Hq), window=100), Mod(cap=30.0)):
        ref, tol = case.reference(m, D ** -0.5, False, "f16 weights")
        for splits in (1, 3):
            assert_within(run_prefill(case, m, D ** -0.5, splits), ref, tol, f"{m}/S{splits}")
    assert int(case.err.item()) == 0


@pytest.mark.parametrize("D,Hq,Hkv,T", [(256, 24, 4, 4), (128, 16, 2, 5)])
@pytest.mark.parametrize("scale", [-0.07, 0.0, 1.0, 1e-6])
def test_any_scale(D, Hq, Hkv, T, scale):
    case = Case(Hq, Hkv, D, [200, 90], [T, T], seed=73).device()
    for m in (Mod(window=80), Mod(cap=9.0), Mod(slopes=slopes(Hq))):
        ref, tol = case.reference(m, scale, True, "f16 weights")
        assert_within(run_decode(case, m, T, scale), ref, tol, f"decode {m}")
        ref, tol = case.reference(m, scale, False, "f16 weights")
        assert_within(run_prefill(case, m, scale), ref, tol, f"prefill {m}")


@pytest.mark.parametrize("D,Hq,Hkv,T", [(256, 24, 4, 4), (128, 16, 2, 2)])
def test_rows_of_large_and_small_elements(D, Hq, Hkv, T):
    """Half of a row's elements 2^20 times the other half, over keys that only
    the small half tells apart: the large ones meet zeros."""
    case = Case(Hq, Hkv, D, [180], [T], seed=74)
    import oracle
    from mod_ref import bits
    rng = np.random.default_rng(75)
    k = rng.standard_normal((180, Hkv, D))
    k[:, :, :D // 2] = 0
    kb = bits(k)
    v = bits(rng.standard_normal((180, Hkv, D)))
    oracle.append(case.pool, Hkv, D, case.pt, np.array([180], np.int32), kb, v, np.array([0, 180], np.int32))
    case.khat, case.vhat = [oracle.qdq_rows(kb)], [oracle.qdq_rows(v)]
    q = rng.standard_normal((T, Hq, D))
    q[:, :, :D // 2] *= 2.0 ** 20
    case.q = bits(q)
    case.device()
    ref, tol = case.reference(Mod(), D ** -0.5, True, "f16 weights")
    assert_within(run_decode(case, Mod(), T, D ** -0.5), ref, tol, "decode")
    assert_within(run_prefill(case, Mod(), D ** -0.5), ref, tol, "prefill")


@pytest.mark.parametrize("gain", [1.0, 1e4])
@pytest.mark.parametrize("T", [2, 4, 8])
def test_an_empty_mod_is_as_exact_as_the_plain_call(T, gain):
    """Verify steps of 12 to 48 rows a pair: the masked and the plain call
    within both their bounds (neither rounds the query to 11 bits)."""
    case = Case(24, 4, 256, [300, 77], [T, T], seed=76, q_gain=gain).device()
    out = run_decode(case, Mod(), T, 1 / 16)
    ws = torch.empty(nv.nvkv_decode_workspace_bytes(2, T, 24, 4, 256, 0), dtype=torch.uint8, device="cuda")
    plain = torch.empty_like(out)
    nv.nvkv_decode_attn(case.cache, case.seqs, case.q_dev, T, 24, 1 / 16, 0, ws)
    nv.nvkv_combine(case.seqs, ws, T, 24, 4, 256, 0, plain)
    ref, tol = case.reference(Mod(), 1 / 16, True, "f16 weights")
    assert_within(out, ref, tol, "masked")
    assert ((out.double() - plain.double()).abs().cpu() <= 2 * tol).all()


def test_a_short_chunk_of_a_group_of_12():
    """12 query heads on one kv-head, a single row."""
    case = Case(12, 1, 256, [190], [1], seed=41).device()
    for m in (Mod(), Mod(window=50, cap=12.0),
              Mod(cap=20.0, window=77, slopes=slopes(12), prefix=[188], starts=[5])):
        ref, tol = case.reference(m, 1 / 16, False, "f16 weights")
        for splits in (0, 1, 3):
            assert_within(run_prefill(case, m, 1 / 16, splits), ref, tol, f"S{splits}")
    assert int(case.err.item()) == 0
