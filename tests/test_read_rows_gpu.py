"""GPU parity of nvkv_read_rows: every cached value of both formats as bf16,
exactly, against the values the oracle's formats define."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_kv_b200 as nv

from mod_ref import Case

pytestmark = pytest.mark.gpu


def read(case, starts, counts, guard=3):
    dev = torch.device("cuda")
    cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=dev)
    total = int(sum(counts))
    k = torch.full((total + guard, case.Hkv, case.D), 7.0, dtype=torch.bfloat16, device=dev)
    v = torch.full_like(k, 9.0)
    nv.nvkv_read_rows(case.cache, case.seqs, torch.tensor(starts, dtype=torch.int32, device=dev), cu, total,
                      max(counts), k, v)
    torch.cuda.synchronize()
    assert (k[total:] == 7.0).all() and (v[total:] == 9.0).all()
    return k[:total].double().cpu(), v[:total].double().cpu()


CASES = [
    # Hkv, D, lens, starts, counts
    (4, 256, [100, 1, 64], [0, 0, 0], [100, 1, 64]),
    (4, 256, [100, 33, 64], [5, 32, 16], [77, 1, 16]),
    (2, 128, [100, 17, 0, 48], [99, 0, 0, 31], [1, 17, 0, 2]),
    (5, 128, [70], [3], [60]),
    (1, 256, [40, 300], [40, 1], [0, 299]),
]


@pytest.mark.parametrize("k8", [False, True], ids=["nvfp4", "k8v4"])
@pytest.mark.parametrize("c", CASES, ids=[f"{c[0]}_{c[1]}_{len(c[2])}" for c in CASES])
def test_rows(c, k8):
    Hkv, D, lens, starts, counts = c
    case = Case(Hkv, Hkv, D, lens, [0] * len(lens), seed=2, k8=k8).device()
    k, v = read(case, starts, counts)
    assert int(case.err.item()) == 0
    at = 0
    for b, n in enumerate(counts):
        s = starts[b]
        want_k, want_v = (torch.from_numpy(t[b][s:s + n]) for t in (case.khat, case.vhat))
        assert torch.equal(v[at:at + n], want_v)
        if k8:  # E4M3 code times an fp32 scale: a product, rounded once to fp32 and once to bf16
            assert ((k[at:at + n] - want_k).abs() <= want_k.abs() * (2.0 ** -8 + 2.0 ** -23)).all()
        else:
            assert torch.equal(k[at:at + n], want_k)
        at += n


def test_every_code_under_every_scale():
    """All 16 codes under all 127 finite scales, K and V, are exact bf16."""
    D, Hkv = 256, 8
    case = Case(Hkv, Hkv, D, [128], [0], seed=1)
    pages = case.pool.reshape(case.num_pages, Hkv, 18 * D)
    code = np.arange(16)
    e2m1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
    e2m1 = np.concatenate([e2m1, -e2m1])
    e4m3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    byte = (code[0::2] | (code[1::2] << 4)).astype(np.uint8)   # the 16 codes in order
    pages[:, :, :8 * D] = np.tile(byte, D)                     # every K group holds all codes
    pages[:, :, 9 * D:17 * D] = np.tile(byte, D)               # every V element row: slots 0..15
    sc = np.arange(case.num_pages * Hkv * D) % 127
    sc = sc.reshape(case.num_pages, Hkv, D).astype(np.uint8)
    pages[:, :, 8 * D:9 * D] = sc
    pages[:, :, 17 * D:] = sc
    case.device()
    k, v = read(case, [0], [128])
    seen = set()
    for pos in range(128):
        p, s = case.pt[0, pos // 16], pos % 16
        for h in range(Hkv):
            for g in range(D // 16):
                ks, vs = sc[p, h, s * (D // 16) + g], sc[p, h, g * 16 + s]
                seen.add(int(ks))
                assert np.array_equal(k[pos, h, 16 * g:16 * g + 16].numpy(), e2m1 * e4m3[ks])
                assert (v[pos, h, 16 * g:16 * g + 16].numpy() == e2m1[s] * e4m3[vs]).all()
    assert len(seen) == 127


def test_bad_ranges_pages_and_lengths():
    case = Case(4, 4, 256, [60, 40, 50], [0, 0, 0], seed=3)
    case.pt[2, 1] = -7
    case.device()
    cu = torch.tensor([0, 10, 20, 70], dtype=torch.int32, device="cuda")
    k = torch.full((70, 4, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, 7.0)
    starts = torch.tensor([-1, 31, 0], dtype=torch.int32, device="cuda")
    nv.nvkv_read_rows(case.cache, case.seqs, starts, cu, 70, 50, k, v)
    torch.cuda.synchronize()
    assert int(case.err.item()) == nv.DEVERR_LENGTH | nv.DEVERR_PAGE_ID
    assert (k[:20] == 7.0).all() and (v[:20] == 7.0).all()       # both ranges leave the cache
    assert (k[36:52] == 7.0).all() and (v[36:52] == 7.0).all()   # the page that is not there
    keep = list(range(20, 36)) + list(range(52, 70))
    assert torch.equal(k[keep].double().cpu(), torch.from_numpy(case.khat[2][[i - 20 for i in keep]]))
    # a bound below the rows asked for, and rows past total_rows, are refused too
    for total, most in ((70, 49), (69, 50)):
        case.err.zero_()
        k.fill_(7.0)
        nv.nvkv_read_rows(case.cache, case.seqs, torch.tensor([0, 0, 0], dtype=torch.int32, device="cuda"), cu,
                          total, most, k, v)
        torch.cuda.synchronize()
        assert int(case.err.item()) & nv.DEVERR_LENGTH
        assert (k[20:] == 7.0).all()


def test_read_then_append_restores_the_bytes():
    """Rows read and appended to a second cache give the same values there."""
    case = Case(4, 4, 256, [90, 33], [0, 0], seed=4).device()
    k, v = read(case, [0, 0], [90, 33])
    dev = torch.device("cuda")
    other = nv.Cache.allocate(case.num_pages, 4, 256, dev, fill=0)
    cu = torch.tensor([0, 90, 123], dtype=torch.int32, device=dev)
    nv.nvkv_append(other, case.seqs, k.bfloat16().to(dev), v.bfloat16().to(dev), cu, 123, 90)
    first = case.cache
    case.cache = other
    k2, v2 = read(case, [0, 0], [90, 33])
    case.cache = first
    assert torch.equal(k, k2) and torch.equal(v, v2)
