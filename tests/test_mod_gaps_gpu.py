"""Chunks whose rows leave keys unseen between the keys that they see: padding
between packed documents (rows whose start lies behind their own position).
Unseen keys are not looked at: their pages may be gone, and their bytes may
hold anything."""
import numpy as np
import pytest
import torch

import nvfp4_quantized_kv_b200 as nv

from mod_ref import Case, Mod, assert_within, interval, run_prefill

pytestmark = pytest.mark.gpu


def unseen_keys(case, mod):
    """[sequence] -> the cached positions that no row of the call sees."""
    out = []
    for b, l in enumerate(case.lens):
        seen = np.zeros(l, bool)
        for i in range(case.n[b]):
            lo, hi = interval(l - case.n[b] + i, l, mod.starts[case.cu[b] + i], mod.window,
                              mod.prefix[b] if mod.prefix else 0)
            seen[lo:max(lo, hi)] = True
        out.append(np.flatnonzero(~seen))
    return out


def spoil(case, mod):
    """NaN patterns in the scale bytes of every unseen key, and no page where
    a page has no other keys (absent, or an id past the pool)."""
    D, blk = case.D, 18 * case.D
    pages = case.pool.reshape(case.num_pages, case.Hkv, blk)
    gone = 0
    for b, keys in enumerate(unseen_keys(case, mod)):
        for pos in keys:
            p, s = case.pt[b, pos // 16], pos % 16
            pages[p, :, 8 * D + s * (D // 16):8 * D + (s + 1) * (D // 16)] = 0x7F
            for g in range(D // 16):
                pages[p, :, 17 * D + g * 16 + s] = 0x7F
        for pg in range(-(-case.lens[b] // 16)):
            if set(range(pg * 16, min(pg * 16 + 16, case.lens[b]))) <= set(keys.tolist()):
                case.pt[b, pg] = -1 if gone % 2 else case.num_pages + 3
                gone += 1
    return gone


def documents(case, lengths, pads):
    """key_starts of every row: documents of the given lengths, each followed
    by rows that see nothing."""
    starts = []
    for b, l in enumerate(case.lens):
        p, at, k = l - case.n[b], [], 0
        while len(at) < case.n[b]:
            doc, pad = lengths[k % len(lengths)], pads[k % len(pads)]
            at += [p + len(at)] * doc + [10 ** 6] * pad
            k += 1
        starts += at[:case.n[b]]
    return starts


SHAPES = [  # Hq, Hkv, D, lens, rows: tiles of 128, of 64 and of 32 rows
    (24, 4, 256, [300, 170], [300, 130]),
    (4, 4, 256, [400], [400]),
    (4, 4, 128, [400, 90], [350, 90]),
    (16, 4, 128, [333], [333]),
    (4, 4, 256, [200, 61], [60, 61]),
    (4, 4, 128, [131, 32], [32, 30]),
    (8, 2, 256, [76], [8]),
]


@pytest.mark.parametrize("masks", ["none", "cap", "bias", "window_prefix"])
@pytest.mark.parametrize("c", SHAPES, ids=[f"{c[0]}_{c[1]}_{c[2]}_{max(c[4])}" for c in SHAPES])
def test_padding_between_documents(c, masks):
    Hq, Hkv, D, lens, n = c
    case = Case(Hq, Hkv, D, lens, n, seed=51)
    starts = documents(case, [5, 37, 3, 1], [41, 19, 2, 23])
    slopes = [2.0 ** (-8 * (i + 1) / Hq) for i in range(Hq)]
    m = {"none": Mod(starts=starts), "cap": Mod(cap=20.0, starts=starts), "bias": Mod(slopes=slopes, starts=starts),
         "window_prefix": Mod(cap=12.0, slopes=slopes, window=30, prefix=[l - n_ + 12 for l, n_ in zip(lens, n)],
                              starts=starts)}[masks]
    gone = spoil(case, m)
    if max(n) > 60:
        assert gone, "the case has no page that nobody sees"
    case.device()
    ref, tol = case.reference(m, D ** -0.5, False, "f16 scores")
    for splits in (0, 1, 3):
        out = run_prefill(case, m, D ** -0.5, splits)
        assert int(case.err.item()) == 0, f"S{splits}"
        assert_within(out, ref, tol, f"S{splits}")


@pytest.mark.parametrize("seed", range(4))
def test_starts_in_any_order(seed):
    """Starts that jump back and forth, most rows seeing nothing, with a
    prefix that some of them see from behind their own position."""
    rng = np.random.default_rng(seed)
    Hq, Hkv, D = ((4, 4, 128), (24, 4, 256), (4, 4, 256), (8, 1, 128))[seed]
    case = Case(Hq, Hkv, D, [420, 150], [390, 140], seed=60 + seed)
    starts = []
    for b, l in enumerate(case.lens):
        p = np.arange(l - case.n[b], l)
        near = p - rng.integers(-3, 12, p.size)
        starts += np.where(rng.random(p.size) < 0.12, near, 10 ** 6).tolist()
    m = Mod(cap=15.0, window=9, prefix=[70, 149], starts=starts)
    assert spoil(case, m) > 0
    case.device()
    ref, tol = case.reference(m, D ** -0.5, False, "f16 scores")
    for splits in (0, 1, 5):
        out = run_prefill(case, m, D ** -0.5, splits)
        assert int(case.err.item()) == 0
        assert_within(out, ref, tol, f"S{splits}")


def test_a_missing_page_that_a_row_sees_is_still_reported():
    case = Case(24, 4, 256, [300], [300], seed=52)
    m = Mod(starts=documents(case, [5, 37, 3, 1], [41, 19, 2, 23]))
    spoil(case, m)
    case.pt[0, 50 // 16] = -1  # position 50 is in the second document
    case.device()
    run_prefill(case, m, 1 / 16)
    assert int(case.err.item()) == nv.DEVERR_PAGE_ID
