"""Refusals of the masked attention, several-axis append and row read calls,
and their host arithmetic, without a GPU."""
import ctypes

import pytest

import nvfp4_quantized_kv_b200 as nv
from nvfp4_quantized_kv_b200 import build as nvbuild

import mod_ref


@pytest.fixture(scope="module")
def lib():
    nvbuild.build()
    return nv.library()


B = ctypes.byref


def cache(pool=0x1000, num_pages=4, hkv=4, d=256):
    return nv._CacheC(pool, num_pages, hkv, d)


def seqs(batch=1, maxp=4, max_len=64):
    return nv._SeqsC(0x2000, maxp, 0x3000, batch, max_len, None)


def mod(cap=0.0, window=0):
    return nv._ScoreModC(cap, window, None, None, None)


@pytest.mark.parametrize("fn", ["nvkv_decode_attn_mod", "nvkv_decode_attn_mod_k8v4"])
def test_decode_refusals(lib, fn):
    f = getattr(lib, fn)
    need = lib.nvkv_decode_workspace_bytes(1, 1, 24, 4, 256, 8)
    ok = dict(c=cache(), s=seqs(), q=0x100, T=1, hq=24, scale=0.1, m=mod(), n=8, ws=0x1000, size=need, out=0x100)

    def call(**kw):
        a = {**ok, **kw}
        m = B(a["m"]) if a["m"] is not None else None
        return f(B(a["c"]), B(a["s"]), a["q"], a["T"], a["hq"], a["scale"], m, a["n"], a["ws"], a["size"], a["out"], None)

    assert call(m=None) == nv.ERR_INVALID_ARG
    for bad in (mod(cap=-1.0), mod(cap=float("nan")), mod(cap=float("inf")), mod(cap=3e38), mod(cap=1e-45),
                mod(window=-1)):
        assert call(m=bad) == nv.ERR_INVALID_ARG
    assert call(out=None) == nv.ERR_INVALID_ARG
    assert call(out=0x108) == nv.ERR_INVALID_ARG
    assert call(q=None) == nv.ERR_INVALID_ARG
    assert call(hq=25) == nv.ERR_INVALID_ARG
    assert call(T=17) == nv.ERR_UNSUPPORTED
    assert call(T=0) == nv.ERR_INVALID_ARG
    assert call(n=-1) == nv.ERR_INVALID_ARG
    assert call(scale=float("inf")) == nv.ERR_INVALID_ARG
    assert call(size=need - 1) == nv.ERR_WORKSPACE
    assert call(ws=0x1008) == nv.ERR_WORKSPACE
    assert call(c=cache(d=64)) == nv.ERR_UNSUPPORTED


@pytest.mark.parametrize("fn", ["nvkv_prefill_attn_mod", "nvkv_prefill_attn_mod_k8v4"])
def test_prefill_refusals(lib, fn):
    f = getattr(lib, fn)

    def call(m=mod(), q=0x100, cu=0x200, total=10, hq=24, n=1, out=0x300, ws=None, size=0):
        return f(B(cache()), B(seqs()), q, cu, total, 10, hq, 0.1, B(m) if m is not None else None, n, ws, size, out, None)

    assert call(m=None) == nv.ERR_INVALID_ARG
    assert call(m=mod(cap=-2.0)) == nv.ERR_INVALID_ARG
    assert call(m=mod(window=-7)) == nv.ERR_INVALID_ARG
    assert call(n=9) == nv.ERR_INVALID_ARG
    assert call(n=-1) == nv.ERR_INVALID_ARG
    assert call(hq=25) == nv.ERR_INVALID_ARG
    assert call(q=None) == nv.ERR_INVALID_ARG
    assert call(out=0x308) == nv.ERR_INVALID_ARG
    assert call(total=0, q=None, cu=None, out=None) == nv.OK
    assert call(total=0, m=None) == nv.ERR_INVALID_ARG


def test_append_axes_refusals(lib):
    f = lib.nvkv_append_rope_axes
    half = 128

    def call(c=cache(), total=3, mx=3, cs=0x400, mp=64, rd=256, pos=0x500, axes=3, axis=bytes(half), q=None, hq=0,
             qo=None, k=0x100, v=0x200, cu=0x300):
        return f(B(c), B(seqs()), k, v, cu, total, mx, cs, mp, rd, pos, axes, axis, q, hq, qo, None)

    assert call(total=0) == nv.OK
    for kw in (dict(cs=None), dict(cs=0x404), dict(mp=0), dict(rd=0), dict(rd=40), dict(rd=288), dict(axes=0),
               dict(axis=None), dict(axis=bytes([0] * 127 + [3])), dict(pos=None), dict(k=None), dict(v=0x208),
               dict(cu=None), dict(q=0x100, qo=None, hq=24), dict(q=0x108, qo=0x100, hq=24),
               dict(q=0x100, qo=0x108, hq=24), dict(q=0x100, qo=0x100, hq=0), dict(total=-1)):
        assert call(**kw) == nv.ERR_INVALID_ARG, kw
    assert call(axes=5) == nv.ERR_UNSUPPORTED
    assert call(c=cache(d=64), rd=64) == nv.ERR_UNSUPPORTED
    assert call(mx=2 ** 31 - 1) == nv.ERR_UNSUPPORTED


@pytest.mark.parametrize("fn", ["nvkv_read_rows", "nvkv_read_rows_k8v4"])
def test_read_refusals(lib, fn):
    f = getattr(lib, fn)

    def call(starts=0x100, cu=0x200, total=3, mx=3, k=0x300, v=0x400):
        return f(B(cache()), B(seqs()), starts, cu, total, mx, k, v, None)

    for kw in (dict(starts=None), dict(cu=None), dict(k=None), dict(v=None), dict(k=0x308), dict(v=0x408),
               dict(total=-1), dict(mx=-1)):
        assert call(**kw) == nv.ERR_INVALID_ARG, kw
    assert call(total=0, starts=None) == nv.OK


def test_more_sequences_than_a_grid_holds(lib):
    """Calls that launch a grid with a side of sequences refuse the count
    that does not fit (the K8V4 prefill's check comes first too)."""
    many = seqs(batch=65536)
    need = lib.nvkv_decode_workspace_bytes(65536, 2, 24, 4, 256, 8)
    assert lib.nvkv_decode_attn_mod(B(cache()), B(many), 0x100, 2, 24, 0.1, B(mod()), 8, 0x1000, need, 0x100,
                                    None) == nv.ERR_UNSUPPORTED
    for f in (lib.nvkv_prefill_attn_mod, lib.nvkv_prefill_attn_mod_k8v4):
        assert f(B(cache()), B(many), 0x100, 0x200, 10, 10, 24, 0.1, B(mod()), 1, None, 0, 0x300,
                 None) == nv.ERR_UNSUPPORTED
        assert f(B(cache()), B(seqs()), 0x100, 0x200, 10, 0, 24, 0.1, B(mod()), 1, None, 0, 0x300, None) == nv.OK
    for f in (lib.nvkv_read_rows, lib.nvkv_read_rows_k8v4):
        assert f(B(cache()), B(many), 0x100, 0x200, 3, 3, 0x300, 0x400, None) == nv.ERR_UNSUPPORTED
    assert lib.nvkv_append_rope_axes(B(cache()), B(many), 0x100, 0x200, 0x300, 3, 3, 0x400, 64, 256, 0x500, 3,
                                     bytes(128), None, 0, None, None) == nv.ERR_UNSUPPORTED


@pytest.mark.parametrize("window", [-1, 2 ** 31, 2 ** 32 + 5])
def test_a_window_that_is_no_int32_is_refused(window):
    with pytest.raises(ValueError, match="window"):
        nv.ScoreMod(window=window)._struct(0, 8, 1, 1)


def test_python_checks():
    import torch
    with pytest.raises(ValueError, match="CUDA"):
        nv.ScoreMod(alibi_slopes=torch.ones(4))
    with pytest.raises(TypeError):
        nv.ScoreMod(key_starts=[1, 2])


def test_interval_equals_the_key_by_key_definition():
    """The interval of visible keys that the 64-bit form uses is the set that
    the definition gives one key at a time."""
    for kv_len in (1, 5, 9):
        for p in range(-2, kv_len):
            for start in (-1, 0, 2, 7, 20):
                for window in (0, 1, 3, 50):
                    for prefix in (-3, 0, 1, 4, 30):
                        lo, hi = mod_ref.interval(p, kv_len, start, window, prefix)
                        assert list(range(lo, max(lo, hi))) == mod_ref.visible(p, kv_len, start, window, prefix), \
                            (p, kv_len, start, window, prefix)
