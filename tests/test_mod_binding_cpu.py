"""What the binding hands to the library in the masked attention, append and
read calls, without a GPU: the calls are caught before they reach it."""
import array
import types

import numpy as np
import pytest
import torch

import nvfp4_quantized_kv_b200 as nv
from nvfp4_quantized_kv_b200 import build as nvbuild

bf16 = torch.bfloat16


@pytest.fixture
def caught(monkeypatch):
    """The arguments of every call that would have gone to the library."""
    nvbuild.build()
    calls = []
    monkeypatch.setattr(nv, "_call", lambda device, fn, what, stream, *args: calls.append(args))
    return calls


def host_cache(hkv=1, d=128):
    """Stand-ins on the CPU (device index -1) for the cache and the batch."""
    cache = types.SimpleNamespace(pool=torch.zeros(1, dtype=torch.uint8), num_pages=4, num_kv_heads=hkv, head_dim=d,
                                  kv_format="nvfp4", _c=nv._CacheC(0x1000, 4, hkv, d))
    seqs = types.SimpleNamespace(page_table=torch.zeros(1, 4, dtype=torch.int32), kv_lens=torch.zeros(1, dtype=torch.int32),
                                 err_word=None, batch=1, _c=nv._SeqsC(0x2000, 4, 0x3000, 1, 64, None))
    return cache, seqs


AXES = [i % 3 for i in range(64)]


def append(axes, rotary=128):
    cache, seqs = host_cache()
    k = torch.zeros(3, 1, 128, dtype=bf16)
    nv.nvkv_append_rope_axes(cache, seqs, k, k, torch.tensor([0, 3], dtype=torch.int32), 3, 3,
                             torch.zeros(64, rotary // 2, 2), rotary, torch.zeros(3, 3, dtype=torch.int32), axes)


@pytest.mark.parametrize("axes", [
    AXES, tuple(AXES), bytes(AXES), bytearray(AXES), memoryview(bytes(AXES)), range(0, 64, 1),
    np.array(AXES, np.uint8), np.array(AXES, np.int32), np.array(AXES, np.int64), np.array(AXES * 2, np.int16)[::2],
    array.array("i", AXES), array.array("B", AXES), torch.tensor(AXES), torch.tensor(AXES, dtype=torch.int32),
], ids=lambda a: f"{type(a).__name__}-{getattr(a, 'dtype', getattr(a, 'typecode', ''))}")
def test_axes_are_the_numbers_of_any_sequence(caught, axes):
    append(axes)
    assert caught[0][12] == bytes([int(a) for a in axes])


@pytest.mark.parametrize("axes", [[0.5] * 64, np.zeros(64), [-1] * 64, [256] * 64, np.full(64, 300), np.zeros((64, 2), np.int32)],
                         ids=["float", "numpy_float", "negative", "past_a_byte", "numpy_past_a_byte", "two_axes"])
def test_axes_that_are_no_bytes_are_refused(caught, axes):
    with pytest.raises((TypeError, ValueError)):
        append(axes)
    assert not caught


def test_a_call_keeps_its_score_mod_while_another_is_made(caught):
    """The library reads a call's struct after the interpreter's lock is
    dropped: a call with other attributes of the same ScoreMod, made
    meanwhile, must not change it."""
    cache, seqs = host_cache()
    q, ws = torch.zeros(1, 2, 128, dtype=bf16), torch.zeros(16, dtype=torch.uint8)
    mod = nv.ScoreMod(softcap=30.0, window=64)
    nv.nvkv_decode_attn_mod(cache, seqs, q, 1, 2, 0.1, mod, 1, ws, q)
    starts = torch.zeros(1, dtype=torch.int32)
    mod.softcap, mod.window, mod.key_starts = 7.0, 5, starts
    nv.nvkv_prefill_attn_mod(cache, seqs, q, torch.tensor([0, 1], dtype=torch.int32), 1, 1, 2, 0.1, mod, 1, None, q)
    first, second = caught[0][6]._obj, caught[1][8]._obj
    assert (first.softcap, first.window, first.key_starts) == (30.0, 64, None)
    assert (second.softcap, second.window, second.key_starts) == (7.0, 5, starts.data_ptr())
