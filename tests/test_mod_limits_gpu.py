"""Sizes at which the masked attention changes its kernel or its indexes."""
import ctypes

import pytest

import nvfp4_quantized_kv_b200 as nv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hkv", [1, 4])
def test_a_pool_past_the_coordinates_of_decode_qk4(hkv):
    """decode_qk4 counts 36 rows a page and kv-head in 32 bits (of 64 bytes at
    head_dim 128: 137 GB).  A larger pool goes to the kernel that counts 18
    rows of 128 bytes.  Names only: nothing is launched and no such pool made."""
    f = nv.library().nvkv_decode_mod_kernel_name
    most = (2 ** 31 - 1) // 36 // hkv
    for pages, want in ((1, b"decode_qk4"), (most, b"decode_qk4"), (most + 1, b"prefill_mod"),
                        (2 * most, b"prefill_mod")):
        assert f(ctypes.byref(nv._CacheC(0x1000, pages, hkv, 128)), 1, 2 * hkv) == want, pages
    # (the largest pool of this GPU's memory stays inside the other kernel's rows)
    assert 192 * 10 ** 9 // (18 * 128) * 18 < 2 ** 31
