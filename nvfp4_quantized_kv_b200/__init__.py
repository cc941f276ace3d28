"""Python binding of libnvkv: attention over an NVFP4-quantised paged KV
cache on B200 (sm_100a).

Argument marshalling only.  Every step of the path (quantise-append, split-K
decode / MTP-verify attention, combine, chunked prefill) runs in the CUDA
kernels of ``libnvkv.so``; the functions here take torch tensors (device
memory and streams come from PyTorch), check dtypes and devices, and pass raw
pointers to the C ABI declared in ``include/nvkv.h``.  There is no CPU or
PyTorch fallback: if the library is missing, every call raises.

Build the library with ``python -m nvfp4_quantized_kv_b200.build``.
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "NvkvError", "Cache", "Seqs", "library", "library_path",
    "nvkv_page_bytes", "nvkv_default_num_splits", "nvkv_decode_workspace_bytes",
    "nvkv_split_plan", "nvkv_append", "nvkv_decode_attn", "nvkv_combine",
    "nvkv_prefill_attn", "nvkv_status_string", "nvkv_decode_attn_static",
    "nvkv_decode_static_scratch_bytes", "nvkv_rope_table", "nvkv_append_rope",
    "nvkv_pages_spill", "nvkv_pages_restore", "nvkv_k8v4_page_bytes", "nvkv_append_k8v4",
    "nvkv_decode_attn_k8v4", "nvkv_prefill_attn_k8v4", "nvkv_pages_spill_k8v4",
    "nvkv_pages_restore_k8v4", "nvkv_prefill_attn_split", "nvkv_prefill_workspace_bytes",
    "nvkv_prefill_num_splits", "ScoreMod", "nvkv_decode_attn_mod",
    "nvkv_decode_mod_kernel_name", "nvkv_prefill_attn_mod",
    "nvkv_append_rope_axes", "nvkv_read_rows",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libnvkv.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA = range(5)
DEVERR_PAGE_ID, DEVERR_LENGTH, DEVERR_TIMEOUT = 1, 2, 4


class NvkvError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {nvkv_status_string(status)} (status {status})")


class _CacheC(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class _SeqsC(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("max_pages_per_seq", ctypes.c_int32),
                ("kv_lens", ctypes.c_void_p), ("batch", ctypes.c_int32),
                ("max_kv_len", ctypes.c_int32), ("err_word", ctypes.c_void_p)]


class _ScoreModC(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("window", ctypes.c_int32),
                ("alibi_slopes", ctypes.c_void_p), ("prefix_lens", ctypes.c_void_p),
                ("key_starts", ctypes.c_void_p)]


_lib = None


def library():
    """Load libnvkv.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise ImportError(
                f"{library_path} is missing: build it with "
                "`python -m nvfp4_quantized_kv_b200.build` (needs nvcc); there is no fallback")
        L = ctypes.CDLL(library_path)
        vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
        cp, sp = ctypes.POINTER(_CacheC), ctypes.POINTER(_SeqsC)
        mp = ctypes.POINTER(_ScoreModC)
        decode_mod = [cp, sp, vp, i32, i32, f32, mp, i32, vp, sz, vp, vp]
        prefill_mod = [cp, sp, vp, vp, i32, i32, i32, f32, mp, i32, vp, sz, vp, vp]
        read_rows = [cp, sp, vp, vp, i32, i32, vp, vp, vp]
        sig = {
            "nvkv_page_bytes": (sz, [i32, i32]),
            "nvkv_default_num_splits": (i32, []),
            "nvkv_decode_workspace_bytes": (sz, [i32, i32, i32, i32, i32, i32]),
            "nvkv_split_plan": (ctypes.c_int, [vp, i32, i32, i32, vp, vp]),
            "nvkv_append": (ctypes.c_int, [cp, sp, vp, vp, vp, i32, i32, vp]),
            "nvkv_decode_attn": (ctypes.c_int, [cp, sp, vp, i32, i32, f32, i32, vp, sz, vp]),
            "nvkv_decode_kernel_name": (ctypes.c_char_p, [cp, i32, i32]),
            "nvkv_decode_kernel_name_k8v4": (ctypes.c_char_p, [cp, i32, i32]),
            "nvkv_combine": (ctypes.c_int, [sp, vp, i32, i32, i32, i32, i32, vp, vp]),
            "nvkv_prefill_attn": (ctypes.c_int, [cp, sp, vp, vp, i32, i32, i32, f32, vp, vp]),
            "nvkv_prefill_workspace_bytes": (sz, [i32, i32, i32, i32]),
            "nvkv_prefill_num_splits": (i32, [cp, i32, i32, i32]),
            "nvkv_prefill_attn_split": (ctypes.c_int, [cp, sp, vp, vp, i32, i32, i32, f32, i32, vp,
                                                       sz, vp, vp]),
            "nvkv_decode_static_scratch_bytes": (sz, []),
            "nvkv_decode_attn_static": (ctypes.c_int, [cp, sp, vp, i32, i32, f32, i32, vp, vp]),
            "nvkv_rope_table": (ctypes.c_int, [vp, i32, i32, ctypes.c_double, ctypes.c_double, vp]),
            "nvkv_append_rope": (ctypes.c_int, [cp, sp, vp, vp, vp, i32, i32, vp, i32, i32, vp]),
            "nvkv_pages_spill": (ctypes.c_int, [cp, vp, vp, i32, vp, ctypes.c_int64, vp, vp]),
            "nvkv_pages_restore": (ctypes.c_int, [cp, vp, vp, i32, vp, ctypes.c_int64, vp, vp]),
            "nvkv_k8v4_page_bytes": (sz, [i32, i32]),
            "nvkv_pages_spill_k8v4": (ctypes.c_int, [cp, vp, vp, i32, vp, ctypes.c_int64, vp, vp]),
            "nvkv_pages_restore_k8v4": (ctypes.c_int, [cp, vp, vp, i32, vp, ctypes.c_int64, vp,
                                                       vp]),
            "nvkv_append_k8v4": (ctypes.c_int, [cp, sp, vp, vp, vp, i32, i32, vp]),
            "nvkv_decode_attn_k8v4": (ctypes.c_int, [cp, sp, vp, i32, i32, f32, i32, vp, sz, vp]),
            "nvkv_prefill_attn_k8v4": (ctypes.c_int, [cp, sp, vp, vp, i32, i32, i32, f32, vp, vp]),
            "nvkv_decode_mod_kernel_name": (ctypes.c_char_p, [cp, i32, i32]),
            "nvkv_decode_attn_mod": (ctypes.c_int, decode_mod),
            "nvkv_decode_attn_mod_k8v4": (ctypes.c_int, decode_mod),
            "nvkv_prefill_attn_mod": (ctypes.c_int, prefill_mod),
            "nvkv_prefill_attn_mod_k8v4": (ctypes.c_int, prefill_mod),
            "nvkv_append_rope_axes": (ctypes.c_int, [cp, sp, vp, vp, vp, i32, i32, vp, i32, i32, vp,
                                                     i32, ctypes.c_char_p, vp, i32, vp, vp]),
            "nvkv_read_rows": (ctypes.c_int, read_rows),
            "nvkv_read_rows_k8v4": (ctypes.c_int, read_rows),
            "nvkv_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def nvkv_status_string(status: int) -> str:
    return library().nvkv_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != OK:
        raise NvkvError(status, what)


def _dev(t: torch.Tensor, dtype: torch.dtype, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


KV_FORMATS = ("nvfp4", "k8v4")


def _page_bytes_of(kv_format: str, num_kv_heads: int, head_dim: int) -> int:
    if kv_format == "nvfp4":
        return nvkv_page_bytes(num_kv_heads, head_dim)
    if kv_format == "k8v4":
        return nvkv_k8v4_page_bytes(num_kv_heads, head_dim)
    raise ValueError(f"kv_format must be one of {KV_FORMATS}, got {kv_format!r}")


class Cache:
    """The paged pool: ``pool`` is a uint8 CUDA tensor of num_pages pages of
    nvkv_page_bytes(num_kv_heads, head_dim) bytes (kv_format "nvfp4") or
    nvkv_k8v4_page_bytes(...) bytes ("k8v4": 8-bit K, NVFP4 V).  A K8V4
    cache is used only with the *_k8v4 calls."""

    def __init__(self, pool: torch.Tensor, num_pages: int, num_kv_heads: int, head_dim: int,
                 kv_format: str = "nvfp4"):
        self.pool, self.num_pages, self.num_kv_heads, self.head_dim = pool, num_pages, num_kv_heads, head_dim
        self.kv_format = kv_format
        need = num_pages * _page_bytes_of(kv_format, num_kv_heads, head_dim)
        if pool.numel() < need:
            raise ValueError(f"pool has {pool.numel()} bytes, needs {need}")
        self._c = _CacheC(_dev(pool, torch.uint8, "pool"), num_pages, num_kv_heads, head_dim)

    @staticmethod
    def allocate(num_pages: int, num_kv_heads: int, head_dim: int, device="cuda", fill=None,
                 kv_format: str = "nvfp4"):
        n = num_pages * _page_bytes_of(kv_format, num_kv_heads, head_dim)
        pool = torch.empty(n, dtype=torch.uint8, device=device)
        if fill is not None:
            pool.fill_(fill)
        return Cache(pool, num_pages, num_kv_heads, head_dim, kv_format)


def _fmt(cache: "Cache", want: str, what: str) -> None:
    if cache.kv_format != want:
        raise ValueError(f"{what} needs a {want} cache, got a {cache.kv_format} cache")


class Seqs:
    """The batch: page_table int32 [batch][max_pages_per_seq] and kv_lens
    int32 [batch] on the device; max_kv_len a host bound; err_word an
    optional int32 device tensor of one element."""

    def __init__(self, page_table: torch.Tensor, kv_lens: torch.Tensor, max_kv_len: int,
                 err_word: torch.Tensor | None = None):
        if page_table.dim() != 2 or kv_lens.dim() != 1 or kv_lens.numel() != page_table.shape[0]:
            raise ValueError("page_table must be [batch][max_pages], kv_lens [batch]")
        self.page_table, self.kv_lens, self.max_kv_len, self.err_word = page_table, kv_lens, max_kv_len, err_word
        self.batch = page_table.shape[0]
        self._c = _SeqsC(_dev(page_table, torch.int32, "page_table"), page_table.shape[1],
                         _dev(kv_lens, torch.int32, "kv_lens"), self.batch, int(max_kv_len),
                         _dev(err_word, torch.int32, "err_word") if err_word is not None else None)


def nvkv_page_bytes(num_kv_heads: int, head_dim: int) -> int:
    return int(library().nvkv_page_bytes(num_kv_heads, head_dim))


def nvkv_default_num_splits() -> int:
    return int(library().nvkv_default_num_splits())


def nvkv_decode_workspace_bytes(batch: int, T: int, num_q_heads: int, num_kv_heads: int,
                                head_dim: int, num_splits: int = 0) -> int:
    n = int(library().nvkv_decode_workspace_bytes(batch, T, num_q_heads, num_kv_heads, head_dim,
                                                  num_splits))
    if n == 0:
        raise NvkvError(ERR_INVALID_ARG, "nvkv_decode_workspace_bytes")
    return n


def nvkv_split_plan(kv_lens_host, num_kv_heads: int, num_splits: int):
    """Host copy of the split plan: (first_split, last_split) per (b, h)."""
    import numpy as np
    kl = np.ascontiguousarray(kv_lens_host, dtype=np.int32)
    n = kl.size * num_kv_heads
    first = np.zeros(n, np.int32)
    last = np.zeros(n, np.int32)
    _check(library().nvkv_split_plan(kl.ctypes.data, kl.size, num_kv_heads, num_splits,
                                     first.ctypes.data, last.ctypes.data), "nvkv_split_plan")
    return first, last


def nvkv_append(cache: Cache, seqs: Seqs, k_new: torch.Tensor, v_new: torch.Tensor,
                cu_new: torch.Tensor, total_new: int, max_new: int, stream=None) -> None:
    _fmt(cache, "nvfp4", "nvkv_append")
    _check(library().nvkv_append(
        ctypes.byref(cache._c), ctypes.byref(seqs._c), _dev(k_new, torch.bfloat16, "k_new"),
        _dev(v_new, torch.bfloat16, "v_new"), _dev(cu_new, torch.int32, "cu_new"), int(total_new),
        int(max_new), _stream(stream)), "nvkv_append")


def nvkv_rope_table(cs: torch.Tensor, rotary_dim: int, base: float, scale: float,
                    stream=None) -> None:
    """Fill cs (float32 CUDA [max_pos][rotary_dim/2][2]) with (cos, sin) of
    (pos / scale) * base^(-2i / rotary_dim)."""
    if cs.dim() != 3 or cs.shape[1] * 2 != rotary_dim or cs.shape[2] != 2:
        raise ValueError("cs must be [max_pos][rotary_dim/2][2]")
    _check(library().nvkv_rope_table(_dev(cs, torch.float32, "cs"), int(cs.shape[0]),
                                     int(rotary_dim), float(base), float(scale), _stream(stream)),
           "nvkv_rope_table")


def nvkv_append_rope(cache: Cache, seqs: Seqs, k_new: torch.Tensor, v_new: torch.Tensor,
                     cu_new: torch.Tensor, total_new: int, max_new: int, rope_cs: torch.Tensor,
                     rotary_dim: int, stream=None) -> None:
    """nvkv_append with K rotated at its position by the rope_cs table."""
    _fmt(cache, "nvfp4", "nvkv_append_rope")
    _check(library().nvkv_append_rope(
        ctypes.byref(cache._c), ctypes.byref(seqs._c), _dev(k_new, torch.bfloat16, "k_new"),
        _dev(v_new, torch.bfloat16, "v_new"), _dev(cu_new, torch.int32, "cu_new"), int(total_new),
        int(max_new), _dev(rope_cs, torch.float32, "rope_cs"), int(rope_cs.shape[0]),
        int(rotary_dim), _stream(stream)), "nvkv_append_rope")


def nvkv_decode_attn(cache: Cache, seqs: Seqs, q: torch.Tensor, T: int, num_q_heads: int,
                     sm_scale: float, num_splits: int, workspace: torch.Tensor,
                     stream=None) -> None:
    _fmt(cache, "nvfp4", "nvkv_decode_attn")
    _check(library().nvkv_decode_attn(
        ctypes.byref(cache._c), ctypes.byref(seqs._c), _dev(q, torch.bfloat16, "q"), int(T),
        int(num_q_heads), float(sm_scale), int(num_splits), _dev(workspace, torch.uint8, "workspace"),
        workspace.numel(), _stream(stream)), "nvkv_decode_attn")


def nvkv_decode_kernel_name(cache: Cache, T: int, num_q_heads: int) -> str:
    """The decode kernel the decode call of this cache's format launches for
    this step shape: "decode_qk4", "decode_tc" or "decode_simt" (NVFP4);
    "decode_qk4_k8v4" or "decode_simt" (K8V4)."""
    if cache.kv_format == "k8v4":
        fn = library().nvkv_decode_kernel_name_k8v4
    else:
        fn = library().nvkv_decode_kernel_name
    return fn(ctypes.byref(cache._c), int(T), int(num_q_heads)).decode()


def nvkv_combine(seqs: Seqs, workspace: torch.Tensor, T: int, num_q_heads: int,
                 num_kv_heads: int, head_dim: int, num_splits: int, out: torch.Tensor,
                 stream=None) -> None:
    _check(library().nvkv_combine(
        ctypes.byref(seqs._c), _dev(workspace, torch.uint8, "workspace"), int(T), int(num_q_heads),
        int(num_kv_heads), int(head_dim), int(num_splits), _dev(out, torch.bfloat16, "out"),
        _stream(stream)), "nvkv_combine")


def nvkv_prefill_attn(cache: Cache, seqs: Seqs, q: torch.Tensor, cu_q: torch.Tensor,
                      total_q: int, max_q: int, num_q_heads: int, sm_scale: float,
                      out: torch.Tensor, stream=None) -> None:
    _fmt(cache, "nvfp4", "nvkv_prefill_attn")
    _check(library().nvkv_prefill_attn(
        ctypes.byref(cache._c), ctypes.byref(seqs._c), _dev(q, torch.bfloat16, "q"),
        _dev(cu_q, torch.int32, "cu_q"), int(total_q), int(max_q), int(num_q_heads),
        float(sm_scale), _dev(out, torch.bfloat16, "out"), _stream(stream)), "nvkv_prefill_attn")


def nvkv_prefill_workspace_bytes(total_q: int, num_q_heads: int, head_dim: int,
                                 num_splits: int) -> int:
    return int(library().nvkv_prefill_workspace_bytes(int(total_q), int(num_q_heads),
                                                      int(head_dim), int(num_splits)))


def nvkv_prefill_num_splits(cache: Cache, batch: int, max_q: int, num_q_heads: int) -> int:
    """The key-split count nvkv_prefill_attn_split takes for num_splits = 0."""
    return int(library().nvkv_prefill_num_splits(ctypes.byref(cache._c), int(batch), int(max_q),
                                                 int(num_q_heads)))


def nvkv_prefill_attn_split(cache: Cache, seqs: Seqs, q: torch.Tensor, cu_q: torch.Tensor,
                            total_q: int, max_q: int, num_q_heads: int, sm_scale: float,
                            num_splits: int, workspace: "torch.Tensor | None", out: torch.Tensor,
                            stream=None) -> None:
    """Chunked prefill with the keys of each query tile split over num_splits
    (1..8) CTAs (0: automatic) and merged; workspace: uint8 device tensor of at least
    nvkv_prefill_workspace_bytes(...) bytes (None when the count is 1)."""
    _fmt(cache, "nvfp4", "nvkv_prefill_attn_split")
    ws = _dev(workspace, torch.uint8, "workspace") if workspace is not None else None
    nbytes = workspace.numel() if workspace is not None else 0
    _check(library().nvkv_prefill_attn_split(
        ctypes.byref(cache._c), ctypes.byref(seqs._c), _dev(q, torch.bfloat16, "q"),
        _dev(cu_q, torch.int32, "cu_q"), int(total_q), int(max_q), int(num_q_heads),
        float(sm_scale), int(num_splits), ws, nbytes, _dev(out, torch.bfloat16, "out"),
        _stream(stream)), "nvkv_prefill_attn_split")


def nvkv_decode_static_scratch_bytes() -> int:
    return int(library().nvkv_decode_static_scratch_bytes())


def nvkv_decode_attn_static(cache: Cache, seqs: Seqs, q: torch.Tensor, T: int, num_q_heads: int,
                            sm_scale: float, num_splits: int, out: torch.Tensor,
                            stream=None) -> None:
    """Decode attention + combine with the library's own device scratch (no
    workspace argument, nothing allocated); see include/nvkv.h."""
    _fmt(cache, "nvfp4", "nvkv_decode_attn_static")
    _check(library().nvkv_decode_attn_static(
        ctypes.byref(cache._c), ctypes.byref(seqs._c), _dev(q, torch.bfloat16, "q"), int(T),
        int(num_q_heads), float(sm_scale), int(num_splits), _dev(out, torch.bfloat16, "out"),
        _stream(stream)), "nvkv_decode_attn_static")


def _dev_or_pinned(t: torch.Tensor, dtype: torch.dtype, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not (t.is_cuda or t.is_pinned()):
        raise ValueError(f"{name} must be on a CUDA device or in pinned host memory")
    return t.data_ptr()


def _pages_args(cache: Cache, page_ids, slot_ids, arena, err_word):
    n = page_ids.numel()
    if slot_ids.numel() != n:
        raise ValueError("page_ids and slot_ids must have the same length")
    pb = _page_bytes_of(cache.kv_format, cache.num_kv_heads, cache.head_dim)
    return (ctypes.byref(cache._c), _dev_or_pinned(page_ids, torch.int32, "page_ids"),
            _dev_or_pinned(slot_ids, torch.int32, "slot_ids"), int(n),
            _dev_or_pinned(arena, torch.uint8, "arena"), arena.numel() // pb,
            _dev(err_word, torch.int32, "err_word") if err_word is not None else None)


def nvkv_pages_spill(cache: Cache, page_ids: torch.Tensor, slot_ids: torch.Tensor,
                     arena: torch.Tensor, err_word: torch.Tensor | None = None, stream=None) -> None:
    """Pool page page_ids[i] -> arena slot slot_ids[i] (arena: uint8, device
    or pinned host, a whole number of page-sized slots of the cache's
    format)."""
    fn = library().nvkv_pages_spill_k8v4 if cache.kv_format == "k8v4" else library().nvkv_pages_spill
    _check(fn(*_pages_args(cache, page_ids, slot_ids, arena, err_word), _stream(stream)),
           "nvkv_pages_spill")


def nvkv_pages_restore(cache: Cache, page_ids: torch.Tensor, slot_ids: torch.Tensor,
                       arena: torch.Tensor, err_word: torch.Tensor | None = None,
                       stream=None) -> None:
    """Arena slot slot_ids[i] -> pool page page_ids[i]."""
    fn = (library().nvkv_pages_restore_k8v4 if cache.kv_format == "k8v4"
          else library().nvkv_pages_restore)
    _check(fn(*_pages_args(cache, page_ids, slot_ids, arena, err_word), _stream(stream)),
           "nvkv_pages_restore")


# ---- K8V4 cache (8-bit K rows with one fp32 scale per row, NVFP4 V) --------

def nvkv_k8v4_page_bytes(num_kv_heads: int, head_dim: int) -> int:
    return int(library().nvkv_k8v4_page_bytes(num_kv_heads, head_dim))


def nvkv_append_k8v4(cache: Cache, seqs: Seqs, k_new: torch.Tensor, v_new: torch.Tensor,
                     cu_new: torch.Tensor, total_new: int, max_new: int, stream=None) -> None:
    _fmt(cache, "k8v4", "nvkv_append_k8v4")
    _check(library().nvkv_append_k8v4(
        ctypes.byref(cache._c), ctypes.byref(seqs._c), _dev(k_new, torch.bfloat16, "k_new"),
        _dev(v_new, torch.bfloat16, "v_new"), _dev(cu_new, torch.int32, "cu_new"), int(total_new),
        int(max_new), _stream(stream)), "nvkv_append_k8v4")


def nvkv_decode_attn_k8v4(cache: Cache, seqs: Seqs, q: torch.Tensor, T: int, num_q_heads: int,
                          sm_scale: float, num_splits: int, workspace: torch.Tensor,
                          stream=None) -> None:
    """Split-K partial results over a K8V4 cache; merge with nvkv_combine."""
    _fmt(cache, "k8v4", "nvkv_decode_attn_k8v4")
    _check(library().nvkv_decode_attn_k8v4(
        ctypes.byref(cache._c), ctypes.byref(seqs._c), _dev(q, torch.bfloat16, "q"), int(T),
        int(num_q_heads), float(sm_scale), int(num_splits), _dev(workspace, torch.uint8, "workspace"),
        workspace.numel(), _stream(stream)), "nvkv_decode_attn_k8v4")


def nvkv_prefill_attn_k8v4(cache: Cache, seqs: Seqs, q: torch.Tensor, cu_q: torch.Tensor,
                           total_q: int, max_q: int, num_q_heads: int, sm_scale: float,
                           out: torch.Tensor, stream=None) -> None:
    _fmt(cache, "k8v4", "nvkv_prefill_attn_k8v4")
    _check(library().nvkv_prefill_attn_k8v4(
        ctypes.byref(cache._c), ctypes.byref(seqs._c), _dev(q, torch.bfloat16, "q"),
        _dev(cu_q, torch.int32, "cu_q"), int(total_q), int(max_q), int(num_q_heads),
        float(sm_scale), _dev(out, torch.bfloat16, "out"), _stream(stream)), "nvkv_prefill_attn_k8v4")


# ---- masked attention, several-axis rotary append, reading rows back -------
# These calls also check that their tensors are on one device and as large as
# the call makes them, and run on that device whatever the current one is.
# A serving step makes a few of them per layer, each shorter than ten
# microseconds on the GPU, so the checks are kept to one test a tensor.

def _arg(t: torch.Tensor, dtype: torch.dtype, device: int, n: int, name: str) -> int:
    """Address of a tensor argument: contiguous, of the dtype, on the device
    and of at least n elements."""
    try:
        if (t.dtype is dtype and t.get_device() == device and t.numel() >= n
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _dev(t, dtype, name)  # raises for a wrong type, dtype, place or layout
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the cache on cuda:{device}")
    raise ValueError(f"{name} has {t.numel()} elements, needs {n}")


def _on(cache: Cache, seqs: Seqs) -> int:
    """The device index of a call's cache and sequences."""
    device = cache.pool.get_device()
    if seqs.page_table.get_device() != device or seqs.kv_lens.get_device() != device:
        raise ValueError(f"the page table is on {seqs.page_table.device}, kv_lens on "
                         f"{seqs.kv_lens.device}, the cache on {cache.pool.device}")
    if seqs.err_word is not None and seqs.err_word.get_device() != device:
        raise ValueError(f"err_word is on {seqs.err_word.device}, the cache on {cache.pool.device}")
    return device


def _call(device: int, fn, what: str, stream, *args) -> None:
    if device == torch._C._cuda_getDevice():
        if stream is None:
            status = fn(*args, torch._C._cuda_getCurrentRawStream(device))
        else:
            status = fn(*args, _stream(stream))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _stream(stream))
    if status != OK:
        raise NvkvError(status, what)


class ScoreMod:
    """How a masked attention call changes its scores and which keys a query
    sees (nvkv_score_mod in include/nvkv.h): scores capped at softcap by a
    tanh, a bias -alibi_slopes[head] * |distance| (float32 [Hq]), a sliding
    window of that many keys, a prefix of prefix_lens[b] tokens (int32
    [batch]) whose queries see all of it, and the first visible key key_starts
    (int32, [batch] for decode, [total_q] for prefill).  Every call takes the
    attributes as they are then, and its kernels read the tensors."""

    def __init__(self, softcap: float = 0.0, window: int = 0,
                 alibi_slopes: torch.Tensor | None = None, prefix_lens: torch.Tensor | None = None,
                 key_starts: torch.Tensor | None = None):
        self.softcap, self.window = float(softcap), int(window)
        self.alibi_slopes, self.prefix_lens, self.key_starts = alibi_slopes, prefix_lens, key_starts
        for t, dtype, name in ((alibi_slopes, torch.float32, "alibi_slopes"),
                               (prefix_lens, torch.int32, "prefix_lens"),
                               (key_starts, torch.int32, "key_starts")):
            if t is not None:
                _dev(t, dtype, name)

    def _struct(self, device: int, num_q_heads: int, batch: int, starts: int) -> _ScoreModC:
        a, p, k = self.alibi_slopes, self.prefix_lens, self.key_starts
        if not 0 <= self.window < 2 ** 31:
            raise ValueError(f"window is {self.window}, must be 0 .. 2^31 - 1")
        # (a struct of its own for each call: the library reads it after the
        # interpreter's lock is dropped, when another thread may make a call)
        return _ScoreModC(
            self.softcap, self.window,
            None if a is None else _arg(a, torch.float32, device, num_q_heads, "alibi_slopes"),
            None if p is None else _arg(p, torch.int32, device, batch, "prefix_lens"),
            None if k is None else _arg(k, torch.int32, device, starts, "key_starts"))


def nvkv_decode_mod_kernel_name(cache: Cache, T: int, num_q_heads: int) -> str:
    """The kernel that nvkv_decode_attn_mod launches for this cache and step
    shape: one of the names of nvkv_decode_kernel_name."""
    if cache.kv_format == "k8v4":
        return nvkv_decode_kernel_name(cache, T, num_q_heads)
    return library().nvkv_decode_mod_kernel_name(ctypes.byref(cache._c), int(T),
                                                 int(num_q_heads)).decode()


def nvkv_decode_attn_mod(cache: Cache, seqs: Seqs, q: torch.Tensor, T: int, num_q_heads: int,
                         sm_scale: float, mod: ScoreMod, num_splits: int,
                         workspace: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    """Decode attention of T queries per sequence with the scores and masks of
    mod, merged into out (bf16 [batch*T][Hq][D]); workspace as for
    nvkv_decode_attn.  For caches of either format."""
    device, L = _on(cache, seqs), _lib or library()
    n = seqs.batch * T * num_q_heads * cache.head_dim
    fn = L.nvkv_decode_attn_mod_k8v4 if cache.kv_format == "k8v4" else L.nvkv_decode_attn_mod
    _call(device, fn, "nvkv_decode_attn_mod", stream, ctypes.byref(cache._c),
          ctypes.byref(seqs._c), _arg(q, torch.bfloat16, device, n, "q"), T, num_q_heads, sm_scale,
          ctypes.byref(mod._struct(device, num_q_heads, seqs.batch, seqs.batch)), num_splits,
          _arg(workspace, torch.uint8, device, 0, "workspace"), workspace.numel(),
          _arg(out, torch.bfloat16, device, n, "out"))


def nvkv_prefill_attn_mod(cache: Cache, seqs: Seqs, q: torch.Tensor, cu_q: torch.Tensor,
                          total_q: int, max_q: int, num_q_heads: int, sm_scale: float,
                          mod: ScoreMod, num_splits: int, workspace: "torch.Tensor | None",
                          out: torch.Tensor, stream=None) -> None:
    """Chunked prefill with the scores and masks of mod; num_splits and
    workspace as for nvkv_prefill_attn_split (0 splits: as many of the
    automatic count as the workspace has room for).  For caches of either
    format."""
    device, L = _on(cache, seqs), _lib or library()
    n = total_q * num_q_heads * cache.head_dim
    fn = L.nvkv_prefill_attn_mod_k8v4 if cache.kv_format == "k8v4" else L.nvkv_prefill_attn_mod
    ws, size = None, 0
    if workspace is not None:
        ws, size = _arg(workspace, torch.uint8, device, 0, "workspace"), workspace.numel()
    _call(device, fn, "nvkv_prefill_attn_mod", stream, ctypes.byref(cache._c),
          ctypes.byref(seqs._c), _arg(q, torch.bfloat16, device, n, "q"),
          _arg(cu_q, torch.int32, device, seqs.batch + 1, "cu_q"), total_q, max_q, num_q_heads,
          sm_scale, ctypes.byref(mod._struct(device, num_q_heads, seqs.batch, total_q)),
          num_splits, ws, size,
          _arg(out, torch.bfloat16, device, n, "out"))


def _axis_bytes(axes) -> bytes:
    """One byte for each number.  Element by element: bytes() of an object with
    a buffer (a numpy array, an array.array) would be its memory, not its numbers."""
    return axes if type(axes) is bytes else bytes(list(axes))


def nvkv_append_rope_axes(cache: Cache, seqs: Seqs, k_new: torch.Tensor, v_new: torch.Tensor,
                          cu_new: torch.Tensor, total_new: int, max_new: int,
                          rope_cs: torch.Tensor, rotary_dim: int, positions: torch.Tensor,
                          axis_of_pair, q: torch.Tensor | None = None,
                          q_out: torch.Tensor | None = None, stream=None) -> None:
    """nvkv_append_rope with the positions of every row on several axes:
    positions int32 [num_axes][total_new], axis_of_pair the axis (a whole
    number) of each of the rotary_dim/2 pairs, as bytes or any sequence of
    whole numbers (a list, a numpy array or array.array of any integer type).  q
    (bf16 [total_new][Hq][D]) is rotated into q_out in the same launch."""
    _fmt(cache, "nvfp4", "nvkv_append_rope_axes")
    device = _on(cache, seqs)
    pos_shape, cs_shape = positions.shape, rope_cs.shape
    if len(pos_shape) != 2 or pos_shape[1] != total_new:
        raise ValueError("positions must be [num_axes][total_new]")
    if len(cs_shape) != 3 or cs_shape[1] * 2 != rotary_dim or cs_shape[2] != 2:
        raise ValueError("rope_cs must be [max_pos][rotary_dim/2][2]")
    if len(axis_of_pair) * 2 != rotary_dim:
        raise ValueError("axis_of_pair must have rotary_dim/2 entries")
    n = total_new * cache.num_kv_heads * cache.head_dim
    hq, qp, qo = 0, None, None
    if q is not None and q_out is not None:
        q_shape = q.shape
        if len(q_shape) != 3 or q_shape[0] != total_new or q_shape[2] != cache.head_dim:
            raise ValueError("q must be [total_new][Hq][D]")
        if q_out.shape != q_shape:
            raise ValueError("q_out must have the shape of q")
        hq = q_shape[1]
        qp, qo = _arg(q, torch.bfloat16, device, 0, "q"), _arg(q_out, torch.bfloat16, device, 0, "q_out")
    elif q is not None or q_out is not None:
        raise ValueError("q and q_out go together")
    _call(device, (_lib or library()).nvkv_append_rope_axes, "nvkv_append_rope_axes", stream,
          ctypes.byref(cache._c), ctypes.byref(seqs._c),
          _arg(k_new, torch.bfloat16, device, n, "k_new"),
          _arg(v_new, torch.bfloat16, device, n, "v_new"),
          _arg(cu_new, torch.int32, device, seqs.batch + 1, "cu_new"), total_new, max_new,
          _arg(rope_cs, torch.float32, device, 0, "rope_cs"), cs_shape[0], rotary_dim,
          _arg(positions, torch.int32, device, 0, "positions"), pos_shape[0],
          _axis_bytes(axis_of_pair), qp, hq, qo)


def nvkv_read_rows(cache: Cache, seqs: Seqs, starts: torch.Tensor, cu_rows: torch.Tensor,
                   total_rows: int, max_rows: int, k_out: torch.Tensor, v_out: torch.Tensor,
                   stream=None) -> None:
    """The cached K and V rows of positions starts[b] .. of every sequence as
    bf16, rows cu_rows[b] .. cu_rows[b+1]-1 of k_out and v_out
    ([total_rows][Hkv][D]).  For caches of either format."""
    device, L = _on(cache, seqs), _lib or library()
    n = total_rows * cache.num_kv_heads * cache.head_dim
    _call(device, L.nvkv_read_rows_k8v4 if cache.kv_format == "k8v4" else L.nvkv_read_rows,
          "nvkv_read_rows", stream, ctypes.byref(cache._c), ctypes.byref(seqs._c),
          _arg(starts, torch.int32, device, seqs.batch, "starts"),
          _arg(cu_rows, torch.int32, device, seqs.batch + 1, "cu_rows"), total_rows, max_rows,
          _arg(k_out, torch.bfloat16, device, n, "k_out"),
          _arg(v_out, torch.bfloat16, device, n, "v_out"))
