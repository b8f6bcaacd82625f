"""Thin Python binding of libvq (ctypes): argument marshalling only.

Every computation runs in the CUDA kernels of libvq.so. This module turns torch
tensors into device pointers and strides, calls the C entry point of the same
name and raises VqError on a non-zero status. PyTorch is used only for device
memory and streams. If libvq.so is missing, importing this module raises: there
is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional, Sequence

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libvq.so")

VQ_OK, VQ_ERR_INVALID_ARGUMENT, VQ_ERR_UNSUPPORTED, VQ_ERR_MISALIGNED, VQ_ERR_CUDA = range(5)
VQ_BF16, VQ_F32, VQ_F16 = 0, 1, 2
VQ_INT8, VQ_E4M3 = 0, 1
VQ_PAGE_TOKENS = 64


class VqError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"libvq status {status}: {message}")
        self.status = status


class vq_cache_desc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("bits", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("block_tokens", ctypes.POINTER(ctypes.c_int32)), ("meta_fp16", ctypes.c_int32)]


class vq_layer_cache(ctypes.Structure):
    _fields_ = [("packed_k", ctypes.c_void_p), ("packed_v", ctypes.c_void_p),
                ("scale_k", ctypes.c_void_p), ("zero_k", ctypes.c_void_p),
                ("scale_v", ctypes.c_void_p), ("zero_v", ctypes.c_void_p)]


class vq_paged_desc(ctypes.Structure):
    _fields_ = [("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("code", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


class vq_paged_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("weight", ctypes.c_void_p)]


class vq_paged_query(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("q_heads", ctypes.c_int32), ("n", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("q", ctypes.c_void_p), ("q_strides", ctypes.c_int64 * 3),
                ("block_table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("q_lens", ctypes.c_void_p),
                ("q_pos", ctypes.c_void_p), ("prefix", ctypes.c_void_p), ("first", ctypes.c_void_p),
                ("slopes", ctypes.c_void_p), ("softmax_scale", ctypes.c_float), ("softcap", ctypes.c_float),
                ("causal", ctypes.c_int32)]


# the same structure packed in one call, for the binding's own use (a fifth of the time that filling fields takes)
_QUERY = struct.Struct("@4iP3q7P2fi")
_I64x3 = ctypes.c_int64 * 3


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is not built; run bit_kv_cache_25_b200.build.build() first")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I32, I64P, VP, F = ctypes.POINTER, ctypes.c_int32, ctypes.POINTER(ctypes.c_int64), ctypes.c_void_p, ctypes.c_float
    SZ = ctypes.c_size_t
    sig = {
        "vq_cache_layout": [P(vq_cache_desc), P(SZ), P(SZ), P(SZ)],
        "vq_quantize_pack_block": [P(vq_cache_desc), I32, VP, I32, I64P, VP, VP, VP, VP],
        "vq_cache_append": [P(vq_cache_desc), P(vq_layer_cache), I32, VP, VP, I32, I64P, I64P, VP],
        "vq_attention_block": [P(vq_cache_desc), P(vq_layer_cache), I32, VP, I64P, F, VP, I32, I64P, VP],
        "vq_append_attention_block": [P(vq_cache_desc), P(vq_layer_cache), I32, VP, VP, I32, I64P, I64P, VP, I64P, F,
                                      VP, I32, I64P, VP],
        "vq_dequantize": [P(vq_cache_desc), I32, VP, VP, VP, VP, VP],
        "vq_paper_layout": [P(vq_cache_desc), P(SZ), P(SZ), P(SZ)],
        "vq_paper_pack": [P(vq_cache_desc), P(vq_layer_cache), VP, VP, VP, VP, VP],
        "vq_paper_unpack": [P(vq_cache_desc), VP, VP, VP, VP, P(vq_layer_cache), VP],
        "vq_paged_append": [P(vq_paged_desc), P(vq_paged_cache), I32, I32, VP, VP, I32, I64P, I64P, VP, VP, VP, VP, VP],
        "vq_paged_read": [P(vq_paged_desc), P(vq_paged_cache), I32, I32, VP, VP, VP, VP, VP, I32, I64P, I64P, VP],
        "vq_paged_attention_workspace": [P(vq_paged_desc), I32, I32, I32, P(SZ)],
        "vq_paged_attention": [P(vq_paged_desc), P(vq_paged_cache), VP, VP, I64P, VP, VP, SZ, VP],
        "vq_paged_weights": [P(vq_paged_desc), P(vq_paged_cache), VP, VP, I32, VP],
        "vq_paged_evict": [P(vq_paged_desc), P(vq_paged_cache), I32, VP, VP, P(vq_paged_desc), P(vq_paged_cache), VP, VP,
                           I32, I32, I32, VP, VP],
        "vq_poll_device_error": [P(ctypes.c_uint32)],
        "vq_check_wait_timeout": [ctypes.c_uint32, VP],
        "vq_status_string": [I32],
        "vq_last_error": [],
        "vq_version": [],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_char_p if name in ("vq_status_string", "vq_last_error") else ctypes.c_int32
    return lib


_lib = _load()

EXPORTED = ("vq_cache_layout", "vq_quantize_pack_block", "vq_cache_append", "vq_attention_block",
            "vq_append_attention_block", "vq_dequantize", "vq_paper_layout", "vq_paper_pack", "vq_paper_unpack",
            "vq_paged_append", "vq_paged_read", "vq_paged_attention_workspace", "vq_paged_attention",
            "vq_paged_weights", "vq_paged_evict",
            "vq_poll_device_error", "vq_check_wait_timeout", "vq_status_string", "vq_last_error", "vq_version")


def _check(status: int):
    if status != VQ_OK:
        raise VqError(status, _lib.vq_last_error().decode() or _lib.vq_status_string(status).decode())


class CacheDesc:
    """Host-side vq_cache_desc plus the int32 block schedule it points to."""

    def __init__(self, batch: int, heads: int, head_dim: int, bits: int, block_tokens: Sequence[int],
                 meta_fp16: bool = False):
        self.block_tokens = list(int(n) for n in block_tokens)
        self._arr = (ctypes.c_int32 * max(1, len(self.block_tokens)))(*self.block_tokens)
        self.c = vq_cache_desc(batch, heads, head_dim, bits, len(self.block_tokens), self._arr, int(bool(meta_fp16)))

    @property
    def batch(self): return self.c.batch

    @property
    def heads(self): return self.c.heads

    @property
    def head_dim(self): return self.c.head_dim

    @property
    def bits(self): return self.c.bits

    @property
    def num_blocks(self): return self.c.num_blocks

    @property
    def meta_fp16(self): return bool(self.c.meta_fp16)

    def word_rows(self, s: int) -> int:
        cpw = 32 // self.bits
        return (self.block_tokens[s] + cpw - 1) // cpw


def _strides(t: torch.Tensor, ndim_expected: int = 4):
    if t.dim() != ndim_expected:
        raise ValueError(f"expected a {ndim_expected}-d [B][H][T][D] tensor, got {tuple(t.shape)}")
    if t.stride(-1) != 1:
        raise ValueError("the channel dimension must be contiguous")
    return (ctypes.c_int64 * 3)(t.stride(0), t.stride(1), t.stride(2))


def _block_tokens(desc: "CacheDesc", block: int) -> int:
    if not 0 <= int(block) < desc.num_blocks:
        raise ValueError(f"block {block} out of range [0, {desc.num_blocks})")
    return desc.block_tokens[int(block)]


def _check_slab(name: str, t: torch.Tensor, desc: "CacheDesc", n: int):
    """t must be a [B][H][n][D] view of the block (any strides, channels contiguous)."""
    want = (desc.batch, desc.heads, n, desc.head_dim)
    if tuple(t.shape) != want:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {want} ([B][H][n_s][D] of this block)")


def _check_flat(name: str, t: torch.Tensor, numel: int, dtypes):
    """t is written or read as a flat array of at least numel elements from data_ptr()."""
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs at least {numel}")


def _check_devices(*named):
    """Every tensor on the same CUDA device (a host pointer would become an
    out-of-bounds device access)."""
    dev = None
    for name, t in named:
        if not t.is_cuda:
            raise ValueError(f"{name} is on {t.device}, not a CUDA device")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the other tensors on {dev}")


_WORDS = (torch.int32, torch.uint32) if hasattr(torch, "uint32") else (torch.int32,)
_F32 = (torch.float32,)


def _check_cache(desc: "CacheDesc", cache: "LayerCache"):
    words, meta, _ = vq_cache_layout(desc)
    for name in ("packed_k", "packed_v"):
        _check_flat(f"cache.{name}", getattr(cache, name), words, _WORDS)
    for name in ("scale_k", "zero_k", "scale_v", "zero_v"):
        _check_flat(f"cache.{name}", getattr(cache, name), meta, _F32)
    ptrs = (cache.packed_k.data_ptr(), cache.packed_v.data_ptr(), cache.scale_k.data_ptr(),
            cache.zero_k.data_ptr(), cache.scale_v.data_ptr(), cache.zero_v.data_ptr())
    if ptrs != (cache.c.packed_k, cache.c.packed_v, cache.c.scale_k, cache.c.zero_k, cache.c.scale_v, cache.c.zero_v):
        raise ValueError("cache tensors were replaced after the LayerCache was built")
    return [(f"cache.{n}", getattr(cache, n)) for n in
            ("packed_k", "packed_v", "scale_k", "zero_k", "scale_v", "zero_v")]


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return VQ_BF16
    if t.dtype == torch.float32:
        return VQ_F32
    raise ValueError(f"unsupported dtype {t.dtype}")


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def vq_cache_layout(desc: CacheDesc):
    """-> (words_per_tensor, meta_per_tensor, block_word_offset list of S+1)."""
    w, m = ctypes.c_size_t(), ctypes.c_size_t()
    offs = (ctypes.c_size_t * (desc.num_blocks + 1))()
    _check(_lib.vq_cache_layout(ctypes.byref(desc.c), ctypes.byref(w), ctypes.byref(m), offs))
    return w.value, m.value, list(offs)


class LayerCache:
    """One layer's cache buffers, allocated by torch (the caller), in the layout
    vq_cache_layout describes."""

    def __init__(self, desc: CacheDesc, device="cuda"):
        words, meta, offs = vq_cache_layout(desc)
        self.desc = desc
        self.block_word_offset = offs
        self.packed_k = torch.empty(words, dtype=torch.int32, device=device)
        self.packed_v = torch.empty(words, dtype=torch.int32, device=device)
        self.scale_k = torch.empty(meta, dtype=torch.float32, device=device)
        self.zero_k = torch.empty(meta, dtype=torch.float32, device=device)
        self.scale_v = torch.empty(meta, dtype=torch.float32, device=device)
        self.zero_v = torch.empty(meta, dtype=torch.float32, device=device)
        self.c = vq_layer_cache(self.packed_k.data_ptr(), self.packed_v.data_ptr(), self.scale_k.data_ptr(),
                                self.zero_k.data_ptr(), self.scale_v.data_ptr(), self.zero_v.data_ptr())

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in
                   (self.packed_k, self.packed_v, self.scale_k, self.zero_k, self.scale_v, self.zero_v))


def vq_quantize_pack_block(desc: CacheDesc, block: int, x: torch.Tensor, packed: torch.Tensor,
                           scale: torch.Tensor, zero: torch.Tensor, stream=None):
    """Quantize + bit-pack one block of one tensor x [B][H][n_s][D] (bf16/fp32)."""
    n = _block_tokens(desc, block)
    _check_slab("x", x, desc, n)
    bhd = desc.batch * desc.heads * desc.head_dim
    _check_flat("packed", packed, bhd * desc.word_rows(block), _WORDS)
    _check_flat("scale", scale, bhd, _F32)
    _check_flat("zero", zero, bhd, _F32)
    _check_devices(("x", x), ("packed", packed), ("scale", scale), ("zero", zero))
    _check(_lib.vq_quantize_pack_block(ctypes.byref(desc.c), block, x.data_ptr(), _dtype(x), _strides(x),
                                       packed.data_ptr(), scale.data_ptr(), zero.data_ptr(), _stream(stream)))


def vq_cache_append(desc: CacheDesc, cache: LayerCache, block: int, k: torch.Tensor, v: torch.Tensor, stream=None):
    """Quantize block `block` of K and V ([B][H][n_s][D] views) into the layer cache."""
    if k.dtype != v.dtype:
        raise ValueError("k and v must have the same dtype")
    n = _block_tokens(desc, block)
    _check_slab("k", k, desc, n)
    _check_slab("v", v, desc, n)
    _check_devices(("k", k), ("v", v), *_check_cache(desc, cache))
    _check(_lib.vq_cache_append(ctypes.byref(desc.c), ctypes.byref(cache.c), block, k.data_ptr(), v.data_ptr(),
                                _dtype(k), _strides(k), _strides(v), _stream(stream)))


def vq_attention_block(desc: CacheDesc, cache: LayerCache, block: int, q: torch.Tensor, softmax_scale: float,
                       out: torch.Tensor, stream=None):
    """Attention of block `block`'s queries q [B][H][n_s][D] (bf16) over the packed
    cache of blocks 0..block; writes out [B][H][n_s][D] (fp32 or bf16)."""
    if q.dtype != torch.bfloat16:
        raise ValueError("q must be bfloat16")
    n = _block_tokens(desc, block)
    _check_slab("q", q, desc, n)
    _check_slab("out", out, desc, n)
    _check_devices(("q", q), ("out", out), *_check_cache(desc, cache))
    _check(_lib.vq_attention_block(ctypes.byref(desc.c), ctypes.byref(cache.c), block, q.data_ptr(), _strides(q),
                                   ctypes.c_float(softmax_scale), out.data_ptr(), _dtype(out), _strides(out),
                                   _stream(stream)))


def vq_append_attention_block(desc: CacheDesc, cache: LayerCache, block: int, k: torch.Tensor, v: torch.Tensor,
                              q: torch.Tensor, softmax_scale: float, out: torch.Tensor, stream=None):
    """Append block `block` of K and V ([B][H][n_s][D]) and attend its queries q
    over blocks 0..block in one call; the same cache and output as
    vq_cache_append followed by vq_attention_block."""
    if k.dtype != v.dtype:
        raise ValueError("k and v must have the same dtype")
    if q.dtype != torch.bfloat16:
        raise ValueError("q must be bfloat16")
    n = _block_tokens(desc, block)
    for name, t in (("k", k), ("v", v), ("q", q), ("out", out)):
        _check_slab(name, t, desc, n)
    _check_devices(("k", k), ("v", v), ("q", q), ("out", out), *_check_cache(desc, cache))
    _check(_lib.vq_append_attention_block(ctypes.byref(desc.c), ctypes.byref(cache.c), block, k.data_ptr(),
                                          v.data_ptr(), _dtype(k), _strides(k), _strides(v), q.data_ptr(),
                                          _strides(q), ctypes.c_float(softmax_scale), out.data_ptr(), _dtype(out),
                                          _strides(out), _stream(stream)))


def vq_paper_layout(desc: CacheDesc):
    """-> (words_per_tensor, meta_words_per_tensor, block_word_offset list of S+1) of the storage
    format the results tables count (one padding-free stream per block, 32-bit metadata pairs)."""
    w, m = ctypes.c_size_t(), ctypes.c_size_t()
    offs = (ctypes.c_size_t * (desc.num_blocks + 1))()
    _check(_lib.vq_paper_layout(ctypes.byref(desc.c), ctypes.byref(w), ctypes.byref(m), offs))
    return w.value, m.value, list(offs)


def vq_paper_pack(desc: CacheDesc, cache: LayerCache, k_words: torch.Tensor, v_words: torch.Tensor,
                  k_meta: torch.Tensor, v_meta: torch.Tensor, stream=None):
    """Write the layer cache in the storage format (lossless when desc.meta_fp16)."""
    words, meta, _ = vq_paper_layout(desc)
    for name, t, n in (("k_words", k_words, words), ("v_words", v_words, words), ("k_meta", k_meta, meta),
                       ("v_meta", v_meta, meta)):
        _check_flat(name, t, n, _WORDS)
    _check_devices(("k_words", k_words), ("v_words", v_words), ("k_meta", k_meta), ("v_meta", v_meta),
                   *_check_cache(desc, cache))
    _check(_lib.vq_paper_pack(ctypes.byref(desc.c), ctypes.byref(cache.c), k_words.data_ptr(), v_words.data_ptr(),
                              k_meta.data_ptr(), v_meta.data_ptr(), _stream(stream)))


def vq_paper_unpack(desc: CacheDesc, k_words: torch.Tensor, v_words: torch.Tensor, k_meta: torch.Tensor,
                    v_meta: torch.Tensor, cache: LayerCache, stream=None):
    """Fill the layer cache from the storage format."""
    words, meta, _ = vq_paper_layout(desc)
    for name, t, n in (("k_words", k_words, words), ("v_words", v_words, words), ("k_meta", k_meta, meta),
                       ("v_meta", v_meta, meta)):
        _check_flat(name, t, n, _WORDS)
    _check_devices(("k_words", k_words), ("v_words", v_words), ("k_meta", k_meta), ("v_meta", v_meta),
                   *_check_cache(desc, cache))
    _check(_lib.vq_paper_unpack(ctypes.byref(desc.c), k_words.data_ptr(), v_words.data_ptr(), k_meta.data_ptr(),
                                v_meta.data_ptr(), ctypes.byref(cache.c), _stream(stream)))


def vq_dequantize(desc: CacheDesc, block: int, packed: torch.Tensor, scale: torch.Tensor, zero: torch.Tensor,
                  out: torch.Tensor, stream=None):
    """Check-only: dequantize one packed block into out [B][H][n_s][D] float32 (contiguous)."""
    if out.dtype != torch.float32 or not out.is_contiguous():
        raise ValueError("out must be contiguous float32")
    n = _block_tokens(desc, block)
    _check_slab("out", out, desc, n)
    bhd = desc.batch * desc.heads * desc.head_dim
    _check_flat("packed", packed, bhd * desc.word_rows(block), _WORDS)
    _check_flat("scale", scale, bhd, _F32)
    _check_flat("zero", zero, bhd, _F32)
    _check_devices(("packed", packed), ("scale", scale), ("zero", zero), ("out", out))
    _check(_lib.vq_dequantize(ctypes.byref(desc.c), block, packed.data_ptr(), scale.data_ptr(), zero.data_ptr(),
                              out.data_ptr(), _stream(stream)))


# ---------------------------------------------------------------- paged 8-bit cache
_CODES = {"int8": VQ_INT8, "e4m3": VQ_E4M3, VQ_INT8: VQ_INT8, VQ_E4M3: VQ_E4M3}
_CODE_DTYPES = {VQ_INT8: (torch.int8, torch.uint8), VQ_E4M3: (torch.float8_e4m3fn, torch.uint8)}
_PAGED_DTYPES = {torch.bfloat16: VQ_BF16, torch.float16: VQ_F16, torch.float32: VQ_F32}


class PagedDesc:
    """Shape of a paged cache: key heads, head_dim, "int8" or "e4m3" codes, pages in
    the pools and pages in a row of the block table."""

    def __init__(self, kv_heads: int, head_dim: int, code, num_pages: int, max_pages: int):
        if code not in _CODES:
            raise ValueError(f"code {code!r}: expected 'int8' or 'e4m3'")
        self.kv_heads, self.head_dim, self.code = int(kv_heads), int(head_dim), _CODES[code]
        self.num_pages, self.max_pages = int(num_pages), int(max_pages)
        self.c = vq_paged_desc(self.kv_heads, self.head_dim, self.code, self.num_pages, self.max_pages)
        self.ref = ctypes.byref(self.c)
        self.shape = (self.kv_heads, self.head_dim, self.code, self.num_pages, self.max_pages)
        self._workspace = {}  # (device, batch, q_heads, n) -> bytes


class PagedCache:
    """The pools of one layer: codes k, v [num_pages][kv_heads][64][head_dim], scales
    [num_pages][kv_heads] and, if asked for, pos and weight [num_pages][kv_heads][64].
    Given tensors are used as they are; the others are allocated here. The tensors of
    a PagedCache stay the same for its life."""

    def __init__(self, desc: PagedDesc, device="cuda", positions: bool = False, weights: bool = False, *, k=None,
                 v=None, k_scale=None, v_scale=None, pos=None, weight=None):
        n, h, d = desc.num_pages, desc.kv_heads, desc.head_dim
        given = [t for t in (k, v, k_scale, v_scale, pos, weight) if t is not None]
        if given:
            device = given[0].device
        slots = (n, h, VQ_PAGE_TOKENS)

        def pool(name, t, shape, dtypes, want=True):
            if t is None:
                return torch.zeros(shape, dtype=dtypes[0], device=device) if want else None
            if t.dtype not in dtypes:
                raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
            if tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{name} has shape {tuple(t.shape)}, expected contiguous {shape}")
            if t.device != device:
                raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")
            return t

        codes = _CODE_DTYPES[desc.code]
        self._desc = desc
        self._k = pool("k", k, slots + (d,), codes)
        self._v = pool("v", v, slots + (d,), codes)
        self._k_scale = pool("k_scale", k_scale, (n, h), _F32)
        self._v_scale = pool("v_scale", v_scale, (n, h), _F32)
        self._pos = pool("pos", pos, slots, (torch.int32,), positions)
        self._weight = pool("weight", weight, slots, _F32, weights)
        self.device = self._k.device
        self.index = self._k.get_device()  # -1: not on a GPU
        self.c = vq_paged_cache(*(None if t is None else t.data_ptr() for t in
                                  (self._k, self._v, self._k_scale, self._v_scale, self._pos, self._weight)))
        self.ref = ctypes.byref(self.c)

    desc = property(lambda self: self._desc)
    k = property(lambda self: self._k)
    v = property(lambda self: self._v)
    k_scale = property(lambda self: self._k_scale)
    v_scale = property(lambda self: self._v_scale)
    pos = property(lambda self: self._pos)
    weight = property(lambda self: self._weight)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in
                   (self._k, self._v, self._k_scale, self._v_scale, self._pos, self._weight) if t is not None)


def _paged_cache_check(desc: PagedDesc, cache: PagedCache) -> int:
    """Index of the cache's device."""
    if cache._desc is not desc and cache._desc.shape != desc.shape:
        raise ValueError("the cache was made for another descriptor")
    if cache.index < 0:
        raise ValueError(f"the cache is on {cache.device}, not a CUDA device")
    return cache.index


_I32 = torch.int32


def _array(name: str, t: Optional[torch.Tensor], shape, device: int, dtype=_I32, optional=True):
    """Device address of a contiguous array argument; None if it is left out."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is missing")
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} is {t.dtype} of shape {tuple(t.shape)}, expected contiguous {dtype} of {tuple(shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not with the cache")
    return t.data_ptr()


def _view(name: str, t: torch.Tensor, shape, device: int):
    """Strides of a [B][H][n][D] argument with channels contiguous."""
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    b, h, n, d = t.stride()
    if d != 1:
        raise ValueError(f"{name}: the channel dimension must be contiguous")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not with the cache")
    return b, h, n


def _paged_dtype(name: str, t: torch.Tensor, allowed) -> int:
    code = _PAGED_DTYPES.get(t.dtype)
    if code not in allowed:
        raise ValueError(f"{name} has unsupported dtype {t.dtype}")
    return code


def _rows(name: str, t: torch.Tensor, heads: Optional[int], desc: PagedDesc):
    shape = t.shape
    if len(shape) != 4 or shape[3] != desc.head_dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected [batch][{heads or 'heads'}][n][{desc.head_dim}]")
    if shape[0] < 1 or shape[2] < 1:
        raise ValueError(f"{name} has shape {tuple(shape)}: batch and n must be at least 1")
    return shape


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the handle without a Stream object around it


def _handle(device: int, stream):
    """The stream a call runs on: the one given, or the device's current one."""
    if stream is None:
        return _raw_stream(device) if _raw_stream is not None else torch.cuda.current_stream(device).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _on(device: int, stream, call):
    """call(stream handle) with `device` current."""
    if device == torch.cuda.current_device():
        _check(call(_handle(device, stream)))
    else:
        with torch.cuda.device(device):
            _check(call(_handle(device, stream)))


def vq_paged_append(desc: PagedDesc, cache: PagedCache, block_table: torch.Tensor, start: torch.Tensor,
                    k: torch.Tensor, v: torch.Tensor, counts: Optional[torch.Tensor] = None,
                    pos: Optional[torch.Tensor] = None, stream=None):
    """Quantize k, v [B][kv_heads][n][D] (bf16, fp16, fp32) into the sequences' pages as
    tokens start[b] .. start[b] + counts[b] - 1 (counts None: n)."""
    dev = _paged_cache_check(desc, cache)
    B, _, n, _ = _rows("k", k, desc.kv_heads, desc)
    if k.dtype != v.dtype:
        raise ValueError("k and v must have the same dtype")
    dt = _paged_dtype("k", k, (VQ_BF16, VQ_F16, VQ_F32))
    ks, vs = _I64x3(*_view("k", k, k.shape, dev)), _I64x3(*_view("v", v, k.shape, dev))
    table = _array("block_table", block_table, (B, desc.max_pages), dev, optional=False)
    start = _array("start", start, (B,), dev, optional=False)
    counts, pos = _array("counts", counts, (B,), dev), _array("pos", pos, (B,), dev)
    _on(dev, stream, lambda s: _lib.vq_paged_append(desc.ref, cache.ref, B, n, k.data_ptr(), v.data_ptr(), dt, ks, vs,
                                                    table, start, counts, pos, s))


def vq_paged_read(desc: PagedDesc, cache: PagedCache, block_table: torch.Tensor, start: torch.Tensor,
                  k_out: torch.Tensor, v_out: torch.Tensor, counts: Optional[torch.Tensor] = None, stream=None):
    """Dequantize tokens start[b] .. start[b] + counts[b] - 1 into k_out, v_out [B][kv_heads][n][D]."""
    dev = _paged_cache_check(desc, cache)
    B, _, n, _ = _rows("k_out", k_out, desc.kv_heads, desc)
    if k_out.dtype != v_out.dtype:
        raise ValueError("k_out and v_out must have the same dtype")
    dt = _paged_dtype("k_out", k_out, (VQ_BF16, VQ_F16, VQ_F32))
    ks = _I64x3(*_view("k_out", k_out, k_out.shape, dev))
    vs = _I64x3(*_view("v_out", v_out, k_out.shape, dev))
    table = _array("block_table", block_table, (B, desc.max_pages), dev, optional=False)
    start = _array("start", start, (B,), dev, optional=False)
    counts = _array("counts", counts, (B,), dev)
    _on(dev, stream, lambda s: _lib.vq_paged_read(desc.ref, cache.ref, B, n, table, start, counts, k_out.data_ptr(),
                                                  v_out.data_ptr(), dt, ks, vs, s))


def _paged_query(desc, block_table, lens, q, softmax_scale, q_lens, q_pos, prefix, first, slopes, softcap, causal, dev):
    """(shape of q, vq_paged_query as bytes)."""
    shape = B, Hq, n, _ = _rows("q", q, None, desc)
    dt = _paged_dtype("q", q, (VQ_BF16, VQ_F16))
    sb, sh, st = _view("q", q, shape, dev)
    per = (B,)
    return shape, _QUERY.pack(
        B, Hq, n, dt, q.data_ptr(), sb, sh, st, _array("block_table", block_table, (B, desc.max_pages), dev, optional=False),
        _array("lens", lens, per, dev, optional=False), _array("q_lens", q_lens, per, dev) or 0,
        _array("q_pos", q_pos, per, dev) or 0, _array("prefix", prefix, per, dev) or 0,
        _array("first", first, (B, n), dev) or 0, _array("slopes", slopes, (Hq,), dev, torch.float32) or 0,
        softmax_scale, softcap, 1 if causal else 0)


def vq_paged_attention_workspace(desc: PagedDesc, batch: int, q_heads: int, n: int) -> int:
    """Bytes of workspace that vq_paged_attention needs on the current device."""
    size = ctypes.c_size_t()
    _check(_lib.vq_paged_attention_workspace(desc.ref, batch, q_heads, n, ctypes.byref(size)))
    return size.value


def vq_paged_attention(desc: PagedDesc, cache: PagedCache, block_table: torch.Tensor, lens: torch.Tensor,
                       q: torch.Tensor, softmax_scale: float, out: torch.Tensor, lse: Optional[torch.Tensor] = None, *,
                       q_lens=None, q_pos=None, prefix=None, first=None, slopes=None, softcap: float = 0.0,
                       causal: bool = False, workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of q [B][Hq][n][D] (bf16 or fp16) over each sequence's first lens[b] cached
    tokens, into out (q's shape and type) and lse [B][Hq][n] float32. The masks and biases are
    vq.h's. workspace: a contiguous uint8 tensor of vq_paged_attention_workspace bytes that no
    call running at the same time uses; None: allocated for this call."""
    dev = _paged_cache_check(desc, cache)
    shape, query = _paged_query(desc, block_table, lens, q, softmax_scale, q_lens, q_pos, prefix, first, slopes, softcap,
                                causal, dev)
    if out.dtype is not q.dtype:
        raise ValueError(f"out is {out.dtype}, q is {q.dtype}: they must have the same dtype")
    os_ = _I64x3(*_view("out", out, shape, dev))
    lse = _array("lse", lse, shape[:3], dev, torch.float32)
    if workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        raise ValueError("workspace must be contiguous and with the cache")
    B, Hq, n, _ = shape

    def call(s):
        size = desc._workspace.get((dev, B, Hq, n))
        if size is None:
            size = desc._workspace[(dev, B, Hq, n)] = vq_paged_attention_workspace(desc, B, Hq, n)
        ws = workspace
        if ws is None and size:
            # from the pool of the stream that the call runs on: memory goes back to it in its order
            if stream is None:
                ws = torch.empty(size, dtype=torch.uint8, device=cache.device)
            else:
                on = stream if hasattr(stream, "cuda_stream") else (
                    torch.cuda.ExternalStream(int(stream), cache.device) if int(stream) else torch.cuda.default_stream(cache.device))
                with torch.cuda.stream(on):
                    ws = torch.empty(size, dtype=torch.uint8, device=cache.device)
        ptr, have = (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())
        return _lib.vq_paged_attention(desc.ref, cache.ref, query, out.data_ptr(), os_, lse, ptr, have, s)

    _on(dev, stream, call)


def vq_paged_weights(desc: PagedDesc, cache: PagedCache, block_table: torch.Tensor, lens: torch.Tensor,
                     q: torch.Tensor, softmax_scale: float, lse: torch.Tensor, *, q_lens=None, q_pos=None, prefix=None,
                     first=None, slopes=None, softcap: float = 0.0, causal: bool = False, accumulate: bool = True,
                     stream=None):
    """Per cached token the sum of its attention weights over these queries (and the query heads
    of its key head), added to cache.weight or put there; lse as vq_paged_attention gave it.
    No two sequences of a call may share a page: call it for them one after the other."""
    dev = _paged_cache_check(desc, cache)
    if cache.weight is None:
        raise ValueError("the cache has no weight")
    shape, query = _paged_query(desc, block_table, lens, q, softmax_scale, q_lens, q_pos, prefix, first, slopes, softcap,
                                causal, dev)
    lse = _array("lse", lse, shape[:3], dev, torch.float32, optional=False)
    _on(dev, stream, lambda s: _lib.vq_paged_weights(desc.ref, cache.ref, query, lse, 1 if accumulate else 0, s))


def vq_paged_evict(desc: PagedDesc, cache: PagedCache, block_table: torch.Tensor, lens: torch.Tensor,
                   to_desc: PagedDesc, to: PagedCache, to_table: torch.Tensor, to_lens: torch.Tensor, keep: int, *,
                   sinks: int = 0, recent: int = 0, kept: torch.Tensor, stream=None):
    """Keep at most `keep` tokens per sequence and key head by cache.weight, moved in order to
    the pages of to_table; writes to_lens [B] and the source slots kept [B][kv_heads][keep]."""
    dev = _paged_cache_check(desc, cache)
    if _paged_cache_check(to_desc, to) != dev:
        raise ValueError(f"the caches are on {cache.device} and {to.device}")
    if cache.weight is None:
        raise ValueError("the cache has no weight")
    if lens.dim() != 1 or lens.shape[0] < 1:
        raise ValueError(f"lens has shape {tuple(lens.shape)}, expected [batch]")
    B = lens.shape[0]
    table = _array("block_table", block_table, (B, desc.max_pages), dev, optional=False)
    lens = _array("lens", lens, (B,), dev, optional=False)
    to_table = _array("to_table", to_table, (B, to_desc.max_pages), dev, optional=False)
    to_lens = _array("to_lens", to_lens, (B,), dev, optional=False)
    kept = _array("kept", kept, (B, desc.kv_heads, int(keep)), dev, optional=False)
    _on(dev, stream, lambda s: _lib.vq_paged_evict(desc.ref, cache.ref, B, table, lens, to_desc.ref, to.ref, to_table,
                                                   to_lens, int(keep), int(sinks), int(recent), kept, s))


def vq_poll_device_error() -> int:
    code = ctypes.c_uint32()
    _check(_lib.vq_poll_device_error(ctypes.byref(code)))
    return code.value


def vq_check_wait_timeout(max_iters: int, stream=None):
    """Launch the self-test whose bounded wait times out (see vq.h); the device
    error word then holds flag 1 once the stream has run it."""
    _check(_lib.vq_check_wait_timeout(max_iters, _stream(stream)))


def vq_version() -> int:
    return _lib.vq_version()


def raw_lib():
    """The ctypes handle (for ABI tests)."""
    return _lib
