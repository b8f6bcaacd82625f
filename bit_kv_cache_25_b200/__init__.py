"""VAR-Q-style packed low-bit KV cache for block-by-block visual AR decoding on B200,
and a paged 8-bit cache for decoding token by token or in chunks.

The compute lives in libvq.so (CUDA, sm_100a); `vq` is its ctypes binding.
"""
from . import vq  # noqa: F401
from .vq import (CacheDesc, LayerCache, PagedCache, PagedDesc, VqError, vq_append_attention_block,  # noqa: F401
                 vq_attention_block, vq_cache_append,
                 vq_cache_layout, vq_dequantize, vq_paged_append, vq_paged_attention,
                 vq_paged_attention_workspace, vq_paged_evict, vq_paged_read, vq_paged_weights,
                 vq_poll_device_error, vq_quantize_pack_block, vq_version)
