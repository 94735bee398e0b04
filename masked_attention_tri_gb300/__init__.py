"""GB300-native (sm_103a) attention: masked, biased triangle attention, packed sequences and a paged cache.

O[b,n,h,q,:] = sum_k softmax_k(s * Q.K + bias[b,h,q,k], or -1e9 where the key
is masked) V[b,n,h,k,:], with the per-row logsumexp and max, as defined on the
cuEquivariance triangle_attention API page; plus a packed-sequence form with a
block-sparse (BlockMask) mask, the backward of both forms, rotary positions, and the
cache that decoding fills (kv_cache_append) and reads (paged_attention).  The work runs in
libtriattn.so (hand-written CUDA, tcgen05 / TMA); this package only marshals tensors into its C ABI.
"""
from . import abi
from .api import (BlockMask, get_status, mask_to_kv_lengths, triangle_attention, triangle_attention_autograd,
                  triangle_attention_backward, varlen_attention, varlen_attention_backward,
                  varlen_attention_kvpacked, varlen_attention_qkvpacked)
from .cache import PagedKVCache, kv_cache_append, paged_attention
from .positions import Rotary, rotary_embedding, rotary_embedding_autograd, rotary_embedding_backward

__all__ = ["abi", "BlockMask", "get_status", "mask_to_kv_lengths", "triangle_attention", "triangle_attention_autograd",
           "triangle_attention_backward", "varlen_attention", "varlen_attention_backward", "varlen_attention_kvpacked",
           "varlen_attention_qkvpacked", "PagedKVCache", "Rotary", "kv_cache_append", "paged_attention",
           "rotary_embedding", "rotary_embedding_autograd", "rotary_embedding_backward"]
