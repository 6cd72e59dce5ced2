"""B200-native int4 KV-cache quantization and decode attention on the packed
cache (compressed-domain attention).  The compute path is libtq.so (CUDA,
sm_100a) behind the C ABI of include/tq.h; this package is its binding.
"""
from ._lib import (TQError, decode_chunk_tokens, decode_workspace_bytes, load,
                   quantize_append, quantize_append_q8, read_q8, sdpa_int4_decode, sdpa_q8,
                   sdpa_q8_decode, sdpa_q8_decode_append, sdpa_q8_workspace_bytes, status_string)
from .cache import BlockKVCache, CodebookKVCache, Int4KVCache, UniformKVCache

__all__ = ["BlockKVCache", "CodebookKVCache", "Int4KVCache", "UniformKVCache", "TQError",
           "decode_chunk_tokens", "decode_workspace_bytes", "load", "quantize_append",
           "quantize_append_q8", "read_q8", "sdpa_int4_decode", "sdpa_q8", "sdpa_q8_decode",
           "sdpa_q8_decode_append", "sdpa_q8_workspace_bytes", "status_string"]
