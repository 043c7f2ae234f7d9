"""Paged-serving operators (include/fia.h): block tables and slot maps, the cache
write, attention with a sliding window and sinks, and decode behind a shared
prefix.

As in _binding.py every step runs in the library's CUDA kernels.  The
marshalling (device and stride checks, tensor descriptions, outputs and the
workspace from torch, the current stream) is compiled (csrc/py_paged.cpp): these
calls take a few microseconds.  Lengths are int32 CUDA tensors, read by the
kernels: no call waits for the GPU or copies to it, and a captured call replays
with new lengths.  There is no fallback: a missing library or a failing call
raises.
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os

from . import build
from ._binding import INT32_MAX, LIB_PATH, FIAError

EXT_PATH = os.path.join(os.path.dirname(LIB_PATH), "_fia_paged.so")
_ext = None


def _load():
    global _ext
    if not os.path.exists(EXT_PATH):
        raise ImportError(f"{os.path.basename(EXT_PATH)} not built at {EXT_PATH}; run attention_fia_prefill_gb300.build.build()")
    import torch   # (its libraries are what the binding links to)
    if build.ext_torch_version() != torch.__version__:
        raise ImportError(f"{os.path.basename(EXT_PATH)} was built against torch {build.ext_torch_version() or '?'}, this is "
                          f"{torch.__version__}; run attention_fia_prefill_gb300.build.build()")
    loader = importlib.machinery.ExtensionFileLoader("_fia_paged", EXT_PATH)
    ext = importlib.util.module_from_spec(importlib.util.spec_from_loader("_fia_paged", loader))
    loader.exec_module(ext)
    ext.set_error(FIAError)
    _ext = ext
    return ext


def fia_block_table_append(context_lens, new_lens, free_blocks, block_table, *, block_size, num_tokens,
                           slot_mapping=None, kv_lens=None, cu_new_lens=None, num_blocks=None):
    """Grows the block tables of a batch to its new lengths and maps every new
    token to its slot of the paged cache.

    context_lens, new_lens: int32 (B), tokens held and to append; free_blocks:
    int32 (F), ids handed out from the front (the list stays as it is: the next
    call takes it without its first num_blocks ids); block_table: int32 (B, W),
    changed in place; num_tokens: slots to write, at least the sum of new_lens.
    Returns (slot_mapping (num_tokens), kv_lens (B), cu_new_lens (B), num_blocks
    (1)), all int32; num_blocks above F says that the list ran out."""
    return (_ext or _load()).block_table_append(context_lens, new_lens, free_blocks, block_table, block_size, num_tokens,
                                                slot_mapping, kv_lens, cu_new_lens, num_blocks)


def fia_cache_write(key, value, key_cache, value_cache, slot_mapping):
    """Copies new keys and values (T, KV_N, D) to the slots slot_mapping (int32,
    T) of the pools ((blocknum, KV_N, block_size, D) or (blocknum, block_size,
    KV_N*D)), in place; negative slots are skipped.  key and value may be slices
    of a fused projection (any token stride).  value and value_cache may be
    None.  Returns (key_cache, value_cache)."""
    return (_ext or _load()).cache_write(key, value, key_cache, value_cache, slot_mapping)


def fia_decode_window(query, key, value, *, actual_seq_kvlen=None, block_table=None, block_size=0, num_heads=1,
                      num_key_value_heads=0, scale_value=1.0, input_layout="BSH", pre_tokens=INT32_MAX, sink_tokens=0,
                      softmax_lse_flag=False, out=None, softmax_lse=None):
    """Incremental attention (Q_S 1..16 new tokens) with a sliding window and
    sink tokens: the token at position p sees key j when j <= p and (j >= p -
    pre_tokens or j < sink_tokens).  actual_seq_kvlen: int32 CUDA tensor (B),
    lengths with the new tokens.  key / value paged or contiguous as for
    fia_decode.  Returns (attention_out, softmax_lse or None)."""
    return (_ext or _load()).decode_window(query, key, value, actual_seq_kvlen, block_table, sink_tokens, num_heads,
                                           num_key_value_heads, scale_value, input_layout, pre_tokens, block_size,
                                           softmax_lse_flag, out, softmax_lse)


def fia_prefill_window(query, key, value, *, actual_seq_qlen=None, actual_seq_kvlen=None, block_table=None, block_size=0,
                       num_heads=1, num_key_value_heads=0, scale_value=1.0, input_layout="BSH", pre_tokens=INT32_MAX,
                       sink_tokens=0, softmax_lse_flag=False, out=None, softmax_lse=None, workspace=None):
    """Prefill (any Q_S) with a sliding window and sink tokens: row i of a batch,
    at position p = i + kv_len - q_len, sees key j when j <= p and (j >= p -
    pre_tokens or j < sink_tokens).  actual_seq_qlen / actual_seq_kvlen: int32
    CUDA tensors (B); for a TND query, and TND keys, running sums.  key / value
    contiguous, or pools with block_table as for fia_prefill_paged.  Returns
    (attention_out, softmax_lse or None)."""
    return (_ext or _load()).prefill_window(query, key, value, actual_seq_qlen, actual_seq_kvlen, block_table, sink_tokens,
                                            num_heads, num_key_value_heads, scale_value, input_layout, pre_tokens, block_size,
                                            softmax_lse_flag, out, softmax_lse, workspace)


def fia_decode_shared_prefix(query, key_cache, value_cache, *, block_table, block_size, actual_seq_kvlen,
                             shared_prefix_len, num_heads=1, num_key_value_heads=0, scale_value=1.0, input_layout="BSH",
                             softmax_lse_flag=False, out=None, softmax_lse=None, workspace=None):
    """Incremental attention (Q_S 1..16 new tokens) for a batch whose block
    tables all begin with the blocks of one shared prefix of shared_prefix_len
    keys (a multiple of block_size), which are read once for the whole batch.
    actual_seq_kvlen: int32 CUDA tensor (B), whole lengths.  Each token sees the
    cache up to itself.  Returns (attention_out, softmax_lse or None)."""
    return (_ext or _load()).decode_shared_prefix(query, key_cache, value_cache, actual_seq_kvlen, block_table,
                                                  shared_prefix_len, num_heads, num_key_value_heads, scale_value,
                                                  input_layout, INT32_MAX, block_size, softmax_lse_flag, out, softmax_lse,
                                                  workspace)
