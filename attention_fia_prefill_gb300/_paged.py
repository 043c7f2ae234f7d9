"""ctypes binding of the paged-serving operators (include/fia.h): block tables
and slot maps, the cache write, attention with a sliding window and sinks, and
decode behind a shared prefix.

As in _binding.py every step runs in the library's CUDA kernels; the functions
here check devices, describe torch tensors, allocate outputs and pass the
current CUDA stream.  Lengths are int32 CUDA tensors, read by the kernels: no
call waits for the GPU or copies to it, and a captured call replays with new
lengths.
"""
from __future__ import annotations

import ctypes
import struct

from ._binding import INT32_MAX, _dtype_code, _lse_shape, _params, _stream_ptr, check, load_library

# fia_tensor: data, dtype, ndim, shape[5].  A packed byte string is passed where
# the call takes a const fia_tensor* (a tenth of the cost of a ctypes struct).
_PACK = struct.Struct("<Qii5q").pack
STATUS_BYTES = 256   # workspace of a call that needs no more than its status word
_PAD = ((0,) * 5, (0,) * 4, (0,) * 3, (0,) * 2, (0,), ())


def _desc(t, name):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _desc_of(t)


def _desc_of(t):
    shape = t.shape
    if len(shape) > 5:
        raise ValueError("at most 5 dims")
    return _PACK(t.data_ptr(), _dtype_code(t), len(shape), *shape, *_PAD[len(shape)])


class _on:
    """Makes the tensors' device current for the call; all must share it."""

    def __init__(self, *ts):
        dev = ts[0].device
        for t in ts:
            if t is not None and t.device != dev:
                raise ValueError("tensors must be on one device")
        if dev.type != "cuda":
            raise ValueError("fia kernels take CUDA tensors")
        self.device = dev
        self.guard = None

    def __enter__(self):
        import torch
        if torch.cuda.current_device() != self.device.index:
            self.guard = torch.cuda.device(self.device)
            self.guard.__enter__()
        return _stream_ptr(self.device)

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def fia_block_table_append(context_lens, new_lens, free_blocks, block_table, *, block_size, num_tokens,
                           slot_mapping=None, kv_lens=None, cu_new_lens=None, num_blocks=None):
    """Grows the block tables of a batch to its new lengths and maps every new
    token to its slot of the paged cache.

    context_lens, new_lens: int32 (B), tokens held and to append; free_blocks:
    int32 (F), ids handed out from the front; block_table: int32 (B, W), changed
    in place; num_tokens: slots to write, at least the sum of new_lens.  Returns
    (slot_mapping (num_tokens), kv_lens (B), cu_new_lens (B), num_blocks (1)),
    all int32; num_blocks above F says that the list ran out."""
    import torch
    for name, t in (("context_lens", context_lens), ("new_lens", new_lens), ("free_blocks", free_blocks)):
        if t.dtype != torch.int32:
            raise TypeError(f"{name} must be int32")
    with _on(context_lens, new_lens, free_blocks, block_table, slot_mapping, kv_lens, cu_new_lens, num_blocks) as stream:
        new = context_lens.new_empty
        if slot_mapping is None:
            slot_mapping = new(num_tokens)
        if slot_mapping.shape[0] != num_tokens:
            raise ValueError("slot_mapping must have num_tokens entries")
        kv_lens = new(context_lens.shape) if kv_lens is None else kv_lens
        cu_new_lens = new(context_lens.shape) if cu_new_lens is None else cu_new_lens
        num_blocks = new(1) if num_blocks is None else num_blocks
        check(load_library().fia_block_table_append(
            _desc(context_lens, "context_lens"), _desc(new_lens, "new_lens"), _desc(free_blocks, "free_blocks"),
            block_size, _desc(block_table, "block_table"), _desc(slot_mapping, "slot_mapping"),
            _desc(kv_lens, "kv_lens"), _desc(cu_new_lens, "cu_new_lens"), _desc(num_blocks, "num_blocks"), stream))
    return slot_mapping, kv_lens, cu_new_lens, num_blocks


def _token_stride(t, name):
    """Elements between the tokens of a (T, N, D) tensor whose heads and columns are contiguous."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be (T, KV_N, D)")
    st, n, d = t.stride(), t.shape[1], t.shape[2]
    if (d > 1 and st[2] != 1) or (n > 1 and st[1] != d):
        raise ValueError(f"{name}: the heads and columns of a token must be contiguous")
    return st[0] if t.shape[0] > 1 else n * d


def fia_cache_write(key, value, key_cache, value_cache, slot_mapping):
    """Copies new keys and values (T, KV_N, D) to the slots slot_mapping (int32,
    T) of the pools ((blocknum, KV_N, block_size, D) or (blocknum, block_size,
    KV_N*D)), in place; negative slots are skipped.  key and value may be slices
    of a fused projection (any token stride).  value and value_cache may be
    None.  Returns (key_cache, value_cache)."""
    with _on(key, value, key_cache, value_cache, slot_mapping) as stream:
        check(load_library().fia_cache_write(
            _desc_of(key), _token_stride(key, "key"), None if value is None else _desc_of(value),
            0 if value is None else _token_stride(value, "value"), _desc(key_cache, "key_cache"),
            _desc(value_cache, "value_cache"), _desc(slot_mapping, "slot_mapping"), stream))
    return key_cache, value_cache


def fia_decode_window(query, key, value, *, actual_seq_kvlen=None, block_table=None, block_size=0, num_heads=1,
                      num_key_value_heads=0, scale_value=1.0, input_layout="BSH", pre_tokens=INT32_MAX, sink_tokens=0,
                      softmax_lse_flag=False, out=None, softmax_lse=None):
    """Incremental attention (Q_S 1..16 new tokens) with a sliding window and
    sink tokens: the token at position p sees key j when j <= p and (j >= p -
    pre_tokens or j < sink_tokens).  actual_seq_kvlen: int32 CUDA tensor (B),
    lengths with the new tokens.  key / value paged or contiguous as for
    fia_decode.  Returns (attention_out, softmax_lse or None)."""
    import torch
    with _on(query, key, value, actual_seq_kvlen, block_table, out, softmax_lse) as stream:
        prm = _params(num_heads=num_heads, num_key_value_heads=num_key_value_heads, scale_value=scale_value,
                      input_layout=input_layout, pre_tokens=pre_tokens, block_size=block_size,
                      softmax_lse_flag=softmax_lse_flag)
        if out is None:
            out = torch.empty_like(query)
        if softmax_lse_flag and softmax_lse is None:
            softmax_lse = query.new_empty(_lse_shape(query, input_layout, num_heads), dtype=torch.float32)
        check(load_library().fia_decode_window(
            _desc(query, "query"), _desc(key, "key"), _desc(value, "value"), _desc(block_table, "block_table"),
            _desc(actual_seq_kvlen, "actual_seq_kvlen"), ctypes.byref(prm.p), sink_tokens, _desc(out, "out"),
            _desc(softmax_lse, "softmax_lse"), stream))
    return out, softmax_lse


def fia_prefill_window(query, key, value, *, actual_seq_qlen=None, actual_seq_kvlen=None, block_table=None, block_size=0,
                       num_heads=1, num_key_value_heads=0, scale_value=1.0, input_layout="BSH", pre_tokens=INT32_MAX,
                       sink_tokens=0, softmax_lse_flag=False, out=None, softmax_lse=None, workspace=None):
    """Prefill (any Q_S) with a sliding window and sink tokens: row i of a batch,
    at position p = i + kv_len - q_len, sees key j when j <= p and (j >= p -
    pre_tokens or j < sink_tokens).  actual_seq_qlen / actual_seq_kvlen: int32
    CUDA tensors (B); for a TND query, and TND keys, running sums.  key / value
    contiguous, or pools with block_table as for fia_prefill_paged.  Returns
    (attention_out, softmax_lse or None)."""
    import torch
    with _on(query, key, value, actual_seq_qlen, actual_seq_kvlen, block_table, out, softmax_lse, workspace) as stream:
        prm = _params(num_heads=num_heads, num_key_value_heads=num_key_value_heads, scale_value=scale_value,
                      input_layout=input_layout, pre_tokens=pre_tokens, block_size=block_size,
                      softmax_lse_flag=softmax_lse_flag)
        if out is None:
            out = torch.empty_like(query)
        if softmax_lse_flag and softmax_lse is None:
            softmax_lse = query.new_empty(_lse_shape(query, input_layout, num_heads), dtype=torch.float32)
        if workspace is None:   # the status word
            workspace = query.new_empty(STATUS_BYTES, dtype=torch.uint8)
        check(load_library().fia_prefill_window(
            _desc(query, "query"), _desc(key, "key"), _desc(value, "value"), _desc(block_table, "block_table"),
            _desc(actual_seq_qlen, "actual_seq_qlen"), _desc(actual_seq_kvlen, "actual_seq_kvlen"), ctypes.byref(prm.p),
            sink_tokens, _desc(out, "out"), _desc(softmax_lse, "softmax_lse"), workspace.data_ptr(), workspace.numel(),
            stream))
    return out, softmax_lse


def fia_decode_shared_prefix(query, key_cache, value_cache, *, block_table, block_size, actual_seq_kvlen,
                             shared_prefix_len, num_heads=1, num_key_value_heads=0, scale_value=1.0, input_layout="BSH",
                             softmax_lse_flag=False, out=None, softmax_lse=None, workspace=None):
    """Incremental attention (Q_S 1..16 new tokens) for a batch whose block
    tables all begin with the blocks of one shared prefix of shared_prefix_len
    keys (a multiple of block_size), which are read once for the whole batch.
    actual_seq_kvlen: int32 CUDA tensor (B), whole lengths.  Each token sees the
    cache up to itself.  Returns (attention_out, softmax_lse or None)."""
    import torch
    with _on(query, key_cache, value_cache, block_table, actual_seq_kvlen, out, softmax_lse, workspace) as stream:
        prm = _params(num_heads=num_heads, num_key_value_heads=num_key_value_heads, scale_value=scale_value,
                      input_layout=input_layout, block_size=block_size, softmax_lse_flag=softmax_lse_flag)
        if out is None:
            out = torch.empty_like(query)
        if softmax_lse_flag and softmax_lse is None:
            softmax_lse = query.new_empty(_lse_shape(query, input_layout, num_heads), dtype=torch.float32)
        lib = load_library()
        args = (_desc(query, "query"), _desc(key_cache, "key_cache"), _desc(value_cache, "value_cache"),
                _desc(block_table, "block_table"), _desc(actual_seq_kvlen, "actual_seq_kvlen"), ctypes.byref(prm.p),
                shared_prefix_len, _desc(out, "out"), _desc(softmax_lse, "softmax_lse"))
        if workspace is None:
            n = ctypes.c_size_t(0)
            check(lib.fia_decode_shared_prefix_get_workspace_size(*args, ctypes.byref(n)))
            workspace = query.new_empty(n.value, dtype=torch.uint8)
        check(lib.fia_decode_shared_prefix(*args, workspace.data_ptr(), workspace.numel(), stream))
    return out, softmax_lse
