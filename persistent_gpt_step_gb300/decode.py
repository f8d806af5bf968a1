"""The operators of a batched decode step on torch CUDA tensors: gpt_kv_append, gpt_decode_attention and
gpt_next_token of the C ABI (also reached as ``binding.kv_append`` and so on).

Every tensor's device, type, shape and strides are checked here before the call; a mismatch raises
GptError(INVALID_ARG).  Indices that live on the device are checked by the kernels and reported in
``status`` (int32 [1], STATUS_* bits of ``binding``, zeroed by the caller).  Calls run on ``stream`` (default:
the current stream) without synchronising; what they return belongs to that stream.

A call's time on the host is that of one small decode step, so the structs are packed as bytes (0.15 us
where building a ctypes structure takes 0.7) and each tensor is looked at once.
"""

from __future__ import annotations

import ctypes
import struct

import torch

from . import binding as B

_CODES = {ctypes.c_void_p: "P", ctypes.c_int64: "q", ctypes.c_size_t: "N", ctypes.c_int32: "i", ctypes.c_float: "f",
          ctypes.c_double: "d"}
_TYPES = {torch.float32: B.DTYPE_FP32, torch.bfloat16: B.DTYPE_BF16}
_I32, _F32 = torch.int32, torch.float32


def _packer(cls):
    """struct.pack for a ctypes structure's fields, in their order."""
    return struct.Struct("@" + "".join(_CODES[t] for _, t in cls._fields_) + "0q").pack


_pack_cache, _pack_append = _packer(B.gpt_paged_cache), _packer(B.gpt_kv_append_args)
_pack_attention, _pack_token = _packer(B.gpt_decode_attention_args), _packer(B.gpt_next_token_args)


def _refuse(msg):
    raise B.GptError(-1, msg)


def _device(name, t):
    """Index of the call's device: that of its first tensor, which must be the current one."""
    if not isinstance(t, torch.Tensor) or t.get_device() < 0:
        _refuse(f"{name} must be a CUDA tensor")
    device = t.get_device()
    if device != torch._C._cuda_getDevice():
        _refuse(f"{name} is on cuda:{device}, not the current device")
    return device


def _ptr(name, t, dtype, shape, device):
    """Address of a tensor of this type and shape on the device, its elements side by side."""
    if t.dtype is not dtype or t.get_device() != device or t.shape != shape or (t.stride()[-1] != 1 and shape[-1] > 1):
        if t.dtype is not dtype:
            _refuse(f"{name} must be {dtype}, got {t.dtype}")
        if t.get_device() != device:
            _refuse(f"{name} is on {t.device}, not on cuda:{device}")
        if t.shape != shape:
            _refuse(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        _refuse(f"the last dimension of {name} must be contiguous")
    return t.data_ptr()


def _strides(t, shape):
    """Row and head stride; 0 where there is one row or head, whose stride says nothing."""
    row, head, _ = t.stride()
    return row if shape[0] > 1 else 0, head if shape[1] > 1 else 0


def _cache(k_cache, v_cache, page_table, device):
    """(packed gpt_paged_cache, sequences, kv heads, head size, type) of a cache."""
    shape, stride, table = k_cache.shape, k_cache.stride(), page_table.shape
    if len(shape) != 4 or len(table) != 2:
        _refuse("k_cache must be [pages, page size, heads, head size], page_table [sequences, pages]")
    dtype = k_cache.dtype
    code = _TYPES.get(dtype)
    if code is None:
        _refuse(f"k_cache must be float32 or bfloat16, got {dtype}")
    pages, page, heads, dim = shape
    if v_cache.stride() != stride:
        _refuse("k_cache and v_cache must have the same strides")
    return (_pack_cache(_ptr("k_cache", k_cache, dtype, shape, device), _ptr("v_cache", v_cache, dtype, shape, device),
                        _ptr("page_table", page_table, _I32, table, device), stride[0] if pages > 1 else 0,
                        stride[1] if page > 1 else 0, stride[2] if heads > 1 else 0, page_table.stride()[0],
                        pages, page, table[0], table[1], heads, dim, code), table[0], heads, dim, dtype)


def _empty(shape, dtype, like, stream):
    """Memory for ``stream``: the allocator hands it out again in that stream's order."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _stream(stream, device):
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def _check(rc):
    if rc:
        raise B.GptError(rc, B.load().gpt_last_error(None).decode())


def kv_append(k, v, k_cache, v_cache, page_table, positions, seq=None, q=None, rope_dims: int = 0,
              rope_base: float = 10000.0, q_out=None, status=None, stream=None):
    """gpt_kv_append: k, v [tokens, kv heads, head size] into the paged cache (k_cache, v_cache [pages, page
    size, kv heads, head size], page_table int32 [sequences, pages]) at ``positions`` (int32 [tokens]) of
    sequences ``seq`` (int32 [tokens]; negative: padding; None: token n is sequence n's), rotated by position
    over the first ``rope_dims`` elements of a head.

    With q [tokens, heads, head size] returns the rotated queries (``q_out``, which may be q, or a new
    tensor), else None."""
    lib = B.load()
    device = _device("k", k)
    cache, _, heads, dim, dtype = _cache(k_cache, v_cache, page_table, device)
    n = k.shape[0]
    kv = (n, heads, dim)
    pk, pv = _ptr("k", k, dtype, kv, device), _ptr("v", v, dtype, kv, device)
    pq = pqo = n_head = 0
    sq = sqo = (0, 0)
    if q is not None:
        if q.dim() != 3:
            _refuse("q must be [tokens, heads, head size]")
        n_head = q.shape[1]
        shape = (n, n_head, dim)
        pq = _ptr("q", q, dtype, shape, device)
        if q_out is None:
            q_out = _empty(shape, dtype, q, stream)
        pqo = _ptr("q_out", q_out, dtype, shape, device)
        sq, sqo = _strides(q, shape), _strides(q_out, shape)
    elif q_out is not None:
        _refuse("q_out goes with q")
    args = _pack_append(pq, pk, pv, pqo, *sq, *_strides(k, kv), *_strides(v, kv), *sqo,
                        _ptr("positions", positions, _I32, (n,), device),
                        0 if seq is None else _ptr("seq", seq, _I32, (n,), device),
                        0 if status is None else _ptr("status", status, _I32, (1,), device), rope_base, n, n_head, rope_dims)
    _check(lib.gpt_kv_append(cache, args, _stream(stream, device)))
    return q_out


def decode_attention(q, k_cache, v_cache, page_table, lens, scale: float | None = None, out=None, status=None,
                     stream=None):
    """gpt_decode_attention: attention of one new token of every sequence, q [sequences, heads, head size],
    over the first ``lens`` (int32 [sequences]) positions of its pages (cache as in kv_append).  ``scale``:
    1/sqrt(head size) unless given.

    Returns (out like q, lse float32 [sequences, heads])."""
    lib = B.load()
    device = _device("q", q)
    cache, n, _, dim, dtype = _cache(k_cache, v_cache, page_table, device)
    if q.dim() != 3:
        _refuse("q must be [sequences, heads, head size]")
    n_head = q.shape[1]
    shape = (n, n_head, dim)
    pq = _ptr("q", q, dtype, shape, device)
    if out is None:
        out = _empty(shape, dtype, q, stream)
    lse = _empty((n, n_head), _F32, q, stream)
    need = lib.gpt_decode_attention_workspace(cache, n_head)
    scratch = _empty((need,), torch.uint8, q, stream).data_ptr() if need else 0
    args = _pack_attention(pq, _ptr("out", out, dtype, shape, device), lse.data_ptr(),
                           _ptr("lens", lens, _I32, (n,), device), *_strides(q, shape), *_strides(out, shape), scratch, need,
                           0 if status is None else _ptr("status", status, _I32, (1,), device),
                           dim ** -0.5 if scale is None else scale, n_head)
    _check(lib.gpt_decode_attention(cache, args, _stream(stream, device)))
    return out, lse


def next_token(logits, history=None, history_lens=None, prompt_lens=None, repetition=None, presence=None,
               frequency=None, bias_ids=None, bias_values=None, allowed=None, out=None, status=None, stream=None):
    """gpt_next_token: logits [rows, vocab] (float32 or bfloat16) with the penalties of ``history`` (int32
    [rows, n]; ``history_lens``, ``prompt_lens`` int32 [rows]; ``repetition``, ``presence``, ``frequency``
    float32 [rows]), the biases ``bias_values`` (float32 [rows, m]) of tokens ``bias_ids`` (int32 [rows, m])
    and the grammar mask ``allowed`` (int32 [rows, ceil(vocab/32)], one bit per token) applied; every
    argument but logits may be None.

    Returns (token int32 [rows], out float32 [rows, vocab], lse float32 [rows]); ``out`` may be float32
    logits themselves."""
    lib = B.load()
    device = _device("logits", logits)
    shape = logits.shape
    if len(shape) != 2:
        _refuse("logits must be [rows, vocab]")
    rows, vocab = shape
    per_row = (rows,)
    code = _TYPES.get(logits.dtype)
    if code is None:
        _refuse(f"logits must be float32 or bfloat16, got {logits.dtype}")
    pz = _ptr("logits", logits, logits.dtype, shape, device)
    ph = phl = ppl = most = s_hist = 0
    if history is not None:
        if history.dim() != 2:
            _refuse("history must be [rows, tokens]")
        most = history.shape[1]
        ph, s_hist = _ptr("history", history, _I32, (rows, most), device), history.stride()[0]
        if history_lens is not None:
            phl = _ptr("history_lens", history_lens, _I32, per_row, device)
        if prompt_lens is not None:
            ppl = _ptr("prompt_lens", prompt_lens, _I32, per_row, device)
        if most == 0:  # a history of no columns has no memory
            ph = phl = ppl = 0
    elif history_lens is not None or prompt_lens is not None:
        _refuse("history_lens and prompt_lens go with history")
    pi = pb = n_bias = s_bias = 0
    if bias_ids is not None and bias_values is not None:
        if bias_ids.dim() != 2 or bias_ids.stride() != bias_values.stride():
            _refuse("bias_ids and bias_values must be [rows, entries] with the same strides")
        n_bias, s_bias = bias_ids.shape[1], bias_ids.stride()[0]
        pi = _ptr("bias_ids", bias_ids, _I32, (rows, n_bias), device)
        pb = _ptr("bias_values", bias_values, _F32, (rows, n_bias), device)
    elif bias_ids is not None or bias_values is not None:
        _refuse("bias_ids and bias_values go together")
    pa = s_mask = 0
    if allowed is not None:
        pa, s_mask = _ptr("allowed", allowed, _I32, (rows, (vocab + 31) // 32), device), allowed.stride()[0]
    if out is None:
        out = _empty(shape, _F32, logits, stream)
    token, lse = _empty(per_row, _I32, logits, stream), _empty(per_row, _F32, logits, stream)
    args = _pack_token(pz, _ptr("out", out, _F32, shape, device), token.data_ptr(), lse.data_ptr(), ph, phl, ppl,
                       0 if repetition is None else _ptr("repetition", repetition, _F32, per_row, device),
                       0 if presence is None else _ptr("presence", presence, _F32, per_row, device),
                       0 if frequency is None else _ptr("frequency", frequency, _F32, per_row, device), pi, pb, pa,
                       0 if status is None else _ptr("status", status, _I32, (1,), device),
                       logits.stride()[0], out.stride()[0], s_hist, s_bias, s_mask, rows, vocab, code, most, n_bias)
    _check(lib.gpt_next_token(args, _stream(stream, device)))
    return token, out, lse
