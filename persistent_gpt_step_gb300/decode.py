"""The operators of a batched decode step on torch CUDA tensors: gpt_kv_append, gpt_decode_attention and
gpt_next_token of the C ABI (also reached as ``binding.kv_append`` and so on).

Every tensor's device, type, shape and strides are checked before the call; a mismatch raises
GptError(INVALID_ARG).  Indices that live on the device are checked by the kernels and reported in
``status`` (int32 [1], STATUS_* bits of ``binding``, zeroed by the caller).  Calls run on ``stream`` (default:
the current stream) without synchronising; what they return belongs to that stream.  Inputs are not recorded on
it: with a stream other than their own, keep them (or call ``record_stream``) until the call has run.  They have
no gradients: a tensor that requires one is refused while gradients are recorded, and the versions of the tensors
that they write move as those of torch's in-place operations do.
The checks and the call itself are the ``_decode`` module (csrc/decode_py.cpp); if it is missing this module raises.
"""

from __future__ import annotations

import ctypes

import torch  # noqa: F401  (its libraries, which _decode needs)

from . import binding as B

try:
    from . import _decode as _C
except ImportError as e:
    raise RuntimeError("the _decode module is missing or does not fit this torch: build it with "
                       "`python -m persistent_gpt_step_gb300.build` (no fallback exists)") from e

_C.init(*(ctypes.cast(getattr(B.load(), f), ctypes.c_void_p).value
          for f in ("gpt_kv_append", "gpt_decode_attention", "gpt_decode_attention_workspace", "gpt_next_token",
                    "gpt_last_error")), B.GptError)


def kv_append(k, v, k_cache, v_cache, page_table, positions, seq=None, q=None, rope_dims: int = 0,
              rope_base: float = 10000.0, q_out=None, status=None, stream=None):
    """gpt_kv_append: k, v [tokens, kv heads, head size] into the paged cache (k_cache, v_cache [pages, page
    size, kv heads, head size], page_table int32 [sequences, pages]) at ``positions`` (int32 [tokens]) of
    sequences ``seq`` (int32 [tokens]; negative: padding; None: token n is sequence n's), rotated by position
    over the first ``rope_dims`` elements of a head.

    With q [tokens, heads, head size] returns the rotated queries (``q_out``, which may be q, or a new
    tensor, whose rows of padding and of bad indices hold nothing), else None."""
    return _C.kv_append(k, v, k_cache, v_cache, page_table, positions, seq, q, rope_dims, rope_base, q_out, status, stream)


def decode_attention(q, k_cache, v_cache, page_table, lens, scale: float | None = None, out=None, status=None,
                     stream=None):
    """gpt_decode_attention: attention of one new token of every sequence, q [sequences, heads, head size],
    over the first ``lens`` (int32 [sequences]) positions of its pages (cache as in kv_append).  ``scale``:
    1/sqrt(head size) unless given.  The kernel is chosen by the table's width: where all sequences are known to be
    short, ``page_table[:, :n]`` is faster than the whole table (a sequence of 513 keys 6.8 us and, in a table of 65,536 positions, 9.8).

    Returns (out like q, lse float32 [sequences, heads])."""
    return _C.decode_attention(q, k_cache, v_cache, page_table, lens, scale, out, status, stream)


def next_token(logits, history=None, history_lens=None, prompt_lens=None, repetition=None, presence=None,
               frequency=None, bias_ids=None, bias_values=None, allowed=None, out=None, status=None, stream=None):
    """gpt_next_token: logits [rows, vocab] (float32 or bfloat16) with the penalties of ``history`` (int32
    [rows, n]; ``history_lens``, ``prompt_lens`` int32 [rows]; ``repetition``, ``presence``, ``frequency``
    float32 [rows]), the biases ``bias_values`` (float32 [rows, m]) of tokens ``bias_ids`` (int32 [rows, m])
    and the grammar mask ``allowed`` (int32 [rows, ceil(vocab/32)], one bit per token) applied; every
    argument but logits may be None.

    Returns (token int32 [rows], out float32 [rows, vocab], lse float32 [rows]); ``out`` may be float32
    logits themselves."""
    return _C.next_token(logits, history, history_lens, prompt_lens, repetition, presence, frequency, bias_ids, bias_values,
                         allowed, out, status, stream)
