"""Binding of include/pq2_attention.h: the paged INT8 key-value cache with the
rotary embedding, attention of new tokens over its pages, and attention over
packed prompts.

Like the rest of the package these functions marshal arguments only (in
``_marshal``, built from csrc/marshal.cpp: with up to eleven tensors a call, checking
them in Python took longer than the kernels run).  Tensors
of heads are [rows][heads][head_dim] with unit stride inside a head (columns of
a projection's output among them); a cache is a contiguous uint8 tensor
[pages][pq2_kv_page_bytes(...)]; index tensors are int32.  All tensors of a call
are on one device; the work goes to that device's current torch stream (or
``stream``), whichever device is current.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

from . import _check, lib
from .block import _raw_stream

ATTENTION_EXPORTED = (
    "pq2_kv_page_bytes",
    "pq2_kv_write",
    "pq2_kv_read",
    "pq2_attention_paged_workspace",
    "pq2_attention_paged",
    "pq2_attention_prompt",
)


class _NoMarshal:
    """In place of ``_marshal`` where it does not load: the rest of the package needs no more than libpq2.so, so only
    the attention calls raise."""

    def __init__(self, reason):
        self._reason = reason

    def __getattr__(self, name):
        raise ImportError(f"{os.path.join(os.path.dirname(__file__), '_marshal.so')}: {self._reason}; the attention "
                          "operators' binding must be built with the installed torch (python gemm_int8_act_amd/build.py); "
                          "there is no fallback path")


def _load_marshal():
    try:
        from . import _marshal
    except ImportError as e:
        return _NoMarshal(str(e))
    # It reads torch's tensors in place, so it holds for the torch that it was compiled against.
    if _marshal.torch_version != torch.__version__:
        return _NoMarshal(f"built for torch {_marshal.torch_version}, not {torch.__version__}")
    return _marshal


_marshal = _load_marshal()


def _bind():
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    for name, args in {
        "pq2_kv_page_bytes": [i64, i64, i64],
        "pq2_attention_paged_workspace": [i64] * 6 + [ctypes.POINTER(i64)] * 2,
        "pq2_kv_write": [ctypes.c_char_p, p],
        "pq2_kv_read": [ctypes.c_char_p, p],
        "pq2_attention_paged": [ctypes.c_char_p, p],
        "pq2_attention_prompt": [ctypes.c_char_p, p],
    }.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = i64 if name == "pq2_kv_page_bytes" else i32


_bind()
_write, _read, _paged, _prompt = lib.pq2_kv_write, lib.pq2_kv_read, lib.pq2_attention_paged, lib.pq2_attention_prompt


def _call(fn, name, stream, args, dev):
    if stream is None:
        s = torch.cuda.current_stream(dev).cuda_stream if _raw_stream is None else _raw_stream(dev)
    else:
        s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if dev == torch.cuda.current_device():
        status = fn(args, s)
    else:
        with torch.cuda.device(dev):
            status = fn(args, s)
    if status:
        _check(status, name)


@functools.lru_cache(maxsize=256)
def pq2_kv_page_bytes(page_tokens: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of one page of the cache (ValueError on a bad size)."""
    size = lib.pq2_kv_page_bytes(page_tokens, kv_heads, head_dim)
    if size < 0:
        raise ValueError(f"pq2_kv_page_bytes: unsupported page_tokens={page_tokens} kv_heads={kv_heads} "
                         f"head_dim={head_dim}")
    return size


@functools.lru_cache(maxsize=256)
def pq2_attention_paged_workspace(seqs: int, max_new: int, heads: int, kv_heads: int, head_dim: int, max_len: int):
    """(floats of `partials`, int32 words of `counters`) of pq2_attention_paged with these sizes."""
    floats, words = ctypes.c_int64(), ctypes.c_int64()
    _check(lib.pq2_attention_paged_workspace(seqs, max_new, heads, kv_heads, head_dim, max_len, ctypes.byref(floats),
                                             ctypes.byref(words)), "pq2_attention_paged_workspace")
    return floats.value, words.value


def pq2_kv_write(k, v, cache, slots, page_tokens: int = 16, *, q=None, q_out=None, k_out=None, v_out=None, cos=None,
                 sin=None, positions=None, interleaved: bool = False, stream=None) -> None:
    """Rotary embedding, then k and v as INT8 codes into the cache, in one launch.

    k, v [m][kv_heads][head_dim] and q [m][heads][head_dim] of one dtype (bf16/f16/f32), e.g. the three parts of a QKV
    projection's output.  cos, sin: float32 [positions][rot_dim / 2] tables (None: no rotation), positions int32 [m];
    interleaved: pairs are neighbouring elements instead of the halves of rot_dim.  cache: uint8 [pages][page bytes], or
    None for the rotation alone; slots int32 [m]: page * page_tokens + offset of each token (outside the cache, e.g.
    -1: not written).  q_out: rotated q (with q); k_out and v_out: rotated k, and v, for a prompt's own attention; one
    dtype of all three; q_out and k_out may be q and k themselves."""
    _call(_write, "pq2_kv_write", stream, *_marshal.kv_write(k, v, cache, slots, page_tokens, q, q_out, k_out, v_out, cos, sin,
                                                             positions, interleaved))


def pq2_kv_read(cache, table, starts, page_tokens: int, k_out, v_out, stream=None) -> None:
    """Tokens 0 .. starts[s + 1] - starts[s] - 1 of each sequence out of the cache, into rows starts[s] .. of k_out and v_out
    [rows][kv_heads][head_dim] (bf16/f16/f32).  table int32 [sequences][pages]; starts int32 [sequences + 1] from 0 on.
    Rows behind the last sequence are left as they were; rows of pages outside the cache or the table are zero."""
    _call(_read, "pq2_kv_read", stream, *_marshal.kv_read(cache, table, starts, page_tokens, k_out, v_out))


def pq2_attention_paged(q, cache, table, lens, page_tokens: int, out, partials=None, counters=None, *, starts=None,
                        max_new: int = 1, max_len=None, scale=None, window: int = 0, stream=None) -> None:
    """Attention of new tokens over the paged cache: q and out [rows][heads][head_dim], bf16 or f16.

    lens int32 [sequences]: tokens of each in the cache, the new ones (already written) among them; table int32
    [sequences][pages].  starts int32 [sequences + 1]: rows of each sequence's new tokens; None: one each.
    max_new goes with starts: the most new tokens of a sequence (the default, 1, too: rows behind a sequence's first max_new are left
    as they were).
    max_len: the longest length expected (None: what the table holds); with seqs, max_new and the heads it gives the
    workspace's sizes, pq2_attention_paged_workspace: partials float32, counters int32, zero before the first call.  scale: 1 /
    sqrt(head_dim) if None.  window: keys that a token sees, itself among them (0: all)."""
    _call(_paged, "pq2_attention_paged", stream, *_marshal.attention_paged(q, cache, table, lens, page_tokens, out, partials,
                                                                           counters, starts, max_new, max_len, scale, window))


def pq2_attention_prompt(q, k, v, out, starts_q, starts_k, *, causal: bool = True, scale=None, window: int = 0,
                         stream=None) -> None:
    """Attention over packed prompts: q and out [rows][heads][head_dim], k and v [key rows][kv_heads][head_dim], bf16 or
    f16.  starts_q, starts_k int32 [sequences + 1] from 0 on: rows of each sequence (more keys than queries behind a prefix:
    the last query is the last key's token).  scale: 1 / sqrt(head_dim) if None.  window (causal only): keys that a
    token sees, itself among them (0: all).  Rows that see no key are zero; rows behind the last sequence are left as
    they were."""
    _call(_prompt, "pq2_attention_prompt", stream, *_marshal.attention_prompt(q, k, v, out, starts_q, starts_k, causal, scale,
                                                                              window))
