"""Binding of include/pq2_attention.h: the paged INT8 key-value cache with the
rotary embedding, attention of new tokens over its pages, and attention over
packed prompts.

Like the rest of the package these functions marshal arguments only.  Tensors
of heads are [rows][heads][head_dim] with unit stride inside a head (columns of
a projection's output among them); a cache is a contiguous uint8 tensor
[pages][pq2_kv_page_bytes(...)]; index tensors are int32.  All tensors of a call
are on one device; the work goes to that device's current torch stream (or
``stream``), whichever device is current.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import PQ2_BF16, PQ2_F16, PQ2_F32, _check, lib
from .block import _raw_stream

ATTENTION_EXPORTED = (
    "pq2_kv_page_bytes",
    "pq2_kv_write",
    "pq2_kv_read",
    "pq2_attention_paged_workspace",
    "pq2_attention_paged",
    "pq2_attention_prompt",
)

# The argument structures of include/pq2_attention.h: the fields in order, with
# their native struct codes.
WRITE_FIELDS = (
    ("q", "P"), ("k", "P"), ("v", "P"),
    ("q_stride", "q"), ("q_head", "q"), ("k_stride", "q"), ("k_head", "q"), ("v_stride", "q"), ("v_head", "q"),
    ("q_out", "P"), ("k_out", "P"), ("v_out", "P"),
    ("qo_stride", "q"), ("qo_head", "q"), ("ko_stride", "q"), ("ko_head", "q"), ("vo_stride", "q"), ("vo_head", "q"),
    ("cos", "P"), ("sin", "P"), ("positions", "P"), ("slots", "P"), ("cache", "P"),
    ("m", "q"), ("heads", "q"), ("kv_heads", "q"), ("head_dim", "q"), ("rot_dim", "q"), ("table_rows", "q"),
    ("pages", "q"), ("page_tokens", "q"),
    ("in_dtype", "i"), ("out_dtype", "i"), ("interleaved", "i"),
)
READ_FIELDS = (
    ("cache", "P"), ("table", "P"), ("starts", "P"), ("k_out", "P"), ("v_out", "P"),
    ("ko_stride", "q"), ("ko_head", "q"), ("vo_stride", "q"), ("vo_head", "q"),
    ("rows", "q"), ("seqs", "q"), ("table_stride", "q"), ("table_pages", "q"), ("kv_heads", "q"), ("head_dim", "q"),
    ("pages", "q"), ("page_tokens", "q"),
    ("out_dtype", "i"),
)
PAGED_FIELDS = (
    ("q", "P"), ("out", "P"), ("q_stride", "q"), ("q_head", "q"), ("out_stride", "q"), ("out_head", "q"),
    ("cache", "P"), ("table", "P"), ("lens", "P"), ("starts", "P"), ("partials", "P"), ("counters", "P"),
    ("rows", "q"), ("seqs", "q"), ("table_stride", "q"), ("table_pages", "q"), ("heads", "q"), ("kv_heads", "q"),
    ("head_dim", "q"), ("pages", "q"), ("page_tokens", "q"), ("max_new", "q"), ("max_len", "q"), ("window", "q"),
    ("scale", "f"), ("dtype", "i"),
)
PROMPT_FIELDS = (
    ("q", "P"), ("k", "P"), ("v", "P"), ("out", "P"),
    ("q_stride", "q"), ("q_head", "q"), ("k_stride", "q"), ("k_head", "q"), ("v_stride", "q"), ("v_head", "q"),
    ("out_stride", "q"), ("out_head", "q"),
    ("starts_q", "P"), ("starts_k", "P"),
    ("rows_q", "q"), ("rows_k", "q"), ("seqs", "q"), ("heads", "q"), ("kv_heads", "q"), ("head_dim", "q"),
    ("window", "q"), ("scale", "f"), ("dtype", "i"), ("causal", "i"),
)


def _packer(fields):
    # The structure ends at a multiple of its widest member, as in C.
    return struct.Struct("@" + "".join(code for _, code in fields) + "0q")


_WRITE, _READ, _PAGED, _PROMPT = (_packer(f) for f in (WRITE_FIELDS, READ_FIELDS, PAGED_FIELDS, PROMPT_FIELDS))

_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8
_DTYPE = {torch.bfloat16: PQ2_BF16, torch.float16: PQ2_F16, torch.float32: PQ2_F32}
_HALF = {torch.bfloat16: PQ2_BF16, torch.float16: PQ2_F16}


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


def _device(first, *rest):
    dev = first.get_device()
    if dev < 0:
        raise ValueError("device tensors expected")
    for t in rest:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors of a call must be on one device")
    return dev


def _call(fn, name, dev, stream, args):
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


# As in block.py the checks run on every call of a decode step and are written
# for few attribute reads.
def _heads(t, name, rows=None, heads=None, dim=None):
    """(pointer, row stride, head stride, rows, heads, head_dim) of a tensor of heads; strides of single rows and heads are
    those of a contiguous tensor, whatever the tensor says."""
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [rows][heads][head_dim]")
    n, h, d = shape
    st, sh, unit = t.stride()
    if unit != 1 or (rows is not None and n != rows) or (heads is not None and h != heads) or \
            (dim is not None and d != dim):
        raise ValueError(f"{name} must be [rows][heads][head_dim] with unit stride, of the call's sizes")
    if h == 1:
        sh = d
    if n == 1:
        st = h * d
    return t.data_ptr(), st, sh, n, h, d


def _index(t, name, n):
    if t.dtype is not _I32 or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} elements")
    return t.data_ptr()


def _pages(cache, page_tokens, kv_heads, head_dim):
    if cache.dtype is not _U8 or cache.dim() != 2 or not cache.is_contiguous() or \
            cache.shape[1] != pq2_kv_page_bytes(page_tokens, kv_heads, head_dim):
        raise ValueError("cache must be a contiguous uint8 tensor [pages][pq2_kv_page_bytes(...)]")
    return cache.data_ptr(), cache.shape[0]


def _table(table, seqs):
    if table.dtype is not _I32 or table.dim() != 2 or table.shape[0] != seqs or table.stride(1) != 1 and table.shape[1] > 1:
        raise ValueError("table must be int32 [sequences][pages] with unit column stride")
    width = table.shape[1]
    return table.data_ptr(), table.stride(0) if seqs > 1 else width, width


def pq2_kv_write(k, v, cache, slots, page_tokens: int = 16, *, q=None, q_out=None, k_out=None, v_out=None, cos=None,
                 sin=None, positions=None, interleaved: bool = False, stream=None) -> None:
    """Rotary embedding, then k and v as INT8 codes into the cache, in one launch.

    k, v [m][kv_heads][head_dim] and q [m][heads][head_dim] of one dtype (bf16/f16/f32), e.g. the three parts of a QKV
    projection's output.  cos, sin: float32 [positions][rot_dim / 2] tables (None: no rotation), positions int32 [m];
    interleaved: pairs are neighbouring elements instead of the halves of rot_dim.  cache: uint8 [pages][page bytes], or
    None for the rotation alone; slots int32 [m]: page * page_tokens + offset of each token (outside the cache, e.g.
    -1: not written).  q_out: rotated q (with q); k_out and v_out: rotated k, and v, for a prompt's own attention; one
    dtype of all three; q_out and k_out may be q and k themselves."""
    kp, kst, kh, m, kv, d = _heads(k, "k")
    vp, vst, vh, _, _, _ = _heads(v, "v", m, kv, d)
    dt = k.dtype
    code = _DTYPE.get(dt)
    if code is None or v.dtype is not dt or (q is not None and q.dtype is not dt):
        raise ValueError("q, k and v must have one dtype, bf16, f16 or f32")
    qp = qst = qh = qop = qos = qoh = kop = kos = koh = vop = vos = voh = 0
    heads = kv
    od = None
    if q is not None:
        qp, qst, qh, _, heads, _ = _heads(q, "q", m, None, d)
    if q_out is not None:
        qop, qos, qoh, _, _, _ = _heads(q_out, "q_out", m, heads, d)
        od = q_out.dtype
    if k_out is not None:
        kop, kos, koh, _, _, _ = _heads(k_out, "k_out", m, kv, d)
        if od is not None and k_out.dtype is not od:
            raise ValueError("q_out, k_out and v_out must have one dtype")
        od = k_out.dtype
    if v_out is not None:
        vop, vos, voh, _, _, _ = _heads(v_out, "v_out", m, kv, d)
        if od is not None and v_out.dtype is not od:
            raise ValueError("q_out, k_out and v_out must have one dtype")
        od = v_out.dtype
    out_code = code if od is None else _DTYPE.get(od)
    if out_code is None:
        raise ValueError(f"unsupported dtype {od}")
    cp = sp = pp = rot = rows = 0
    if cos is not None or sin is not None:
        if cos is None or sin is None or positions is None or cos.dim() != 2 or cos.shape != sin.shape or \
                cos.dtype is not _F32 or sin.dtype is not _F32 or not cos.is_contiguous() or not sin.is_contiguous():
            raise ValueError("cos and sin must be contiguous float32 [positions][rot_dim / 2] tables, with positions")
        rows, rot = cos.shape
        rot *= 2
        cp, sp, pp = cos.data_ptr(), sin.data_ptr(), _index(positions, "positions", m)
    else:
        positions = None
    bp = pages = lp = 0
    if cache is not None:
        bp, pages = _pages(cache, page_tokens, kv, d)
        lp = _index(slots, "slots", m)
    else:
        slots = None
    args = _WRITE.pack(qp, kp, vp, qst, qh, kst, kh, vst, vh, qop, kop, vop, qos, qoh, kos, koh, vos, voh, cp, sp, pp, lp,
                       bp, m, heads, kv, d, rot, rows, pages, page_tokens, code, out_code, 1 if interleaved else 0)
    _call(lib.pq2_kv_write, "pq2_kv_write",
          _device(k, v, cache, slots, q, q_out, k_out, v_out, cos, sin, positions), stream, args)


def pq2_kv_read(cache, table, starts, page_tokens: int, k_out, v_out, stream=None) -> None:
    """Tokens 0 .. starts[s + 1] - starts[s] - 1 of each sequence out of the cache, into rows starts[s] .. of k_out and v_out
    [rows][kv_heads][head_dim] (bf16/f16/f32).  table int32 [sequences][pages]; starts int32 [sequences + 1] from 0 on.
    Rows behind the last sequence are left as they were; rows of pages outside the cache or the table are zero."""
    kp, kst, kh, rows, kv, d = _heads(k_out, "k_out")
    vp, vst, vh, _, _, _ = _heads(v_out, "v_out", rows, kv, d)
    code = _DTYPE.get(k_out.dtype)
    if code is None or v_out.dtype is not k_out.dtype:
        raise ValueError("k_out and v_out must have one dtype, bf16, f16 or f32")
    seqs = table.shape[0]
    tp, tst, width = _table(table, seqs)
    sp = _index(starts, "starts", seqs + 1)
    cp, pages = _pages(cache, page_tokens, kv, d)
    args = _READ.pack(cp, tp, sp, kp, vp, kst, kh, vst, vh, rows, seqs, tst, width, kv, d, pages, page_tokens, code)
    _call(lib.pq2_kv_read, "pq2_kv_read", _device(k_out, v_out, cache, table, starts), stream, args)


def pq2_attention_paged(q, cache, table, lens, page_tokens: int, out, partials=None, counters=None, *, starts=None,
                        max_new: int = 1, max_len=None, scale=None, window: int = 0, stream=None) -> None:
    """Attention of new tokens over the paged cache: q and out [rows][heads][head_dim], bf16 or f16.

    lens int32 [sequences]: tokens of each in the cache, the new ones (already written) among them; table int32
    [sequences][pages].  starts int32 [sequences + 1]: rows of each sequence's new tokens, at most max_new each; None: one each.
    max_len: the longest length expected (None: what the table holds); with seqs, max_new and the heads it gives the
    workspace's sizes, pq2_attention_paged_workspace: partials float32, counters int32, zero before the first call.  scale: 1 /
    sqrt(head_dim) if None.  window: keys that a token sees, itself among them (0: all)."""
    qp, qst, qh, rows, heads, d = _heads(q, "q")
    op, ost, oh, _, _, _ = _heads(out, "out", rows, heads, d)
    code = _HALF.get(q.dtype)
    if code is None or out.dtype is not q.dtype:
        raise ValueError("q and out must have one dtype, bf16 or f16")
    seqs = lens.shape[0]
    lp = _index(lens, "lens", seqs)
    tp, tst, width = _table(table, seqs)
    kv = cache.shape[1] // pq2_kv_page_bytes(page_tokens, 1, d)
    cp, pages = _pages(cache, page_tokens, kv, d)
    sp = 0
    if starts is not None:
        sp = _index(starts, "starts", seqs + 1)
    elif rows != seqs:
        raise ValueError("without starts, q has one row a sequence")
    if max_len is None:
        max_len = width * page_tokens
    floats, words = pq2_attention_paged_workspace(seqs, max_new, heads, kv, d, max_len)
    wp = np = 0
    if words:
        if partials is None or counters is None or partials.dtype is not _F32 or counters.dtype is not _I32 or \
                partials.numel() < floats or counters.numel() < words or not partials.is_contiguous() or \
                not counters.is_contiguous():
            raise ValueError("partials float32 and counters int32 of pq2_attention_paged_workspace(...) expected")
        wp, np = partials.data_ptr(), counters.data_ptr()
    else:
        partials = counters = None
    args = _PAGED.pack(qp, op, qst, qh, ost, oh, cp, tp, lp, sp, wp, np, rows, seqs, tst, width, heads, kv, d, pages,
                       page_tokens, max_new, max_len, window, d ** -0.5 if scale is None else scale, code)
    _call(lib.pq2_attention_paged, "pq2_attention_paged",
          _device(q, out, cache, table, lens, starts, partials, counters), stream, args)


def pq2_attention_prompt(q, k, v, out, starts_q, starts_k, *, causal: bool = True, scale=None, window: int = 0,
                         stream=None) -> None:
    """Attention over packed prompts: q and out [rows][heads][head_dim], k and v [key rows][kv_heads][head_dim], bf16 or
    f16.  starts_q, starts_k int32 [sequences + 1] from 0 on: rows of each sequence (more keys than queries behind a prefix:
    the last query is the last key's token).  scale: 1 / sqrt(head_dim) if None.  window (causal only): keys that a
    token sees, itself among them (0: all).  Rows that see no key are zero; rows behind the last sequence are left as
    they were."""
    qp, qst, qh, rows_q, heads, d = _heads(q, "q")
    op, ost, oh, _, _, _ = _heads(out, "out", rows_q, heads, d)
    kp, kst, kh, rows_k, kv, _ = _heads(k, "k", None, None, d)
    vp, vst, vh, _, _, _ = _heads(v, "v", rows_k, kv, d)
    dt = q.dtype
    code = _HALF.get(dt)
    if code is None or out.dtype is not dt or k.dtype is not dt or v.dtype is not dt:
        raise ValueError("q, k, v and out must have one dtype, bf16 or f16")
    seqs = starts_q.shape[0] - 1
    a, b = _index(starts_q, "starts_q", seqs + 1), _index(starts_k, "starts_k", seqs + 1)
    args = _PROMPT.pack(qp, kp, vp, op, qst, qh, kst, kh, vst, vh, ost, oh, a, b, rows_q, rows_k, seqs, heads, kv, d, window,
                        d ** -0.5 if scale is None else scale, code, 1 if causal else 0)
    _call(lib.pq2_attention_prompt, "pq2_attention_prompt", _device(q, k, v, out, starts_q, starts_k), stream, args)
