"""Binding of include/pq2_block.h: products with 4-bit weights, the gated
feed-forward product, and the norms around a block with the INT8 quantiser.

Like the rest of the package these functions marshal arguments only.  All
tensors of a call are on one device; the work goes to that device's current
torch stream (or ``stream``), whichever device is current.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import PQ2_BF16, PQ2_F16, PQ2_F32, _check, lib, pq2_tiles_bytes

_tiles_bytes = functools.lru_cache(maxsize=256)(pq2_tiles_bytes)

ACT_SILU, ACT_GELU_TANH = 0, 1

BLOCK_EXPORTED = (
    "pq2_w4_tiles_bytes",
    "pq2_prepare_w4_tiles",
    "pq2_matmul_w4",
    "pq2_linear_w4",
    "pq2_gated_matmul_tiles",
    "pq2_gated_matmul_w4",
    "pq2_gated_linear_tiles",
    "pq2_gated_linear_w4",
    "pq2_block_norm",
)

_DTYPE = {torch.bfloat16: PQ2_BF16, torch.float16: PQ2_F16, torch.float32: PQ2_F32}


# pq2_block_norm_args of include/pq2_block.h: the fields in order, with their
# native struct codes.
NORM_FIELDS = (
    ("r", "P"), ("r_stride", "q"),
    ("block", "P"), ("block_stride", "q"),
    ("post_w", "P"),
    ("gate", "P"), ("gate_stride", "q"),
    ("w", "P"),
    ("r_out", "P"), ("r_out_stride", "q"),
    ("x_out", "P"), ("x_out_stride", "q"),
    ("q", "P"), ("xs", "P"),
    ("m", "q"), ("k", "q"), ("agroup", "q"),
    ("eps", "d"), ("alpha", "f"),
    ("r_dtype", "i"), ("block_dtype", "i"), ("w_dtype", "i"), ("x_dtype", "i"), ("unit_offset", "i"),
)
_NORM = struct.Struct("@" + "".join(code for _, code in NORM_FIELDS))


def _bind():
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    product = [p, p, p, i64, i64, i64]
    for name, args in {
        "pq2_w4_tiles_bytes": [i64, i64, i64],
        "pq2_prepare_w4_tiles": [p, i64, p, i64, i64, i64, i64, p, p],
        "pq2_matmul_w4": product + [i64, p, p],
        "pq2_linear_w4": [p, i32, i64, p, i64, i64, i64, i64, p, p, p, p],
        "pq2_gated_matmul_tiles": [p, p, p, p, i64, i64, i64, i32, p, i32, p],
        "pq2_gated_matmul_w4": [p, p, p, p, i64, i64, i64, i64, i32, p, i32, p],
        "pq2_gated_linear_tiles": [p, i32, i64, p, p, i64, i64, i64, i32, p, i32, p, p, p],
        "pq2_gated_linear_w4": [p, i32, i64, p, p, i64, i64, i64, i64, i32, p, i32, p, p, p],
        "pq2_block_norm": [ctypes.c_char_p, p],
    }.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = i64 if name == "pq2_w4_tiles_bytes" else i32


_bind()


def _dtype(t, name):
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: unsupported dtype {t.dtype}")
    return code


def _device(first, *rest):
    """Index of the one GPU that holds the call's tensors."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError("device tensors expected")
    for t in rest:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors of a call must be on one device")
    return dev


def _call(name, dev, stream, *args):
    """Calls the entry point on device ``dev``: its current stream unless one is given."""
    if stream is None:
        s = torch.cuda.current_stream(dev).cuda_stream if _raw_stream is None else _raw_stream(dev)
    else:
        s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    fn = _FN[name]
    if dev == torch.cuda.current_device():
        status = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, s)
    if status:
        _check(status, name)


# The current stream's handle without a Stream object around it (a call's
# host time is near the decode kernels' own).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_FN = {name: getattr(lib, name) for name in BLOCK_EXPORTED}


@functools.lru_cache(maxsize=256)
def pq2_w4_tiles_bytes(n: int, k: int, wgroup: int) -> int:
    """Bytes of the w4 tile layout of an n x k weight matrix (ValueError on a bad shape or group)."""
    size = lib.pq2_w4_tiles_bytes(n, k, wgroup)
    if size < 0:
        raise ValueError(f"pq2_w4_tiles_bytes: unsupported shape n={n} k={k} wgroup={wgroup}")
    return size


def pq2_prepare_w4_tiles(codes, scales, wgroup: int, tiles, stream=None) -> None:
    """codes: uint8 [n][>= k/2], two 4-bit codes a byte (the even weight in the low half, weight = code - 8);
    scales: float16 [n][k/wgroup]; both with unit column stride.  tiles: contiguous uint8 of
    pq2_w4_tiles_bytes(n, k, wgroup) bytes.  n and k come from scales."""
    if codes.dtype != torch.uint8 or scales.dtype != torch.float16 or tiles.dtype != torch.uint8:
        raise ValueError("codes uint8, scales float16, tiles uint8 expected")
    if codes.dim() != 2 or scales.dim() != 2 or codes.stride(1) != 1 or scales.stride(1) != 1:
        raise ValueError("codes and scales must be 2-D with unit column stride")
    n, k = scales.shape[0], scales.shape[1] * wgroup
    if codes.shape[0] != n or codes.shape[1] < k // 2:
        raise ValueError("shape mismatch between codes and scales")
    if not tiles.is_contiguous() or tiles.numel() < pq2_w4_tiles_bytes(n, k, wgroup):
        raise ValueError("tiles must be a contiguous uint8 tensor of pq2_w4_tiles_bytes(n, k, wgroup) bytes")
    _call("pq2_prepare_w4_tiles", _device(codes, scales, tiles), stream, codes.data_ptr(),
          _row_stride(codes), scales.data_ptr(), _row_stride(scales), n, k, wgroup, tiles.data_ptr())


# The checks below run on every call of a decode step and are written for few
# attribute reads (a tensor attribute costs about 0.1 us of host time).
_F32, _I8, _U8 = torch.float32, torch.int8, torch.uint8
_Y = (_F32,)
_H = tuple(_DTYPE)


def _row_stride(t):
    """Row stride in elements; a single row's is its length, whatever the tensor says."""
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _weights(tiles, need):
    if tiles.dtype is not _U8 or tiles.numel() < need or not tiles.is_contiguous():
        raise ValueError("weights: contiguous uint8 tensor of the prepared layout's size expected")
    return tiles.data_ptr()


def _codes(q, xs, m):
    if q.dtype is not _I8 or xs.dtype is not _F32 or not q.is_contiguous() or not xs.is_contiguous():
        raise ValueError("q contiguous int8 and xs contiguous float32 expected")
    rows, k = q.shape
    if rows != m or xs.numel() * 128 != m * k:
        raise ValueError("shape mismatch: q [m][k], xs [m][k/128] expected")
    return k


def _out(t, name, dtypes):
    if t.dtype not in dtypes or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous 2-D tensor of {', '.join(str(d) for d in dtypes)} expected")
    m, n = t.shape
    return m, n


def _x(x, m, k):
    rows, width = x.shape
    stride, unit = x.stride()
    if unit != 1 or rows != m or width < k:
        raise ValueError("x must be [m][>= k] with unit column stride")
    return x.data_ptr(), _dtype(x, "x"), stride if m > 1 else max(stride, width)


def pq2_matmul_w4(q, xs, tiles, y, wgroup: int, stream=None) -> None:
    """y [m][n] (float32) = 4-bit weights x INT8 activations, any m >= 1; q int8 [m][k] and xs float32 [m][k/128]
    from pq2_quantize_act_i8 or pq2_block_norm."""
    m, n = _out(y, "y", _Y)
    k = _codes(q, xs, m)
    w = _weights(tiles, pq2_w4_tiles_bytes(n, k, wgroup))
    _call("pq2_matmul_w4", _device(q, xs, tiles, y), stream, q.data_ptr(), xs.data_ptr(), w, m, n, k, wgroup,
          y.data_ptr())


def pq2_linear_w4(x, tiles, y, wgroup: int, q_work, xs_work, stream=None) -> None:
    """The complete call: x [m][>= k] bf16/f16/f32 quantised into q_work / xs_work (scratch, int8 [m][k] and float32
    [m][k/128]), then pq2_matmul_w4."""
    m, n = _out(y, "y", _Y)
    k = _codes(q_work, xs_work, m)
    w = _weights(tiles, pq2_w4_tiles_bytes(n, k, wgroup))
    _call("pq2_linear_w4", _device(x, tiles, y, q_work, xs_work), stream, *_x(x, m, k), w, m, n, k, wgroup,
          y.data_ptr(), q_work.data_ptr(), xs_work.data_ptr())


def pq2_gated_matmul_tiles(q, xs, gate, up, h, act: int = ACT_SILU, stream=None) -> None:
    """h [m][n] (bf16/f16/f32) = act(gate product) * up product in one kernel; gate and up are ternary tile layouts of
    one shape, q / xs as pq2_matmul_w4."""
    m, n = _out(h, "h", _H)
    k = _codes(q, xs, m)
    need = _tiles_bytes(n, k)
    _call("pq2_gated_matmul_tiles", _device(q, xs, gate, up, h), stream, q.data_ptr(), xs.data_ptr(),
          _weights(gate, need), _weights(up, need), m, n, k, act, h.data_ptr(), _DTYPE[h.dtype])


def pq2_gated_matmul_w4(q, xs, gate, up, h, wgroup: int, act: int = ACT_SILU, stream=None) -> None:
    """pq2_gated_matmul_tiles with 4-bit weights in the w4 tile layout."""
    m, n = _out(h, "h", _H)
    k = _codes(q, xs, m)
    need = pq2_w4_tiles_bytes(n, k, wgroup)
    _call("pq2_gated_matmul_w4", _device(q, xs, gate, up, h), stream, q.data_ptr(), xs.data_ptr(),
          _weights(gate, need), _weights(up, need), m, n, k, wgroup, act, h.data_ptr(), _DTYPE[h.dtype])


def pq2_gated_linear_tiles(x, gate, up, h, q_work, xs_work, act: int = ACT_SILU, stream=None) -> None:
    """The complete call of pq2_gated_matmul_tiles: x quantised into the scratch first."""
    m, n = _out(h, "h", _H)
    k = _codes(q_work, xs_work, m)
    need = _tiles_bytes(n, k)
    _call("pq2_gated_linear_tiles", _device(x, gate, up, h, q_work, xs_work), stream, *_x(x, m, k),
          _weights(gate, need), _weights(up, need), m, n, k, act, h.data_ptr(), _DTYPE[h.dtype], q_work.data_ptr(),
          xs_work.data_ptr())


def pq2_gated_linear_w4(x, gate, up, h, wgroup: int, q_work, xs_work, act: int = ACT_SILU, stream=None) -> None:
    """The complete call of pq2_gated_matmul_w4: x quantised into the scratch first."""
    m, n = _out(h, "h", _H)
    k = _codes(q_work, xs_work, m)
    need = pq2_w4_tiles_bytes(n, k, wgroup)
    _call("pq2_gated_linear_w4", _device(x, gate, up, h, q_work, xs_work), stream, *_x(x, m, k),
          _weights(gate, need), _weights(up, need), m, n, k, wgroup, act, h.data_ptr(), _DTYPE[h.dtype],
          q_work.data_ptr(), xs_work.data_ptr())


def _rows(t, name, shape):
    st = t.stride()
    if t.shape != shape or st[1] != 1:
        raise ValueError(f"{name} must be [m][k] with unit column stride")
    return t.data_ptr(), st[0] if shape[0] > 1 else max(st[0], shape[1])


def _vector(t, name, k, dtype):
    if t.shape != (k,) or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [k] tensor of the norm weights' dtype")
    return t.data_ptr()


def pq2_block_norm(r, w, eps: float, *, block=None, post_w=None, gate=None, alpha: float = 1.0,
                   unit_offset: bool = False, r_out=None, x_out=None, x_dtype=None, q=None, xs=None,
                   agroup: int = 128, stream=None) -> None:
    """Between two blocks, one launch: r' = r + alpha * gate * norm(block), x = norm(r'), codes of x.

    r [m][k]; block [m][k] (the block's output) or None; post_w [k]: weights of the norm after the block, or None for
    none; gate [k] or [m][k]; w [k]: weights of the norm before the next block.  Outputs, each optional: r_out (r's
    dtype; may be r itself), x_out (x_dtype), and q int8 [m][k] with xs float32 [m][k/agroup].  x is rounded to
    x_dtype (x_out's dtype if not given, else r's) before it is quantised, so q and xs are those of
    pq2_quantize_act_i8_g on x_out.  post_w and gate have w's dtype."""
    shape = r.shape
    m, k = shape
    rt, wt = r.dtype, w.dtype
    rp, rs = _rows(r, "r", shape)
    wp = _vector(w, "w", k, wt)
    bp = bs = bd = pp = gp = gs = op = os_ = xp = xst = qp = sp = 0
    if block is not None:
        bp, bs = _rows(block, "block", shape)
        bd = _dtype(block, "block")
    if post_w is not None:
        pp = _vector(post_w, "post_w", k, wt)
    if gate is not None:
        if len(gate.shape) == 1:
            gp = _vector(gate, "gate", k, wt)
        elif gate.dtype is not wt:
            raise ValueError("gate must have the norm weights' dtype")
        else:
            gp, gs = _rows(gate, "gate", shape)
    if r_out is not None:
        if r_out.dtype is not rt:
            raise ValueError("r_out must have r's dtype")
        op, os_ = _rows(r_out, "r_out", shape)
    if x_out is not None:
        if x_dtype is not None and x_out.dtype is not x_dtype:
            raise ValueError("x_out must have x_dtype")
        xp, xst = _rows(x_out, "x_out", shape)
        x_dtype = x_out.dtype
    xd = _DTYPE.get(rt if x_dtype is None else x_dtype)
    if xd is None:
        raise ValueError(f"unsupported x_dtype {x_dtype}")
    if q is not None:
        if q.dtype is not _I8 or q.shape != shape or not q.is_contiguous():
            raise ValueError("q must be a contiguous int8 [m][k] tensor")
        qp = q.data_ptr()
    if xs is not None:
        if xs.dtype is not _F32 or agroup not in (128, 64, 32) or xs.numel() * agroup != m * k or \
                not xs.is_contiguous():
            raise ValueError("xs must be a contiguous float32 [m][k/agroup] tensor, agroup 128, 64 or 32")
        sp = xs.data_ptr()
    args = _NORM.pack(rp, rs, bp, bs, pp, gp, gs, wp, op, os_, xp, xst, qp, sp, m, k, agroup, eps, alpha,
                      _dtype(r, "r"), bd, _dtype(w, "w"), xd, 1 if unit_offset else 0)
    _call("pq2_block_norm", _device(r, w, block, post_w, gate, r_out, x_out, q, xs), stream, args)
