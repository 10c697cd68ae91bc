"""The block operators' C ABI without a GPU: the symbols of pq2_block.h are
exported and bound, and bad arguments are refused on the host (every case
fails validation or the device check, so nothing is launched)."""
import ctypes
import functools
import math
import os
import re
from fractions import Fraction

import numpy as np
import pytest
import torch

import block_reference as ref
import gemm_int8_act_amd as pq2
from gemm_int8_act_amd.block import NORM_FIELDS, _NORM

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, ESHAPE, EALIGN, EDEVICE = pq2.PQ2_OK, pq2.PQ2_EINVAL, pq2.PQ2_ESHAPE, pq2.PQ2_EALIGN, pq2.PQ2_EDEVICE

# Fake device addresses, never dereferenced: validation fails first.
A, B, C, D, E, F = (0x7F0000000000 + (i << 36) for i in range(6))



class BlockNormArgs(ctypes.Structure):
    _fields_ = [(name, {"P": ctypes.c_void_p, "q": ctypes.c_int64, "d": ctypes.c_double, "f": ctypes.c_float,
                        "i": ctypes.c_int}[code]) for name, code in NORM_FIELDS]


no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="the device check passes on a GPU")


def test_header_symbols_exported():
    text = open(os.path.join(ROOT, "include", "pq2_block.h")).read()
    names = set(re.findall(r"^(?:int|int64_t)\s+(pq2_\w+)\s*\(", text, re.M))
    assert names == set(pq2.BLOCK_EXPORTED)
    for name in names:
        assert hasattr(pq2.lib, name) and hasattr(pq2, name), name


def test_args_struct_matches_the_header(tmp_path):
    """Field order and offsets of the binding's structure, by the C compiler."""
    import subprocess
    fields = [f for f, _ in BlockNormArgs._fields_]
    src = tmp_path / "offsets.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "pq2_block.h"\nint main(void) {\n'
                   + "".join(f'printf("%zu\\n", offsetof(pq2_block_norm_args, {f}));\n' for f in fields)
                   + 'printf("%zu\\n", sizeof(pq2_block_norm_args)); return 0; }\n')
    exe = tmp_path / "offsets"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(BlockNormArgs, f).offset for f in fields] + [ctypes.sizeof(BlockNormArgs)]
    # What the binding packs is that structure, byte for byte.
    a = BlockNormArgs()
    values = [i + 1 if code in "Pq" else (i + 1) / 2 if code in "df" else i + 1 for i, (_, code) in enumerate(NORM_FIELDS)]
    for (name, _), v in zip(NORM_FIELDS, values):
        setattr(a, name, v)
    assert _NORM.pack(*values) == bytes(a)


def test_w4_tiles_bytes():
    f = pq2.pq2_w4_tiles_bytes
    assert f(10240, 5120, 128) == 10240 * 5120 // 2 + 10240 * 40 * 2
    assert f(1, 128, 32) == 8192 + 1024
    assert f(17, 1152, 64) == 2 * 2 * (8192 + 512)
    for n, k, g in ((0, 128, 128), (1, 100, 128), (1, 0, 64), (1, 1 << 17, 32), ((1 << 30) + 1, 128, 128),
                    (1, 128, 16), (1, 128, 0), (1, 128, 256)):
        with pytest.raises(ValueError):
            f(n, k, g)


def test_reference_layout_is_a_permutation():
    """The scatter of the reference layout read back weight by weight."""
    n, k, wg = 19, 1152, 64
    _, scales, c = ref.make_w4(n, k, wg, 3)
    t = ref.w4_tiles(c, scales, wg)
    unit = 8192 + 512
    for row, kk in ((0, 0), (18, 1151), (5, 77), (16, 1024), (7, 200), (3, 95)):
        base = (row // 16 * 2 + kk // 1024) * unit + kk % 1024 // 128 * 1024
        lane = row % 16 + 16 * (kk % 64 // 16)
        u = 2 * (kk % 128 // 64) + kk % 16 // 8
        byte = int(t[base + 16 * lane + 4 * u + kk % 4])
        nib = (byte >> 4) if kk % 8 >= 4 else (byte & 15)
        assert (nib ^ 8) == int(c[row, kk]), (row, kk)


def test_prepare_w4_validation():
    f = pq2.lib.pq2_prepare_w4_tiles
    assert f(None, 64, B, 1, 4, 128, 128, C, None) == EINVAL
    assert f(A, 64, None, 1, 4, 128, 128, C, None) == EINVAL
    assert f(A, 64, B, 1, 4, 128, 128, None, None) == EINVAL
    assert f(A, 64, B, 1, 4, 128, 48, C, None) == EINVAL
    assert f(A, 64, B, 1, 0, 128, 128, C, None) == ESHAPE
    assert f(A, 64, B, 1, 4, 192, 128, C, None) == ESHAPE
    assert f(A, 63, B, 1, 4, 128, 128, C, None) == ESHAPE
    assert f(A, 64, B, 3, 4, 128, 32, C, None) == ESHAPE
    assert f(A, 1 << 40, B, 1, 4, 128, 128, C, None) == ESHAPE and f(A, 64, B, 1 << 40, 4, 128, 128, C, None) == ESHAPE
    assert f(A, 64, B, 1, 4, 128, 128, C + 8, None) == EALIGN
    assert f(A, 64, B + 1, 1, 4, 128, 128, C, None) == EALIGN
    assert f(A, 64, B, 1, 4, 128, 128, A + 128, None) == EINVAL
    assert f(A, 64, B, 1, 4, 128, 128, B - 16, None) == EINVAL


@pytest.mark.parametrize("kind", ["w4", "gated_tiles", "gated_w4"])
def test_product_validation(kind):
    def f(q=A, xs=B, w=C, m=1, n=8, k=128, wg=128, y=D, up=E, act=0, dt=2):
        if kind == "w4":
            return pq2.lib.pq2_matmul_w4(q, xs, w, m, n, k, wg, y, None)
        if kind == "gated_w4":
            return pq2.lib.pq2_gated_matmul_w4(q, xs, w, up, m, n, k, wg, act, y, dt, None)
        return pq2.lib.pq2_gated_matmul_tiles(q, xs, w, up, m, n, k, act, y, dt, None)
    for name in ("q", "xs", "w", "y"):
        assert f(**{name: None}) == EINVAL
    assert f(m=0) == ESHAPE and f(m=65535 * 16 + 1) == ESHAPE
    assert f(n=0) == ESHAPE and f(n=(1 << 30) + 1) == ESHAPE
    assert f(k=0) == ESHAPE and f(k=200) == ESHAPE and f(k=1 << 17) == ESHAPE
    assert f(q=A + 8) == EALIGN and f(xs=B + 2) == EALIGN and f(w=C + 8) == EALIGN and f(y=D + 2) == EALIGN
    assert f(y=C + 64) == EINVAL and f(y=A) == EINVAL and f(y=B) == EINVAL
    if kind != "gated_tiles":
        assert f(wg=0) == EINVAL and f(wg=16) == EINVAL and f(wg=-128) == EINVAL
    if kind != "w4":
        assert f(up=None) == EINVAL and f(up=E + 8) == EALIGN and f(y=E) == EINVAL
        assert f(act=2) == EINVAL and f(act=-1) == EINVAL and f(dt=3) == EINVAL and f(dt=-1) == EINVAL
        assert f(y=D + 1, dt=0) == EALIGN
    if torch.cuda.device_count() == 0:
        assert f() == EDEVICE and f(m=65535 * 16) == EDEVICE and f(up=C) == EDEVICE


@pytest.mark.parametrize("kind", ["w4", "gated_tiles", "gated_w4"])
def test_linear_validation(kind):
    def f(x=F, dt=0, stride=128, w=C, m=2, n=8, k=128, wg=64, y=D, up=E, q=A, xs=B):
        if kind == "w4":
            return pq2.lib.pq2_linear_w4(x, dt, stride, w, m, n, k, wg, y, q, xs, None)
        if kind == "gated_w4":
            return pq2.lib.pq2_gated_linear_w4(x, dt, stride, w, up, m, n, k, wg, 0, y, 0, q, xs, None)
        return pq2.lib.pq2_gated_linear_tiles(x, dt, stride, w, up, m, n, k, 0, y, 0, q, xs, None)
    for name in ("x", "q", "xs", "w", "y"):
        assert f(**{name: None}) == EINVAL
    assert f(dt=3) == EINVAL and f(stride=127) == ESHAPE and f(m=0) == ESHAPE and f(k=64) == ESHAPE
    assert f(stride=(1 << 31) + 1) == ESHAPE and f(stride=(1 << 62) + 64) == ESHAPE
    assert f(m=65535 * 16, k=32768, stride=32768) == ESHAPE
    assert f(x=F + 1) == EALIGN and f(dt=2, x=F + 2) == EALIGN and f(q=A + 8) == EALIGN
    assert f(q=F) == EINVAL and f(xs=F) == EINVAL and f(y=F) == EINVAL    # x overlapped
    assert f(q=C) == EINVAL and f(xs=C + 64) == EINVAL                    # the weights overlapped
    assert f(xs=A + 16) == EINVAL and f(y=A) == EINVAL and f(y=B) == EINVAL
    if kind != "w4":
        assert f(q=E) == EINVAL and f(xs=E + 64) == EINVAL
    if torch.cuda.device_count() == 0:
        assert f() == EDEVICE and f(x=F + 2) == EDEVICE


@pytest.mark.parametrize("m", [1, 33, 65535 * 16])
def test_the_largest_n_is_one_that_every_kernel_can_launch(m):
    """Wider matrices are refused on the host (a complete call would have quantised x by the time its product has no
    launch); the widest accepted one passes every check."""
    most = (1 << 30) - 512          # 2^24 - 8 blocks of 64 columns; 2^24 workgroups of 256 threads are too many for a launch
    far = [i << 52 for i in range(1, 7)]
    def calls(n):
        q, xs, w, u, y, x = far
        return (pq2.lib.pq2_matmul_w4(q, xs, w, m, n, 128, 32, y, None),
                pq2.lib.pq2_linear_w4(x, 0, 128, w, m, n, 128, 128, y, q, xs, None),
                pq2.lib.pq2_gated_matmul_w4(q, xs, w, u, m, n, 128, 64, 0, y, 0, None),
                pq2.lib.pq2_gated_matmul_tiles(q, xs, w, u, m, n, 128, 0, y, 0, None),
                pq2.lib.pq2_gated_linear_w4(x, 0, 128, w, u, m, n, 128, 32, 1, y, 2, q, xs, None),
                pq2.lib.pq2_gated_linear_tiles(x, 0, 128, w, u, m, n, 128, 1, y, 2, q, xs, None),
                pq2.lib.pq2_prepare_w4_tiles(q, 64, xs, 4, n, 128, 32, w, None))
    assert set(calls(most + 1)) == {ESHAPE} and set(calls(1 << 30)) == {ESHAPE}
    assert pq2.lib.pq2_w4_tiles_bytes(most + 1, 128, 128) == -1
    assert pq2.lib.pq2_w4_tiles_bytes(most, 128, 128) == most // 16 * (8192 + 256)
    if torch.cuda.device_count() == 0:
        assert set(calls(most)) == {EDEVICE}


def norm_args(**kw):
    a = BlockNormArgs()
    a.r, a.r_stride, a.w, a.r_out, a.r_out_stride = A, 128, B, C, 128
    a.m, a.k, a.agroup, a.eps, a.alpha = 4, 128, 128, 1e-6, 1.0
    for name, v in kw.items():
        setattr(a, name, v)
    return pq2.lib.pq2_block_norm(bytes(a), None)


def test_block_norm_validation():
    f = norm_args
    assert pq2.lib.pq2_block_norm(None, None) == EINVAL
    assert f(r=None) == EINVAL and f(w=None) == EINVAL and f(r_out=None) == EINVAL
    assert f(q=D) == EINVAL and f(xs=D) == EINVAL
    assert f(post_w=D) == EINVAL and f(gate=D) == EINVAL               # no block
    assert f(r_dtype=3) == EINVAL and f(w_dtype=-1) == EINVAL and f(x_dtype=9) == EINVAL
    assert f(block=D, block_stride=128, block_dtype=4) == EINVAL
    assert f(q=D, xs=E, agroup=16) == EINVAL
    for eps in (0.0, -1e-6, 1e-71, float("inf"), float("nan")):
        assert f(eps=eps) == EINVAL
    assert f(alpha=float("nan")) == EINVAL and f(alpha=float("inf")) == EINVAL and f(unit_offset=2) == EINVAL
    assert f(m=0) == ESHAPE and f(m=65535 * 16 + 1) == ESHAPE and f(m=1 << 31) == ESHAPE and f(k=64) == ESHAPE and f(k=1 << 17) == ESHAPE
    assert f(r_stride=127) == ESHAPE and f(r_out_stride=1) == ESHAPE
    assert f(r_stride=(1 << 31) + 1) == ESHAPE and f(r_out_stride=1 << 62) == ESHAPE
    assert f(block=D, block_stride=1 << 61) == ESHAPE and f(x_out=D, x_out_stride=1 << 40) == ESHAPE
    assert f(block=D, block_stride=128, gate=E, gate_stride=1 << 60) == ESHAPE
    assert f(block=D, block_stride=0) == ESHAPE
    assert f(block=D, block_stride=128, gate=E, gate_stride=5) == ESHAPE
    assert f(x_out=D, x_out_stride=100) == ESHAPE
    assert f(r=A + 1) == EALIGN and f(w=B + 1) == EALIGN and f(r_out=C + 1) == EALIGN
    assert f(q=D + 4, xs=E) == EALIGN and f(q=D, xs=E + 2) == EALIGN
    assert f(block=D + 2, block_stride=128, block_dtype=2) == EALIGN
    assert f(r_out=A + 256) == EINVAL and f(r_out=A, r_out_stride=256) == EINVAL   # partly over r
    assert f(r_out=B) == EINVAL and f(x_out=A, x_out_stride=128) == EINVAL
    assert f(x_out=C, x_out_stride=128) == EINVAL and f(q=C, xs=E) == EINVAL and f(q=D, xs=D) == EINVAL
    assert f(block=C, block_stride=128) == EINVAL
    if torch.cuda.device_count() == 0:
        assert f() == EDEVICE and f(r_out=A) == EDEVICE
        assert f(block=D, block_stride=128, gate=E, gate_stride=0, post_w=F) == EDEVICE


def test_block_norm_columns_of_one_buffer():
    """Rows that lie between each other do not overlap; rows that share a byte, or have other strides, do."""
    f = functools.partial(norm_args, r_stride=512, r_out_stride=512)            # 256 of each 1024 bytes
    shared = [f(r_out=A + d) for d in (1024, 254, -254, 1022, 1026, 2048 + 128)]
    shared += [f(r_out=A + 256, r_out_stride=513), f(r_out=A + 256, r_out_stride=1024),
               f(r_out=A + 256, x_out=A + 256, x_out_stride=512), f(r_out=A + 256, x_out=A + 510, x_out_stride=512),
               f(r_out=A + 256, block=A + 384, block_stride=512), f(r_out=A + 256, w=A + 256),
               f(r_out=A + 256, x_out=A + 512, x_out_stride=256, x_dtype=2)]    # 512 bytes of each 1024, up to 1024: fits
    assert shared[:-1] == [EINVAL] * (len(shared) - 1)
    apart = [shared[-1]] + [f(r_out=A + d) for d in (256, 768, -256, -768, 2048 + 512)]
    apart += [f(r_out=A + 256, x_out=A + 512, x_out_stride=512, block=A + 768, block_stride=512),
              f(r_out=A, x_out=A + 512, x_out_stride=512, block=A + 256, block_stride=512, gate=A + 768, gate_stride=512)]
    if torch.cuda.device_count() == 0:
        assert apart == [EDEVICE] * len(apart)


def rn32(v):
    """A positive Fraction rounded to 24 significant bits, ties to even."""
    e = v.numerator.bit_length() - v.denominator.bit_length()
    while v >= Fraction(2) ** e:
        e += 1
    while v < Fraction(2) ** (e - 1):
        e -= 1
    unit = Fraction(2) ** (e - 24)
    return round(v / unit) * unit        # (Python's round: ties to even)


def test_quantiser_codes_at_the_hardest_quotients():
    """The steps of quantise_bits in exact arithmetic, on every quotient where they might miss the correctly rounded one
    at a border of the codes: the same codes."""
    xs, ds, _ = ref.hard_quotients()
    assert len(xs) > 1000
    differ = 0
    for x, d in zip(map(Fraction, xs), map(Fraction, ds)):
        y = rn32(1 / d)
        t0 = rn32(x * y)
        e = x - t0 * d
        e = (rn32(e) if e > 0 else -rn32(-e)) if e else e
        t, q = rn32(t0 + e * y), rn32(x / d)
        assert abs(t0 - x / d) <= 2 * Fraction(float(np.spacing(np.float32(float(q))))), (float(x), float(d))
        differ += t != q
        assert round(t) == round(q), (float(x), float(d))
    print(f"{len(xs)} quotients, {differ} rounded otherwise")


def test_hard_quotients_are_all_there_are():
    """Found by their residue, against all 2^23 divisors tried for some of the midpoints."""
    xs, ds, mids = ref.hard_quotients()
    den = np.arange(1 << 23, 1 << 24, dtype=np.int64)
    for mid in np.unique(mids)[::23]:
        e = math.frexp(mid)[1] - 1
        product = int(math.ldexp(mid, 24 - e)) * den
        tried = set()
        for s in (24, 25):
            num = (product + (1 << s >> 1)) >> s
            hit = (np.abs((num << s) - product) < 8) & (num >= 1 << 23) & (num <= 1 << 24)
            tried |= {(math.ldexp(int(a), s + e - 47), math.ldexp(int(b), -23)) for a, b in zip(num[hit], den[hit])}
        assert tried == set(zip(xs[mids == mid].tolist(), ds[mids == mid].tolist()))


def test_quantiser_codes_next_to_the_borders():
    """The same steps in float arithmetic, for random divisors and the four x around each border and the midpoints
    beside it.  (Products of floats are exact in doubles, and x - t0 d is a double; t0 + e y, rounded to a double
    first, could only differ within 2^-28 ulp of a midpoint: the cases of the test above.)"""
    rng = np.random.default_rng(1)
    f32, f64 = np.float32, np.float64
    for h in range(127):
        d = (rng.integers(1 << 23, 1 << 24, 4000) * 2.0 ** -23).astype(f32)
        border = f32(h + 0.5)
        for mid in (f64(border), (f64(border) + f64(np.nextafter(border, f32(0)))) / 2,
                    (f64(border) + f64(np.nextafter(border, f32(1000)))) / 2):
            x = (mid * d.astype(f64)).astype(f32)
            for step in (x, np.nextafter(x, f32(0)), np.nextafter(x, f32(1000))):
                q = (step.astype(f64) / d).astype(f32)
                y = f32(1) / d
                t0 = step * y
                e = (step.astype(f64) - t0.astype(f64) * d).astype(f32)
                t = (t0.astype(f64) + e.astype(f64) * y).astype(f32)
                assert np.array_equal(np.rint(t), np.rint(q)), h


@no_gpu
def test_binding_refuses_host_tensors_and_shapes():
    t = torch.zeros
    with pytest.raises(ValueError):
        pq2.pq2_block_norm(t((2, 128)), t(128), 1e-6, r_out=t((2, 128)))
    with pytest.raises(ValueError):
        pq2.pq2_block_norm(t((2, 128)), t(64), 1e-6, r_out=t((2, 128)))
    with pytest.raises(ValueError):
        pq2.pq2_block_norm(t((2, 128)), t(128), 1e-6, q=t((2, 128), dtype=torch.int8), xs=t((2, 4)), agroup=16)
    with pytest.raises(ValueError):
        pq2.pq2_matmul_w4(t((2, 128), dtype=torch.int8), t((2, 1)), t(9216, dtype=torch.uint8), t((3, 5)), 32)
    with pytest.raises(ValueError):
        pq2.pq2_matmul_w4(t((2, 128), dtype=torch.int8), t((2, 1)), t(9215, dtype=torch.uint8), t((2, 5)), 32)
    with pytest.raises(ValueError):
        pq2.pq2_linear_w4(t((2, 127)), t(9216, dtype=torch.uint8), t((2, 5)), 32, t((2, 128), dtype=torch.int8), t((2, 1)))
