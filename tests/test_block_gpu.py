"""The block operators on the GPU against plain 64-bit references: products
with 4-bit weights, the gated feed-forward product, the block norms.  Bounds
are those of tests/block_reference.py; outputs are poisoned before a call and
followed by guard elements that must not change."""
import functools
import math

import pytest
import torch

import block_reference as ref
import workloads

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@functools.lru_cache(maxsize=None)
def _pq2():
    import gemm_int8_act_amd as pq2
    return pq2


def announce(msg):
    print(f"[gpu-case] {msg}", flush=True)


class Guarded:
    """A poisoned contiguous output of a shape, with guard elements behind it."""

    def __init__(self, shape, dtype):
        self.count = 1
        for s in shape:
            self.count *= s
        value = -77 if dtype == torch.int8 else float("nan")
        self.all = torch.full((self.count + 64,), value, dtype=dtype, device=DEV)
        self.all[self.count:] = 42
        self.t = self.all[:self.count].view(shape)

    def read(self):
        torch.cuda.synchronize()
        assert bool((self.all[self.count:] == 42).all()), "wrote behind the output"
        return self.t.cpu()


def within(got, want, bound, what):
    got = got.double()
    assert bool(torch.isfinite(got).all()), f"{what}: non-finite output"
    excess = (got - want).abs() - bound
    worst = int(excess.argmax())
    assert float(excess.max()) <= 0, (f"{what}: off by {float((got - want).abs().flatten()[worst]):.3e}, bound "
                                      f"{float(bound.flatten()[worst]):.3e} at {worst}")


def activations(m, k, seed, dtype=torch.bfloat16, pad=0):
    x = workloads.make_activations(m, k + pad, seed, "normal+outliers").to(dtype)
    return x


def w4(n, k, wg, seed, pad=0):
    pq2 = _pq2()
    codes, scales, c = ref.make_w4(n, k, wg, seed, pad)
    out = torch.full((pq2.pq2_w4_tiles_bytes(n, k, wg),), 0xA5, dtype=torch.uint8, device=DEV)
    cd, sd = codes.to(DEV), scales.to(DEV)
    pq2.pq2_prepare_w4_tiles(cd, sd[:, :k // wg], wg, out)
    return out, c, scales


def quantise(x, k):
    pq2 = _pq2()
    q = torch.empty((x.shape[0], k), dtype=torch.int8, device=DEV)
    xs = torch.empty((x.shape[0], k // 128), dtype=torch.float32, device=DEV)
    pq2.pq2_quantize_act_i8(x.to(DEV), q, xs)
    return q, xs


# ---------------------------------------------------------------- 4-bit layout
@pytest.mark.parametrize("wg", [128, 64, 32])
@pytest.mark.parametrize("n,k,pad", [(1, 128, 0), (19, 1152, 0), (37, 384, 5), (256, 5120, 3), (16, 17408, 0)])
def test_prepare_w4_byte_exact(n, k, pad, wg):
    announce(f"prepare w4 n={n} k={k} wg={wg} pad={pad}")
    tiles, c, scales = w4(n, k, wg, n + k, pad)
    torch.cuda.synchronize()
    assert torch.equal(tiles.cpu(), ref.w4_tiles(c, scales, wg))


# ---------------------------------------------------------------- 4-bit products
W4_SHAPES = [(1, 1, 128), (1, 200, 512), (2, 17, 384), (3, 33, 1024), (4, 300, 1152), (5, 16, 128), (4, 40, 16384),
             (9, 150, 2176), (16, 64, 5120), (16, 31, 17408), (17, 100, 640), (33, 70, 5120), (64, 128, 1024),
             (100, 257, 1152), (131, 40, 3200), (1, 24, 65536), (300, 600, 1280),
             # decode: LDS full of activations, several segments a wave, each place the activations of a wide pass sit in
             (4, 33, 32768), (3, 20, 65536), (8, 40, 17408), (13, 24, 12288), (16, 20, 24576), (7, 18, 65536),
             # prefill: low-latency, 32-row and 64-row kernels, ragged rows and columns, groups behind the last segment
             (130, 1400, 384), (700, 300, 1152), (1400, 130, 2176), (33, 1400, 384), (257, 300, 1152), (500, 130, 2176), (1000, 1001, 256), (2100, 1100, 384), (2201, 2083, 128)]


@pytest.mark.parametrize("wg", [128, 64, 32])
@pytest.mark.parametrize("m,n,k", W4_SHAPES)
def test_matmul_w4(m, n, k, wg):
    announce(f"matmul w4 m={m} n={n} k={k} wg={wg}")
    tiles, c, scales = w4(n, k, wg, m + n)
    x = activations(m, k, m + k)
    q, xs = quantise(x, k)
    y = Guarded((m, n), torch.float32)
    _pq2().pq2_matmul_w4(q, xs, tiles, y.t, wg)
    want, bound = ref.product(*ref.quantised(x, k), (c - 8).double(), scales, wg)
    within(y.read(), want, bound, "y")


@pytest.mark.parametrize("wg", [128, 64, 32])
@pytest.mark.parametrize("k", [1152, 17408])
def test_matmul_w4_columns_do_not_depend_on_the_batch(k, wg):
    announce(f"w4 batch invariance k={k} wg={wg}")
    n = 90
    tiles, _, _ = w4(n, k, wg, 5)
    q, xs = quantise(activations(16, k, 6), k)
    whole = torch.empty((16, n), device=DEV)
    _pq2().pq2_matmul_w4(q, xs, tiles, whole, wg)
    for m in (1, 2, 3, 4, 5, 11):
        y = torch.empty((m, n), device=DEV)
        _pq2().pq2_matmul_w4(q[16 - m:].clone(), xs[16 - m:].clone(), tiles, y, wg)
        torch.cuda.synchronize()
        assert torch.equal(y, whole[16 - m:]), m


@pytest.mark.parametrize("wg", [128, 64, 32])
@pytest.mark.parametrize("m,n,k", [(16, 4100, 17408), (9, 8192, 17408), (16, 8300, 12288), (12, 4128, 26624), (5, 4200, 65536),
                                   (16, 4097, 9728)])
def test_matmul_w4_rows_do_not_depend_on_the_matrix(m, n, k, wg):
    """A row's bits in a matrix of more than 256 tiles (in pairs, for some of these) and in a slice of it."""
    announce(f"w4 slices m={m} n={n} k={k} wg={wg}")
    pq2 = _pq2()
    gen = torch.Generator(device=DEV).manual_seed(n + k + wg)
    w = torch.empty(pq2.pq2_w4_tiles_bytes(n, k, wg), dtype=torch.uint8, device=DEV)
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, generator=gen, device=DEV)
    pq2.pq2_prepare_w4_tiles(codes, (torch.rand((n, k // wg), generator=gen, device=DEV) * 0.05).half(), wg, w)
    q, xs = quantise(activations(m, k, 5), k)
    y = Guarded((m, n), torch.float32)
    pq2.pq2_matmul_w4(q, xs, w, y.t, wg)
    got = y.read()
    assert bool(torch.isfinite(got).all())
    for first in (0, 2000, n // 16 * 16 - 48):      # whole tiles; the last slice ends with the matrix
        rows = min(2000, n - first)
        size = pq2.pq2_w4_tiles_bytes(rows, k, wg)
        start = pq2.pq2_w4_tiles_bytes(first, k, wg) if first else 0
        part = torch.empty((m, rows), device=DEV)
        pq2.pq2_matmul_w4(q, xs, w[start:start + size], part, wg)
        torch.cuda.synchronize()
        assert torch.equal(got[:, first:first + rows], part.cpu()), f"rows from {first}"


@pytest.mark.parametrize("m", [3, 16, 150])
def test_w4_extreme_codes(m):
    """All weights -8 or 7 against codes of +-127: the largest dots, exact as floats."""
    announce(f"w4 extremes m={m}")
    n, k, wg = 48, 1024, 128
    c = torch.zeros((n, k), dtype=torch.uint8)
    c[n // 2:] = 15
    tiles = torch.empty(_pq2().pq2_w4_tiles_bytes(n, k, wg), dtype=torch.uint8, device=DEV)
    scales = torch.full((n, k // wg), 0.5, dtype=torch.float16)
    _pq2().pq2_prepare_w4_tiles((c[:, 0::2] | (c[:, 1::2] << 4)).contiguous().to(DEV), scales.to(DEV), wg, tiles)
    x = torch.full((m, k), 127.0).to(torch.bfloat16)
    x[1::2] *= -1
    q, xs = quantise(x, k)
    y = torch.empty((m, n), device=DEV)
    _pq2().pq2_matmul_w4(q, xs, tiles, y, wg)
    torch.cuda.synchronize()
    sign = torch.ones(m, 1)
    sign[1::2] = -1
    want = sign * torch.where(torch.arange(n) < n // 2, -8.0, 7.0) * 0.5 * 127 * k
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,k,pad", [(1, 50, 1024, 0), (3, 130, 640, 5), (20, 33, 1152, 8)])
def test_linear_w4_is_quantise_then_matmul(dtype, m, n, k, pad):
    announce(f"linear w4 {dtype} m={m} pad={pad}")
    tiles, _, _ = w4(n, k, 64, 9)
    x = activations(m, k, 4, DT[dtype], pad).to(DEV)
    q, xs = quantise(x, k)
    want = torch.empty((m, n), device=DEV)
    _pq2().pq2_matmul_w4(q, xs, tiles, want, 64)
    y, qw, sw = Guarded((m, n), torch.float32), torch.zeros_like(q), torch.zeros_like(xs)
    _pq2().pq2_linear_w4(x, tiles, y.t, 64, qw, sw)
    assert torch.equal(y.read(), want.cpu())


def hard_activations(m, k, dtype, seed):
    """Values at and next to rounding borders of their group's scale, over the exponent range: ties (c + 1/2) * scale
    and their neighbours, subnormal and huge groups, all-zero groups, single elements."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randint(-127, 128, (m, k // 128, 128), generator=gen).double() + 0.5 * torch.randint(0, 2, (m, k // 128, 128), generator=gen)
    lo, hi = {"bf16": (-130, 118), "f16": (-22, 6), "f32": (-145, 118)}[dtype]
    exp = torch.randint(lo, hi, (m, k // 128, 1), generator=gen).double()
    frac = 1 + torch.rand((m, k // 128, 1), generator=gen).double() * torch.randint(0, 2, (m, k // 128, 1), generator=gen)
    x[..., 0] = 127
    x = x * frac * torch.exp2(exp)
    x[0, 0] = 0
    if k > 128:
        x[0, 1] = 0
        x[0, 1, 77] = x.abs().max()
    x = x.reshape(m, k).to(DT[dtype])
    step = torch.randint(-1, 2, (m, k), generator=gen)
    raw = x.view(torch.int16 if dtype != "f32" else torch.int32)
    near = (raw + step.to(raw.dtype)).view(DT[dtype])
    return torch.where(torch.isfinite(near) & (x != 0), near, x)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,k", [(1, 1024), (2, 5120), (4, 2176), (3, 17408)])
def test_linear_w4_codes_at_rounding_borders(m, k, dtype):
    """The in-kernel quantiser's codes: the same y, bit for bit, as from pq2_quantize_act_i8's q and xs, which are
    those of the definition, with one weight column standing out per row so that single codes show."""
    announce(f"linear w4 rounding borders {dtype} m={m} k={k}")
    n = 256
    x = hard_activations(m, k, dtype, m + k)
    want_q, want_s = ref.quantised(x, k)
    xd = x.to(DEV)
    q, xs = quantise(xd, k)
    assert torch.equal(q.cpu().double().view(want_q.shape), want_q) and torch.equal(xs.cpu().double(), want_s)
    tiles, _, _ = w4(n, k, 32, 77)
    y, z = torch.empty((m, n), device=DEV), torch.empty((m, n), device=DEV)
    _pq2().pq2_matmul_w4(q, xs, tiles, y, 32)
    _pq2().pq2_linear_w4(xd, tiles, z, 32, torch.zeros_like(q), torch.zeros_like(xs))
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int32), z.view(torch.int32))


@pytest.mark.parametrize("m,n", [(4, 40), (16, 40), (64, 40), (60, 1200), (200, 1200), (2200, 2100)])
def test_w4_a_bad_row_stays_alone(m, n):
    """NaN scales in one row of xs reach that row's outputs only (k ends inside a segment)."""
    announce(f"w4 one bad row m={m} n={n}")
    k = 1152
    tiles, _, _ = w4(n, k, 128, 2)
    q, xs = quantise(activations(m, k, 3), k)
    y = torch.empty((m, n), device=DEV)
    _pq2().pq2_matmul_w4(q, xs, tiles, y, 128)
    xs[2] = float("nan")
    z = torch.empty((m, n), device=DEV)
    _pq2().pq2_matmul_w4(q, xs, tiles, z, 128)
    torch.cuda.synchronize()
    rows = [i for i in range(m) if i != 2]
    assert torch.equal(y[rows], z[rows]) and bool(torch.isnan(z[2]).all())


def poisoned_scratch(m, k):
    return (torch.full((m, k), -77, dtype=torch.int8, device=DEV),
            torch.full((m, k // 128), -3.0, dtype=torch.float32, device=DEV))


def untouched(qw, sw):
    return bool((qw == -77).all()) and bool((sw == -3.0).all())


def test_linear_w4_codes_at_the_hardest_quotients():
    """The in-kernel quantiser on every quotient where its steps might miss a border, one to a group (the group's
    largest element gives its divisor), over exponents and signs; a row of weights picks each group's code."""
    announce("linear w4 hardest quotients")
    xs, ds, _ = ref.hard_quotients()
    amax = (ds * 127).astype("float32")
    fits = ((amax.astype("float64") / 127).astype("float32") == ds) & (amax >= xs)
    xs, ds, amax = (torch.from_numpy(v[fits].astype("float64")) for v in (xs, ds, amax))
    assert len(xs) > 1000
    k = 49152
    groups = k // 128
    codes = torch.full((groups, k // 2), 0x88, dtype=torch.uint8)
    codes[torch.arange(groups), 64 * torch.arange(groups)] = 0x98           # weight 1 at the group's second element
    tiles = torch.empty(_pq2().pq2_w4_tiles_bytes(groups, k, 32), dtype=torch.uint8, device=DEV)
    _pq2().pq2_prepare_w4_tiles(codes.to(DEV), torch.ones((groups, k // 32), dtype=torch.float16, device=DEV), 32, tiles)
    for first in range(0, len(xs), groups):
        part = slice(first, min(first + groups, len(xs)))
        some = part.stop - first
        scale = torch.exp2((torch.arange(some) * 37 % 201 - 100).double()) * (1 - 2 * (torch.arange(some) % 2)).double()
        x = torch.zeros((1, groups, 128), dtype=torch.float64)
        x[0, :some, 0], x[0, :some, 1] = amax[part] * scale, xs[part] * scale
        x = x.float().view(1, k)
        q, s = ref.quantised(x, k)
        assert torch.equal(s[0, :some], ds[part] * scale.abs())
        y, (qw, sw) = Guarded((1, groups), torch.float32), poisoned_scratch(1, k)
        _pq2().pq2_linear_w4(x.to(DEV), tiles, y.t, 32, qw, sw)
        assert torch.equal(y.read()[0], (q[0, :, 1] * s[0]).float()) and untouched(qw, sw)


# Complete calls that one launch does (block_takes_x in block_small_m.hip: m times the 12288-weight parts of k is at
# most four), with one to five segments of k a wave, ragged ends, and passes of fewer columns than m (K > 32768).
ONE_LAUNCH = [(1, 640), (4, 1152), (3, 11392), (4, 12288), (1, 12416), (2, 12416), (2, 17408), (2, 24576), (1, 24704),
              (1, 33024), (1, 36864), (1, 40960), (1, 49152)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,k", ONE_LAUNCH)
def test_linear_w4_in_one_launch(m, k, dtype):
    """The bits of quantiser and product, from the launch that leaves the scratch alone."""
    n = 77
    x = hard_activations(m, k, dtype, m + k).to(DEV)
    q, xs = quantise(x, k)
    for wg in (128, 64, 32):
        announce(f"linear w4 in one launch {dtype} m={m} k={k} wg={wg}")
        tiles, _, _ = w4(n, k, wg, k)
        want, y = Guarded((m, n), torch.float32), Guarded((m, n), torch.float32)
        _pq2().pq2_matmul_w4(q, xs, tiles, want.t, wg)
        scratch = poisoned_scratch(m, k)
        _pq2().pq2_linear_w4(x, tiles, y.t, wg, *scratch)
        assert torch.equal(y.read().view(torch.int32), want.read().view(torch.int32)), wg
        assert untouched(*scratch), "took two launches"


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,k", ONE_LAUNCH)
def test_gated_linear_in_one_launch(m, k, dtype):
    pq2 = _pq2()
    n = 45
    x = activations(m, k, m + k, DT[dtype]).to(DEV)
    q, xs = quantise(x, k)
    for wg in (0, 128, 64, 32):
        announce(f"gated linear in one launch {dtype} m={m} k={k} wg={wg}")
        a, b = (w4(n, k, wg, i)[0] if wg else ternary_tiles(n, k, i)[0] for i in (3, 4))
        want, h = Guarded((m, n), torch.float32), Guarded((m, n), torch.float32)
        scratch = poisoned_scratch(m, k)
        if wg:
            pq2.pq2_gated_matmul_w4(q, xs, a, b, want.t, wg, pq2.ACT_GELU_TANH)
            pq2.pq2_gated_linear_w4(x, a, b, h.t, wg, *scratch, pq2.ACT_GELU_TANH)
        else:
            pq2.pq2_gated_matmul_tiles(q, xs, a, b, want.t)
            pq2.pq2_gated_linear_tiles(x, a, b, h.t, *scratch)
        assert bool(torch.isfinite(want.t).all())
        assert torch.equal(h.read().view(torch.int32), want.read().view(torch.int32)), wg
        assert untouched(*scratch), "took two launches"


@pytest.mark.parametrize("m,k", [(3, 17408), (4, 24576), (2, 36864), (1, 61440), (5, 640)])
def test_linear_w4_in_two_launches(m, k):
    """Past that rule, and for rows that 16-byte loads do not reach: the scratch holds the quantiser's results."""
    announce(f"linear w4 in two launches m={m} k={k}")
    n, wg = 33, 64
    tiles, _, _ = w4(n, k, wg, 6)
    for mm, shift in ((m, 0), (1, 1)):
        x = torch.zeros(mm * k + 8, dtype=torch.bfloat16, device=DEV)[shift:shift + mm * k].view(mm, k)
        x.copy_(activations(mm, k, 7))
        q, xs = quantise(x, k)
        want, y = torch.empty((mm, n), device=DEV), torch.empty((mm, n), device=DEV)
        _pq2().pq2_matmul_w4(q, xs, tiles, want, wg)
        qw, sw = poisoned_scratch(mm, k)
        _pq2().pq2_linear_w4(x, tiles, y, wg, qw, sw)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        assert torch.equal(qw, q) and torch.equal(sw, xs), (mm, shift)


# m, n, k: decode of up to four and of more columns, each prefill kernel.
HUGE_SHAPES = [(1, 40, 1152), (4, 40, 17408), (7, 40, 1152), (16, 40, 17408), (12, 4130, 17408), (60, 1200, 384), (200, 1200, 1152),
               (2100, 1100, 256), (2201, 2083, 256)]


def huge_weights(n, k, wg, seed):
    """(tiles, c, scales) with, by row modulo three, positive weights, negative ones, and positive ones in the first half
    of k against negative ones in the second."""
    gen = torch.Generator().manual_seed(seed)
    c = torch.randint(9, 16, (n, k), generator=gen, dtype=torch.uint8)
    c[1::3] = 16 - c[1::3]
    c[2::3, k // 2:] = 16 - c[2::3, k // 2:]
    scales = (torch.rand((n, k // wg), generator=gen) * 0.5 + 0.5).half()
    tiles = torch.empty(_pq2().pq2_w4_tiles_bytes(n, k, wg), dtype=torch.uint8, device=DEV)
    _pq2().pq2_prepare_w4_tiles((c[:, 0::2] | (c[:, 1::2] << 4)).contiguous().to(DEV), scales.to(DEV), wg, tiles)
    return tiles, c.long(), scales


def huge_activations(m, k, wg, c, scales):
    """Positive FP32 activations whose sums of magnitudes end between 2^126 and 2^127, so that no order of adding the
    terms passes the largest float."""
    x = workloads.make_activations(m, k, 3, "normal+outliers").float().abs() + 0.25
    q, xs = ref.quantised(x, k)
    per_group = (q.reshape(m, k // wg, wg).sum(2) * xs.repeat_interleave(128 // wg, 1))
    most = float((per_group.abs() @ (scales.double() * (c - 8).abs().amax(1, keepdim=True)).t()).max())
    return x * 2.0 ** (126 - math.floor(math.log2(most)))


@pytest.mark.parametrize("wg", [128, 64, 32])
@pytest.mark.parametrize("m,n,k", HUGE_SHAPES)
def test_w4_sums_near_the_largest_float(m, n, k, wg):
    """y, and every sum on the way, stays below the largest float: the result is finite and within the bound."""
    announce(f"w4 huge m={m} n={n} k={k} wg={wg}")
    tiles, c, scales = huge_weights(n, k, wg, n + k)
    x = huge_activations(m, k, wg, c, scales)
    q, xs = quantise(x, k)
    y, z = Guarded((m, n), torch.float32), Guarded((m, n), torch.float32)
    _pq2().pq2_matmul_w4(q, xs, tiles, y.t, wg)
    _pq2().pq2_linear_w4(x.to(DEV), tiles, z.t, wg, torch.empty_like(q), torch.empty_like(xs))
    want, bound = ref.product(*ref.quantised(x, k), (c - 8).double(), scales, wg)
    assert float(want.abs().max()) > 2.0 ** 124
    within(y.read(), want, bound, "y")
    assert torch.equal(y.t, z.t)


@pytest.mark.parametrize("wg", [128, 64, 32])
@pytest.mark.parametrize("m,n,k", [(2, 40, 1152), (13, 40, 1152), (60, 1200, 384), (2201, 2083, 256)])
def test_gated_w4_sums_near_the_largest_float(m, n, k, wg):
    """A gate or an up product near the largest float against one that is zero: zero, not inf * 0."""
    announce(f"gated w4 huge m={m} n={n} k={k} wg={wg}")
    tiles, c, scales = huge_weights(n, k, wg, n + k)
    x = huge_activations(m, k, wg, c, scales)
    q, xs = quantise(x, k)
    zero = torch.empty_like(tiles)
    _pq2().pq2_prepare_w4_tiles(torch.full((n, k // 2), 0x88, dtype=torch.uint8, device=DEV), scales.to(DEV), wg, zero)
    for gate, up in ((tiles, zero), (zero, tiles)):
        h = Guarded((m, n), torch.float32)
        _pq2().pq2_gated_matmul_w4(q, xs, gate, up, h.t, wg)
        assert bool((h.read() == 0).all())


@pytest.mark.parametrize("m,n", [(1, 48), (4, 48), (9, 48), (64, 48), (200, 1200), (2200, 2083)])
def test_w4_subnormal_scales_and_sums(m, n):
    """One group: y = RN(RN(dot * ws) * xs) bit for bit, with subnormal fp16 weight scales, and activation scales down
    to where y is subnormal."""
    announce(f"w4 subnormals m={m} n={n}")
    k = 128
    codes, scales, c = ref.make_w4(n, k, k, 5)
    scales = (torch.arange(1, n + 1)[:, None] % 1500 * 2.0 ** -24).half()
    tiles = torch.empty(_pq2().pq2_w4_tiles_bytes(n, k, k), dtype=torch.uint8, device=DEV)
    _pq2().pq2_prepare_w4_tiles(codes.to(DEV), scales.to(DEV), k, tiles)
    x = workloads.make_activations(m, k, 6, "normal").float() * torch.exp2(-(torch.arange(m) * 29 % 130).float())[:, None]
    q, xs = ref.quantised(x, k)
    dot = q[:, 0] @ (c - 8).double().t()
    want = (dot * scales.double().t()).float() * xs.float()
    y = Guarded((m, n), torch.float32)
    _pq2().pq2_matmul_w4(*quantise(x, k), tiles, y.t, k)
    assert torch.equal(y.read(), want)
    assert m < 64 or bool(((want != 0) & (want.abs() < 2.0 ** -126)).any())


def test_w4_zero_activations():
    announce("w4 zero activations")
    tiles, _, _ = w4(30, 640, 32, 1)
    for m in (1, 7, 40):
        q, xs = quantise(torch.zeros((m, 640), dtype=torch.bfloat16), 640)
        y = Guarded((m, 30), torch.float32)
        _pq2().pq2_matmul_w4(q, xs, tiles, y.t, 32)
        assert bool((y.read() == 0).all())


# ---------------------------------------------------------------- gated product
def ternary_tiles(n, k, seed):
    pq2 = _pq2()
    raw = workloads.make_raw_weights(n, k, seed=seed, codes="ternary+3")
    tiles = torch.empty(pq2.pq2_tiles_bytes(n, k), dtype=torch.uint8, device=DEV)
    pq2.pq2_prepare_tiles(torch.from_numpy(raw).to(DEV), n, k, tiles)
    return tiles, raw


GATED_SHAPES = [(1500, 1999, 128), (600, 2100, 256), (40, 1500, 1152), (4, 33, 32768), (8, 17, 17408), (1, 1, 128), (1, 200, 1024), (2, 40, 384), (4, 33, 5120), (6, 17, 1152), (16, 100, 2176),
                (13, 24, 17408), (37, 65, 1152), (70, 130, 640), (129, 300, 1024), (4, 20, 16384),
                (300, 700, 640), (200, 400, 8192), (70, 1100, 8192)]


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("h", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("wg", [0, 128, 64, 32])
@pytest.mark.parametrize("m,n,k", GATED_SHAPES)
def test_gated(m, n, k, wg, h, act):
    announce(f"gated m={m} n={n} k={k} wg={wg} h={h} act={act}")
    x = activations(m, k, m + n)
    q, xs = quantise(x, k)
    codes = ref.quantised(x, k)
    out = Guarded((m, n), DT[h])
    if wg:
        (wa, ca, sa), (wb, cb, sb) = w4(n, k, wg, 11), w4(n, k, wg, 12)
        _pq2().pq2_gated_matmul_w4(q, xs, wa, wb, out.t, wg, act)
        ga, gb = ((ref.product(*codes, (c - 8).double(), s, wg)) for c, s in ((ca, sa), (cb, sb)))
    else:
        (wa, ra), (wb, rb) = ternary_tiles(n, k, 21), ternary_tiles(n, k, 22)
        _pq2().pq2_gated_matmul_tiles(q, xs, wa, wb, out.t, act)
        ga, gb = (ref.product(*codes, *ref.ternary(r, n, k), 128) for r in (ra, rb))
    want, bound = ref.gated(*ga, *gb, act, DT[h])
    within(out.read(), want, bound, "h")


@pytest.mark.parametrize("m,n,k", [(1, 50, 1024), (4, 33, 5120), (7, 100, 8192), (16, 20, 17408)])
def test_gated_tiles_has_the_bits_of_the_two_products(m, n, k):
    """With large positive gates SiLU(g) = g exactly in FP32, so h = fl(yg * yu) of the library's two matmuls."""
    announce(f"gated bits m={m} n={n} k={k}")
    pq2 = _pq2()
    raw = workloads.make_raw_weights(n, k, seed=5, codes="ternary")
    raw.reshape(n, k // 128, 34)[:, :, 2:] |= 0xAA        # codes 2 and 3: weights +1 and +2
    x = activations(m, k, 8).abs() + 0.5
    gate = torch.empty(pq2.pq2_tiles_bytes(n, k), dtype=torch.uint8, device=DEV)
    pq2.pq2_prepare_tiles(torch.from_numpy(raw).to(DEV), n, k, gate)
    up, _ = ternary_tiles(n, k, 6)
    q, xs = quantise(x, k)
    yg, yu, h = (torch.empty((m, n), device=DEV) for _ in range(3))
    pq2.pq2_matmul_small_m_tiles(q, xs, gate, yg)
    pq2.pq2_matmul_small_m_tiles(q, xs, up, yu)
    pq2.pq2_gated_matmul_tiles(q, xs, gate, up, h, pq2.ACT_SILU)
    torch.cuda.synchronize()
    big = yg > 20                                        # exp(-g) < 2^-25: 1 + exp(-g) = 1
    assert float(big.float().mean()) > 0.9
    assert torch.equal(h[big], (yg * yu)[big])


@pytest.mark.parametrize("m", [2, 12, 80])
def test_gated_one_matrix_for_both_and_linear(m):
    announce(f"gated shared matrix m={m}")
    pq2 = _pq2()
    n, k = 60, 1152
    x = activations(m, k, 3, torch.float16, 8).to(DEV)
    q, xs = quantise(x, k)
    for wg in (0, 32):
        w = w4(n, k, wg, 4)[0] if wg else ternary_tiles(n, k, 4)[0]
        a, b = (torch.empty((m, n), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        qw, sw = torch.empty_like(q), torch.empty_like(xs)
        if wg:
            pq2.pq2_gated_matmul_w4(q, xs, w, w, a, wg, pq2.ACT_GELU_TANH)
            pq2.pq2_gated_linear_w4(x, w, w, b, wg, qw, sw, pq2.ACT_GELU_TANH)
        else:
            pq2.pq2_gated_matmul_tiles(q, xs, w, w, a, pq2.ACT_GELU_TANH)
            pq2.pq2_gated_linear_tiles(x, w, w, b, qw, sw, pq2.ACT_GELU_TANH)
        torch.cuda.synchronize()
        assert torch.equal(a, b) and bool(torch.isfinite(a).all())


def test_gated_more_rows_than_one_launch_takes():
    """2^24 workgroups of 256 threads and more: the rows of several launches have the bits of a small call's."""
    m, n, k, wg = 65535 * 16, 32768, 128, 32
    part = m // 257
    if torch.cuda.mem_get_info()[0] < 100e9:
        pytest.skip("needs 70 GB for the output")
    announce(f"gated m={m} n={n} k={k} wg={wg}")
    pq2 = _pq2()
    w = w4(n, k, wg, 5)[0]
    q, xs = quantise(activations(part, k, 6), k)
    want = torch.empty((part, n), dtype=torch.bfloat16, device=DEV)
    pq2.pq2_gated_matmul_w4(q, xs, w, w, want, wg)
    h = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device=DEV)
    pq2.pq2_gated_matmul_w4(q.repeat(257, 1), xs.repeat(257, 1), w, w, h, wg)
    torch.cuda.synchronize()
    for i in range(257):
        assert torch.equal(h[i * part:(i + 1) * part], want), f"rows of part {i}"
    del h
    torch.cuda.empty_cache()


@pytest.mark.parametrize("act", [0, 1])
def test_gated_far_ends_of_the_activation(act):
    """Gates far below and above zero: act(g) goes to 0 and g, never NaN."""
    announce(f"gated extremes act={act}")
    pq2 = _pq2()
    n, k, m = 32, 1024, 4
    w, _, _ = w4(n, k, 128, 8)
    x = activations(m, k, 5).float() * torch.tensor([1.0, 1e3, 1e8, 1e16])[:, None]
    q, xs = quantise(x, k)
    y, h = torch.empty((m, n), device=DEV), torch.empty((m, n), device=DEV)
    pq2.pq2_matmul_w4(q, xs, w, y, 128)
    pq2.pq2_gated_matmul_w4(q, xs, w, w, h, 128, act)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(h).all())
    far = y.abs() > 200
    assert bool(far.any())
    assert torch.equal(h[far], torch.where(y > 0, y * y, torch.zeros_like(y))[far].abs())


# ---------------------------------------------------------------- block norm
def rand(shape, seed, dtype, mul=1.0, add=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * mul + add).to(dtype)


NORM_CASES = [
    # m, k, r, block, w, x, post, gate, unit_offset, agroup
    (1, 128, "bf16", "f32", "bf16", "bf16", False, None, False, 128),
    (3, 5120, "bf16", "f32", "bf16", "bf16", True, "row", False, 128),
    (2, 1152, "f32", "f32", "f32", "bf16", True, "full", True, 32),
    (5, 384, "f16", "f16", "f16", "f16", False, "full", False, 64),
    (4, 8320, "bf16", "bf16", "f32", "f32", True, None, True, 128),
    (2, 17408, "f32", "bf16", "bf16", "f32", False, "row", False, 64),
    (1, 65536, "bf16", "f32", "bf16", "bf16", True, "full", False, 32),
    (3, 20480, "f16", "f32", "bf16", "bf16", True, "row", False, 128),
    (257, 640, "bf16", "f32", "bf16", "bf16", True, "full", False, 128),
    (3, 5120, "bf16", None, "bf16", "bf16", False, None, False, 128),
    (2, 256, "f32", None, "bf16", "f16", False, None, True, 32),
]


def check_norm(case, pad=0, shift=0, in_place=False, seed=1):
    m, k, r, b, w, x, post, gate, unit, ag = case
    pq2 = _pq2()

    def rows(t):
        """The rows of t inside a larger buffer: row stride k + pad, base shifted by `shift` elements."""
        wide = torch.full((m * (k + pad) + shift + 16,), 7.0, dtype=t.dtype, device=DEV)
        v = wide[shift:shift + m * (k + pad)].view(m, k + pad)[:, :k]
        v.copy_(t)
        return v
    rr = rand((m, k), seed, DT[r], 1.5)
    kw = {}
    if b:
        kw["block"] = rand((m, k), seed + 1, DT[b], 0.7)
    mean = 0.0 if unit else 1.0
    if post:
        kw["post_w"] = rand((k,), seed + 2, DT[w], 0.1, mean)
    if gate:
        kw["gate"] = rand((k,) if gate == "row" else (m, k), seed + 3, DT[w], 0.5)
    ww = rand((k,), seed + 4, DT[w], 0.1, mean)
    want_r, want_x = ref.block_norm(rr, ww, 1e-5, alpha=0.37, unit_offset=unit, x_dtype=DT[x], **kw)

    dev = {n: (rows(t) if t.dim() == 2 else t.to(DEV)) for n, t in kw.items()}
    rd = rows(rr)
    r_out = rd if in_place else rows(torch.full((m, k), float("nan"), dtype=DT[r]))
    x_out = rows(torch.full((m, k), float("nan"), dtype=DT[x]))
    q, xs = Guarded((m, k), torch.int8), Guarded((m, k // ag), torch.float32)
    pq2.pq2_block_norm(rd, ww.to(DEV), 1e-5, alpha=0.37, unit_offset=unit, r_out=r_out, x_out=x_out, q=q.t, xs=xs.t,
                       agroup=ag, **dev)
    torch.cuda.synchronize()
    assert torch.equal(r_out.cpu(), want_r), "r'"
    assert torch.equal(x_out.cpu(), want_x), "x"
    q2 = torch.empty((m, k), dtype=torch.int8, device=DEV)
    s2 = torch.empty((m, k // ag), dtype=torch.float32, device=DEV)
    pq2.pq2_quantize_act_i8_g(x_out, q2, s2, ag)
    assert torch.equal(q.read(), q2.cpu()) and torch.equal(xs.read(), s2.cpu())
    want_q, want_s = ref.quantised(want_x, k, ag)
    assert torch.equal(q2.cpu().double().view(m, -1, ag), want_q) and torch.equal(s2.cpu().double(), want_s)
    if pad:
        for t in (r_out, x_out):
            between = t.as_strided((m - 1, pad), (k + pad, 1), t.storage_offset() + k)
            assert bool((between == 7.0).all()), "wrote between the rows"


@pytest.mark.parametrize("case", NORM_CASES, ids=lambda c: "-".join(str(v) for v in c))
def test_block_norm_bits(case):
    announce(f"block norm {case}")
    check_norm(case)


def guarded_rows(m, k, pad, dtype, shift):
    """(m rows of k elements, the buffer they lie in, where they lie in it): poisoned rows, 64 elements of 42 in front of
    the first and behind the last, and 42 between them."""
    wide = torch.full((64 + shift + (m - 1) * (k + pad) + k + 64,), 42.0, dtype=dtype, device=DEV)
    where = (torch.arange(m)[:, None] * (k + pad) + torch.arange(k)[None, :] + 64 + shift).flatten()
    rows = wide.as_strided((m, k), (k + pad, 1), 64 + shift)
    rows.fill_(float("nan"))
    return rows, wide, where


@pytest.mark.parametrize("m,k", [(3, 128), (2, 5120), (800, 1152), (769, 2176), (2, 8320), (770, 9216), (3, 20480), (2, 33024),
                                 (2, 65536)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (0, 1), (3, 1)])
def test_block_norm_writes_its_rows_only(m, k, pad, shift):
    """Workgroups of one, two, four and eight chunks a thread, the last chunks partial: what lies in front of, between
    and behind the rows of r_out and x_out stays, as does what lies behind q and xs."""
    announce(f"block norm guards m={m} k={k} pad={pad} shift={shift}")
    r, b, w = rand((m, k), 1, torch.bfloat16), rand((m, k), 2, torch.float32), rand((k,), 3, torch.bfloat16, 0.1, 1)
    want_r, want_x = ref.block_norm(r, w, 1e-5, block=b, alpha=0.5, x_dtype=torch.float16)
    r_out, r_wide, where = guarded_rows(m, k, pad, torch.bfloat16, shift)
    x_out, x_wide, _ = guarded_rows(m, k, pad, torch.float16, shift)
    q, xs = Guarded((m, k), torch.int8), Guarded((m, k // 32), torch.float32)
    _pq2().pq2_block_norm(r.to(DEV), w.to(DEV), 1e-5, block=b.to(DEV), alpha=0.5, r_out=r_out, x_out=x_out, q=q.t, xs=xs.t,
                          agroup=32)
    q.read(), xs.read()
    assert torch.equal(r_out.cpu(), want_r) and torch.equal(x_out.cpu(), want_x)
    for wide in (r_wide, x_wide):
        rest = torch.ones(wide.numel(), dtype=torch.bool)
        rest[where] = False
        assert bool((wide.cpu()[rest] == 42).all()), "wrote outside its rows"


@pytest.mark.parametrize("pad,shift", [(8, 0), (16, 8), (3, 1), (0, 1), (5, 0)])
@pytest.mark.parametrize("case", NORM_CASES[1:4], ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}")
def test_block_norm_strides(case, pad, shift):
    announce(f"block norm pad={pad} shift={shift} {case}")
    check_norm(case, pad, shift)


@pytest.mark.parametrize("case", NORM_CASES[:5], ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}")
def test_block_norm_in_place(case):
    announce(f"block norm in place {case}")
    check_norm(case, in_place=True)


@pytest.mark.parametrize("m,k,pad", [(5, 1152, 0), (3, 640, 3), (800, 5120, 8)])
def test_block_norm_columns_of_one_buffer(m, k, pad):
    """Stream, block, gate and outputs side by side in the rows of one buffer."""
    announce(f"block norm columns of one buffer m={m} k={k} pad={pad}")
    pq2 = _pq2()
    wide = torch.full((m, 5 * k + pad), 7.0, dtype=torch.bfloat16, device=DEV)
    r, b, g, ro, xo = (wide[:, i * k:(i + 1) * k] for i in range(5))
    for i, t in enumerate((r, b, g)):
        t.copy_(rand((m, k), i, torch.bfloat16, 0.8))
    w = rand((k,), 5, torch.bfloat16, 0.1, 1)
    before = wide.cpu()
    want_r, want_x = ref.block_norm(before[:, :k], w, 1e-5, block=before[:, k:2 * k], post_w=w,
                                    gate=before[:, 2 * k:3 * k], alpha=0.5)
    pq2.pq2_block_norm(r, w.to(DEV), 1e-5, block=b, post_w=w.to(DEV), gate=g, alpha=0.5, r_out=ro, x_out=xo)
    torch.cuda.synchronize()
    after = wide.cpu()
    assert torch.equal(after[:, 3 * k:4 * k], want_r) and torch.equal(after[:, 4 * k:5 * k], want_x)
    assert torch.equal(after[:, :3 * k], before[:, :3 * k]) and bool((after[:, 5 * k:] == 7.0).all())


def test_block_norm_single_outputs():
    """Each output alone has the bits it has beside the others."""
    announce("block norm single outputs")
    pq2 = _pq2()
    m, k = 5, 1152
    r, b = rand((m, k), 1, torch.bfloat16).to(DEV), rand((m, k), 2, torch.float32).to(DEV)
    w = rand((k,), 3, torch.bfloat16, 0.1, 1).to(DEV)
    new = lambda dt: torch.empty((m, k), dtype=dt, device=DEV)  # noqa: E731
    ro, xo, q = new(torch.bfloat16), new(torch.bfloat16), new(torch.int8)
    xs = torch.empty((m, 9), device=DEV)
    pq2.pq2_block_norm(r, w, 1e-6, block=b, post_w=w, r_out=ro, x_out=xo, q=q, xs=xs)
    r1, x1, q1, s1 = new(torch.bfloat16), new(torch.bfloat16), new(torch.int8), torch.empty_like(xs)
    pq2.pq2_block_norm(r, w, 1e-6, block=b, post_w=w, r_out=r1)
    pq2.pq2_block_norm(r, w, 1e-6, block=b, post_w=w, x_out=x1)
    pq2.pq2_block_norm(r, w, 1e-6, block=b, post_w=w, q=q1, xs=s1)
    torch.cuda.synchronize()
    assert torch.equal(ro, r1) and torch.equal(xo, x1) and torch.equal(q, q1) and torch.equal(xs, s1)


@pytest.mark.parametrize("m,k", [(767, 2048), (768, 2048), (800, 1152), (770, 9216), (769, 128), (9, 33024)])
def test_block_norm_many_rows(m, k):
    """Both sides of the workgroup shape's rule, and rows of two to eight chunks a thread."""
    announce(f"block norm many rows m={m} k={k}")
    check_norm((m, k, "bf16", "f32", "bf16", "bf16", True, "row", False, 64))


def test_block_norm_zero_and_tiny_rows():
    announce("block norm zero and tiny rows")
    pq2 = _pq2()
    k = 384
    r = torch.zeros((4, k), dtype=torch.float32)
    r[1] = 2.0 ** -140
    r[2, 5] = 3e38
    r[3] = 1e-30
    w = torch.ones(k, dtype=torch.float32)
    want_r, want_x = ref.block_norm(r, w, 1e-6)
    x, q, xs = torch.empty((4, k), device=DEV), torch.empty((4, k), dtype=torch.int8, device=DEV), torch.empty((4, 3), device=DEV)
    pq2.pq2_block_norm(r.to(DEV), w.to(DEV), 1e-6, x_out=x, q=q, xs=xs)
    torch.cuda.synchronize()
    assert torch.equal(x.cpu(), want_x)
    want_q, want_s = ref.quantised(want_x, k)
    assert torch.equal(q.cpu().double().view(4, 3, 128), want_q) and torch.equal(xs.cpu().double(), want_s)


def test_block_norm_gate_broadcast_by_a_zero_stride():
    announce("block norm expanded gate")
    pq2 = _pq2()
    m, k = 6, 640
    r, b = rand((m, k), 1, torch.float16).to(DEV), rand((m, k), 2, torch.float32).to(DEV)
    w, g = rand((k,), 3, torch.float16, 0.1, 1).to(DEV), rand((k,), 4, torch.float16).to(DEV)
    a, c = torch.empty_like(r), torch.empty_like(r)
    pq2.pq2_block_norm(r, w, 1e-6, block=b, gate=g, x_out=a)
    pq2.pq2_block_norm(r, w, 1e-6, block=b, gate=g.expand(m, k), x_out=c)
    torch.cuda.synchronize()
    assert torch.equal(a, c)


# ---------------------------------------------------------------- together
class Block:
    """A feed-forward block between two norms, as a decoder runs it: gated
    product on ternary weights, down product on 4-bit weights."""

    def __init__(self, m, hidden, inner, wg, seed=1):
        pq2 = _pq2()
        self.m, self.wg = m, wg
        self.gate, self.raw_gate = ternary_tiles(inner, hidden, seed)
        self.up, self.raw_up = ternary_tiles(inner, hidden, seed + 1)
        self.down, self.c, self.s = w4(hidden, inner, wg, seed + 2)
        self.w_in, self.w_out, self.w_post = (rand((hidden,), seed + i, torch.bfloat16, 0.1, 1).to(DEV)
                                              for i in (3, 4, 5))
        e = lambda shape, dt: torch.empty(shape, dtype=dt, device=DEV)  # noqa: E731
        self.q, self.xs = e((m, hidden), torch.int8), e((m, hidden // 128), torch.float32)
        self.qh, self.xh = e((m, inner), torch.int8), e((m, inner // 128), torch.float32)
        self.h, self.y = e((m, inner), torch.bfloat16), e((m, hidden), torch.float32)
        self.r, self.x = e((m, hidden), torch.bfloat16), e((m, hidden), torch.bfloat16)

    def run(self, r, stream=None):
        pq2 = _pq2()
        pq2.pq2_block_norm(r, self.w_in, 1e-6, q=self.q, xs=self.xs, stream=stream)
        pq2.pq2_gated_matmul_tiles(self.q, self.xs, self.gate, self.up, self.h, stream=stream)
        pq2.pq2_linear_w4(self.h, self.down, self.y, self.wg, self.qh, self.xh, stream=stream)
        pq2.pq2_block_norm(r, self.w_out, 1e-6, block=self.y, post_w=self.w_post, alpha=0.5, r_out=self.r,
                           x_out=self.x, stream=stream)

    def check(self, r):
        """Every step against its reference on the step's own inputs."""
        torch.cuda.synchronize()
        hidden, inner = self.q.shape[1], self.qh.shape[1]
        _, x = ref.block_norm(r.cpu(), self.w_in.cpu(), 1e-6)
        q, xs = ref.quantised(x, hidden)
        assert torch.equal(self.q.cpu().double().view(q.shape), q) and torch.equal(self.xs.cpu().double(), xs)
        parts = [ref.product(q, xs, *ref.ternary(w, inner, hidden), 128) for w in (self.raw_gate, self.raw_up)]
        within(self.h.cpu(), *ref.gated(*parts[0], *parts[1], 0, torch.bfloat16), "h")
        within(self.y.cpu(), *ref.product(*ref.quantised(self.h.cpu(), inner), (self.c - 8).double(), self.s, self.wg),
               "y")
        want_r, want_x = ref.block_norm(r.cpu(), self.w_out.cpu(), 1e-6, block=self.y.cpu(),
                                        post_w=self.w_post.cpu(), alpha=0.5)
        assert torch.equal(self.r.cpu(), want_r) and torch.equal(self.x.cpu(), want_x)


@pytest.mark.parametrize("m", [1, 4, 16, 70, 300, 400])
def test_block_together(m):
    announce(f"block together m={m}")
    b = Block(m, 640, 1152, 32)
    r = rand((m, 640), 9, torch.bfloat16).to(DEV)
    b.run(r)
    b.check(r)


def test_block_on_another_stream():
    announce("block on a side stream")
    b = Block(3, 384, 512, 128)
    r = rand((3, 384), 9, torch.bfloat16).to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b.run(r, stream=side)
    side.synchronize()
    b.check(r)
    with torch.cuda.stream(side):
        b.r.zero_()
        b.run(r)
    side.synchronize()
    b.check(r)


@pytest.mark.parametrize("m", [2, 9, 40, 300, 400])
def test_block_captured_and_replayed(m):
    """Replays with new inputs, eager runs of the same buffers between them."""
    announce(f"block captured m={m}")
    b, eager = Block(m, 640, 1152, 64), Block(m, 640, 1152, 64)
    r = rand((m, 640), 9, torch.bfloat16).to(DEV)
    b.run(r)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run(r)
    for i in range(4):
        r.copy_(rand((m, 640), 20 + i, torch.bfloat16).to(DEV))
        graph.replay()
        eager.run(r)
        torch.cuda.synchronize()
        for name in ("q", "xs", "h", "y", "r", "x"):
            assert torch.equal(getattr(b, name), getattr(eager, name)), (i, name)
    b.check(r)
