"""Plain 64-bit references of the block operators, and their error bounds.

y: every FP32 term float(dot) * ws * xs carries at most S + 1 roundings (S
weight groups per 128 activations) and is then part of at most G + 16 FP32
additions (G activation groups, 16 slices), so
    |y - exact| <= (G + S + 20) * 2^-24 * sum |xs * ws * dot|.
A gated output adds the activation's own error: expf within two units and the
division and products around it, with the exponent's relative error entering
times |z| (z the sigmoid's argument); |act'| <= 1.13 for SiLU and GELU.
"""
import math

import numpy as np
import torch

U24 = 2.0 ** -24


def make_w4(n, k, wg, seed, pad=0):
    """(codes uint8 [n][k/2 + pad], scales float16 [n][k/wg + pad], c int64 [n][k])."""
    gen = torch.Generator().manual_seed(seed)
    c = torch.randint(0, 16, (n, k), generator=gen, dtype=torch.uint8)
    codes = c[:, 0::2] | (c[:, 1::2] << 4)
    scales = (torch.rand((n, k // wg), generator=gen) * 0.045 + 0.005).to(torch.float16)
    if pad:
        codes = torch.cat([codes, torch.full((n, pad), 0xEE, dtype=torch.uint8)], 1)
        scales = torch.cat([scales, torch.full((n, pad), float("nan"), dtype=torch.float16)], 1)
    return codes.contiguous(), scales.contiguous(), c.long()


def w4_tiles(c, scales, wg):
    """The w4 tile layout as a scatter over single weights (uint8 tensor)."""
    n, k = c.shape
    s = 128 // wg
    t, s8 = (n + 15) // 16, (k + 1023) // 1024
    unit = 8192 + 256 * s
    nib = np.zeros((t * s8 * unit, 2), dtype=np.uint8)
    row, kk = np.meshgrid(np.arange(n), np.arange(k), indexing="ij")
    in_block = kk % 128
    lane = row % 16 + 16 * (in_block % 64 // 16)
    e = in_block % 16
    byte = ((row // 16 * s8 + kk // 1024) * unit + kk % 1024 // 128 * 1024 + 16 * lane + 8 * (in_block // 64)
            + 4 * (e // 8) + e % 4)
    nib[byte, e // 4 % 2] = (c.numpy() - 8) & 15
    out = nib[:, 0] | (nib[:, 1] << 4)
    view = out.view(np.uint16)
    g = np.arange(k // wg)
    rows = np.arange(n)[:, None]
    at = (rows // 16 * s8 + g // (8 * s)) * unit + 8192 + 16 * s * (rows % 16) + 2 * (g % (8 * s))
    view[at // 2] = scales[:, :k // wg].contiguous().view(torch.int16).numpy().view(np.uint16)
    return torch.from_numpy(out)


def quantised(x, k, group=128):
    """Codes and scales by the definition, as float64 [m][k/group][group] and [m][k/group]."""
    v = x[:, :k].double().reshape(x.shape[0], k // group, group)
    xs = (v.abs().amax(2) / 127).float().double()
    d = torch.where(xs > 0, xs, torch.ones_like(xs))
    q = (v / d[:, :, None]).float().double().round().clamp(-127, 127)
    return q, xs


def product(q, xs, weights, scales, wg):
    """(y, bound) [m][n] in float64: weights float64 [n][k] (c - 8 or c - 1), scales [n][k/wg]."""
    m, n = q.shape[0], weights.shape[0]
    k = weights.shape[1]
    s = 128 // wg
    qs = q.reshape(m, k // wg, wg).permute(1, 0, 2).contiguous()
    wt = weights.reshape(n, k // wg, wg).permute(1, 2, 0).contiguous()
    dots = torch.bmm(qs, wt)                                   # [k/wg][m][n], float64: exact
    terms = dots * xs.repeat_interleave(s, 1).t()[:, :, None] * scales[:, :k // wg].double().t()[:, None, :]
    return terms.sum(0), (k // 128 + s + 20) * U24 * terms.abs().sum(0) + 1e-30


def ternary(raw, n, k):
    """(weights float64 [n][k], scales [n][k/128]) of raw 34-byte blocks."""
    b = torch.from_numpy(np.ascontiguousarray(raw[:, :k // 128 * 34])).view(n, k // 128, 34)
    ws = b[:, :, :2].contiguous().view(torch.float16)[:, :, 0]
    c = b[:, :, 2:]
    w = torch.stack([c & 3, (c >> 2) & 3, (c >> 4) & 3, c >> 6], 3).reshape(n, k).double() - 1
    return w, ws


def gated(g, dg, u, du, act, dtype):
    """(h, bound) in float64 from the two products and their bounds."""
    z = g if act == 0 else 1.5957691216057308 * (g + 0.044715 * g ** 3)
    a = g * torch.sigmoid(z)
    da = 1.13 * dg + a.abs() * (8 + 8 * z.abs()) * U24
    h = a * u
    bound = da * (u.abs() + du) + a.abs() * du + h.abs() * 2 * U24
    half_step = torch.finfo(dtype).eps / 2
    return h, bound + (h.abs() + bound) * half_step + torch.finfo(dtype).tiny * torch.finfo(dtype).eps + 1e-30


def hard_quotients():
    """Every (x, d, M), x and d float32 with 1 <= d < 2, whose quotient q = x / d lies next to a border h + 1/2 of the codes
    (0 <= h <= 126) and so near the FP32 midpoint M beside it that quantise_bits might round it to the other side.

    Its t = RN(t0 + e y), with y = RN(1 / d), t0 = RN(x y), e = RN(x - t0 d), is RN(q + delta).  y is within 2^-24 of
    1 / d, relative; x y hence within one ulp of q and t0 within two.  e and y bring a relative error of 2^-24 each into
    e y ~ q - t0, so |delta| <= 2 ulp * 2^-23 * (1 + 2^-25).  t is RN(q) unless a midpoint lies between q and q + delta,
    and the code is that of RN(q) unless this midpoint is beside a border.  With M = M' 2^(m-24), M' odd and of 25 bits,
    d = D 2^-23 and x = X 2^(s+m-47), s = 24 or 25: x - M d = (X 2^s - M' D) 2^(m-47), and |q - M| <= |delta| leaves
    |X 2^s - M' D| < 8: zero never (M' is odd, D of at most 24 bits), so for each M and s seven values of either sign,
    each with one D modulo 2^s."""
    x, d, mids = [], [], []
    for h in range(127):
        border = np.float32(h + 0.5)
        for side in (np.float32(0), np.float32(1000)):
            mid = (float(border) + float(np.nextafter(border, side))) / 2
            e = math.frexp(mid)[1] - 1
            big = int(math.ldexp(mid, 24 - e))
            assert big % 2 == 1 and 1 << 24 <= big < 1 << 25
            for s in (24, 25):
                inverse = pow(big, -1, 1 << s)
                for rest in (r for r in range(-7, 8) if r):
                    den = -rest * inverse % (1 << s)
                    num = (rest + big * den) >> s
                    if 1 << 23 <= den < 1 << 24 and 1 << 23 <= num <= 1 << 24:
                        d.append(math.ldexp(den, -23))
                        x.append(math.ldexp(num, s + e - 47))
                        mids.append(mid)
    return np.array(x), np.array(d), np.array(mids)


def block_norm(r, w, eps, block=None, post_w=None, gate=None, alpha=1.0, unit_offset=False, x_dtype=None):
    """(r', x) on the CPU: single FP32 operations, sums in FP64."""
    def rstd(v):
        return (1 / torch.sqrt(v.double().square().sum(1, keepdim=True) / v.shape[1] + eps)).float()

    def weight(t):
        return 1 + t.float() if unit_offset else t.float()
    if block is not None:
        t = block.float()
        if post_w is not None:
            t = t * rstd(t) * weight(post_w)
        if gate is not None:
            t = t * gate.float()
        t = t * torch.tensor(alpha, dtype=torch.float32)
        r = (r.float() + t).to(r.dtype)
    v = r.float()
    return r, (v * rstd(v) * weight(w)).to(x_dtype or r.dtype)
