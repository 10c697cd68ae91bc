"""Plain references of the attention operators, and their error bounds.

The cache's codes and scales, and everything that pq2_kv_write and pq2_kv_read
put out, follow from single FP32 operations: the references below give the
same bits.

Attention is computed in 64 bits.  Bounds, with u = 2^-24 and half = eps / 2 of
the 16-bit type:
- a score is a sum of head_dim exact products in FP32 (products of two 8- or
  11-bit numbers are exact), scaled with at most four roundings: off by at
  most d_j = (head_dim + 4) u A_j + 4 u |s_j|, A_j = scale * sum |q k_j|;
  paged: the products are q (c + 1152), |c + 1152| <= 1279, with 1152 sum q taken off, so that A_j is joined by
  2 * 1279 / 127 * scale * max|k_j| * sum |q|, a bound for the worst order of signs (for random ones the
  norm of the whole error is held to that of the last rounding);
- a weight exp(s_j - m), with the subtraction and exp2 (two units), is then
  off by e_j = d_j + d_m + 8 u + 2 u (|s_j| + |m|) of itself, d_m the same bound of the row's largest A;
- paged: the weight times the value's scale is kept as two bf16, 2^-16 of itself
  at most (half a step of the second, on a remainder of half a step of the first, is 2^-18);
  prompt: it is rounded to the 16-bit type, half of itself, or, as an fp16 below the
  normal range, 2^-25 where the row's largest weight is 1;
- sums run over at most 256 + n / 32 roundings from one end to the other (a step
  takes 64 or 256 keys, with a rescaling and two products; 128 parts and 8 waves at most are joined);
- o = sum w v / sum w is then off by at most (e + sums) (sum w |v| + |o|), and rounded once.
"""
import torch

U = 2.0 ** -24
DIMS = (64, 128, 256)


def parts(cache, page, kv, d):
    """Views of a cache: key codes, value codes [pages][kv][page][d], key scales, value scales [pages][kv][page]."""
    c = cache.view(cache.shape[0], kv, page * (2 * d + 8))
    codes = c[:, :, :2 * page * d].view(torch.int8).unflatten(2, (2, page, d))
    scales = c[:, :, 2 * page * d:].view(torch.float32).unflatten(2, (2, page))
    return codes[:, :, 0], codes[:, :, 1], scales[:, :, 0], scales[:, :, 1]


def rotated(x, cos, sin, positions, interleaved):
    """x [m][heads][d] in FP32 with its first elements rotated, single FP32 operations."""
    x = x.float().clone()
    if cos is None:
        return x
    half = cos.shape[1]
    p = positions.long().clamp(0, cos.shape[0] - 1)
    c, s = cos[p][:, None], sin[p][:, None]
    i = torch.arange(half)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = x[..., first], x[..., second]
    x[..., first], x[..., second] = a * c - b * s, b * c + a * s
    return x


def codes(x):
    """(int8 codes, float32 scales) of rows, by the definition."""
    v = x.double()
    scale = (v.abs().amax(-1) / 127).float()
    by = torch.where(scale > 0, scale, torch.ones_like(scale)).double()
    return (v / by[..., None]).float().double().round().clamp(-127, 127).to(torch.int8), scale


def tables(rows, rot, base=1e4):
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    angle = torch.arange(rows, dtype=torch.float64)[:, None] * freq
    return angle.cos().float(), angle.sin().float()


def make_cache(pages, page, kv, d, seed, device):
    """Random codes, scales about 1/45."""
    gen = torch.Generator().manual_seed(seed)
    cache = torch.zeros((pages, kv * page * (2 * d + 8)), dtype=torch.uint8)
    kc, vc, ks, vs = parts(cache, page, kv, d)
    for c in (kc, vc):
        c.copy_(torch.randint(-127, 128, c.shape, generator=gen, dtype=torch.int8))
    for s in (ks, vs):
        s.copy_((torch.rand(s.shape, generator=gen) + 0.5) / 70)
    return cache.to(device)


def rows_of(cache, page, kv, d, table_row, length):
    """Keys and values [length][kv][d] of one sequence in float64 (codes * scales), and which tokens are there."""
    kc, vc, ks, vs = parts(cache, page, kv, d)
    t = torch.arange(length, device=cache.device)
    idx = t // page
    inside = idx < table_row.shape[0]
    pg = table_row.long()[idx.clamp(max=table_row.shape[0] - 1)]
    there = inside & (pg >= 0) & (pg < cache.shape[0])
    pg = torch.where(there, pg, torch.zeros_like(pg))
    at = t % page
    return [(c[pg, :, at].double() * s[pg, :, at].double()[..., None]) for c, s in ((kc, ks), (vc, vs))] + [there]


def attention(q, k, v, first, *, scale, causal=True, window=0, there=None, paged=False, dtype):
    """(o, bound) [n][heads][d] in float64: queries q at positions first, first + 1, ... among the keys."""
    n, heads, d = q.shape
    o = torch.zeros((n, heads, d), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(o)
    nk = k.shape[0]
    half = torch.finfo(dtype).eps / 2
    if not n or not nk:
        return o, bound + 1e-30
    gap = first + torch.arange(n, device=q.device)[:, None] - torch.arange(nk, device=q.device)[None]
    seen = gap >= 0 if causal else torch.ones_like(gap, dtype=torch.bool)
    if window:
        seen = seen & (gap < window)
    if there is not None:
        seen = seen & there[None]
    some = seen.any(1)
    inf = float("inf")
    for h in range(heads):
        g = h // (heads // k.shape[1])
        qh, kh, vh = q[:, h].double(), k[:, g].double(), v[:, g].double()
        s = (qh @ kh.t().contiguous()) * scale
        a = (qh.abs() @ kh.abs().t().contiguous()) * scale
        s = torch.where(seen, s, torch.full_like(s, -inf))
        a = torch.where(seen, a, torch.zeros_like(a))
        top = torch.where(some, s.amax(1), torch.zeros_like(s[:, 0]))
        w = torch.exp(s - top[:, None])
        total = w.sum(1).clamp(min=1e-300)
        sa = torch.where(seen, s.abs(), torch.zeros_like(s))
        if paged:
            a = a + 20.2 * scale * qh.abs().sum(1)[:, None] * kh.abs().amax(1)[None]
        dj = (d + 4) * U * a + 4 * U * sa
        e = dj + dj.amax(1, keepdim=True) + 8 * U + 2 * U * (sa + top.abs()[:, None]) + (256 + nk / 32) * U
        e = e + (2.0 ** -16 if paged else half)
        vv = torch.where(seen.any(0)[:, None], vh, torch.zeros_like(vh))
        oh = (w @ vv) / total[:, None]
        spread = ((w * e) @ vv.abs()) / total[:, None] + oh.abs() * ((w * e).sum(1) / total)[:, None]
        if not paged and dtype == torch.float16:
            spread = spread + (seen.double() * 2.0 ** -25) @ (vv.abs() + oh.abs().amax()) / total[:, None]
        o[:, h] = oh
        bound[:, h] = spread + (oh.abs() + spread) * half + torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    return o, bound + 1e-30
