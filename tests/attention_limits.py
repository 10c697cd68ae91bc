"""Limits of the attention tests that see a single lost or doubled key.

Counting.  With queries of zero every score is 0 and every weight 1, and with
values that are small integers times one power of two every product and sum is
an integer below 2^24 times that power: exact in FP32, in whatever order and
however the keys are split.  The result is the mean of the values that a row
sees, with one rounding each of 1 / n, of the product and of the output:

    |o - mean| <= (half + 4 u) |mean| + the type's smallest subnormal / 2

u = 2^-24, half = eps / 2 of the output's type.  A key that is missing or
counted twice moves every column by |v - mean| / n, which is 1 / sqrt(n) of the
mean's typical size: seen up to some 100 000 keys.

Norms.  Over a sequence's outputs, the last rounding is off by at most half |o|.
The keys' own errors (of a score, of a rounded weight) are independent, e of
the weight each: they move o by about e sqrt(sum w^2 (v - o)^2) / sum w, taken
twice here (as if four keys in a row erred alike).  FP32 sums err by u of the
running sum a step, sqrt(steps) u |o| together: less than 2^-16 |o| for up to 2^16
steps.  So

    |got - o| <= (half + 2^-16) |o| + 2 e |sqrt(sum w^2 (v - o)^2) / sum w|

with e = half for prompts, whose weights are rounded to the type, and over the
pages 2^-17 (a weight as two bf16) plus what a score is off, 2 sqrt(d) u A: d
roundings of at most u of the sum's largest magnitude A = scale * max sum |q k|,
as a random walk, with four sigma for the largest of them in place of one in
two places.  A lost key of n is about 1 / sqrt(n) of |o|.
"""
import torch

U = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


def seen_keys(n, nk, first, *, causal=True, window=0, there=None, device=None):
    """[n][nk]: the keys that queries at positions first, first + 1, ... see."""
    gap = first + torch.arange(n, device=device)[:, None] - torch.arange(nk, device=device)[None]
    seen = gap >= 0 if causal else torch.ones_like(gap, dtype=torch.bool)
    if window:
        seen = seen & (gap < window)
    return seen if there is None else seen & there[None]


def mean_of_seen(v, seen, heads):
    """[n][heads][d] in float64: the mean of the values that each row sees, zero where it sees none."""
    nk, kv, d = v.shape
    total = (seen.double() @ v.double().reshape(nk, kv * d)).view(seen.shape[0], kv, d)
    mean = total / seen.sum(1).clamp(min=1).double()[:, None, None]
    return mean.repeat_interleave(heads // kv, 1)


def check_counts(got, mean, dtype, what):
    got = got.double()
    assert bool(torch.isfinite(got).all()), f"{what}: non-finite output"
    bound = (half(dtype) + 4 * U) * mean.abs() + torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2
    over = (got - mean).abs() - bound
    worst = int(over.argmax())
    assert float(over.max()) <= 0, (f"{what}: {float(got.flatten()[worst])!r} instead of {float(mean.flatten()[worst])!r} at "
                                    f"{worst}, {int((over > 0).sum())} of {over.numel()} off")


def exact_and_spread(q, k, v, seen, scale):
    """(o, sqrt(sum w^2 (v - o)^2) / sum w [n][heads][d], the largest A) in float64."""
    n, heads, d = q.shape
    o = torch.zeros((n, heads, d), dtype=torch.float64, device=q.device)
    spread = torch.zeros_like(o)
    largest = 0.0
    some = seen.any(1)
    for h in range(heads):
        g = h // (heads // k.shape[1])
        qh, kh, vh = q[:, h].double(), k[:, g].double(), v[:, g].double()
        kt = kh.t().contiguous()
        s = (qh @ kt) * scale
        s = torch.where(seen, s, torch.full_like(s, -float("inf")))
        top = torch.where(some, s.amax(1), torch.zeros_like(s[:, 0]))
        w = torch.exp(s - top[:, None])
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        vh = torch.where(seen.any(0)[:, None], vh, torch.zeros_like(vh))
        o[:, h] = w @ vh
        w2 = w * w
        spread[:, h] = (w2 @ (vh * vh) - 2 * o[:, h] * (w2 @ vh) + o[:, h] ** 2 * w2.sum(1, keepdim=True)).clamp(min=0).sqrt()
        a = (qh.abs() @ kt.abs()) * scale
        largest = max(largest, float(torch.where(seen, a, torch.zeros_like(a)).max()))
    return o, spread, largest


def check_norm(got, q, k, v, seen, *, scale, dtype, paged, what):
    """One sequence's outputs [n][heads][d] against the limit above."""
    got = got.double()
    assert bool(torch.isfinite(got).all()), f"{what}: non-finite output"
    if not seen.numel():
        assert not bool(got.any()), what
        return
    o, spread, largest = exact_and_spread(q, k, v, seen, scale)
    e = 2.0 ** -17 + 2 * q.shape[2] ** 0.5 * U * largest if paged else half(dtype)
    limit = (half(dtype) + 2.0 ** -16) * float(o.norm()) + 2 * e * float(spread.norm()) + 1e-30
    if not paged and dtype == torch.float16:
        # Weights below the normal range of fp16 are off by at most 2^-32 where the row's largest is 1.
        limit += 2.0 ** -32 * v.shape[0] ** 0.5 * float(o.numel() ** 0.5 * v.double().abs().nan_to_num(0.0, 0.0, 0.0).max())
    off = float((got - o).norm())
    assert off <= limit, f"{what}: off by {off:.3e} in the norm, limit {limit:.3e} ({off / float(o.norm()):.2e} of it)"
