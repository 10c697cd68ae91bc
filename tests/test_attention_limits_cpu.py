"""The limits of tests/attention_limits.py see a key that is missing or counted twice, and accept correctly rounded results."""
import pytest
import torch

import attention_limits as lim
import attention_reference as ref

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def case(n, d, dt):
    gen = torch.Generator().manual_seed(n + d)
    q = torch.randn((2, 4, d), generator=gen).mul(1.2).to(DT[dt])
    k = torch.randn((n, 2, d), generator=gen).to(DT[dt])
    v = torch.randint(-127, 128, (n, 2, d), generator=gen).double() / 64
    return q, k, v


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("d", ref.DIMS)
@pytest.mark.parametrize("n,lost", [(33, 32), (700, 255), (5000, 4999), (6000, 255), (33000, 2048)])
def test_counts_see_one_key(n, lost, d, dt):
    _, _, v = case(n, d, dt)
    seen = lim.seen_keys(2, n, n - 2)
    mean = lim.mean_of_seen(v, seen, 4)
    lim.check_counts(mean.to(DT[dt]), mean, DT[dt], "whole")
    less, total = seen.clone(), seen.sum(1)[:, None, None].double()
    less[:, lost] = False
    if int((less != seen).sum()) == 0:
        return
    for wrong in (lim.mean_of_seen(v, less, 4),                                            # not seen at all
                  lim.mean_of_seen(v, less, 4) * (total - 1) / total,                      # its value dropped
                  (mean * total + (mean * total - lim.mean_of_seen(v, less, 4) * (total - 1))) / (total + 1)):  # twice
        with pytest.raises(AssertionError):
            lim.check_counts(wrong.to(DT[dt]), mean, DT[dt], "one key off")


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("d", ref.DIMS)
@pytest.mark.parametrize("n,lost", [(700, slice(255, 256)), (6000, slice(255, 256)), (5000, slice(16, 32)), (5000, slice(4984, 5000))])
def test_norms_see_lost_keys(n, lost, d, dt, paged):
    """One ordinary key, or a half step of them; of a prompt in bf16, whose weights are rounded to 8 bits, four keys."""
    q, k, v = case(n, d, dt)
    if not paged:
        v = v.to(DT[dt])
    seen = lim.seen_keys(2, n, n - 1)
    args = dict(scale=d ** -0.5, dtype=DT[dt], paged=paged)
    o, _, _ = lim.exact_and_spread(q, k, v, seen, d ** -0.5)
    lim.check_norm(o.to(DT[dt]), q, k, v, seen, what="whole", **args)
    less = seen.clone()
    less[:, lost] = False
    if not paged and dt == "bf16" and lost.stop - lost.start == 1:
        less[:, lost.start:lost.start + 4] = False
    wrong, _, _ = lim.exact_and_spread(q, k, v, less, d ** -0.5)
    with pytest.raises(AssertionError):
        lim.check_norm(wrong.to(DT[dt]), q, k, v, seen, what="keys lost", **args)
