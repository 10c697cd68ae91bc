"""The attention operators on the GPU where a single key, a scale or a rounding
decides (limits and their derivation in tests/attention_limits.py)."""
import functools

import pytest
import torch

import attention_limits as lim
import attention_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@functools.lru_cache(maxsize=None)
def _pq2():
    import gemm_int8_act_amd as pq2
    return pq2


def announce(msg):
    print(f"[gpu-case] {msg}", flush=True)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def starts_of(lengths):
    s = [0]
    for n in lengths:
        s.append(s[-1] + n)
    return ints(s)


def randn(shape, seed, scale=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale


def randint(lo, hi, shape, seed):
    return torch.randint(lo, hi + 1, shape, generator=torch.Generator().manual_seed(seed))


# ---------------------------------------------------------------- scales
@pytest.mark.parametrize("scale", [1.5e-45, 1e-40, 1.2e-38, 1.7e-38])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("d", ref.DIMS)
def test_smallest_scales(d, dt, scale):
    """Scales so small that every weight is 1: the mean of the values, exactly summed, over many tiles."""
    announce(f"smallest scales d={d} {dt} {scale}")
    pq2 = _pq2()
    # (The second: workgroups of eight waves, where there are any.)
    for n, heads, kv, causal in ((300, 4, 2, True), (4200, 32, 2, False)):
        q = randn((n, heads, d), 1).to(DT[dt]).to(DEV)
        k = randn((n, kv, d), 2).to(DT[dt]).to(DEV)
        v = randint(-100, 100, (n, kv, d), 3).to(DT[dt]).to(DEV)
        out = torch.full_like(q, float("nan"))
        s = starts_of([n])
        pq2.pq2_attention_prompt(q, k, v, out, s, s, causal=causal, scale=scale)
        torch.cuda.synchronize()
        seen = lim.seen_keys(n, n, 0, causal=causal, device=DEV)
        lim.check_counts(out, lim.mean_of_seen(v, seen, heads), DT[dt], f"prompt of {n}")
    cache = ref.make_cache(90, 16, 2, d, 4, DEV)
    ref.parts(cache, 16, 2, d)[3].fill_(2.0 ** -6)
    table = torch.arange(90, dtype=torch.int32, device=DEV).view(1, 90)
    q = randn((2, 8, d), 5).to(DT[dt]).to(DEV)
    out = torch.full_like(q, float("nan"))
    floats, words = pq2.pq2_attention_paged_workspace(1, 2, 8, 2, d, 1440)
    pq2.pq2_attention_paged(q, cache, table, ints([1400]), 16, out, torch.empty(floats, device=DEV),
                            torch.zeros(words, dtype=torch.int32, device=DEV), starts=ints([0, 2]), max_new=2, scale=scale)
    torch.cuda.synchronize()
    _, v, _ = ref.rows_of(cache, 16, 2, d, table[0], 1400)
    lim.check_counts(out, lim.mean_of_seen(v, lim.seen_keys(2, 1400, 1398, device=DEV), 8), DT[dt], "paged")


# ---------------------------------------------------------------- large max_new
@pytest.mark.parametrize("d", ref.DIMS)
@pytest.mark.parametrize("seqs,heads,kv,max_new", [(1, 64, 1, 1 << 20), (3, 16, 1, 1 << 20), (2, 15, 3, 1 << 19), (1, 1, 1, 1 << 24), (5, 24, 3, 5000)])
def test_paged_room_for_many_new_tokens(seqs, heads, kv, max_new, d):
    """Calls with room for far more new tokens than there are: nearly all their workgroups find no rows.  Fewer than
    eight places among them, whose row tiles go to all XCDs."""
    announce(f"paged max_new={max_new} seqs={seqs} heads={heads}/{kv} d={d}")
    lengths, new = [700, 45, 300, 16, 1][:seqs], [3, 1, 2, 0, 1][:seqs]
    page = 16
    cache = ref.make_cache(seqs * 44, page, kv, d, d, DEV)
    ref.parts(cache, page, kv, d)[3].fill_(2.0 ** -6)
    table = torch.arange(seqs * 44, dtype=torch.int32, device=DEV).view(seqs, 44)
    q = randn((sum(new), heads, d), 2).bfloat16().to(DEV)
    pq2 = _pq2()
    floats, words = pq2.pq2_attention_paged_workspace(seqs, max_new, heads, kv, d, 700)
    assert floats < 1 << 29
    work = torch.empty(floats, device=DEV), torch.zeros(words, dtype=torch.int32, device=DEV)
    zero, got = (torch.full_like(q, float("nan")) for _ in range(2))
    for x, out in ((torch.zeros_like(q), zero), (q, got)):
        pq2.pq2_attention_paged(x, cache, table, ints(lengths), page, out, *work, starts=starts_of(new), max_new=max_new, max_len=700)
    torch.cuda.synchronize()
    at = 0
    for i, (n, t) in enumerate(zip(lengths, new)):
        k, v, _ = ref.rows_of(cache, page, kv, d, table[i], n)
        seen = lim.seen_keys(t, n, n - t, device=DEV)
        if t:
            lim.check_counts(zero[at:at + t], lim.mean_of_seen(v, seen, heads), torch.bfloat16, f"sequence {i}")
            lim.check_norm(got[at:at + t], q[at:at + t], k, v, seen, scale=d ** -0.5, dtype=torch.bfloat16, paged=True, what=f"sequence {i}")
        at += t
