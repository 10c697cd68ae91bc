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


# ---------------------------------------------------------------- scores over the pages
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("d", ref.DIMS)
def test_paged_scores_of_queries_with_an_offset(d, dt):
    """Queries with a common offset, as projections with a bias give them, and keys with an outlier channel, whose other
    codes are small: scores are off by no more than FP32 sums of q k are."""
    announce(f"paged, queries with an offset d={d} {dt}")
    pq2 = _pq2()
    heads, kv, page, lengths = 16, 2, 16, [300, 77, 1000]
    width = 63
    cache = ref.make_cache(3 * width, page, kv, d, 6, DEV)
    kc, _, ks, _ = ref.parts(cache, page, kv, d)
    small = (randn(kc.shape, 7) * 5).round().clamp(-127, 127)
    small[..., 3] = 127 * randint(0, 1, kc.shape[:-1], 8) * 2 - 127
    kc.copy_(small.to(torch.int8))
    ks.fill_(0.25)
    table = torch.arange(3 * width, dtype=torch.int32, device=DEV).view(3, width)
    sign = 2.0 * randint(0, 1, (1, heads, 1), 9) - 1
    q = randn((3, heads, d), 10) + 8 * sign
    q[..., 3] = 0.1
    q = q.to(DT[dt]).to(DEV)
    out = torch.full_like(q, float("nan"))
    floats, words = pq2.pq2_attention_paged_workspace(3, 1, heads, kv, d, width * page)
    pq2.pq2_attention_paged(q, cache, table, ints(lengths), page, out, torch.empty(floats, device=DEV),
                            torch.zeros(words, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    for i, n in enumerate(lengths):
        k, v, _ = ref.rows_of(cache, page, kv, d, table[i], n)
        seen = lim.seen_keys(1, n, n - 1, device=DEV)
        o, spread, largest = lim.exact_and_spread(q[i:i + 1], k, v, seen, d ** -0.5)
        print(f"  n={n} off {float((out[i:i + 1].double() - o).norm() / o.norm()):.2e} A={largest:.1f}", flush=True)
        lim.check_norm(out[i:i + 1], q[i:i + 1], k, v, seen, scale=d ** -0.5, dtype=DT[dt], paged=True, what=f"sequence {i}")


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("d", ref.DIMS)
def test_paged_elements_far_below_the_largest(d, dt):
    """Elements of q between 2^-24 and 2^-14 of the row's largest count as multiples of 2^-24 of it: here they alone make
    the scores, the largest meets codes of zero."""
    announce(f"paged, small elements of q d={d} {dt}")
    pq2 = _pq2()
    heads, page, n = 8, 16, 130
    cache = ref.make_cache(9, page, 1, d, 6, DEV)
    kc, _, ks, _ = ref.parts(cache, page, 1, d)
    kc[..., 5] = 0
    ks.fill_(2.0 ** 8)
    table = torch.arange(9, dtype=torch.int32, device=DEV).view(1, 9)
    q = (randint(-31, 31, (1, heads, d), 9) * 2.0 ** -22).to(DT[dt]).to(DEV)     # multiples of 2^-24 of 1
    q[..., 5] = 1.0
    out = torch.full_like(q, float("nan"))
    pq2.pq2_attention_paged(q, cache, table, ints([n]), page, out, max_len=144, scale=0.5)
    torch.cuda.synchronize()
    k, v, _ = ref.rows_of(cache, page, 1, d, table[0], n)
    lim.check_norm(out, q, k, v, lim.seen_keys(1, n, n - 1, device=DEV), scale=0.5, dtype=DT[dt], paged=True, what="o")


# ---------------------------------------------------------------- small weights of prompts
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("d", ref.DIMS)
@pytest.mark.parametrize("below", [14, 15, 16, 18, 20, 23, 24, 25, 26, 28, 30])
def test_prompt_weights_far_below_the_largest(below, d, dt):
    """One leading key whose value is zero, thousands of others with weights 2^-below of its: the output is theirs alone.
    Weights are powers of two (the scale is ln 2), exact in 16 bits as far as they reach; the sums err by at most n u, the
    scores by 4 roundings of `below`."""
    announce(f"prompt, weights 2^-{below} d={d} {dt}")
    pq2 = _pq2()
    for n, nq, heads, kv in ((4000, 40, 2, 1), (8200, 4100, 32, 1)):      # the second: eight waves
        if nq > 1000 and below not in (16, 26):
            continue
        for lead in (0, n - 5, n // 2):
            q = torch.zeros((nq, heads, d), dtype=DT[dt], device=DEV)
            q[..., 0] = 1.0
            k = randn((n, kv, d), 2).to(DT[dt]).to(DEV)
            k[..., 0] = -below
            k[lead, :, 0] = 0.0
            v = randint(100, 250, (n, kv, d), 3).to(DT[dt]).to(DEV)
            v[lead] = 0.0
            out = torch.full_like(q, float("nan"))
            pq2.pq2_attention_prompt(q, k, v, out, starts_of([nq]), starts_of([n]), causal=False, scale=0.6931471805599453)
            torch.cuda.synchronize()
            w = 2.0 ** -below
            want = (v.double().sum(0) * w / (1 + (n - 1) * w)).repeat_interleave(heads // kv, 0)[None]
            limit = (lim.half(DT[dt]) + (n + 16 + 8 * below) * lim.U) * want
            over = (out.double() - want).abs() - limit
            assert float(over.max()) <= 0, (f"n={n} leading key {lead}: {float(out[0, 0, 0])!r} instead of {float(want[0, 0, 0])!r}")


# ---------------------------------------------------------------- every key, once
PAGES = [
    # lengths, new tokens, heads, kv, page, window, more
    ([1], [1], 1, 1, 16, 0, {}),
    ([0, 1, 2, 15, 16, 17, 31, 32, 33, 255, 256, 257], [1] * 12, 8, 2, 16, 0, {}),
    ([517, 700, 2000], [1, 1, 1], 10, 2, 16, 0, {}),
    ([700, 90, 1500], [2, 1, 3], 6, 2, 16, 0, dict(bad_page=True)),
    ([6000, 3], [1, 1], 4, 2, 32, 0, dict(max_len=600)),
    ([600, 3], [1, 1], 4, 2, 32, 0, dict(max_len=100000, max_new=5)),
    ([700, 100, 490], [4, 3, 2], 4, 2, 16, 0, dict(table_pages=30)),
    ([700, 100, 490], [4, 3, 2], 4, 2, 16, 250, dict(table_pages=30)),
    ([600, 20, 3, 0], [16, 9, 5, 2], 10, 2, 64, 0, {}),
    ([3000, 100, 7], [4, 7, 1], 24, 4, 32, 0, {}),
    ([1000, 900], [2, 1], 34, 2, 64, 0, {}),
    ([4000, 300, 50], [3, 1, 8], 5, 5, 128, 100, {}),
    ([9000, 40], [8, 8], 8, 1, 256, 1024, {}),
    ([2500, 2500], [1, 0], 16, 2, 16, 1, {}),
    ([20000, 17, 9000], [1, 1, 1], 8, 8, 32, 0, {}),
    ([33000], [1], 16, 2, 64, 0, {}),
    ([70000], [1], 4, 1, 256, 0, {}),
    ([5000 if i == 3 else 2600 if i == 70 else 4100 if i == 149 else 7 * i * i % 300 for i in range(150)],
     [1 + i % 3 if i % 11 else 0 for i in range(150)], 4, 2, 16, 0, {}),
]


def paged_call(lengths, new, heads, kv, d, page, dt, window, q, cache, table, max_new=None, max_len=None, scale=None):
    pq2 = _pq2()
    out = torch.full_like(q, float("nan"))
    max_new, max_len = max_new or max(max(new), 1), max_len or max(1, max(lengths))
    floats, words = pq2.pq2_attention_paged_workspace(len(lengths), max_new, heads, kv, d, max_len)
    pq2.pq2_attention_paged(q, cache, table, ints(lengths), page, out, torch.full((floats,), float("nan"), device=DEV),
                            torch.zeros(words, dtype=torch.int32, device=DEV), starts=starts_of(new), max_new=max_new, max_len=max_len,
                            window=window, scale=scale)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("d", ref.DIMS)
@pytest.mark.parametrize("lengths,new,heads,kv,page,window,more", PAGES)
def test_paged_every_key_once(lengths, new, heads, kv, page, window, more, d, dt):
    """Every key of a row counts once (queries of zero), and with ordinary queries no sequence's norm misses one."""
    announce(f"paged counts lengths={lengths[:12]} new={new[:8]} heads={heads}/{kv} d={d} page={page} {dt} window={window} {more}")
    more = dict(more)
    width = max(1, max((n + page - 1) // page for n in lengths))
    pages = len(lengths) * width + 3
    cache = ref.make_cache(pages, page, kv, d, d + 1, DEV)
    _, _, ks, vs = ref.parts(cache, page, kv, d)
    vs.fill_(2.0 ** -6)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(5))[:len(lengths) * width].to(torch.int32).view(-1, width).to(DEV)
    for i, n in enumerate(lengths):                 # behind the lengths: anything
        last = table[i, n // page:].long() if n % page == 0 else table[i, n // page + 1:].long()
        ks[last], vs[last] = float("nan"), float("inf")
        if n % page:
            ks[int(table[i, n // page]), :, n % page:], vs[int(table[i, n // page]), :, n % page:] = float("nan"), float("inf")
    if more.pop("bad_page", False):
        table[0, 0], table[-1, -1] = -1, pages
    table = table[:, :more.pop("table_pages", width)]
    rows = sum(new)
    q = randn((rows, heads, d), 9, 1.2).to(DT[dt]).to(DEV)
    zero, got = (paged_call(lengths, new, heads, kv, d, page, dt, window, x, cache, table, **more) for x in (torch.zeros_like(q), q))
    at = 0
    for i, (n, t) in enumerate(zip(lengths, new)):
        k, v, there = ref.rows_of(cache, page, kv, d, table[i], n)
        k, v = (torch.where(there[:, None, None], x, torch.zeros_like(x)) for x in (k, v))
        seen = lim.seen_keys(t, n, n - t, window=window, there=there, device=DEV)
        if t:
            lim.check_counts(zero[at:at + t], lim.mean_of_seen(v, seen, heads), DT[dt], f"sequence {i}")
            if len(lengths) < 100 or n > 2000 or i % 10 == 1:
                lim.check_norm(got[at:at + t], q[at:at + t], k, v, seen, scale=d ** -0.5, dtype=DT[dt], paged=True, what=f"sequence {i}")
        at += t


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("d", ref.DIMS)
@pytest.mark.parametrize("n,page,max_len", [(300, 16, 300), (2000, 32, 2000), (5000, 64, 5000), (5000, 16, 300), (40000, 256, 40000)])
def test_paged_needles(n, page, max_len, d, dt):
    """Each head's query is one key's codes, and its output that key's value: at the edges of pages, tiles, steps and
    parts.  The key's score leads by far more than ln n, so that all but the last rounding is below 2^-8 of the largest value."""
    announce(f"paged needles n={n} page={page} d={d} {dt}")
    heads, kv = 64, 4
    width = (n + page - 1) // page
    cache = ref.make_cache(width, page, kv, d, 3, DEV)
    kc, vc, ks, vs = ref.parts(cache, page, kv, d)
    ks.fill_(1.0 / 64)
    vs.fill_(1.0 / 64)
    table = torch.randperm(width, generator=torch.Generator().manual_seed(4)).to(torch.int32).view(1, -1).to(DEV)
    edges = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 127, 128, 129, 255, 256, 257, 383, 384, 511, 512, 1023, 1024, 2047, 2048, 4095, 4096]
    edges = [e for e in edges if e < n] + [n - 1, n - 2, n // 2, (n - 1) // 128 * 128, (n - 1) // page * page, (n - 1) // page * page - 1]
    at = torch.tensor((edges * heads)[:heads], device=DEV)
    k, v, _ = ref.rows_of(cache, page, kv, d, table[0], n)
    g = torch.arange(heads, device=DEV) // (heads // kv)
    q = k[at, g][None].to(DT[dt])
    got = paged_call([n], [1], heads, kv, d, page, dt, 0, q, cache, table, max_len=max_len, scale=4 / d ** 0.5)
    assert float((got[0].double() - v[at, g]).abs().max()) <= 2 * 2.0 ** -8 * float(v.abs().max())


PROMPTS = [
    # queries, keys, heads, kv, causal, window
    ([1], [1], 1, 1, True, 0),
    ([64, 1, 0, 129, 65, 31], [64, 1, 0, 129, 65, 31], 4, 2, True, 0),
    ([5, 100, 130, 0], [300, 100, 513, 70], 6, 2, True, 0),
    ([40, 90], [7, 0], 2, 1, True, 0),
    ([300, 77], [300, 500], 4, 4, False, 0),
    ([10, 3], [0, 65], 4, 1, False, 0),
    ([700, 20], [700, 400], 5, 1, True, 100),
    ([300, 150], [333, 150], 2, 2, True, 1),
    ([3] * 150, [4] * 150, 2, 1, True, 0),
    ([4100, 100], [8300, 133], 32, 4, True, 3000),
    ([4200], [4200], 32, 2, True, 0),
]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("d", ref.DIMS)
@pytest.mark.parametrize("nq,nk,heads,kv,causal,window", PROMPTS)
def test_prompt_every_key_once(nq, nk, heads, kv, causal, window, d, dt):
    announce(f"prompt counts nq={nq[:6]} nk={nk[:6]} heads={heads}/{kv} d={d} {dt} causal={causal} window={window}")
    pq2 = _pq2()
    rq, rk = sum(nq), max(1, sum(nk))
    q = randn((rq, heads, d), d, 1.2).to(DT[dt]).to(DEV)
    k = randn((rk, kv, d), d + 1).to(DT[dt]).to(DEV)
    v = randint(-127, 127, (rk, kv, d), d + 2).to(DT[dt]).to(DEV)
    zero, got = (torch.full_like(q, 7.0) for _ in range(2))
    for x, out in ((torch.zeros_like(q), zero), (q, got)):
        pq2.pq2_attention_prompt(x, k, v, out, starts_of(nq), starts_of(nk), causal=causal, window=window)
    torch.cuda.synchronize()
    a = b = 0
    for i, (n, m) in enumerate(zip(nq, nk)):
        seen = lim.seen_keys(n, m, m - n, causal=causal, window=window, device=DEV)
        if n:
            lim.check_counts(zero[a:a + n], lim.mean_of_seen(v[b:b + m], seen, heads), DT[dt], f"sequence {i}")
            if n < 1000 or d == 128:
                lim.check_norm(got[a:a + n], q[a:a + n], k[b:b + m], v[b:b + m], seen, scale=d ** -0.5, dtype=DT[dt], paged=False,
                               what=f"sequence {i}")
        a, b = a + n, b + m


# ---------------------------------------------------------------- large scores
@pytest.mark.parametrize("dt,size", [("f16", 30.0), ("f16", 1000.0), ("f16", 15000.0), ("bf16", 1000.0), ("bf16", 1e6), ("bf16", 1e15)])
@pytest.mark.parametrize("d", ref.DIMS)
def test_large_scores(d, dt, size):
    """Scores from 1e3 to 1e30 times ln 2, far apart: rows whose largest leads by more than FP32 sums may be off, and by 40, are
    that key's value."""
    announce(f"large scores d={d} {dt} {size}")
    pq2 = _pq2()
    for n, heads, kv, causal in ((300, 4, 2, True), (4200, 32, 2, False)):
        q, k = ((randn((n, h, d), i).clamp(-4, 4) * size).to(DT[dt]).to(DEV) for i, h in ((1, heads), (2, kv)))
        v = randint(-100, 100, (n, kv, d), 3).to(DT[dt]).to(DEV)
        out = torch.full_like(q, float("nan"))
        pq2.pq2_attention_prompt(q, k, v, out, starts_of([n]), starts_of([n]), causal=causal)
        torch.cuda.synchronize()
        led = 0
        for h in range(0, heads, 7):
            led += leading_values(out[:, h], q[:, h], k[:, h // (heads // kv)], v[:, h // (heads // kv)], causal)
        assert led > n // 2
    cache = ref.make_cache(90, 16, 2, d, 4, DEV)
    _, _, ks, vs = ref.parts(cache, 16, 2, d)
    ks.mul_(size)
    vs.fill_(1.0)
    table = torch.arange(90, dtype=torch.int32, device=DEV).view(1, 90)
    q = (randn((2, 8, d), 5).clamp(-4, 4) * size).to(DT[dt]).to(DEV)
    out = torch.full_like(q, float("nan"))
    floats, words = pq2.pq2_attention_paged_workspace(1, 2, 8, 2, d, 1440)
    pq2.pq2_attention_paged(q, cache, table, ints([1400]), 16, out, torch.empty(floats, device=DEV),
                            torch.zeros(words, dtype=torch.int32, device=DEV), starts=ints([0, 2]), max_new=2)
    torch.cuda.synchronize()
    k, v, _ = ref.rows_of(cache, 16, 2, d, table[0], 1400)
    assert sum(leading_values(out[1:, h], q[1:, h], k[:, h // 4], v[:, h // 4], False) for h in range(8)) > 4


def leading_values(out, q, k, v, causal):
    """Checks the rows whose largest score leads; how many these are."""
    a = q.double() @ k.double().t().contiguous() * q.shape[1] ** -0.5
    if causal:
        a = a.masked_fill(~lim.seen_keys(a.shape[0], a.shape[1], 0, device=DEV), -float("inf"))
    most = (q.double().abs() @ k.double().abs().t().contiguous()).amax(1) * q.shape[1] ** -0.5
    top = a.topk(min(2, a.shape[1]), dim=1)
    lead = top.values[:, 0] - top.values[:, 1] > 40 + 2 * (q.shape[1] + 8) * lim.U * most
    got, want = out[lead].double(), v.double()[top.indices[lead, 0]]
    # (bf16 and fp16 hold the values; weights 2^-57 of the largest and less move nothing.)
    assert torch.equal(got, want), (f"{int((got != want).any(1).sum())} of {int(lead.sum())} rows, first "
                                    f"{got[(got != want).any(1)][0, :4].tolist()} instead of {want[(got != want).any(1)][0, :4].tolist()}")
    return int(lead.sum())


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("d", ref.DIMS)
@pytest.mark.parametrize("common", [2.0 ** 10, 2.0 ** 18, 2.0 ** 22, 2.0 ** 23])
def test_prompt_large_scores_in_common(common, d, dt):
    """Scores of a large common part and small integers, exact in FP32, under a scale of ln 2: weights are powers of two, and
    the common part has no influence, also while the reference moves."""
    announce(f"prompt, common score {common} d={d} {dt}")
    pq2 = _pq2()
    n = 700
    for order in (1, -1):
        small = torch.arange(n) * 3 // 100               # 0 .. 20
        small = small.flip(0) if order < 0 else small
        k = torch.zeros((n, 1, d))
        k[:, 0, 0], k[:, 0, 1] = 2.0 ** (int(common).bit_length() // 2), small
        q = torch.zeros((40, 2, d))
        q[..., 0], q[..., 1] = common / k[0, 0, 0], 1.0
        q, k = q.to(DT[dt]).to(DEV), k.to(DT[dt]).to(DEV)
        v = randint(50, 250, (n, 1, d), 3).to(DT[dt]).to(DEV)
        out = torch.full_like(q, float("nan"))
        pq2.pq2_attention_prompt(q, k, v, out, starts_of([40]), starts_of([n]), causal=False, scale=0.6931471805599453)
        torch.cuda.synchronize()
        w = torch.exp2(small.double() - 20).to(DEV)
        want = ((w[:, None, None] * v.double()).sum(0) / w.sum())[None]
        # The scale's own rounding, three units of a difference of 20; sums of n terms; the output.  Up to 1024 the exponent of
        # a weight is a product with the common part, two roundings to 2^-14.
        limit = (lim.half(DT[dt]) + (n + 100) * lim.U + (2.0 ** -13 if common <= 2.0 ** 10 else 0)) * want
        over = (out.double() - want).abs() - limit
        assert float(over.max()) <= 0, f"{float(out[0, 0, 0])!r} instead of {float(want[0, 0, 0])!r}"


# ---------------------------------------------------------------- the ends of the ranges
@pytest.mark.parametrize("heads,kv,d", [(1024, 1, 64), (200, 1, 128), (1024, 1024, 64), (999, 27, 256), (1024, 8, 128)])
def test_many_heads(heads, kv, d):
    announce(f"many heads {heads}/{kv} d={d}")
    pq2 = _pq2()
    nq, nk = [5, 0, 40], [77, 9, 40]
    q = torch.zeros((sum(nq), heads, d), dtype=torch.bfloat16, device=DEV)
    k = randn((sum(nk), kv, d), 1).bfloat16().to(DEV)
    v = randint(-127, 127, (sum(nk), kv, d), 2).bfloat16().to(DEV)
    out = torch.full_like(q, float("nan"))
    pq2.pq2_attention_prompt(q, k, v, out, starts_of(nq), starts_of(nk))
    cache = ref.make_cache(12, 16, kv, d, 4, DEV)
    ref.parts(cache, 16, kv, d)[3].fill_(2.0 ** -6)
    table = torch.arange(12, dtype=torch.int32, device=DEV).view(2, 6)
    lengths, new = [90, 33], [2, 1]
    got = paged_call(lengths, new, heads, kv, d, 16, "bf16", 0, q[:3], cache, table)
    a = b = at = 0
    for n, m in zip(nq, nk):
        if n:
            seen = lim.seen_keys(n, m, m - n, device=DEV)
            lim.check_counts(out[a:a + n], lim.mean_of_seen(v[b:b + m], seen, heads), torch.bfloat16, "prompt")
        a, b = a + n, b + m
    for i, (n, t) in enumerate(zip(lengths, new)):
        _, vv, _ = ref.rows_of(cache, 16, kv, d, table[i], n)
        lim.check_counts(got[at:at + t], lim.mean_of_seen(vv, lim.seen_keys(t, n, n - t, device=DEV), heads), torch.bfloat16, "paged")
        at += t


def test_most_sequences():
    """65535 sequences of none to three tokens."""
    announce("65535 sequences")
    pq2 = _pq2()
    heads, kv, d, seqs = 2, 1, 64, 65535
    n = randint(0, 3, (seqs,), 1).to(DEV)
    starts = torch.zeros(seqs + 1, dtype=torch.int32, device=DEV)
    starts[1:] = n.cumsum(0)
    rows = int(starts[-1])
    seq = torch.repeat_interleave(torch.arange(seqs, device=DEV), n)
    t = torch.arange(rows, device=DEV) - starts[seq]
    v = randint(-127, 127, (rows, kv, d), 2).to(DEV)
    # Row t of a sequence sees t + 1 values: their mean.
    sums = v.double().cumsum(0)
    before = torch.cat([torch.zeros_like(sums[:1]), sums])[starts[seq].long()]
    mean = ((sums - before) / (t + 1).double()[:, None, None]).repeat_interleave(heads, 1)
    q = torch.zeros((rows, heads, d), dtype=torch.bfloat16, device=DEV)
    k = randn((rows, kv, d), 3).bfloat16().to(DEV)
    out = torch.full_like(q, float("nan"))
    pq2.pq2_attention_prompt(q, k, v.bfloat16(), out, starts, starts)
    torch.cuda.synchronize()
    lim.check_counts(out, mean, torch.bfloat16, "prompt")
    # The same tokens in a cache, a page for each sequence.
    page = 16
    cache = torch.zeros((seqs, pq2.pq2_kv_page_bytes(page, kv, d)), dtype=torch.uint8, device=DEV)
    kc, vc, ks, vs = ref.parts(cache, page, kv, d)
    vc[seq, :, t] = v.to(torch.int8)
    vs[seq, :, t] = 1.0
    table = torch.arange(seqs, dtype=torch.int32, device=DEV).flip(0).contiguous().view(seqs, 1)
    cache = cache.flip(0).contiguous()
    got = torch.full_like(q, float("nan"))
    floats, words = pq2.pq2_attention_paged_workspace(seqs, 3, heads, kv, d, 16)
    assert (floats, words) == (0, 0)
    pq2.pq2_attention_paged(q, cache, table, n.int(), page, got, starts=starts, max_new=3, max_len=16)
    back = [torch.full((rows, kv, d), float("nan"), device=DEV) for _ in "kv"]
    pq2.pq2_kv_read(cache, table, starts, page, *back)
    torch.cuda.synchronize()
    lim.check_counts(got, mean, torch.bfloat16, "paged")
    assert torch.equal(back[1], v.float()) and not bool(back[0].any())


@pytest.mark.parametrize("d", ref.DIMS)
def test_kv_write_rows_of_every_size(d):
    """Rows from the smallest FP32 numbers to the largest: codes and scales by the definition."""
    announce(f"kv write, rows of every size d={d}")
    pq2 = _pq2()
    sizes = [2.0 ** e for e in range(-149, 127, 3)]
    m = len(sizes)
    x = randn((m, 2, d), 1).clamp(-2, 2).double() * torch.tensor(sizes, dtype=torch.float64)[:, None, None]
    x = x.float()
    assert bool(torch.isfinite(x).all())
    page = 16
    pages = (m + page - 1) // page
    cache = torch.full((pages, pq2.pq2_kv_page_bytes(page, 1, d)), 0xA5, dtype=torch.uint8, device=DEV)
    xd = x.to(DEV)
    pq2.pq2_kv_write(xd[:, :1], xd[:, 1:], cache, torch.arange(m, dtype=torch.int32, device=DEV), page)
    torch.cuda.synchronize()
    want = torch.full(cache.shape, 0xA5, dtype=torch.uint8)
    kc, vc, ks, vs = ref.parts(want, page, 1, d)
    pg, at = torch.arange(m) // page, torch.arange(m) % page
    (kc[pg, :, at], ks[pg, :, at]), (vc[pg, :, at], vs[pg, :, at]) = ref.codes(x[:, :1]), ref.codes(x[:, 1:])
    got = ref.parts(cache.cpu(), page, 1, d)
    for name, a, b in zip(("k codes", "v codes", "k scales", "v scales"), got, (kc, vc, ks, vs)):
        a, b = a[pg, :, at], b[pg, :, at]
        bad = (a != b).flatten(1).any(1)
        assert not bool(bad.any()), f"{name} of rows of size {[sizes[i] for i in bad.nonzero().flatten().tolist()][:6]}"
