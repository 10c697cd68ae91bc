"""The attention operators on the GPU against plain references (bounds and
references in tests/attention_reference.py): the cache bit for bit, attention
within its bound.  Outputs are poisoned before a call."""
import functools

import pytest
import torch

import attention_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


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


def same_bits(a, b):
    view = {2: torch.int16, 4: torch.int32, 1: torch.uint8}[a.element_size()]
    return torch.equal(a.contiguous().view(view), b.contiguous().view(view))


def within(got, want, bound, what):
    got = got.double()
    assert bool(torch.isfinite(got).all()), f"{what}: non-finite output"
    excess = (got - want).abs() - bound
    worst = int(excess.argmax())
    assert float(excess.max()) <= 0, (f"{what}: off by {float((got - want).abs().flatten()[worst]):.3e}, bound "
                                      f"{float(bound.flatten()[worst]):.3e} at {worst}")


# ---------------------------------------------------------------- the cache
WRITES = [
    # m, heads, kv, d, rot, interleaved, page, in, out
    (1, 64, 8, 128, 128, False, 16, "f32", "bf16"),
    (1, 1, 1, 64, 64, True, 16, "bf16", "f16"),
    (5, 24, 4, 256, 64, True, 64, "f32", "f16"),
    (17, 6, 3, 64, 16, False, 32, "f16", "bf16"),
    (33, 5, 5, 128, 32, False, 128, "bf16", "f32"),
    (16, 8, 2, 256, 256, False, 256, "bf16", "bf16"),
    (700, 10, 2, 128, 128, False, 16, "f32", "bf16"),
    (1025, 4, 1, 64, 0, False, 64, "f16", "f16"),
    (600, 3, 1, 256, 200, True, 32, "f32", "f32"),
]


@pytest.mark.parametrize("m,heads,kv,d,rot,inter,page,xin,xout", WRITES)
def test_kv_write_bits(m, heads, kv, d, rot, inter, page, xin, xout):
    announce(f"kv write m={m} heads={heads}/{kv} d={d} rot={rot} inter={inter} page={page} {xin}->{xout}")
    gen = torch.Generator().manual_seed(m + d)
    x = randn((m, heads + 2 * kv, d), m, 2.0)
    x[torch.rand(x.shape, generator=gen) < 0.01] = 0.0
    x[0, -1] = 0.0                                   # a value row of zeros: scale 0
    x = x.to(DT[xin])
    pages = (m + page - 1) // page + 3
    slots = torch.randperm(pages * page, generator=gen)[:m].to(torch.int32)
    if m > 4:
        slots[1], slots[3] = -1, pages * page        # not written
    rows = 50
    positions = torch.randint(0, rows, (m,), generator=gen, dtype=torch.int32)
    if m > 4:
        positions[2], positions[4] = -7, rows + 3    # nearest row
    cos, sin = ref.tables(rows, rot) if rot else (None, None)
    xd = x.to(DEV)
    cache = torch.full((pages, _pq2().pq2_kv_page_bytes(page, kv, d)), 0xA5, dtype=torch.uint8, device=DEV)
    outs = [torch.full((m, h, d), float("nan"), dtype=DT[xout], device=DEV) for h in (heads, kv, kv)]
    _pq2().pq2_kv_write(xd[:, heads:heads + kv], xd[:, heads + kv:], cache, slots.to(DEV), page, q=xd[:, :heads], q_out=outs[0],
                        k_out=outs[1], v_out=outs[2], cos=None if cos is None else cos.to(DEV),
                        sin=None if sin is None else sin.to(DEV), positions=positions.to(DEV), interleaved=inter)
    torch.cuda.synchronize()
    q, k = (ref.rotated(t, cos, sin, positions, inter) for t in (x[:, :heads], x[:, heads:heads + kv]))
    v = x[:, heads + kv:].float()
    for name, got, want in zip("qkv", outs, (q, k, v)):
        assert same_bits(got.cpu(), want.to(DT[xout])), name
    want = torch.full(cache.shape, 0xA5, dtype=torch.uint8)
    kc, vc, ks, vs = ref.parts(want, page, kv, d)
    ok = (slots >= 0) & (slots < pages * page)
    pg, at = slots[ok].long() // page, slots[ok].long() % page
    (kc[pg, :, at], ks[pg, :, at]), (vc[pg, :, at], vs[pg, :, at]) = ref.codes(k[ok]), ref.codes(v[ok])
    assert torch.equal(cache.cpu(), want)


def test_kv_write_in_place_and_layouts():
    """Rotation in place inside one QKV buffer, and heads outside the rows."""
    announce("kv write in place, head-major")
    pq2 = _pq2()
    m, heads, kv, d, page = 37, 6, 2, 128, 16
    cos, sin = ref.tables(64, d)
    positions = torch.arange(m, dtype=torch.int32)
    x = randn((m, heads + 2 * kv, d), 1).bfloat16()
    slots = torch.arange(m, dtype=torch.int32, device=DEV)
    caches = [torch.zeros((3, pq2.pq2_kv_page_bytes(page, kv, d)), dtype=torch.uint8, device=DEV) for _ in range(3)]
    kw = dict(cos=cos.to(DEV), sin=sin.to(DEV), positions=positions.to(DEV))
    a = x.to(DEV)
    plain = torch.empty_like(a)
    pq2.pq2_kv_write(a[:, heads:heads + kv], a[:, heads + kv:], caches[0], slots, page, q=a[:, :heads], q_out=plain[:, :heads],
                     k_out=plain[:, heads:heads + kv], v_out=plain[:, heads + kv:], **kw)
    b = x.to(DEV)
    k = b[:, heads:heads + kv]
    pq2.pq2_kv_write(k, b[:, heads + kv:], caches[1], slots, page, q=b[:, :heads], q_out=b[:, :heads], k_out=k, **kw)
    c = x.to(DEV).transpose(0, 1).contiguous().transpose(0, 1)      # [heads][rows][d] in memory
    out = torch.empty_like(c)
    pq2.pq2_kv_write(c[:, heads:heads + kv], c[:, heads + kv:], caches[2], slots, page, q=c[:, :heads], q_out=out[:, :heads], **kw)
    torch.cuda.synchronize()
    assert torch.equal(b, plain) and torch.equal(out[:, :heads], plain[:, :heads])
    assert torch.equal(caches[0], caches[1]) and torch.equal(caches[0], caches[2])


READS = [
    # lengths, kv, d, page, out
    ([1], 1, 64, 16, "f32"),
    ([0, 5, 0, 0, 33, 64, 1], 3, 64, 16, "bf16"),
    ([100, 0, 257], 2, 128, 32, "f16"),
    ([31] * 70 + [0] * 70 + [3], 1, 128, 16, "bf16"),
    ([300], 4, 256, 256, "f32"),
    ([0, 77, 12], 5, 256, 64, "bf16"),
    # two rows a lane
    ([3000, 0, 2300], 8, 128, 16, "bf16"),
    ([2100, 1, 33], 8, 256, 64, "f32"),
    ([9001, 77], 8, 64, 32, "f16"),
]


@pytest.mark.parametrize("lengths,kv,d,page,out", READS)
def test_kv_read_bits(lengths, kv, d, page, out):
    announce(f"kv read {len(lengths)} sequences kv={kv} d={d} page={page} {out}")
    width = max(1, max((n + page - 1) // page for n in lengths))
    pages = len(lengths) * width + 2
    cache = ref.make_cache(pages, page, kv, d, 3, DEV)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(4))[:len(lengths) * width].to(torch.int32).view(-1, width)
    bad = len(lengths) > 1 and lengths[1] > 0
    if bad:
        table[1, 0] = pages                          # outside the cache: zeros
    longest = max(range(len(lengths)), key=lambda i: lengths[i])
    used = width
    if lengths[longest] > page:
        used = width - 1                             # the last page of the longest lies beyond the table: zeros
    rows = sum(lengths)
    k, v = (torch.full((rows + 9, kv, d), 7.0, dtype=DT[out], device=DEV) for _ in "kv")
    td = table.to(DEV)
    _pq2().pq2_kv_read(cache, td[:, :used], starts_of(lengths), page, k, v)
    torch.cuda.synchronize()
    host = cache.cpu()
    at = 0
    for i, n in enumerate(lengths):
        if not n:
            continue
        kk, vv, there = ref.rows_of(host, page, kv, d, table[i, :used], n)
        for got, want in ((k, kk), (v, vv)):
            want = torch.where(there[:, None, None], want, torch.zeros_like(want)).float().to(DT[out])
            assert same_bits(got[at:at + n].cpu(), want), i
        at += n
    assert bool((k[rows:] == 7).all()) and bool((v[rows:] == 7).all())


# ---------------------------------------------------------------- attention over the pages
def paged_case(lengths, new, heads, kv, d, page, dt, window, seed=0, spare=3, max_len=None, max_new=None, garbage=True, strided=False,
               bad_page=False, scale=None, table_pages=None):
    """(got, want, bound) of one call; what the pages hold behind a length is garbage with NaN scales."""
    pq2 = _pq2()
    width = max(1, max((max(n, 0) + page - 1) // page for n in lengths))
    pages = len(lengths) * width + spare
    cache = ref.make_cache(pages, page, kv, d, seed + 1, DEV)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(seed + 2))[:len(lengths) * width].to(torch.int32).view(-1, width).to(DEV)
    if garbage:
        _, _, ks, vs = ref.parts(cache, page, kv, d)
        for i, n in enumerate(lengths):
            for p in range(width):
                first = max(0, n - p * page)
                if first < page:
                    ks[int(table[i, p]), :, first:] = float("nan")
                    vs[int(table[i, p]), :, first:] = float("inf")
    if bad_page:
        table[0, 0], table[-1, -1] = -1, pages
    if table_pages:
        table = table[:, :table_pages]              # lengths go beyond what the table holds
    starts = starts_of(new)
    rows = sum(new)
    q = randn((rows, heads, d), seed, 1.5).to(DT[dt]).to(DEV)
    if strided:
        buf = torch.zeros((rows, heads + 3, d), dtype=DT[dt], device=DEV)
        buf[:, 2:2 + heads] = q
        q = buf[:, 2:2 + heads]
        out = torch.full((heads, rows, d), float("nan"), dtype=DT[dt], device=DEV).transpose(0, 1)
    else:
        out = torch.full((rows, heads, d), float("nan"), dtype=DT[dt], device=DEV)
    max_new = max_new or max(max(new), 1)
    max_len = max_len or max(1, max(lengths))
    floats, words = pq2.pq2_attention_paged_workspace(len(lengths), max_new, heads, kv, d, max_len)
    partials = torch.full((floats + 16,), float("nan"), device=DEV)
    counters = torch.zeros(words, dtype=torch.int32, device=DEV)
    kw = dict(starts=starts, max_new=max_new, max_len=max_len, window=window, scale=scale)
    pq2.pq2_attention_paged(q, cache, table, ints(lengths), page, out, partials, counters, **kw)
    again = torch.full_like(out, float("nan"))
    pq2.pq2_attention_paged(q, cache, table, ints(lengths), page, again, partials, counters, **kw)
    torch.cuda.synchronize()
    assert same_bits(out, again), "a second call on the same workspace differs"
    assert not words or int(counters.abs().sum()) == 0
    assert bool(torch.isnan(partials[floats:]).all()), "wrote behind the workspace"
    want, bound = [], []
    at = 0
    for i, (n, t) in enumerate(zip(lengths, new)):
        k, v, there = ref.rows_of(cache, page, kv, d, table[i], max(n, 0))
        k, v = (torch.where(there[:, None, None], x, torch.zeros_like(x)) for x in (k, v))
        o, b = ref.attention(q[at:at + t], k, v, n - t, scale=scale or d ** -0.5, window=window, there=there, paged=True, dtype=DT[dt])
        want.append(o)
        bound.append(b)
        at += t
    return out, torch.cat(want), torch.cat(bound)


PAGED = [
    # lengths, new tokens, heads, kv, d, page, type, window
    ([1], [1], 1, 1, 64, 16, "bf16", 0),
    ([517], [1], 40, 8, 128, 16, "bf16", 0),
    ([0, 1, 2, 15, 16, 17, 31, 32, 33, 255, 256, 257], [1] * 12, 8, 2, 128, 16, "f16", 0),
    ([300, 40, 700], [1, 1, 1], 7, 1, 64, 32, "bf16", 0),
    ([1000, 900], [1, 1], 34, 2, 64, 64, "f16", 0),                      # 17 grouped heads: two tiles of rows
    ([5000, 2, 0, 900], [1] * 4, 6, 1, 256, 64, "f16", 0),
    ([3000, 100, 7], [4, 7, 1], 24, 4, 256, 32, "bf16", 0),
    ([600, 20, 3, 0], [16, 9, 5, 2], 10, 2, 128, 16, "bf16", 0),         # more new tokens than keys: rows that see none
    ([4000, 300, 50], [3, 1, 8], 5, 5, 128, 128, "f16", 100),
    ([9000, 40], [8, 8], 8, 1, 64, 256, "bf16", 1024),
    ([2500, 2500], [1, 0], 16, 2, 128, 16, "bf16", 1),
    ([33000], [1], 64, 8, 128, 64, "bf16", 0),
    ([20000, 17, 9000], [1, 1, 1], 8, 8, 128, 32, "f16", 0),
]


@pytest.mark.parametrize("lengths,new,heads,kv,d,page,dt,window", PAGED)
def test_attention_paged(lengths, new, heads, kv, d, page, dt, window):
    announce(f"paged lengths={lengths} new={new} heads={heads}/{kv} d={d} page={page} {dt} window={window}")
    got, want, bound = paged_case(lengths, new, heads, kv, d, page, dt, window, seed=heads + d)
    within(got, want, bound, "o")
    # The last rounding is off by at most half of each value; all other errors together are a tenth of that.
    assert float((got.double() - want).norm()) <= 1.1 * torch.finfo(DT[dt]).eps / 2 * float(want.norm())


@pytest.mark.parametrize("d", ref.DIMS)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_attention_paged_strides_bad_pages_bounds(d, dt):
    announce(f"paged strided, bad pages d={d} {dt}")
    within(*paged_case([700, 90, 1500], [2, 1, 3], 6, 2, d, 16, dt, 0, strided=True, garbage=False, bad_page=True), "bad pages")
    # Lengths far beyond max_len are computed; so are workspaces for far longer ones.
    within(*paged_case([6000, 3], [1, 1], 4, 2, d, 32, dt, 0, max_len=600), "beyond max_len")
    within(*paged_case([600, 3], [1, 1], 4, 2, d, 32, dt, 0, max_len=100000, max_new=5), "roomy workspace")
    within(*paged_case([800, 40], [1, 2], 4, 1, d, 32, dt, 0, scale=3.0), "sharp softmax")
    within(*paged_case([700, 100, 490], [4, 3, 2], 4, 2, d, 16, dt, 0, table_pages=30), "beyond the table")
    within(*paged_case([700, 100, 490], [4, 3, 2], 4, 2, d, 16, dt, 250, table_pages=30), "beyond the table, window")


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("f16", 64)])
def test_attention_paged_many_sequences(dt, d):
    """More sequences than one group of 64 workgroups' places; some empty, some long."""
    announce(f"paged many sequences d={d} {dt}")
    lengths = [(7 * i * i) % 300 for i in range(150)]
    lengths[3], lengths[70], lengths[149] = 5000, 2600, 4100
    new = [1 + i % 3 if i % 11 else 0 for i in range(150)]
    within(*paged_case(lengths, new, 4, 2, d, 16, dt, 0, max_new=3), "o")


def test_attention_paged_rows_do_not_depend_on_the_batch():
    announce("paged batch invariance")
    pq2 = _pq2()
    heads, kv, d, page = 8, 2, 128, 16
    lens = [900, 20, 3000, 1]
    cache = ref.make_cache(800, page, kv, d, 1, DEV)
    table = torch.arange(4 * 190, dtype=torch.int32, device=DEV).view(4, 190)
    q = randn((4, heads, d), 2).bfloat16().to(DEV)
    floats, words = pq2.pq2_attention_paged_workspace(4, 1, heads, kv, d, 3040)
    work = torch.empty(floats, device=DEV), torch.zeros(words, dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    pq2.pq2_attention_paged(q, cache, table, ints(lens), page, out, *work, max_len=3040)
    swapped = torch.empty_like(q)
    order = torch.tensor([2, 0, 3, 1], device=DEV)
    pq2.pq2_attention_paged(q[order], cache, table[order].contiguous(), ints([lens[i] for i in order.tolist()]), page, swapped, *work,
                            max_len=3040)
    torch.cuda.synchronize()
    assert torch.equal(swapped, out[order])


def test_attention_paged_leaves_other_rows():
    """Rows of no sequence, and new tokens beyond max_new, keep what out held."""
    announce("paged untouched rows")
    pq2 = _pq2()
    cache = ref.make_cache(8, 16, 1, 64, 1, DEV)
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(2, 4)
    q = randn((9, 16, 64), 3).bfloat16().to(DEV)
    out = torch.full_like(q, 7.0)
    starts = ints([1, 4, 6])                        # row 0 and rows 6.. belong to none
    pq2.pq2_attention_paged(q, cache, table, ints([40, 50]), 16, out, starts=starts, max_new=2, max_len=64)
    torch.cuda.synchronize()
    held = [bool((out[i] == 7).all()) for i in range(9)]
    assert held == [True, False, False, True, False, False, True, True, True]


# ---------------------------------------------------------------- attention over prompts
def prompt_case(nq, nk, heads, kv, d, dt, causal, window, seed=0, layout="packed", tail=0, scale=None):
    pq2 = _pq2()
    rq, rk = sum(nq) + tail, max(1, sum(nk) + tail)
    q, k, v = (randn((r, h, d), seed + i, s).to(DT[dt]).to(DEV) for i, (r, h, s) in enumerate(((rq, heads, 1.5), (rk, kv, 1.0), (rk, kv, 1.0))))
    if tail:                                         # rows of no sequence: anything
        k[sum(nk):], v[sum(nk):] = float("nan"), float("inf")
    out = torch.full_like(q, 7.0)
    if layout == "columns":
        qb = torch.full((rq, heads + 2, d), 3.0, dtype=DT[dt], device=DEV)
        kb = torch.full((rk, 3 * kv, d), float("nan"), dtype=DT[dt], device=DEV)
        qb[:, 1:1 + heads], kb[:, :kv], kb[:, 2 * kv:] = q, k, v
        q, k, v = qb[:, 1:1 + heads], kb[:, :kv], kb[:, 2 * kv:]
    elif layout == "heads first":
        q, k, v, out = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v, out))
    pq2.pq2_attention_prompt(q, k, v, out, starts_of(nq), starts_of(nk), causal=causal, window=window, scale=scale)
    torch.cuda.synchronize()
    want, bound, a, b = [], [], 0, 0
    for n, m in zip(nq, nk):
        o, e = ref.attention(q[a:a + n], k[b:b + m], v[b:b + m], m - n, scale=scale or d ** -0.5, causal=causal, window=window, dtype=DT[dt])
        want.append(o)
        bound.append(e)
        a, b = a + n, b + m
    assert bool((out[a:] == 7).all()), "wrote rows of no sequence"
    return out[:a], torch.cat(want), torch.cat(bound)


PROMPTS = [
    # queries, keys, heads, kv, type, causal, window
    ([1], [1], 1, 1, "bf16", True, 0),
    ([128], [128], 2, 1, "bf16", True, 0),
    ([200], [200], 3, 3, "f16", True, 0),
    ([64, 1, 0, 129, 65, 31], [64, 1, 0, 129, 65, 31], 4, 2, "bf16", True, 0),
    ([5, 100, 130, 0], [300, 100, 513, 70], 6, 2, "f16", True, 0),       # behind prefixes
    ([40, 90], [7, 0], 2, 1, "bf16", True, 0),                           # fewer keys than queries: rows that see none
    ([300, 77], [300, 500], 4, 4, "bf16", False, 0),
    ([10, 3], [0, 65], 4, 1, "f16", False, 0),
    ([700, 20], [700, 400], 5, 1, "bf16", True, 100),
    ([300, 150], [333, 150], 2, 2, "f16", True, 1),
    ([3] * 150, [4] * 150, 2, 1, "bf16", True, 0),
    ([1500], [1500], 2, 1, "bf16", True, 0),
]


@pytest.mark.parametrize("d", ref.DIMS)
@pytest.mark.parametrize("nq,nk,heads,kv,dt,causal,window", PROMPTS)
def test_attention_prompt(nq, nk, heads, kv, dt, causal, window, d):
    announce(f"prompt nq={nq[:6]} nk={nk[:6]} heads={heads}/{kv} d={d} {dt} causal={causal} window={window}")
    within(*prompt_case(nq, nk, heads, kv, d, dt, causal, window, seed=d), "o")


@pytest.mark.parametrize("nq,nk,heads,kv,d,dt,causal,window", [
    ([4200], [4200], 32, 2, 128, "bf16", True, 0),
    ([4100, 100], [8300, 133], 32, 4, 128, "f16", True, 3000),
    ([4100], [4133], 33, 3, 128, "bf16", False, 0),
    ([2400, 0, 77, 333], [2500, 5, 77, 300], 24, 4, 256, "f16", True, 0),
    ([900, 1900], [1000, 1900], 24, 3, 256, "bf16", True, 500),
    ([2900], [40], 24, 2, 256, "bf16", False, 0),
    ([3000], [3000], 16, 16, 64, "bf16", True, 0),
])
def test_attention_prompt_large(nq, nk, heads, kv, d, dt, causal, window):
    """The workgroups of eight waves, many steps."""
    announce(f"prompt large nq={nq} nk={nk} heads={heads}/{kv} d={d} {dt} causal={causal} window={window}")
    within(*prompt_case(nq, nk, heads, kv, d, dt, causal, window, seed=d), "o")


@pytest.mark.parametrize("d", ref.DIMS)
@pytest.mark.parametrize("layout", ["columns", "heads first", "packed"])
def test_attention_prompt_layouts(layout, d):
    announce(f"prompt layout {layout} d={d}")
    within(*prompt_case([70, 200], [70, 290], 6, 2, d, "bf16", True, 0, layout=layout, tail=33), "o")
    within(*prompt_case([90], [90], 2, 1, d, "f16", True, 0, layout=layout, tail=5, scale=3.0), "sharp softmax")


def test_attention_prompt_growing_scores():
    """Scores that rise by far along the keys: every step moves the running maximum."""
    announce("prompt growing scores")
    pq2 = _pq2()
    n, d = 900, 128
    q = torch.ones((n, 1, d), dtype=torch.bfloat16, device=DEV)
    k = (torch.linspace(-8, 8, n)[:, None, None] * torch.ones(1, 1, d)).bfloat16().to(DEV)
    v = randn((n, 1, d), 3).bfloat16().to(DEV)
    for flip in (False, True):
        kk = k.flip(0).contiguous() if flip else k
        out = torch.empty_like(q)
        s = starts_of([n])
        pq2.pq2_attention_prompt(q, kk, v, out, s, s, causal=False)
        want, bound = ref.attention(q, kk, v, 0, scale=d ** -0.5, causal=False, dtype=torch.bfloat16)
        torch.cuda.synchronize()
        within(out, want, bound, f"flip={flip}")


# ---------------------------------------------------------------- as they are used
def test_operators_in_a_row():
    """A prompt in two pieces (the second behind the first as its prefix, read back from the cache), then decoded tokens:
    the cache's attention agrees with the prompt's on the same keys."""
    announce("operators in a row")
    pq2 = _pq2()
    heads, kv, d, page, n1, n2 = 8, 2, 128, 16, 200, 75
    n = n1 + n2
    cos, sin = (t.to(DEV) for t in ref.tables(400, d))
    cache = torch.zeros((20, pq2.pq2_kv_page_bytes(page, kv, d)), dtype=torch.uint8, device=DEV)
    table = torch.randperm(20, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(1, 20).to(DEV)
    x = randn((n, heads + 2 * kv, d), 2).to(DEV)

    def slots(a, b):
        t = torch.arange(a, b, device=DEV)
        return (table[0].long()[t // page] * page + t % page).to(torch.int32)

    def piece(a, b):
        part = x[a:b]
        out = [torch.empty((b - a, h, d), dtype=torch.bfloat16, device=DEV) for h in (heads, kv, kv)]
        pq2.pq2_kv_write(part[:, heads:heads + kv], part[:, heads + kv:], cache, slots(a, b), page, q=part[:, :heads], q_out=out[0],
                         k_out=out[1], v_out=out[2], cos=cos, sin=sin, positions=torch.arange(a, b, dtype=torch.int32, device=DEV))
        return out
    q1, k1, v1 = piece(0, n1)
    o1 = torch.empty_like(q1)
    pq2.pq2_attention_prompt(q1, k1, v1, o1, starts_of([n1]), starts_of([n1]))
    q2, k2, v2 = piece(n1, n)
    kb, vb = (torch.empty((n, kv, d), dtype=torch.bfloat16, device=DEV) for _ in "kv")
    pq2.pq2_kv_read(cache, table, starts_of([n1]), page, kb, vb)
    kb[n1:], vb[n1:] = k2, v2
    o2 = torch.empty_like(q2)
    pq2.pq2_attention_prompt(q2, kb, vb, o2, starts_of([n2]), starts_of([n]))
    o3 = torch.empty_like(q2)
    pq2.pq2_attention_paged(q2, cache, table, ints([n]), page, o3, starts=ints([0, n2]), max_new=n2, max_len=n,
                            partials=torch.empty(1 << 20, device=DEV), counters=torch.zeros(4096, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    for got, q, k, v, first in ((o1, q1, k1, v1, 0), (o2, q2, kb, vb, n1)):
        want, bound = ref.attention(q, k, v, first, scale=d ** -0.5, dtype=torch.bfloat16)
        within(got, want, bound, "prompt")
    kk, vv, there = ref.rows_of(cache, page, kv, d, table[0], n)
    want, bound = ref.attention(q2, kk, vv, n1, scale=d ** -0.5, paged=True, there=there, dtype=torch.bfloat16)
    within(o3, want, bound, "paged")
    # Codes are off by half a step: scores and values by about 1/254 of a row's largest element.
    assert float((o3.double() - o2.double()).norm() / o2.double().norm()) < 0.02


def test_captured_and_replayed():
    """A decode step (write, attention over the pages) in a graph, replayed on new inputs and lengths between eager calls."""
    announce("captured decode step")
    pq2 = _pq2()
    heads, kv, d, page, seqs, width = 16, 2, 128, 16, 3, 200
    cos, sin = (t.to(DEV) for t in ref.tables(4000, d))
    cache = ref.make_cache(seqs * width, page, kv, d, 1, DEV)
    table = torch.arange(seqs * width, dtype=torch.int32, device=DEV).view(seqs, width)
    x = torch.zeros((seqs, heads + 2 * kv, d), device=DEV)
    lens, slots, positions = (torch.zeros(seqs, dtype=torch.int32, device=DEV) for _ in range(3))
    q = torch.empty((seqs, heads, d), dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(q)
    floats, words = pq2.pq2_attention_paged_workspace(seqs, 1, heads, kv, d, width * page)
    work = [(torch.empty(floats, device=DEV), torch.zeros(words, dtype=torch.int32, device=DEV)) for _ in range(2)]

    def step(cache, out, w):
        pq2.pq2_kv_write(x[:, heads:heads + kv], x[:, heads + kv:], cache, slots, page, q=x[:, :heads], q_out=q, cos=cos, sin=sin,
                         positions=positions)
        pq2.pq2_attention_paged(q, cache, table, lens, page, out, *w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cache, out, work[0])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, out, work[0])
    for turn, now in enumerate(([5, 900, 3199], [1, 1, 1], [3100, 17, 640], [3200, 2000, 3])):
        x.copy_(randn(x.shape, turn))
        lens.copy_(ints(now))
        positions.copy_(lens - 1)
        slots.copy_(torch.arange(seqs, device=DEV, dtype=torch.int32) * width * page + positions)
        eager_cache, eager = cache.clone(), torch.empty_like(out)
        step(eager_cache, eager, work[1])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cache, eager_cache) and torch.equal(out, eager), turn


def test_offsets_beyond_32_bits():
    """A cache of more than 4 GiB, its last pages used, and keys whose rows are 16 MiB apart."""
    announce("offsets beyond 32 bits")
    pq2 = _pq2()
    heads, kv, d, page, n = 8, 4, 256, 256, 700
    big = torch.empty((9000, pq2.pq2_kv_page_bytes(page, kv, d)), dtype=torch.uint8, device=DEV)
    small = torch.zeros((4, big.shape[1]), dtype=torch.uint8, device=DEV)
    big[-4:] = 0
    assert big.numel() > 1 << 32
    k, v, q = (randn((n, h, d), i).half().to(DEV) for i, h in enumerate((kv, kv, heads)))
    t = torch.arange(n, device=DEV, dtype=torch.int32)
    got = []
    for cache, first in ((small, 0), (big, 8996)):
        pq2.pq2_kv_write(k, v, cache, t + first * page, page)
        table = torch.arange(4, dtype=torch.int32, device=DEV).view(1, 4) + first
        out = torch.empty_like(q[-3:])
        pq2.pq2_attention_paged(q[-3:], cache, table, ints([n]), page, out, starts=ints([0, 3]), max_new=3, max_len=n,
                                partials=torch.empty(1 << 20, device=DEV), counters=torch.zeros(4096, dtype=torch.int32, device=DEV))
        back = [torch.empty((n, kv, d), device=DEV) for _ in "kv"]
        pq2.pq2_kv_read(cache, table, starts_of([n]), page, *back)
        got.append([out, *back])
    torch.cuda.synchronize()
    assert torch.equal(small, big[-4:]) and all(torch.equal(a, b) for a, b in zip(*got))
    del big
    wide = torch.empty((300, 1 << 23), dtype=torch.half, device=DEV)
    far = wide[:, 512:512 + kv * d].unflatten(1, (kv, d))
    far.copy_(k[:300])
    s = starts_of([300])
    outs = [torch.empty_like(q[:300]) for _ in range(2)]
    pq2.pq2_attention_prompt(q[:300], k[:300], v[:300], outs[0], s, s)
    pq2.pq2_attention_prompt(q[:300], far, v[:300], outs[1], s, s)
    torch.cuda.synchronize()
    assert torch.equal(*outs)


def test_prompt_captured_and_replayed():
    announce("captured prompt")
    pq2 = _pq2()
    heads, kv, d, page = 4, 2, 128, 16
    cache = ref.make_cache(60, page, kv, d, 1, DEV)
    table = torch.arange(60, dtype=torch.int32, device=DEV).view(2, 30)
    k, v = (torch.empty((900, kv, d), dtype=torch.bfloat16, device=DEV) for _ in "kv")
    q = torch.empty((700, heads, d), dtype=torch.bfloat16, device=DEV)
    out = torch.zeros_like(q)
    starts_q, starts_k = (torch.zeros(3, dtype=torch.int32, device=DEV) for _ in range(2))

    def step(k, v, out):
        pq2.pq2_kv_read(cache, table, starts_k, page, k, v)
        pq2.pq2_attention_prompt(q, k, v, out, starts_q, starts_k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(k, v, out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(k, v, out)
    for turn, (a, b) in enumerate((([300, 400], [450, 450]), ([1, 0], [1, 0]), ([0, 700], [0, 480]))):
        q.copy_(randn(q.shape, turn))
        starts_q.copy_(starts_of(a))
        starts_k.copy_(starts_of(b))
        eager = [k.clone(), v.clone(), out.clone()]
        step(*eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((k, v, out), eager)), turn


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own, beside each other."""
    announce("two paged calls at once")
    pq2 = _pq2()
    heads, kv, d, page, n = 16, 2, 128, 16, 20000
    cache = ref.make_cache(1300, page, kv, d, 1, DEV)
    table = torch.arange(1250, dtype=torch.int32, device=DEV).view(1, 1250)
    floats, words = pq2.pq2_attention_paged_workspace(1, 1, heads, kv, d, n)
    lens = ints([n])
    q = [randn((1, heads, d), i).bfloat16().to(DEV) for i in range(2)]
    work = [(torch.empty(floats, device=DEV), torch.zeros(words, dtype=torch.int32, device=DEV)) for _ in range(2)]
    want = [torch.empty_like(x) for x in q]
    for i in range(2):
        pq2.pq2_attention_paged(q[i], cache, table, lens, page, want[i], *work[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[torch.zeros_like(x) for _ in range(20)] for x in q]
    torch.cuda.synchronize()
    for turn in range(20):
        for i in range(2):
            pq2.pq2_attention_paged(q[i], cache, table, lens, page, got[i][turn], *work[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i]) for i in range(2) for x in got[i])


def test_other_stream():
    """On a stream that is not the current one, with inputs made on it."""
    announce("other stream")
    pq2 = _pq2()
    q = randn((300, 4, 64), 1).half().to(DEV)
    k, v = (randn((300, 2, 64), 2 + i).half().to(DEV) for i in range(2))
    s = starts_of([300])
    want = torch.empty_like(q)
    pq2.pq2_attention_prompt(q, k, v, want, s, s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    pq2.pq2_attention_prompt(q, k, v, out, s, s, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
