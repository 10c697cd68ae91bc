"""Measured cases of the attention operators: keys and values quantised into a
paged INT8 cache and read back, attention of new tokens over the pages, and
attention over packed prompts.

Where ``own`` is false every operator runs in its plain form (elementary torch
operations); where it is true the library's entry points run.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEV = "cuda"
TABLE_ROWS = 40960          # positions in the rotary tables


# ---------------------------------------------------------------- cases
def listed():
    return [
        # One decoded token: its query rotated, its key and value into the cache, from the projection's FP32 output.
        dict(name="write 1", op="write", m=1, heads=64, kv=8, d=128, rot=128, inter=False, page=16, x="f32", o="bf16", dense=False),
        # Verification of 16 tokens, wide heads rotated in part, neighbouring pairs.
        dict(name="write 16", op="write", m=16, heads=24, kv=4, d=256, rot=64, inter=True, page=64, x="f32", o="f16", dense=False),
        # A prompt of 4096 tokens: the cache, and rotated queries, keys and values for the prompt's own attention.
        dict(name="write 4096", op="write", m=4096, heads=64, kv=8, d=128, rot=128, inter=False, page=16, x="f32", o="bf16", dense=True),
        # Prefixes of a ragged batch of prompts, small heads.
        dict(name="read ragged 19", op="read", seqs=19, lo=0, hi=700, kv=5, d=64, page=16, o="f32"),
        # The prefix of a long document, before its next piece of prompt.
        dict(name="read 32768", op="read", seqs=1, lo=32768, hi=32768, kv=8, d=128, page=64, o="bf16"),
        # One sequence in decode, a short cache: latency only.
        dict(name="paged 1 short", op="paged", seqs=1, new=1, lo=517, hi=517, heads=40, kv=8, d=128, page=16, window=0, x="bf16"),
        # One sequence in decode behind a very long document.
        dict(name="paged 1 long", op="paged", seqs=1, new=1, lo=131071, hi=131071, heads=64, kv=8, d=128, page=64, window=0, x="bf16"),
        # A serving batch of 64 sequences of very different lengths, one new token each.
        dict(name="paged 64 ragged", op="paged", seqs=64, new=1, lo=1, hi=16384, heads=40, kv=8, d=128, page=16, window=0, x="bf16"),
        # Drafted tokens of eight sequences verified together, wide heads, a sliding window.
        dict(name="paged 8 verify", op="paged", seqs=8, new=8, lo=1000, hi=9000, heads=24, kv=4, d=256, page=32, window=4096, x="f16"),
        # A short prompt alone.
        dict(name="prompt 512", op="prompt", seqs=1, lo=512, hi=512, prefix=0, heads=40, kv=8, d=128, causal=True, window=0, x="bf16"),
        # A ragged batch of prompts packed together, some behind a prefix, wide heads.
        dict(name="prompt packed 24", op="prompt", seqs=24, lo=0, hi=1500, prefix=700, heads=24, kv=4, d=256, causal=True, window=0, x="f16"),
        # A long prompt.
        dict(name="prompt 8192", op="prompt", seqs=1, lo=8192, hi=8192, prefix=0, heads=40, kv=8, d=128, causal=True, window=0, x="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lengths(count, lo, hi, salt=""):
    """Lengths of a ragged batch, the same ones for the same case: between lo and hi, spread over their logarithm, the longest one hi."""
    rng = random.Random("%d %d %d %s" % (count, lo, hi, salt))
    n = [max(lo, _log(rng, lo + 1, hi + 1) - 1) for _ in range(count)]
    n[rng.randrange(count)] = hi
    return n


def draw(rng):
    op = rng.choice(["write", "read", "paged", "prompt"])
    d = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 3, 4, 5, 8])
    heads = kv * rng.choice([1, 2, 4, 5, 6, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    half = rng.choice(["bf16", "f16"])
    if op == "write":
        m = max(1, min(_log(rng, 1, 4096), 4096 * 10240 // ((heads + 2 * kv) * d)))
        return dict(op=op, m=m, heads=heads, kv=kv, d=d, rot=rng.choice([0, d // 4, d // 2, d]), inter=rng.random() < 0.5,
                    page=page, x=rng.choice(["bf16", "f16", "f32"]), o=half, dense=rng.random() < 0.5)
    if op == "read":
        seqs = _log(rng, 1, 40)
        hi = max(1, min(_log(rng, 1, 32768), 32768 * 8 * 128 // (seqs * kv * d)))
        return dict(op=op, seqs=seqs, lo=rng.choice([0, 1, hi // 2, hi]), hi=hi, kv=kv, d=d, page=page,
                    o=rng.choice(["bf16", "f16", "f32"]))
    if op == "paged":
        seqs, new = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 4, 7, 16])
        hi = max(1, min(_log(rng, 1, 131071), 2 ** 30 // (seqs * kv * d), 2 ** 28 // (seqs * heads * new)))
        return dict(op=op, seqs=seqs, new=new, lo=rng.choice([0, 1, hi // 2, hi]), hi=hi, heads=heads, kv=kv, d=d, page=page,
                    window=rng.choice([0, 0, 0, 100, 1024]), x=half)
    seqs = _log(rng, 1, 40)
    prefix = rng.choice([0, 0, 100, 1000])
    causal = rng.random() < 0.8
    room = 8192 * 8192 * 40 * 128 // (2 * seqs * heads * d)
    hi = max(1, min(_log(rng, 1, 8192), int(math.sqrt(room)) - prefix))
    return dict(op=op, seqs=seqs, lo=rng.choice([0, 1, hi // 2, hi]), hi=hi, prefix=prefix, heads=heads, kv=kv, d=d,
                causal=causal, window=rng.choice([0, 0, 0, 300]) if causal else 0, x=half)


def _size(t):
    return 4 if t == "f32" else 2


def _new_tokens(c):
    return _lengths(c["seqs"], 1, c["new"], "new")


def _prompt_lengths(c):
    """(queries, keys) of each sequence: the keys hold the prefix and the prompt itself."""
    nq = _lengths(c["seqs"], c["lo"], c["hi"])
    rng = random.Random("prefix %d %d" % (c["seqs"], c["prefix"]))
    return nq, [n + (rng.randrange(c["prefix"] + 1) if c["prefix"] else 0) for n in nq]


def _visible(first, count, window):
    """Keys that `count` queries from position `first` on see, in all."""
    total = 0
    for p in range(max(first, 0), first + count):
        total += min(p + 1, window) if window else p + 1
    return total


def work(c):
    d, kv = c["d"], c["kv"]
    if c["op"] == "write":
        m, heads = c["m"], c["heads"]
        cache = m * kv * (2 * d + 8)
        values = m * (heads + (2 * kv if c["dense"] else 0)) * d * 2
        # The cache is written and read, the values that it holds come back in FP32.
        return {"bytes": m * (heads + 2 * kv) * d * _size(c["x"]) + values + 4 * m * c["rot"] + 2 * cache + 8 * m * kv * d,
                "flops": 3 * m * (heads + kv) * c["rot"] + 4 * m * kv * d}
    if c["op"] == "read":
        n = sum(_lengths(c["seqs"], c["lo"], c["hi"]))
        return {"bytes": max(1, n * kv * (2 * d + 8) + 2 * n * kv * d * _size(c["o"])), "flops": 2 * n * kv * d}
    heads = c["heads"]
    if c["op"] == "paged":
        read, pairs, tokens = 0, 0, 0
        for n, t in zip(_lengths(c["seqs"], c["lo"], c["hi"]), _new_tokens(c)):
            pairs += _visible(n - t, t, c["window"])
            read += min(n, c["window"] + t - 1) if c["window"] else n
            tokens += t
        return {"bytes": read * kv * (2 * d + 8) + 2 * tokens * heads * d * 2, "flops": 4 * pairs * heads * d}
    nq, nk = _prompt_lengths(c)
    pairs = sum(_visible(b - a, a, c["window"]) if c["causal"] else a * b for a, b in zip(nq, nk))
    return {"bytes": max(1, (2 * sum(nq) * heads + 2 * sum(nk) * kv) * d * 2), "flops": 4 * pairs * heads * d}


# ---------------------------------------------------------------- inputs
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _starts(lengths):
    s = [0]
    for n in lengths:
        s.append(s[-1] + n)
    return _ints(s)


def _page_table(gen, lengths, page):
    """(table [sequences][most pages of one], pages): pages of the sequences shuffled over the cache, as after a while of serving."""
    width = max(1, max((n + page - 1) // page for n in lengths))
    used = len(lengths) * width
    order = torch.randperm(used + 3, generator=gen, device=DEV)[:used]
    return order.to(torch.int32).view(len(lengths), width), used + 3


def _parts(cache, page, kv, d):
    """Views of a cache [pages][page bytes]: key and value codes [pages][kv][page][d], their scales [pages][kv][page]."""
    c = cache.view(cache.shape[0], kv, page * (2 * d + 8))
    codes = c[:, :, :2 * page * d].view(torch.int8).unflatten(2, (2, page, d))
    scales = c[:, :, 2 * page * d:].view(torch.float32).unflatten(2, (2, page))
    return codes[:, :, 0], codes[:, :, 1], scales[:, :, 0], scales[:, :, 1]


def _filled_cache(gen, pages, page, kv, d):
    cache = torch.empty((pages, kv * page * (2 * d + 8)), dtype=torch.uint8, device=DEV)
    parts = _parts(cache, page, kv, d)
    for codes, spread in ((parts[0], 45.0), (parts[1], 40.0)):
        for at in range(0, pages, 4096):
            some = codes[at:at + 4096]
            some.copy_(torch.randn(some.shape, generator=gen, device=DEV).mul_(spread).round_().clamp_(-127, 127))
    for scales, typical in ((parts[2], 1.0 / 45), (parts[3], 1.0 / 40)):
        scales.copy_((torch.rand(scales.shape, generator=gen, device=DEV) + 0.5) * typical)
    return cache


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    s = dict(c)
    d, kv = c["d"], c["kv"]
    if c["op"] == "write":
        m, heads, page = c["m"], c["heads"], c["page"]
        x = torch.randn((m, heads + 2 * kv, d), generator=gen, device=DEV)
        hit = torch.rand(x.shape, generator=gen, device=DEV) < 0.001          # outliers, as projections have them
        x = torch.where(hit, 20.0 * x.sign(), x).to(DTYPES[c["x"]])
        s["q"], s["k"], s["v"] = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
        s["positions"] = torch.randint(0, TABLE_ROWS, (m,), generator=gen, device=DEV, dtype=torch.int32)
        s["cos"] = s["sin"] = None
        if c["rot"]:
            freq = 1e6 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEV) / c["rot"])
            angle = torch.arange(TABLE_ROWS, dtype=torch.float64, device=DEV)[:, None] * freq
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["table"], pages = _page_table(gen, [m], page)
        at = torch.arange(m, device=DEV)
        s["slots"] = (s["table"][0, at // page] * page + at % page).to(torch.int32)
        s["starts"] = _starts([m])
        s["cache"] = torch.zeros((pages, kv * page * (2 * d + 8)), dtype=torch.uint8, device=DEV)
        half = DTYPES[c["o"]]
        s["q_out"] = torch.empty((m, heads, d), dtype=half, device=DEV)
        s["k_out"], s["v_out"] = (torch.empty((m, kv, d), dtype=half, device=DEV) if c["dense"] else None for _ in "kv")
        s["k_back"], s["v_back"] = (torch.empty((m, kv, d), device=DEV) for _ in "kv")
        return s
    if c["op"] == "read":
        lengths = _lengths(c["seqs"], c["lo"], c["hi"])
        s["table"], pages = _page_table(gen, lengths, c["page"])
        s["cache"] = _filled_cache(gen, pages, c["page"], kv, d)
        s["starts"], s["rows"] = _starts(lengths), sum(lengths)
        s["k_out"], s["v_out"] = (torch.empty((s["rows"], kv, d), dtype=DTYPES[c["o"]], device=DEV) for _ in "kv")
        return s
    heads, dt = c["heads"], DTYPES[c["x"]]
    if c["op"] == "paged":
        lengths, new = _lengths(c["seqs"], c["lo"], c["hi"]), _new_tokens(c)
        s["table"], pages = _page_table(gen, lengths, c["page"])
        s["cache"] = _filled_cache(gen, pages, c["page"], kv, d)
        s["lens"], s["starts"] = _ints(lengths), _starts(new)
        s["q"] = (1.5 * torch.randn((sum(new), heads, d), generator=gen, device=DEV)).to(dt)
        s["out"] = torch.empty_like(s["q"])
        s["longest"] = max(lengths)
        if own:
            import gemm_int8_act_amd as pq2
            floats, words = pq2.pq2_attention_paged_workspace(c["seqs"], c["new"], heads, kv, d, max(1, s["longest"]))
            s["partials"] = torch.empty(floats, device=DEV)
            s["counters"] = torch.zeros(words, dtype=torch.int32, device=DEV)
        return s
    s["nq"], s["nk"] = _prompt_lengths(c)
    s["starts_q"], s["starts_k"] = _starts(s["nq"]), _starts(s["nk"])
    s["q"] = (1.5 * torch.randn((sum(s["nq"]), heads, d), generator=gen, device=DEV)).to(dt)
    s["k"] = torch.randn((sum(s["nk"]), kv, d), generator=gen, device=DEV).to(dt)
    s["v"] = torch.randn((sum(s["nk"]), kv, d), generator=gen, device=DEV).to(dt)
    s["out"] = torch.empty_like(s["q"])
    return s


# ---------------------------------------------------------------- plain forms
def _rotated(x, s):
    """x [m][heads][d] in FP32, its first rot elements turned by the position's angles."""
    rot = s["rot"]
    if not rot:
        return x.float()
    at = s["positions"].long()
    c, n = s["cos"][at][:, None], s["sin"][at][:, None]
    v = x.float()
    turned, rest = v[..., :rot], v[..., rot:]
    if s["inter"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * c - b * n, b * c + a * n], dim=-1).flatten(-2)
    else:
        a, b = turned[..., :rot // 2], turned[..., rot // 2:]
        turned = torch.cat([a * c - b * n, b * c + a * n], dim=-1)
    return torch.cat([turned, rest], dim=-1)


def _quantised(x):
    """INT8 codes and scales of rows; quotients go through 64 bits (values next to a border)."""
    scale = (x.abs().amax(dim=-1).double() / 127).float()
    by = torch.where(scale > 0, scale, torch.ones_like(scale)).double()
    return (x.double() / by[..., None]).float().round().clamp(-127, 127).to(torch.int8), scale


def _tokens_of(s):
    """(page, offset) in the cache of each row that a read gives."""
    starts = s["starts"].long()
    row = torch.arange(s["k_out"].shape[0] if s["op"] == "read" else s["m"], device=DEV)
    seq = torch.searchsorted(starts, row, right=True) - 1
    t = row - starts[seq]
    return s["table"].long()[seq, t // s["page"]], t % s["page"]


def _plain_read(s, dtype):
    kc, vc, ks, vs = _parts(s["cache"], s["page"], s["kv"], s["d"])
    page, at = _tokens_of(s)
    return [(c[page, :, at].float() * sc[page, :, at][..., None]).to(dtype) for c, sc in ((kc, ks), (vc, vs))]


def _plain_write(s):
    half = DTYPES[s["o"]]
    q, k, v = _rotated(s["q"], s), _rotated(s["k"], s), s["v"].float()
    parts = _parts(s["cache"], s["page"], s["kv"], s["d"])
    slot = s["slots"].long()
    page, at = slot // s["page"], slot % s["page"]
    kc, ks = _quantised(k)
    vc, vs = _quantised(v)
    parts[0][page, :, at], parts[1][page, :, at], parts[2][page, :, at], parts[3][page, :, at] = kc, vc, ks, vs
    out = [q.to(half)] + ([k.to(half), v.to(half)] if s["dense"] else [])
    return out + _plain_read(s, torch.float32)


def _softmax_rows(scores, seen):
    """Softmax over the seen columns; rows that see none are zero."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(dim=-1, keepdim=True)
    return p / torch.where(total > 0, total, torch.ones_like(total))


def _plain_paged(s):
    seqs, heads, kv, d, page, new = s["seqs"], s["heads"], s["kv"], s["d"], s["page"], s["new"]
    group, width = heads // kv, s["table"].shape[1] * s["page"]
    kc, vc, ks, vs = _parts(s["cache"], page, kv, d)
    table = s["table"].long()

    def gathered(codes, scales):                       # [seqs][kv][width][d] in FP32
        x = codes[table].float() * scales[table][..., None]
        return x.transpose(1, 2).reshape(seqs, kv, width, d)
    starts, lens = s["starts"].long(), s["lens"].long()
    i = torch.arange(new, device=DEV)
    there = i[None] < (starts[1:] - starts[:-1])[:, None]
    row = (starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(seqs, new, kv, group, d).permute(0, 2, 3, 1, 4).reshape(seqs, kv, group * new, d)
    position = lens[:, None] - (starts[1:] - starts[:-1])[:, None] + i                          # [seqs][new]
    j = torch.arange(width, device=DEV)
    seen = (j <= position[..., None]) & (j < lens[:, None, None])
    if s["window"]:
        seen = seen & (j > position[..., None] - s["window"])
    scores = (q @ gathered(kc, ks).transpose(2, 3).contiguous()) / math.sqrt(d)
    p = _softmax_rows(scores.view(seqs, kv, group, new, width), seen[:, None, None])
    o = p.view(seqs, kv, group * new, width) @ gathered(vc, vs)
    o = o.view(seqs, kv, group, new, d).permute(0, 3, 1, 2, 4).reshape(seqs, new, heads, d)
    return o[there].to(s["q"].dtype)


def _plain_prompt(s):
    heads, kv, d = s["heads"], s["kv"], s["d"]
    group = heads // kv
    out = s["out"]
    for q, k, v, o in zip(s["q"].split(s["nq"]), s["k"].split(s["nk"]), s["v"].split(s["nk"]), out.split(s["nq"])):
        nq, nk = q.shape[0], k.shape[0]
        if not nq:
            continue
        qf = q.float().view(nq, kv, group, d).permute(1, 2, 0, 3).reshape(kv, group * nq, d)
        kf = k.float().permute(1, 2, 0).contiguous()
        vf = v.float().transpose(0, 1).contiguous()
        i, j = torch.arange(nq, device=DEV)[:, None] + (nk - nq), torch.arange(nk, device=DEV)[None]
        seen = (j <= i) if s["causal"] else torch.ones((nq, nk), dtype=torch.bool, device=DEV)
        if s["window"]:
            seen = seen & (j > i - s["window"])
        p = _softmax_rows(((qf @ kf) / math.sqrt(d)).view(kv, group, nq, nk), seen).view(kv, group * nq, nk)
        o.copy_((p @ vf).view(kv, group, nq, d).permute(2, 0, 1, 3).reshape(nq, heads, d))
    return out


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "write":
        return _plain_write(s)
    if s["op"] == "read":
        return _plain_read(s, DTYPES[s["o"]])
    return _plain_paged(s) if s["op"] == "paged" else _plain_prompt(s)


# ---------------------------------------------------------------- the library's calls
def _run_own(s):
    import gemm_int8_act_amd as pq2
    if s["op"] == "write":
        pq2.pq2_kv_write(s["k"], s["v"], s["cache"], s["slots"], s["page"], q=s["q"], q_out=s["q_out"], k_out=s["k_out"],
                         v_out=s["v_out"], cos=s["cos"], sin=s["sin"], positions=s["positions"], interleaved=s["inter"])
        # The codes as the values they stand for.
        pq2.pq2_kv_read(s["cache"], s["table"], s["starts"], s["page"], s["k_back"], s["v_back"])
        return [s["q_out"]] + ([s["k_out"], s["v_out"]] if s["dense"] else []) + [s["k_back"], s["v_back"]]
    if s["op"] == "read":
        pq2.pq2_kv_read(s["cache"], s["table"], s["starts"], s["page"], s["k_out"], s["v_out"])
        return [s["k_out"], s["v_out"]]
    if s["op"] == "paged":
        pq2.pq2_attention_paged(s["q"], s["cache"], s["table"], s["lens"], s["page"], s["out"], s["partials"], s["counters"],
                                starts=s["starts"], max_new=s["new"], max_len=max(1, s["longest"]), window=s["window"])
        return s["out"]
    pq2.pq2_attention_prompt(s["q"], s["k"], s["v"], s["out"], s["starts_q"], s["starts_k"], causal=s["causal"],
                             window=s["window"])
    return s["out"]


# ---------------------------------------------------------------- 64 bits
def _exact_rotated(x, s):
    """By the definition: products and their sum are FP32 values, formed here from 64-bit ones."""
    v = x.double().clone()
    half = s["rot"] // 2
    if not half:
        return v
    step = lambda t: t.to(torch.float32).to(torch.float64)  # noqa: E731
    pos = s["positions"].tolist()
    cos, sin = (torch.stack([t[p] for p in pos]).double().unsqueeze(1) for t in (s["cos"], s["sin"]))
    first = torch.arange(half, device=DEV) * (2 if s["inter"] else 1)
    second = first + (1 if s["inter"] else half)
    a, b = v[:, :, first], v[:, :, second]
    v[:, :, first] = step(step(a * cos) - step(b * sin))
    v[:, :, second] = step(step(b * cos) + step(a * sin))
    return v


def _exact_codes_value(x):
    scale = (x.abs().max(dim=2).values / 127.0).to(torch.float32).to(torch.float64)
    by = torch.where(scale == 0, torch.ones_like(scale), scale).unsqueeze(2)
    return torch.round((x / by).to(torch.float32)).clamp(-127, 127).double() * scale.unsqueeze(2)


def _exact_rows(s, seq, length):
    """Keys and values [length][kv][d] of one sequence, page by page order of its table."""
    page, kv, d = s["page"], s["kv"], s["d"]
    n = (length + page - 1) // page
    raw = s["cache"][s["table"][seq, :n].long()].view(n, kv, page * (2 * d + 8))
    got = []
    for which in range(2):
        codes = raw[:, :, which * page * d:(which + 1) * page * d].contiguous().view(torch.int8).view(n, kv, page, d)
        at = 2 * page * d + which * page * 4
        scales = raw[:, :, at:at + page * 4].contiguous().view(torch.float32).view(n, kv, page, 1)
        rows = (codes.double() * scales.double()).permute(0, 2, 1, 3).reshape(n * page, kv, d)
        got.append(rows[:length])
    return got


def _exact_attention(q, k, v, first, window, causal=True):
    """o [n][heads][d] of queries at positions first, first + 1, ... among the keys, a head at a time."""
    n, heads, d = q.shape
    out = torch.zeros((n, heads, d), dtype=torch.float64, device=DEV)
    if not n or not k.shape[0]:
        return out
    gap = (first + torch.arange(n, device=DEV)).unsqueeze(1) - torch.arange(k.shape[0], device=DEV).unsqueeze(0)
    hidden = (gap < 0) if causal else torch.zeros_like(gap, dtype=torch.bool)
    if window:
        hidden = hidden | (gap >= window)
    for h in range(heads):
        g = h // (heads // k.shape[1])
        z = torch.mm(q[:, h].double(), k[:, g].double().t().contiguous()) * d ** -0.5
        z[hidden] = -math.inf
        w = torch.exp(z - torch.logsumexp(z, dim=1, keepdim=True)).nan_to_num(0.0)
        out[:, h] = torch.mm(w, v[:, g].double())
    return out


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "write":
        q, k, v = _exact_rotated(s["q"], s), _exact_rotated(s["k"], s), s["v"].double()
        return [q] + ([k, v] if c["dense"] else []) + [_exact_codes_value(k), _exact_codes_value(v)]
    if c["op"] == "read":
        rows = [_exact_rows(s, i, n) for i, n in enumerate(_lengths(c["seqs"], c["lo"], c["hi"]))]
        return [torch.cat([r[w] for r in rows]) for w in range(2)]
    if c["op"] == "paged":
        lengths, new, out, at = _lengths(c["seqs"], c["lo"], c["hi"]), _new_tokens(c), [], 0
        for i, (n, t) in enumerate(zip(lengths, new)):
            k, v = _exact_rows(s, i, n)
            out.append(_exact_attention(s["q"][at:at + t], k, v, n - t, c["window"]))
            at += t
        return torch.cat(out)
    out, q0, k0 = [], 0, 0
    for a, b in zip(s["nq"], s["nk"]):
        out.append(_exact_attention(s["q"][q0:q0 + a], s["k"][k0:k0 + b], s["v"][k0:k0 + b], b - a, c["window"], c["causal"]))
        q0, k0 = q0 + a, k0 + b
    return torch.cat(out)
