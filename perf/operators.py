"""Measured cases of the operators around the packed matmul: products with 4-bit
weights, the gated feed-forward product, and the block norms with their
quantiser.

Where ``own`` is false every operator runs in its plain form (elementary torch
operations); where it is true the library's entry points run.
"""
import math

import torch

own = False

GROUP = 128                 # activations per INT8 scale in the two products
BLOCK_BYTES = 34            # raw ternary block: fp16 scale, 32 code bytes
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
DEV = "cuda"


# ---------------------------------------------------------------- cases
def listed():
    return [
        # The smallest correctness shape of the repository's workloads, one token: latency only.
        dict(name="w4 tiny 1", op="w4", m=1, n=1024, k=512, wg=32, x="bf16"),
        # Attention QKV projection in decode, one token.
        dict(name="w4 qkv 1", op="w4", m=1, n=10240, k=5120, wg=128, x="bf16"),
        # FFN down projection, four tokens verified together, fine weight groups.
        dict(name="w4 down 4", op="w4", m=4, n=5120, k=17408, wg=32, x="f32"),
        # The same projection at the widest verification batch.
        dict(name="w4 down 16", op="w4", m=16, n=5120, k=17408, wg=64, x="bf16"),
        # Gate-sized projection of a prompt of 512 tokens.
        dict(name="w4 gate 512", op="w4", m=512, n=6144, k=5120, wg=128, x="bf16"),
        # Ternary feed-forward in decode, one token: gate and up together.
        dict(name="gated ternary 1", op="gated", m=1, n=17408, k=5120, wg=0, x="bf16", act="silu", h="bf16"),
        # 4-bit feed-forward, eight tokens verified together.
        dict(name="gated w4 8", op="gated", m=8, n=17408, k=5120, wg=128, x="bf16", act="silu", h="bf16"),
        # A short prompt through a small odd layer: ragged rows, groups and tokens.
        dict(name="gated w4 ragged 37", op="gated", m=37, n=1000, k=1152, wg=32, x="f16", act="gelu", h="f16"),
        # Ternary feed-forward of a prompt of 1024 tokens.
        dict(name="gated ternary 1024", op="gated", m=1024, n=17408, k=5120, wg=0, x="bf16", act="silu", h="bf16"),
        # Between two blocks in decode: add the block's output to the stream, norm it, quantise it.
        dict(name="norm 1", op="norm", m=1, k=5120, ag=128, r="bf16", post=False, gate="none", out="q"),
        # Verification of 16 tokens through a model with norms on both sides and a gate per channel.
        dict(name="norm 16 post", op="norm", m=16, k=5120, ag=32, r="f32", post=True, gate="row", out="q"),
        # A long prompt, norms on both sides, a gate per token and channel, activations out for another reader.
        dict(name="norm 4096 post", op="norm", m=4096, k=5120, ag=128, r="bf16", post=True, gate="full", out="x"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["w4", "gated", "norm"])
    k = 128 * _log(rng, 1, 136)
    if op == "norm":
        m = min(_log(rng, 1, 4096), 4096 * 5120 // k)
        return dict(op=op, m=m, k=k, ag=rng.choice([128, 64, 32]), r=rng.choice(["bf16", "f16", "f32"]),
                    post=rng.random() < 0.5, gate=rng.choice(["none", "row", "full"]), out=rng.choice(["q", "x"]))
    n = _log(rng, 1, 17408)
    m = max(1, min(_log(rng, 1, 1024), 1024 * 17408 * 5120 // (n * k)))
    if op == "w4":
        return dict(op=op, m=m, n=n, k=k, wg=rng.choice([128, 64, 32]), x=rng.choice(["bf16", "f16", "f32"]))
    return dict(op=op, m=m, n=n, k=k, wg=rng.choice([0, 128, 64, 32]), x=rng.choice(["bf16", "f16", "f32"]),
                act=rng.choice(["silu", "gelu"]), h=rng.choice(["bf16", "f16", "f32"]))


def work(c):
    m, k = c["m"], c["k"]
    size = lambda t: 4 if t == "f32" else 2  # noqa: E731
    if c["op"] == "norm":
        # Block output and stream in, stream and codes (or activations) out, the weights once.
        per = 4 + 2 * size(c["r"]) + (2 if c["gate"] == "full" else 0)
        out = m * k + 4 * m * (k // c["ag"]) if c["out"] == "q" else 2 * m * k
        weights = 2 * k * (1 + (1 if c["post"] else 0) + (1 if c["gate"] == "row" else 0))
        return {"bytes": m * k * per + out + weights, "flops": m * k * (12 + (4 if c["post"] else 0))}
    n = c["n"]
    if c["wg"]:
        weight = n * k // 2 + 2 * n * (k // c["wg"])
    else:
        weight = n * (k // GROUP) * BLOCK_BYTES
    if c["op"] == "w4":
        return {"bytes": weight + m * k * size(c["x"]) + 4 * m * n, "flops": 2 * m * n * k}
    return {"bytes": 2 * weight + m * k * size(c["x"]) + m * n * size(c["h"]), "flops": 4 * m * n * k}


# ---------------------------------------------------------------- inputs
def _weights(gen, n, k, wg):
    """(codes, scales) of 4-bit weights, two codes a byte (the even weight in the low half), or (raw blocks, None) of
    ternary ones."""
    if wg:
        c = torch.randn((n, k), generator=gen, device=DEV).mul_(2.5).round_().add_(8).clamp_(0, 15).to(torch.uint8)
        codes = (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()
        scales = (torch.rand((n, k // wg), generator=gen, device=DEV) * 0.045 + 0.005).to(torch.float16)
        return codes, scales
    g = k // GROUP
    c = torch.randint(0, 3, (n, g, 32, 4), generator=gen, device=DEV, dtype=torch.uint8)
    code_bytes = c[..., 0] | (c[..., 1] << 2) | (c[..., 2] << 4) | (c[..., 3] << 6)
    scales = (torch.rand((n, g, 1), generator=gen, device=DEV) * 0.045 + 0.005).to(torch.float16)
    return torch.cat([scales.view(torch.uint8), code_bytes], dim=2).reshape(n, g * BLOCK_BYTES).contiguous(), None


def _prepared(weights, n, k, wg):
    """The library's layout of a weight matrix, made once when a model is loaded."""
    import gemm_int8_act_amd as pq2
    codes, scales = weights
    if wg:
        tiles = torch.empty(pq2.pq2_w4_tiles_bytes(n, k, wg), dtype=torch.uint8, device=DEV)
        pq2.pq2_prepare_w4_tiles(codes, scales, wg, tiles)
    else:
        tiles = torch.empty(pq2.pq2_tiles_bytes(n, k), dtype=torch.uint8, device=DEV)
        pq2.pq2_prepare_tiles(codes, n, k, tiles)
    return tiles


def prepare(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    m, k = c["m"], c["k"]
    s = dict(c)
    if c["op"] == "norm":
        dt = DTYPES[c["r"]]
        vec = lambda: (1 + 0.1 * torch.randn(k, generator=gen, device=DEV)).to(torch.bfloat16)  # noqa: E731
        s["stream_in"] = (torch.randn((m, k), generator=gen, device=DEV) * 1.5).to(dt)
        s["block"] = torch.randn((m, k), generator=gen, device=DEV) * 0.7
        s["w"] = vec()
        s["w_post"] = vec() if c["post"] else None
        s["gate"] = None
        if c["gate"] != "none":
            shape = (k,) if c["gate"] == "row" else (m, k)
            s["gate"] = (0.5 * torch.randn(shape, generator=gen, device=DEV)).to(torch.bfloat16)
        s["alpha"], s["eps"] = 0.25, 1e-6
        s["stream_out"] = torch.empty_like(s["stream_in"])
        if c["out"] == "q":
            s["q"] = torch.empty((m, k), dtype=torch.int8, device=DEV)
            s["xs"] = torch.empty((m, k // c["ag"]), dtype=torch.float32, device=DEV)
        else:
            s["x_out"] = torch.empty((m, k), dtype=torch.bfloat16, device=DEV)
        return s
    n, wg = c["n"], c["wg"]
    x = torch.randn((m, k), generator=gen, device=DEV)
    hit = torch.rand((m, k), generator=gen, device=DEV) < 0.001      # outliers, as the attention inputs have them
    s["input"] = torch.where(hit, 20.0 * x.sign(), x).to(DTYPES[c["x"]])
    names = ("w",) if c["op"] == "w4" else ("gate", "up")
    s["raw"] = [_weights(gen, n, k, wg) for _ in names]
    s["out"] = torch.empty((m, n), dtype=torch.float32 if c["op"] == "w4" else DTYPES[c["h"]], device=DEV)
    s["q_work"] = torch.empty((m, k), dtype=torch.int8, device=DEV)
    s["xs_work"] = torch.empty((m, k // GROUP), dtype=torch.float32, device=DEV)
    if own:
        s["tiles"] = [_prepared(w, n, k, wg) for w in s["raw"]]
    return s


# ---------------------------------------------------------------- plain forms
def _quantised(x, group):
    """INT8 codes [m][groups][group] and scales [m][groups]; quotients go through 64 bits (values next to a border)."""
    v = x.float().view(x.shape[0], -1, group)
    xs = (v.abs().amax(dim=2).double() / 127).float()
    d = torch.where(xs > 0, xs, torch.ones_like(xs)).double()
    q = (v.double() / d.unsqueeze(2)).float().round().clamp(-127, 127)
    return q, xs


def _dequantised(weights, k, wg):
    codes, scales = weights
    n = codes.shape[0]
    if wg:
        w = torch.stack([codes & 15, codes >> 4], dim=2).view(n, k // wg, wg).float() - 8
        return (w * scales.float().unsqueeze(2)).view(n, k)
    blocks = codes.view(n, k // GROUP, BLOCK_BYTES)
    ws = blocks[:, :, :2].contiguous().view(torch.float16).float()
    b = blocks[:, :, 2:]
    w = torch.stack([b & 3, (b >> 2) & 3, (b >> 4) & 3, b >> 6], dim=3).view(n, k // GROUP, GROUP).float() - 1
    return (w * ws).view(n, k)


def _plain_product(a, weights, k, wg):
    return a @ _dequantised(weights, k, wg).t()


def _activation(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g)))


def _rstd(v, eps):
    """1 / root of the mean square, summed in 64 bits, rounded once: the codes behind it are compared one by one."""
    return (1 / torch.sqrt(v.double().square().mean(dim=1, keepdim=True) + eps)).float()


def _plain_norm(s):
    t = s["block"]
    if s["w_post"] is not None:
        t = t * _rstd(t, s["eps"]) * s["w_post"].float()
    if s["gate"] is not None:
        t = t * s["gate"].float()
    t = t * s["alpha"]
    stream = (s["stream_in"].float() + t).to(s["stream_in"].dtype)
    v = stream.float()
    x = (v * _rstd(v, s["eps"]) * s["w"].float()).to(torch.bfloat16)
    if "x_out" in s:
        return [stream, x]
    q, xs = _quantised(x, s["ag"])
    return [stream, xs, q * xs.unsqueeze(2)]


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "norm":
        return _plain_norm(s)
    k, wg = s["k"], s["wg"]
    q, xs = _quantised(s["input"], GROUP)
    a = (q * xs.unsqueeze(2)).view(-1, k)
    y = _plain_product(a, s["raw"][0], k, wg)
    if s["op"] == "w4":
        return y
    return (_activation(y, s["act"]) * _plain_product(a, s["raw"][1], k, wg)).to(DTYPES[s["h"]])


# ---------------------------------------------------------------- the library's calls
def _run_own(s):
    import gemm_int8_act_amd as pq2
    if s["op"] == "norm":
        pq2.pq2_block_norm(s["stream_in"], s["w"], s["eps"], x_dtype=torch.bfloat16, block=s["block"],
                           post_w=s["w_post"], gate=s["gate"], alpha=s["alpha"], r_out=s["stream_out"],
                           q=s.get("q"), xs=s.get("xs"), agroup=s["ag"], x_out=s.get("x_out"))
        if "x_out" in s:
            return [s["stream_out"], s["x_out"]]
        # The codes as the values they stand for.
        return [s["stream_out"], s["xs"], s["q"].view(s["m"], -1, s["ag"]) * s["xs"].unsqueeze(2)]
    if s["op"] == "w4":
        pq2.pq2_linear_w4(s["input"], s["tiles"][0], s["out"], s["wg"], s["q_work"], s["xs_work"])
        return s["out"]
    act = pq2.ACT_SILU if s["act"] == "silu" else pq2.ACT_GELU_TANH
    if s["wg"]:
        pq2.pq2_gated_linear_w4(s["input"], s["tiles"][0], s["tiles"][1], s["out"], s["wg"], s["q_work"],
                                s["xs_work"], act)
    else:
        pq2.pq2_gated_linear_tiles(s["input"], s["tiles"][0], s["tiles"][1], s["out"], s["q_work"], s["xs_work"], act)
    return s["out"]


# ---------------------------------------------------------------- 64 bits
def _exact_codes(x, group):
    """Codes and scales by the definition: both quotients are FP32 values, formed here from 64-bit ones."""
    m, k = x.shape
    v = x.to(torch.float64).reshape(m, k // group, group)
    scale = (v.abs().max(dim=2).values / 127.0).to(torch.float32).to(torch.float64)
    by = torch.where(scale == 0, torch.ones_like(scale), scale)
    codes = torch.clamp(torch.round((v / by[:, :, None]).to(torch.float32)), -127, 127).to(torch.float64)
    return codes, scale


def _exact_product(codes, scale, weights, k, wg):
    """Sum over weight groups of (exact dot) * (activation scale) * (weight scale)."""
    raw, ws = weights
    n = raw.shape[0]
    step = wg or GROUP
    per = GROUP // step
    y = torch.zeros((codes.shape[0], n), dtype=torch.float64, device=DEV)
    for i in range(k // step):
        a = codes[:, i // per, (i % per) * step:(i % per + 1) * step]
        if wg:
            b = raw[:, i * step // 2:(i + 1) * step // 2].to(torch.int64)
            c = torch.empty((n, step), dtype=torch.float64, device=DEV)
            c[:, 0::2], c[:, 1::2] = (b % 16 - 8).double(), (b // 16 - 8).double()
            f = ws[:, i].double()
        else:
            b = raw[:, i * BLOCK_BYTES:(i + 1) * BLOCK_BYTES]
            c = torch.empty((n, step), dtype=torch.float64, device=DEV)
            for field in range(4):
                c[:, field::4] = (b[:, 2:].to(torch.int64) // 4 ** field % 4 - 1).double()
            f = b[:, :2].contiguous().view(torch.float16)[:, 0].double()
        y += (a.contiguous() @ c.t().contiguous()) * scale[:, i // per, None] * f[None, :]
    return y


def exact(c, seed):
    s = prepare(c, seed)
    k = c["k"]
    if c["op"] == "norm":
        def normed(v, w):
            return v / torch.sqrt((v * v).sum(1, keepdim=True) / k + s["eps"]) * w.double()
        t = s["block"].double()
        if s["w_post"] is not None:
            t = normed(t, s["w_post"])
        if s["gate"] is not None:
            t = t * s["gate"].double()
        stream = s["stream_in"].double() + s["alpha"] * t
        x = normed(stream.to(s["stream_in"].dtype).double(), s["w"])
        if c["out"] == "x":
            return [stream, x]
        codes, scale = _exact_codes(x.to(torch.bfloat16), c["ag"])
        return [stream, scale, codes * scale[:, :, None]]
    codes, scale = _exact_codes(s["input"], GROUP)
    y = _exact_product(codes, scale, s["raw"][0], k, c["wg"])
    if c["op"] == "w4":
        return y
    u = _exact_product(codes, scale, s["raw"][1], k, c["wg"])
    if c["act"] == "silu":
        return y * u * torch.sigmoid(y)
    return y * u * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
