"""The attention operators' C ABI without a GPU: the symbols of
pq2_attention.h are exported and bound, the argument structures are the
header's, and bad arguments are refused on the host (every case fails
validation or the device check, so nothing is launched)."""
import ctypes
import os
import re
import struct
import subprocess

import pytest
import torch

import attention_reference as ref
import gemm_int8_act_amd as pq2
from gemm_int8_act_amd import _marshal

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, EINVAL, ESHAPE, EALIGN, EDEVICE = pq2.PQ2_OK, pq2.PQ2_EINVAL, pq2.PQ2_ESHAPE, pq2.PQ2_EALIGN, pq2.PQ2_EDEVICE

# Fake device addresses, never dereferenced: validation fails first.
A, B, C, D, E, F, G, H, I, J, K, L = (0x7F0000000000 + (i << 38) for i in range(12))
CTYPES = {"P": ctypes.c_void_p, "q": ctypes.c_int64, "f": ctypes.c_float, "i": ctypes.c_int}

no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="the device check passes on a GPU")


# The argument structures of include/pq2_attention.h: the fields in order, with
# their native struct codes.
WRITE_FIELDS = (
    ("q", "P"), ("k", "P"), ("v", "P"),
    ("q_stride", "q"), ("q_head", "q"), ("k_stride", "q"), ("k_head", "q"), ("v_stride", "q"), ("v_head", "q"),
    ("q_out", "P"), ("k_out", "P"), ("v_out", "P"),
    ("qo_stride", "q"), ("qo_head", "q"), ("ko_stride", "q"), ("ko_head", "q"), ("vo_stride", "q"), ("vo_head", "q"),
    ("cos", "P"), ("sin", "P"), ("positions", "P"), ("slots", "P"), ("cache", "P"),
    ("m", "q"), ("heads", "q"), ("kv_heads", "q"), ("head_dim", "q"), ("rot_dim", "q"), ("table_rows", "q"),
    ("pages", "q"), ("page_tokens", "q"),
    ("in_dtype", "i"), ("out_dtype", "i"), ("interleaved", "i"),
)
READ_FIELDS = (
    ("cache", "P"), ("table", "P"), ("starts", "P"), ("k_out", "P"), ("v_out", "P"),
    ("ko_stride", "q"), ("ko_head", "q"), ("vo_stride", "q"), ("vo_head", "q"),
    ("rows", "q"), ("seqs", "q"), ("table_stride", "q"), ("table_pages", "q"), ("kv_heads", "q"), ("head_dim", "q"),
    ("pages", "q"), ("page_tokens", "q"),
    ("out_dtype", "i"),
)
PAGED_FIELDS = (
    ("q", "P"), ("out", "P"), ("q_stride", "q"), ("q_head", "q"), ("out_stride", "q"), ("out_head", "q"),
    ("cache", "P"), ("table", "P"), ("lens", "P"), ("starts", "P"), ("partials", "P"), ("counters", "P"),
    ("rows", "q"), ("seqs", "q"), ("table_stride", "q"), ("table_pages", "q"), ("heads", "q"), ("kv_heads", "q"),
    ("head_dim", "q"), ("pages", "q"), ("page_tokens", "q"), ("max_new", "q"), ("max_len", "q"), ("window", "q"),
    ("scale", "f"), ("dtype", "i"),
)
PROMPT_FIELDS = (
    ("q", "P"), ("k", "P"), ("v", "P"), ("out", "P"),
    ("q_stride", "q"), ("q_head", "q"), ("k_stride", "q"), ("k_head", "q"), ("v_stride", "q"), ("v_head", "q"),
    ("out_stride", "q"), ("out_head", "q"),
    ("starts_q", "P"), ("starts_k", "P"),
    ("rows_q", "q"), ("rows_k", "q"), ("seqs", "q"), ("heads", "q"), ("kv_heads", "q"), ("head_dim", "q"),
    ("window", "q"), ("scale", "f"), ("dtype", "i"), ("causal", "i"),
)


def packer(fields):
    # The structure ends at a multiple of its widest member, as in C.
    return struct.Struct("@" + "".join(code for _, code in fields) + "0q")


def structure(name, fields):
    return type(name, (ctypes.Structure,), {"_fields_": [(f, CTYPES[c]) for f, c in fields]})


STRUCTS = {"pq2_kv_write_args": (WRITE_FIELDS, packer(WRITE_FIELDS)),
           "pq2_kv_read_args": (READ_FIELDS, packer(READ_FIELDS)),
           "pq2_attention_paged_args": (PAGED_FIELDS, packer(PAGED_FIELDS)),
           "pq2_attention_prompt_args": (PROMPT_FIELDS, packer(PROMPT_FIELDS))}


def test_header_symbols_exported():
    text = open(os.path.join(ROOT, "include", "pq2_attention.h")).read()
    names = set(re.findall(r"^(?:int|int64_t)\s+(pq2_\w+)\s*\(", text, re.M))
    assert names == set(pq2.ATTENTION_EXPORTED)
    for name in names:
        assert hasattr(pq2.lib, name) and hasattr(pq2, name), name


@pytest.mark.parametrize("name", list(STRUCTS))
def test_args_struct_matches_the_header(tmp_path, name):
    """Field order and offsets of the structures used here, by the C compiler."""
    fields, packer = STRUCTS[name]
    cls = structure(name, fields)
    src = tmp_path / "offsets.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "pq2_attention.h"\nint main(void) {\n'
                   + "".join(f'printf("%zu\\n", offsetof({name}, {f}));\n' for f, _ in fields)
                   + f'printf("%zu\\n", sizeof({name})); return 0; }}\n')
    exe = tmp_path / "offsets"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [getattr(cls, f).offset for f, _ in fields] + [ctypes.sizeof(cls)]
    values = [i + 1 if code != "f" else (i + 1) / 2 for i, (_, code) in enumerate(fields)]
    a = cls(**{f: v for (f, _), v in zip(fields, values)})
    assert packer.pack(*values) == bytes(a)


def test_page_bytes():
    f = pq2.pq2_kv_page_bytes
    assert f(16, 8, 128) == 8 * 16 * 264 and f(256, 1, 64) == 256 * 136 and f(32, 4, 256) == 4 * 32 * 520
    for p, kv, d in ((8, 1, 64), (24, 1, 64), (512, 1, 64), (16, 0, 64), (16, 1025, 64), (16, 1, 96), (16, 1, 512)):
        with pytest.raises(ValueError):
            f(p, kv, d)


def test_reference_cache_views():
    """The reference's views address the layout that the header states."""
    page, kv, d = 32, 3, 64
    cache = torch.arange(2 * kv * page * (2 * d + 8), dtype=torch.int64).remainder(251).to(torch.uint8).view(2, -1)
    kc, vc, ks, vs = ref.parts(cache, page, kv, d)
    flat = cache.flatten()
    block = page * (2 * d + 8)
    for p, h, t, e in ((0, 0, 0, 0), (1, 2, 31, 63), (1, 1, 7, 20)):
        at = (p * kv + h) * block
        assert int(kc[p, h, t, e]) == int(flat[at + t * d + e].view(torch.int8))
        assert int(vc[p, h, t, e]) == int(flat[at + page * d + t * d + e].view(torch.int8))
        for s, o in ((ks, 2 * page * d), (vs, 2 * page * d + 4 * page)):
            assert torch.equal(s[p, h, t].contiguous().view(torch.int32), flat[at + o + 4 * t:at + o + 4 * t + 4].view(torch.int32)[0])


def call(name, **over):
    fields, packer = STRUCTS[name + "_args"]
    base = {
        "pq2_kv_write": dict(q=A, k=B, v=C, q_stride=1024, q_head=128, k_stride=256, k_head=128, v_stride=256, v_head=128,
                             q_out=D, k_out=E, v_out=F, qo_stride=1024, qo_head=128, ko_stride=256, ko_head=128,
                             vo_stride=256, vo_head=128, cos=G, sin=H, positions=I, slots=J, cache=K, m=5, heads=8, kv_heads=2,
                             head_dim=128, rot_dim=128, table_rows=100, pages=7, page_tokens=16, in_dtype=2, out_dtype=0,
                             interleaved=0),
        "pq2_kv_read": dict(cache=A, table=B, starts=C, k_out=D, v_out=E, ko_stride=256, ko_head=128, vo_stride=256,
                            vo_head=128, rows=9, seqs=2, table_stride=4, table_pages=4, kv_heads=2, head_dim=128, pages=7,
                            page_tokens=16, out_dtype=2),
        "pq2_attention_paged": dict(q=A, out=B, q_stride=1024, q_head=128, out_stride=1024, out_head=128, cache=C, table=D, lens=E,
                                    starts=F, partials=G, counters=H, rows=6, seqs=3, table_stride=300, table_pages=300, heads=8,
                                    kv_heads=2, head_dim=128, pages=700, page_tokens=16, max_new=2, max_len=4800, window=0,
                                    scale=0.1, dtype=0),
        "pq2_attention_prompt": dict(q=A, k=B, v=C, out=D, q_stride=1024, q_head=128, k_stride=256, k_head=128, v_stride=256,
                                     v_head=128, out_stride=1024, out_head=128, starts_q=E, starts_k=F, rows_q=50, rows_k=60,
                                     seqs=3, heads=8, kv_heads=2, head_dim=128, window=0, scale=0.1, dtype=0, causal=1),
    }[name]
    base.update(over)
    return getattr(pq2.lib, name)(packer.pack(*[base[f] or 0 for f, _ in fields]), None)


GOOD = ("pq2_kv_write", "pq2_kv_read", "pq2_attention_paged", "pq2_attention_prompt")


@no_gpu
@pytest.mark.parametrize("name", GOOD)
def test_good_arguments_reach_the_device_check(name):
    assert call(name) == EDEVICE


@pytest.mark.parametrize("name", GOOD)
def test_null_args(name):
    assert getattr(pq2.lib, name)(None, None) == EINVAL


REFUSED = {
    "pq2_kv_write": [
        (EINVAL, dict(k=0)), (EINVAL, dict(v=0)), (EINVAL, dict(q=0)), (EINVAL, dict(q_out=0)), (EINVAL, dict(cos=0)),
        (EINVAL, dict(sin=0)), (EINVAL, dict(positions=0)), (EINVAL, dict(slots=0)),
        (EINVAL, dict(cache=0, q=0, q_out=0, k_out=0, v_out=0)), (EINVAL, dict(in_dtype=3)), (EINVAL, dict(out_dtype=-1)),
        (EINVAL, dict(interleaved=2)), (ESHAPE, dict(m=0)), (ESHAPE, dict(m=(1 << 24) + 1)), (ESHAPE, dict(heads=7)),
        (ESHAPE, dict(heads=1)), (ESHAPE, dict(heads=2048)), (ESHAPE, dict(kv_heads=0)), (ESHAPE, dict(head_dim=96)),
        (ESHAPE, dict(rot_dim=4)), (ESHAPE, dict(rot_dim=136)), (ESHAPE, dict(rot_dim=-8)), (ESHAPE, dict(table_rows=0)),
        (ESHAPE, dict(table_rows=1 << 31)), (ESHAPE, dict(pages=0)), (ESHAPE, dict(pages=1 << 28)), (ESHAPE, dict(page_tokens=24)),
        (ESHAPE, dict(q_stride=1000)), (ESHAPE, dict(k_stride=64)), (ESHAPE, dict(v_head=64)), (ESHAPE, dict(q_stride=1 << 24)),
        (ESHAPE, dict(vo_head=(1 << 31) + 4)), (EALIGN, dict(k_stride=258)), (EALIGN, dict(qo_stride=1028)),
        (EALIGN, dict(k=B + 8)), (EALIGN, dict(v_out=F + 2)), (EALIGN, dict(cache=K + 8)), (EALIGN, dict(cos=G + 4)),
        (EALIGN, dict(slots=J + 2)), (EALIGN, dict(positions=I + 1)),
        (EINVAL, dict(q_out=A)), (EINVAL, dict(k_out=B, out_dtype=2, ko_stride=512)), (EINVAL, dict(q_out=B)), (EINVAL, dict(v_out=E)),
        (EINVAL, dict(cache=A)), (EINVAL, dict(k_out=J)), (EINVAL, dict(k_out=G)), (EINVAL, dict(q_out=K)),
        # one buffer's columns: the next row of q_out would meet k's
        (EINVAL, dict(q=A, k=A + 4096, v=A + 5120, q_stride=1536, k_stride=1536, v_stride=1536, q_out=A + 16, qo_stride=1536, out_dtype=2)),
    ],
    "pq2_kv_read": [
        (EINVAL, dict(cache=0)), (EINVAL, dict(table=0)), (EINVAL, dict(starts=0)), (EINVAL, dict(k_out=0)), (EINVAL, dict(v_out=0)),
        (EINVAL, dict(out_dtype=5)), (ESHAPE, dict(rows=0)), (ESHAPE, dict(seqs=0)), (ESHAPE, dict(seqs=65536)),
        (ESHAPE, dict(table_pages=0)), (ESHAPE, dict(table_stride=3)), (ESHAPE, dict(table_pages=1 << 27, table_stride=1 << 27)),
        (ESHAPE, dict(head_dim=32)), (ESHAPE, dict(kv_heads=0)), (ESHAPE, dict(pages=0)), (ESHAPE, dict(page_tokens=0)),
        (ESHAPE, dict(ko_stride=200)), (EALIGN, dict(ko_stride=257)), (EALIGN, dict(k_out=D + 4)), (EALIGN, dict(cache=A + 4)),
        (EALIGN, dict(table=B + 2)), (EALIGN, dict(starts=C + 3)), (EINVAL, dict(k_out=E)), (EINVAL, dict(k_out=A)),
        (EINVAL, dict(v_out=B)), (EINVAL, dict(v_out=C)),
    ],
    "pq2_attention_paged": [
        (EINVAL, dict(q=0)), (EINVAL, dict(out=0)), (EINVAL, dict(cache=0)), (EINVAL, dict(table=0)), (EINVAL, dict(lens=0)),
        (EINVAL, dict(dtype=2)), (EINVAL, dict(scale=0.0)), (EINVAL, dict(scale=-1.0)), (EINVAL, dict(scale=float("nan"))),
        (EINVAL, dict(scale=float("inf"))), (EINVAL, dict(window=-1)), (EINVAL, dict(partials=0)), (EINVAL, dict(counters=0)),
        (ESHAPE, dict(starts=0)), (ESHAPE, dict(seqs=0)), (ESHAPE, dict(seqs=65536)), (ESHAPE, dict(max_new=0)),
        (ESHAPE, dict(max_len=0)), (ESHAPE, dict(heads=9)), (ESHAPE, dict(kv_heads=3)), (ESHAPE, dict(head_dim=80)),
        (ESHAPE, dict(rows=0)), (ESHAPE, dict(page_tokens=20)), (ESHAPE, dict(pages=0)), (ESHAPE, dict(table_pages=0)),
        (ESHAPE, dict(table_stride=299)), (ESHAPE, dict(table_pages=1 << 27, table_stride=1 << 27)), (ESHAPE, dict(q_stride=512)),
        (ESHAPE, dict(max_new=1 << 24, seqs=65535)), (EALIGN, dict(q_stride=1028)), (EALIGN, dict(q=A + 8)), (EALIGN, dict(out=B + 4)),
        (EALIGN, dict(cache=C + 8)), (EALIGN, dict(table=D + 2)), (EALIGN, dict(lens=E + 1)), (EALIGN, dict(starts=F + 2)),
        (EALIGN, dict(partials=G + 4)), (EALIGN, dict(counters=H + 2)), (EINVAL, dict(out=A)), (EINVAL, dict(out=C)),
        (EINVAL, dict(out=E)), (EINVAL, dict(partials=A)), (EINVAL, dict(counters=G)), (EINVAL, dict(counters=D)),
    ],
    "pq2_attention_prompt": [
        (EINVAL, dict(q=0)), (EINVAL, dict(k=0)), (EINVAL, dict(v=0)), (EINVAL, dict(out=0)), (EINVAL, dict(starts_q=0)),
        (EINVAL, dict(starts_k=0)), (EINVAL, dict(dtype=2)), (EINVAL, dict(causal=2)), (EINVAL, dict(scale=0.0)),
        (EINVAL, dict(scale=float("inf"))), (EINVAL, dict(window=-5)), (EINVAL, dict(window=5, causal=0)), (ESHAPE, dict(rows_q=0)),
        (ESHAPE, dict(rows_k=0)), (ESHAPE, dict(rows_q=(1 << 24) + 1)), (ESHAPE, dict(rows_q=1 << 24, heads=128, kv_heads=1, q_stride=1 << 14, out_stride=1 << 14)), (ESHAPE, dict(seqs=0)), (ESHAPE, dict(seqs=65536)),
        (ESHAPE, dict(heads=5)), (ESHAPE, dict(head_dim=160)), (ESHAPE, dict(k_stride=200)), (ESHAPE, dict(v_stride=1 << 24)),
        (EALIGN, dict(v_stride=260)), (EALIGN, dict(k=B + 2)), (EALIGN, dict(out=D + 8)), (EALIGN, dict(starts_q=E + 2)),
        (EINVAL, dict(out=A)), (EINVAL, dict(out=B)), (EINVAL, dict(out=C)), (EINVAL, dict(out=F)),
    ],
}


@pytest.mark.parametrize("name,status,over", [(n, s, o) for n, cases in REFUSED.items() for s, o in cases])
def test_refused(name, status, over):
    assert call(name, **over) == status


@no_gpu
@pytest.mark.parametrize("name,over", [
    # no q, no rotation, no dense outputs: their fields are not read
    ("pq2_kv_write", dict(q=0, q_out=0, heads=0, k_out=0, v_out=0, rot_dim=0, cos=0, sin=0, positions=0, table_rows=0)),
    # the rotation alone
    ("pq2_kv_write", dict(cache=0, slots=0, pages=0, page_tokens=0, v_out=0)),
    # in place; columns of one buffer; heads outside the rows
    ("pq2_kv_write", dict(q_out=A, k_out=B, out_dtype=2)),
    ("pq2_kv_write", dict(q=A, k=A + 4096, v=A + 5120, q_stride=1536, k_stride=1536, v_stride=1536, q_out=A, qo_stride=1536, k_out=A + 4096,
                          ko_stride=1536, v_out=0, out_dtype=2)),
    ("pq2_kv_write", dict(q_stride=128, q_head=640, k_stride=128, k_head=640)),
    # nothing is split: no workspace
    ("pq2_attention_paged", dict(max_len=200, partials=0, counters=0)),
    ("pq2_attention_paged", dict(starts=0, rows=3)),
    # q and out columns of one buffer
    ("pq2_attention_paged", dict(out=A + 2048, q_stride=2048, out_stride=2048)),
    ("pq2_attention_prompt", dict(out=A + 2048, q_stride=2048, out_stride=2048)),
    ("pq2_attention_prompt", dict(causal=0, k_stride=128, k_head=128 * 60)),
])
def test_accepted(name, over):
    assert call(name, **over) == EDEVICE


def test_workspace():
    f = pq2.pq2_attention_paged_workspace
    assert f(1, 1, 8, 8, 128, 100) == (0, 0)
    floats, words = f(2, 3, 40, 8, 128, 40000)
    assert words > 0 and words % 16 == 0 and floats % (16 * 15 * 130) == 0 and floats >= 16 * 15 * 130 * 2
    for bad in ((0, 1, 8, 8, 128, 100), (1, 0, 8, 8, 128, 100), (1, 1, 9, 8, 128, 100), (1, 1, 8, 8, 100, 100), (1, 1, 8, 8, 128, 0)):
        with pytest.raises(ValueError):
            f(*bad)


def test_binding_refuses():
    """What the binding checks itself, on CPU tensors: types and shapes before the device."""
    k = torch.zeros(3, 2, 64)
    i = torch.zeros(3, dtype=torch.int32)
    cache = torch.zeros(4, pq2.pq2_kv_page_bytes(16, 2, 64), dtype=torch.uint8)
    h = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    table = torch.zeros(3, 4, dtype=torch.int32)
    starts = torch.zeros(4, dtype=torch.int32)
    kh = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    bad = [
        lambda: pq2.pq2_kv_write(k, k.double(), cache, i),
        lambda: pq2.pq2_kv_write(k, k[:2], cache, i),
        lambda: pq2.pq2_kv_write(k[:, :, ::2], k[:, :, ::2], None, None, k_out=k[:, :, ::2]),
        lambda: pq2.pq2_kv_write(k, k, cache[:, :-8], i),
        lambda: pq2.pq2_kv_write(k, k, cache, i.long()),
        lambda: pq2.pq2_kv_write(k, k, cache, i[:2]),
        lambda: pq2.pq2_kv_write(k, k, cache, i, 32),
        lambda: pq2.pq2_kv_write(k, k, cache, i, cos=torch.zeros(5, 16), positions=i),
        lambda: pq2.pq2_kv_write(k, k, cache, i, cos=torch.zeros(5, 16), sin=torch.zeros(5, 16)),
        lambda: pq2.pq2_kv_write(k, k, cache, i, cos=torch.zeros(5, 16), sin=torch.zeros(5, 8), positions=i),
        lambda: pq2.pq2_kv_write(k, k, cache, i, q=torch.zeros(3, 4, 64), q_out=h, k_out=torch.zeros(3, 2, 64)),
        lambda: pq2.pq2_kv_read(cache, table, starts, 16, k, h[:, :2]),
        lambda: pq2.pq2_kv_read(cache, table, starts[:3], 16, k, k.clone()),
        lambda: pq2.pq2_kv_read(cache, table[:, ::2], starts, 16, k, k.clone()),
        lambda: pq2.pq2_attention_paged(h, cache, table, i, 16, torch.zeros(3, 4, 64)),
        lambda: pq2.pq2_attention_paged(h.float(), cache, table, i, 16, h.float()),
        lambda: pq2.pq2_attention_paged(h, cache, table, i[:2], 16, h.clone()),
        lambda: pq2.pq2_attention_paged(h, cache, table[:2], i, 16, h.clone()),
        lambda: pq2.pq2_attention_paged(h, cache, table, i, 16, h.clone(), max_len=50000),
        lambda: pq2.pq2_attention_prompt(h, kh, kh[:2], h.clone(), starts, starts),
        lambda: pq2.pq2_attention_prompt(h, kh.half(), kh, h.clone(), starts, starts),
        lambda: pq2.pq2_attention_prompt(h, kh, kh, h.clone(), starts, starts[:2]),
        lambda: pq2.pq2_attention_prompt(h, kh, kh, h.clone(), starts, starts),          # CPU tensors
    ]
    for n, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            print("accepted", n)
