"""Without the attention operators' argument marshaller, or with one of another torch, the rest of the package works and
the attention calls say what to do."""
import os
import subprocess
import sys

import pytest
import torch

from gemm_int8_act_amd import _marshal

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CALLS = """
import torch
import gemm_int8_act_amd as pq2
assert pq2.lib.pq2_layout_version() > 0 and pq2.pq2_kv_page_bytes(16, 2, 64) > 0
assert pq2.pq2_attention_paged_workspace(1, 1, 8, 8, 128, 100) == (0, 0)
x, i, s = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
for call in (lambda: pq2.pq2_kv_write(x, x, None, i, q=x, q_out=x), lambda: pq2.pq2_kv_read(x, x, s, 16, x, x),
             lambda: pq2.pq2_attention_paged(x, x, x, i, 16, x), lambda: pq2.pq2_attention_prompt(x, x, x, x, s, s)):
    try:
        call()
    except ImportError as e:
        assert "_marshal.so" in str(e) and "build.py" in str(e), e
    else:
        raise SystemExit("no ImportError")
print("said so")
"""


def run(before):
    res = subprocess.run([sys.executable, "-c", before + CALLS], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "said so" in res.stdout, res.stdout + res.stderr


def test_marshal_is_of_this_torch():
    assert _marshal.torch_version == torch.__version__


@pytest.mark.parametrize("before", [
    "import sys\nsys.modules['gemm_int8_act_amd._marshal'] = None\n",
    "import sys, types\nm = types.ModuleType('gemm_int8_act_amd._marshal')\nm.torch_version = '1.0'\n"
    "sys.modules['gemm_int8_act_amd._marshal'] = m\n",
], ids=["missing", "another torch"])
def test_without_a_marshaller_of_this_torch(before):
    run(before)
