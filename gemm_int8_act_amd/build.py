"""Build libpq2.so (the gfx950 HIP kernels and their C ABI) in-tree.

    python gemm_int8_act_amd/build.py

(run it as a script: importing the package would load the library it builds).

Each .hip source compiles to an object in parallel, then hipcc links the
shared library next to this file.  Packed-FP32 instruction selection is
switched off for the device code (-target-feature -packed-fp32-ops).
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libpq2.so")
MARSHAL = os.path.join(HERE, "_marshal.so")  # host code only: arguments from torch tensors
BUILD_DIR = os.path.join(HERE, "_build")
SOURCES = ["api.hip", "quantize.hip", "small_m.hip", "small_m_wg.hip", "tiles.hip", "prefill.hip", "probe.hip",
           "block_api.hip", "w4.hip", "block_small_m.hip", "block_prefill.hip",
           "norm.hip", "attention_api.hip", "kv_cache.hip", "attention_paged.hip", "attention_prompt.hip"]
ARCH = "gfx950"

COMMON_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def _hipcc() -> str:
    path = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(path):
        raise RuntimeError("hipcc not found: a ROCm toolchain is needed to build libpq2")
    return path


# Per-source extra flags.  The prefill kernel rescales every MFMA result on
# the vector ALU; asking the backend for the VGPR form of the MFMA keeps the
# accumulators out of AGPRs and saves one register move per output and group.
EXTRA_FLAGS = {
    "prefill.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
    "block_prefill.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
}


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [_hipcc(), *COMMON_FLAGS, *EXTRA_FLAGS.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    return obj


def _marshal_module() -> None:
    """Compile the binding's argument marshaller (csrc/marshal.cpp) against torch's headers; it finds libpq2.so next to
    itself."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    tmp = MARSHAL + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-DUSE_ROCM",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DPQ2_TORCH_VERSION="{torch.__version__}"',
           "-I", sysconfig.get_path("include"), "-isystem", os.path.join(root, "include"),
           os.path.join(CSRC, "marshal.cpp"), "-o", tmp, "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-L", HERE, "-lpq2", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for marshal.cpp:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, MARSHAL)


def build(verbose: bool = False) -> str:
    """Compile every HIP source for gfx950, link libpq2.so and build the argument marshaller; returns libpq2's path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    workers = min(len(SOURCES), max(1, (os.cpu_count() or 1)))
    with concurrent.futures.ThreadPoolExecutor(max_workers=workers) as pool:
        objs = list(pool.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    _marshal_module()
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
