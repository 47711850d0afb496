"""Build the HIP library libmoe_fp4.so in-tree for gfx950 with hipcc, and the
attention binding's native half _attn_binding.so.

Usage: python block_scaled_fp4_sqrtsoftplus_amd/build.py   (or __graft_entry__.build()); it
does not import the package, whose import loads the library.
Every call recompiles all sources (a few seconds each, in parallel).
"""

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "libmoe_fp4.so")
BINDING = os.path.join(PKG, "_attn_binding.so")
BUILD = os.path.join(ROOT, "_build")
SOURCES = ["api.cpp", "quant_act.hip", "route.hip", "expert_gemm.hip", "expert_gemm_nv.hip", "expert_gemm_w4.hip",
           "bf16_gemm.hip", "combine.hip", "cast_fp8.hip", "attn_api.cpp", "kv_append.hip", "attn_decode.hip",
           "attn_prefill.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-fPIC", "-std=c++17",
    # packed fp32 instructions are not generated (see the design notes)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # no floating-point contraction: routing weights and scores must round
    # exactly as written
    "-ffp-contract=off",
    "-Wno-unused-result",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]


def _compile(src):
    obj = os.path.join(BUILD, src + ".o")
    cmd = [HIPCC] + FLAGS + (["-x", "hip"] if src.endswith(".cpp") else []) + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stderr}")
    return obj


def _compile_binding():
    """The binding's native half: host code against torch's and Python's headers."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD, "attn_binding.cpp.o")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-fPIC", "-std=c++17", "-Wno-unused-parameter",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"],
           "-c", os.path.join(CSRC, "attn_binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the binding's compilation failed:\n{r.stderr}")
    return obj, os.path.join(root, "lib")


def _link_binding(obj, torch_lib):
    tmp = BINDING + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", PKG, "-l:libmoe_fp4.so",
           "-L", torch_lib, "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{torch_lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the binding's link failed:\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(verbose=False):
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(8, len(SOURCES) + 1)) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(_compile, SOURCES))
        binding = binding.result()
    tmp = OUT + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, OUT)
    _link_binding(*binding)
    if verbose:
        print("built", OUT, BINDING)
    return OUT


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
