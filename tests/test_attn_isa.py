"""Properties of the attention kernels' generated AMD assembly that their
inline assembly relies on: the asynchronous load into LDS takes its address from m0,
which the compiler is not told about, so nothing else may use m0; and no packed
fp32 arithmetic appears.  CPU-only: hipcc cross-compiles."""

import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_scaled_fp4_sqrtsoftplus_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not installed")
@pytest.mark.parametrize("src,loads", [("attn_prefill.hip", True), ("attn_decode.hip", True), ("kv_append.hip", False)])
def test_m0_belongs_to_the_loads_into_lds(src, loads, tmp_path):
    out = str(tmp_path / "k.s")
    subprocess.run([HIPCC, "--offload-arch=gfx950", "--cuda-device-only", "-S", "-O3", "-std=c++17", "-Xclang",
                    "-target-feature", "-Xclang", "-packed-fp32-ops", "-ffp-contract=off", "-I",
                    os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(CSRC, src), "-o", out],
                   check=True, capture_output=True)
    lines = [t.split(";")[0].strip() for t in open(out).read().split("\n")]
    lines = [t for t in lines if t and not t.startswith(".") and not t.endswith(":")]
    found = 0
    for i, t in enumerate(lines):
        assert not re.match(r"v_pk_(add|mul|fma)_f32", t), t
        if t.startswith("global_load_lds"):
            found += 1
            assert lines[i - 1].startswith("s_nop") and re.match(r"s_mov_b32 m0, ", lines[i - 2]), lines[i - 2:i + 1]
        elif re.search(r"\bm0\b", t):
            assert t.startswith("s_mov_b32 m0, ") and lines[i + 2].startswith("global_load_lds"), t
    assert (found > 0) == loads
