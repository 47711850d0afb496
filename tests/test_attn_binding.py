"""The attention operators' Python binding on a host without a GPU."""

import os
import shutil
import subprocess
import sys

import pytest

moe = pytest.importorskip("block_scaled_fp4_sqrtsoftplus_amd",
                          reason="libmoe_fp4.so not built (run __graft_entry__.build())")


@pytest.mark.parametrize("at", range(5))
def test_workspace_of_sizes_past_32_bits(at):
    sizes = [4, 32, 8, 128, 1]       # batch, heads_q, heads_kv, head_dim, q_len
    assert moe.attn_workspace_size(*sizes) > 0
    sizes[at] += 1 << 32             # an invalid configuration, not the one of the lower bits
    assert moe.attn_workspace_size(*sizes) == 0


@pytest.mark.parametrize("native", ["missing", "unloadable"])
def test_layer_without_the_native_half(native, tmp_path):
    # the MoE layer's entry points need the library alone; the attention names say what is wrong
    name = moe.__name__
    src = os.path.dirname(moe.__file__)
    os.mkdir(tmp_path / name)
    for f in ("__init__.py", "attention.py", "libmoe_fp4.so"):
        shutil.copy(os.path.join(src, f), tmp_path / name / f)
    if native == "unloadable":
        (tmp_path / name / "_attn_binding.so").write_bytes(b"not a library")
    code = f"""
import {name} as moe
assert moe.__file__.startswith({str(tmp_path)!r})
cfg = moe.Config(tokens=4, hidden=512, inter=256, n_experts=8, top_k=2)
assert moe.workspace_size(cfg, moe.OP_LAYER) > 0 and moe.Layer and moe.layer
for n in ("KVCache", "Rope", "DecodeAttention", "kv_append", "attn_decode", "attn_prefill", "attn_workspace_size"):
    try:
        getattr(moe, n)
    except ImportError as e:
        assert "_attn_binding" in str(e) and "build.py" in str(e), e
    else:
        raise SystemExit(n)
try:
    moe.nothing
except AttributeError:
    print("fine")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip().endswith("fine"), r.stderr
