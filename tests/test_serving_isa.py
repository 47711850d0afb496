"""What test_attn_isa states of the attention kernels' assembly, for those of include/moe_serving.h."""

import os

import pytest

import test_attn_isa


@pytest.mark.skipif(not os.path.exists(test_attn_isa.HIPCC), reason="hipcc not installed")
@pytest.mark.parametrize("src,loads", [("attn_tree.hip", True), ("attn_prefill_sinks.hip", True), ("kv_move.hip", False),
                                       ("page_pool.hip", False)])
def test_m0_and_packed_arithmetic(src, loads, tmp_path):
    test_attn_isa.test_m0_belongs_to_the_loads_into_lds(src, loads, tmp_path)


@pytest.mark.skipif(not os.path.exists(test_attn_isa.HIPCC), reason="hipcc not installed")
def test_m0_and_packed_arithmetic_of_the_trees_own_kernel(tmp_path):
    test_attn_isa.test_m0_belongs_to_the_loads_into_lds("attn_tree_rows.hip", True, tmp_path)
