"""The attention operators' Python binding on a host without a GPU."""

import pytest

moe = pytest.importorskip("block_scaled_fp4_sqrtsoftplus_amd",
                          reason="libmoe_fp4.so not built (run __graft_entry__.build())")


@pytest.mark.parametrize("at", range(5))
def test_workspace_of_sizes_past_32_bits(at):
    sizes = [4, 32, 8, 128, 1]       # batch, heads_q, heads_kv, head_dim, q_len
    assert moe.attn_workspace_size(*sizes) > 0
    sizes[at] += 1 << 32             # an invalid configuration, not the one of the lower bits
    assert moe.attn_workspace_size(*sizes) == 0
