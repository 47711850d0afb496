"""The example block: a token decoded over the cache attends as it does inside
its whole prompt, in both cache formats, and the MoE layer follows."""

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("block_scaled_fp4_sqrtsoftplus_amd")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("window", [0, 40])
def test_tokens_continue_prompts(fmt, window):
    from decoder_block import DecoderBlock
    lengths, steps = [70, 1, 33], 5
    kv = moe.KV_FP8 if fmt == "fp8" else moe.KV_BF16
    xs = torch.randn(3, 80, 1024, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    one, whole = DecoderBlock(kv_format=kv, window=window), DecoderBlock(window=window)
    one.attend_prompts(torch.cat([xs[b, :n] for b, n in enumerate(lengths)]), lengths)
    got = [one.attend_tokens(torch.stack([xs[b, n + i] for b, n in enumerate(lengths)])) for i in range(steps)]
    longer = [n + steps for n in lengths]
    packed = torch.cat([xs[b, :n] for b, n in enumerate(longer)])
    want = whole.attend_prompts(packed, longer).float()
    v_max = whole._qkv(packed)[2].float().abs().max()
    ends = torch.tensor(longer).cumsum(0)
    for i in range(steps):
        w = want[(ends - steps + i).cuda()]
        err = (got[i].float() - w).abs()
        # each side rounds its weights and its result to bf16: 2^-8 of sum p |v| <= max |v| and of the
        # result, twice.  An FP8 row is off by 2^-4 of each element: v by that directly, and a
        # score by 2^-4 sum |q k| / sqrt(128), which for normal q and k stays below 2^-4 * 0.64 * 128 / 11.3
        # < 0.5 and moves every weight by less than e^0.5 - 1 either way.
        tol = 2 * 2.0 ** -8 * (w.abs() + v_max) * 1.05
        if fmt == "fp8":
            tol = tol + (2.0 ** -4 + 2 * 0.65) * v_max
            # far below that bound on the average: the errors of 128 elements and of many keys are not aligned
            assert (err.square().mean() / w.square().mean()).sqrt() < 0.1
        assert (err <= tol).all(), err.max()
    y = one.tokens(xs[:, 79])
    assert y.shape == (3, 1024) and torch.isfinite(y.float()).all()


def test_block_rest_is_the_moe_layer():
    from decoder_block import DecoderBlock
    b = DecoderBlock()
    x = torch.randn(9, 1024, device="cuda").bfloat16()
    att = torch.randn(9, 16, 128, device="cuda").bfloat16()
    x1 = x + torch.nn.functional.linear(att.flatten(1), b.w_o)
    y = b._rest(x, att)
    assert torch.equal(y, x1 + moe.layer(moe.Config(tokens=9, **b.moe_sizes), x1, b.experts, w_gate=b.w_gate))
    b.pages.free.clear()
    with pytest.raises(RuntimeError, match="page"):
        b.attend_prompts(x, [9, 0, 0])
