"""include/moe_attn.h on a host without a GPU: every entry point is exported,
workspaces are sized, and invalid arguments get their documented status before
any HIP call."""

import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

moe = pytest.importorskip("block_scaled_fp4_sqrtsoftplus_amd",
                          reason="libmoe_fp4.so not built (run __graft_entry__.build())")
from block_scaled_fp4_sqrtsoftplus_amd import attention as A  # noqa: E402

lib, ref = moe.lib, ctypes.byref
NULL, SHAPE, ALIGN, SMALL = 1, 2, 3, 4


def test_exports_every_declared_symbol():
    src = open(os.path.join(ROOT, "include", "moe_attn.h")).read()
    names = set(re.findall(r"^(?:size_t|moe_status)\s+(moe_\w+)\(", src, re.M))
    assert names == {"moe_kv_append", "moe_attn_workspace_size", "moe_attn_decode", "moe_attn_prefill"}
    for n in names:
        assert hasattr(lib, n), n


def _rows(**kw):
    return A.MoeRowsC(**{**dict(p=16, stride_token=4096, stride_head=128), **kw})


def _cache(**kw):
    d = dict(k=16, v=32, k_scale=None, v_scale=None, pages=9, stride_page=16384, stride_head=2048, stride_token=128,
             page_size=16, heads=8, head_dim=128, format=0)
    return A.MoeKvCacheC(**{**d, **kw})


def _cfg(**kw):
    d = dict(tokens=4, tokens_kv=4, batch=4, q_len=1, heads_q=32, heads_kv=8, head_dim=128, causal=1, window=0,
             scale=0.1)
    return A.MoeAttnConfigC(**{**d, **kw})


def _rope(**kw):
    d = dict(cos_sin=16, positions=10, rot_dim=128, rot_offset=0, interleaved=0, reserved=0)
    return A.MoeRopeC(**{**d, **kw})


def _append(cache=None, rope=None, tokens=3, slots=16, positions=16, k=None, v=None, hq=4, q=None, q_out=None,
            k_out=None, no_v=False):
    r = lambda x: None if x is None else ref(x)  # noqa: E731
    return lib.moe_kv_append(ref(cache or _cache()), r(rope), tokens, slots, positions, ref(k or _rows()),
                             None if no_v else ref(v or _rows()), hq, r(q), r(q_out), r(k_out), None)


@pytest.mark.parametrize("status,kw", [
    (SHAPE, dict(tokens=-1)), (NULL, dict(slots=None)), (ALIGN, dict(slots=20)),
    (SHAPE, dict(cache=_cache(head_dim=96))), (SHAPE, dict(cache=_cache(page_size=24))),
    (SHAPE, dict(cache=_cache(page_size=8))), (SHAPE, dict(cache=_cache(heads=0))),
    (SHAPE, dict(cache=_cache(format=2))), (SHAPE, dict(cache=_cache(pages=-1))),
    (SHAPE, dict(cache=_cache(stride_page=-16))), (ALIGN, dict(cache=_cache(stride_token=132))),
    (SHAPE, dict(cache=_cache(stride_token=(1 << 23) + 16))), (ALIGN, dict(cache=_cache(k=20))), (NULL, dict(cache=_cache(v=None))),
    (NULL, dict(cache=_cache(format=1))), (ALIGN, dict(cache=_cache(format=1, k_scale=16, v_scale=17))),
    (ALIGN, dict(cache=_cache(format=1, k_scale=16, v_scale=16, stride_token=136))),
    (NULL, dict(k=_rows(p=None))), (ALIGN, dict(k=_rows(p=24))), (ALIGN, dict(v=_rows(stride_head=4))),
    (SHAPE, dict(k=_rows(stride_token=-8))), (SHAPE, dict(k=_rows(stride_token=1 << 41))),
    (NULL, dict(no_v=True)), (NULL, dict(cache=_cache(v=16))),           # v exactly when the cache has two tensors
    (NULL, dict(q=_rows())), (NULL, dict(q_out=_rows())), (SHAPE, dict(q=_rows(), q_out=_rows(), hq=0)),
    (ALIGN, dict(k_out=_rows(p=8))),
    (SHAPE, dict(rope=_rope(rot_dim=24))), (SHAPE, dict(rope=_rope(rot_dim=0))),
    (SHAPE, dict(rope=_rope(rot_offset=8))), (SHAPE, dict(rope=_rope(rot_dim=16, rot_offset=4))),
    (SHAPE, dict(rope=_rope(positions=0))), (NULL, dict(rope=_rope(cos_sin=None))),
    (NULL, dict(rope=_rope(), positions=None)), (ALIGN, dict(rope=_rope(cos_sin=20))),
    (ALIGN, dict(rope=_rope(), positions=18)),
])
def test_append_refusals(status, kw):
    assert _append(**kw) == status


def test_append_of_nothing_is_a_no_op():
    assert _append(tokens=0, slots=None, k=_rows(p=None), v=_rows(p=None)) == 0
    assert lib.moe_kv_append(None, None, 0, None, None, None, None, 0, None, None, None, None) == NULL


def test_workspace_size():
    a = lib.moe_attn_workspace_size(ref(_cfg()))
    assert a > 0 and a % 256 == 0
    # it grows with the sequences, not with their lengths, and holds a row of each
    b = lib.moe_attn_workspace_size(ref(_cfg(batch=1000, tokens=1000)))
    assert b - a >= 996 * 32 * 128 * 4
    assert lib.moe_attn_workspace_size(None) == 0
    assert lib.moe_attn_workspace_size(ref(_cfg(tokens=5))) == 0
    assert moe.attn_workspace_size(4, 32, 8, 128) == a
    assert moe.attn_workspace_size(4, 30, 8, 128) == 0


BAD_CFG = [dict(head_dim=96), dict(heads_kv=0), dict(heads_q=30), dict(heads_q=4), dict(heads_q=2048),
           dict(batch=-1), dict(batch=70000, tokens=70000), dict(tokens=-1), dict(window=-1),
           dict(window=(1 << 30) + 1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf"))]


def _decode(cfg=None, q=None, cache=None, table=16, width=4, lens=16, out=None, lse=None, ws=256, ws_bytes=1 << 40):
    return lib.moe_attn_decode(ref(cfg or _cfg()), ref(q or _rows()), ref(cache or _cache()), table, width, lens,
                               ref(out or _rows()), lse, ws, ws_bytes, None)


@pytest.mark.parametrize("status,kw", [(SHAPE, dict(cfg=_cfg(**c))) for c in BAD_CFG] + [
    (SHAPE, dict(cfg=_cfg(q_len=0))), (SHAPE, dict(cfg=_cfg(q_len=17, tokens=68))), (SHAPE, dict(cfg=_cfg(tokens=8))),
    (SHAPE, dict(cache=_cache(heads=4))), (SHAPE, dict(cache=_cache(head_dim=64))), (NULL, dict(cache=_cache(k=None))),
    (SHAPE, dict(width=-1)), (SHAPE, dict(width=1 << 27)), (NULL, dict(table=None)), (NULL, dict(lens=None)),
    (ALIGN, dict(table=18)), (ALIGN, dict(lens=17)), (ALIGN, dict(lse=2)), (NULL, dict(q=_rows(p=None))),
    (ALIGN, dict(out=_rows(p=20))), (SMALL, dict(ws_bytes=100)), (NULL, dict(ws=None)), (ALIGN, dict(ws=24)),
])
def test_decode_refusals(status, kw):
    assert _decode(**kw) == status


def test_decode_of_nothing_is_a_no_op():
    assert _decode(cfg=_cfg(batch=0, tokens=0), q=_rows(p=None), out=_rows(p=None), table=None, lens=None) == 0


def _prefill(cfg=None, q=None, k=None, v=None, cu_q=16, cu_k=None, out=None, lse=None):
    return lib.moe_attn_prefill(ref(cfg or _cfg()), ref(q or _rows()), ref(k or _rows()), ref(v or _rows()), cu_q,
                                cu_k, ref(out or _rows()), lse, None)


@pytest.mark.parametrize("status,kw", [(SHAPE, dict(cfg=_cfg(**c))) for c in BAD_CFG] + [
    (SHAPE, dict(cfg=_cfg(causal=2))), (SHAPE, dict(cfg=_cfg(tokens_kv=-1))), (SHAPE, dict(cfg=_cfg(tokens_kv=1 << 30))),
    (NULL, dict(cu_q=None)), (ALIGN, dict(cu_q=18)), (ALIGN, dict(cu_k=18)), (ALIGN, dict(lse=6)),
    (NULL, dict(k=_rows(p=None))), (NULL, dict(out=_rows(p=None))), (ALIGN, dict(v=_rows(p=8))),
    (ALIGN, dict(q=_rows(stride_token=12))), (SHAPE, dict(k=_rows(stride_token=(1 << 23) + 8))),
])
def test_prefill_refusals(status, kw):
    assert _prefill(**kw) == status


def test_prefill_of_nothing_is_a_no_op():
    empty = _rows(p=None)
    assert _prefill(cfg=_cfg(tokens=0, tokens_kv=0), q=empty, k=empty, v=empty, out=empty, cu_q=None) == 0
