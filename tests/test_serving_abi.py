"""include/moe_serving.h on a host without a GPU: every entry point is exported, workspaces are sized, and invalid
arguments get their documented status before any HIP call."""

import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

moe = pytest.importorskip("block_scaled_fp4_sqrtsoftplus_amd",
                          reason="libmoe_fp4.so not built (run __graft_entry__.build())")
from block_scaled_fp4_sqrtsoftplus_amd import attention as A  # noqa: E402
from block_scaled_fp4_sqrtsoftplus_amd import serving as S  # noqa: E402

lib, ref = moe.lib, ctypes.byref
NULL, SHAPE, ALIGN, SMALL, UNSUPPORTED = 1, 2, 3, 4, 5


def test_exports_every_declared_symbol():
    src = open(os.path.join(ROOT, "include", "moe_serving.h")).read()
    names = set(re.findall(r"^(?:size_t|moe_status)\s+(moe_\w+)\(", src, re.M))
    assert names == {"moe_attn_decode_sinks", "moe_attn_prefill_sinks", "moe_tree_masks",
                     "moe_attn_tree_workspace_size", "moe_attn_tree", "moe_kv_compact", "moe_kv_copy_pages",
                     "moe_pool_workspace_size", "moe_pool_grow", "moe_pool_fork", "moe_pool_trim"}
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


def _pool(**kw):
    d = dict(refs=16, table=16, lens=16, pages=100, batch=4, width=8, page_size=16, reserved=0)
    return S.MoePagePoolC(**{**d, **kw})


BAD_CFG = [dict(head_dim=96), dict(heads_kv=0), dict(heads_q=30), dict(heads_q=4), dict(heads_q=2048),
           dict(batch=-1), dict(batch=70000, tokens=70000), dict(tokens=-1), dict(window=-1),
           dict(window=(1 << 30) + 1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf"))]


def _decode(cfg=None, sinks=4, q=None, cache=None, table=16, width=4, lens=16, out=None, lse=None, ws=256,
            ws_bytes=1 << 40):
    return lib.moe_attn_decode_sinks(ref(cfg or _cfg(window=8)), sinks, ref(q or _rows()), ref(cache or _cache()), table,
                                     width, lens, ref(out or _rows()), lse, ws, ws_bytes, None)


COMMON = [
    (SHAPE, dict(sinks=-1)), (SHAPE, dict(sinks=(1 << 30) + 1)),
    (SHAPE, dict(cache=_cache(heads=4))), (SHAPE, dict(cache=_cache(head_dim=64))), (NULL, dict(cache=_cache(k=None))),
    (SHAPE, dict(width=-1)), (SHAPE, dict(width=1 << 27)), (NULL, dict(table=None)), (NULL, dict(lens=None)),
    (ALIGN, dict(table=18)), (ALIGN, dict(lens=17)), (ALIGN, dict(lse=2)), (NULL, dict(q=_rows(p=None))),
    (ALIGN, dict(out=_rows(p=20))), (SMALL, dict(ws_bytes=100)), (NULL, dict(ws=None)), (ALIGN, dict(ws=24)),
]


@pytest.mark.parametrize("status,kw", [(SHAPE, dict(cfg=_cfg(**c))) for c in BAD_CFG] + COMMON + [
    (SHAPE, dict(cfg=_cfg(q_len=0))), (SHAPE, dict(cfg=_cfg(q_len=17, tokens=68))), (SHAPE, dict(cfg=_cfg(tokens=8)))])
def test_decode_sinks_refusals(status, kw):
    assert _decode(**kw) == status


def _prefill(cfg=None, sinks=4, q=None, k=None, v=None, cu_q=16, cu_k=None, out=None, lse=None):
    return lib.moe_attn_prefill_sinks(ref(cfg or _cfg(window=8)), sinks, ref(q or _rows()), ref(k or _rows()),
                                      ref(v or _rows()), cu_q, cu_k, ref(out or _rows()), lse, None)


@pytest.mark.parametrize("status,kw", [(SHAPE, dict(cfg=_cfg(**c))) for c in BAD_CFG] + [
    (SHAPE, dict(sinks=-1)), (SHAPE, dict(sinks=(1 << 30) + 1)), (SHAPE, dict(cfg=_cfg(causal=2))),
    (SHAPE, dict(cfg=_cfg(tokens_kv=-1))), (NULL, dict(cu_q=None)), (ALIGN, dict(cu_q=18)), (ALIGN, dict(cu_k=18)),
    (ALIGN, dict(lse=6)), (NULL, dict(k=_rows(p=None))), (ALIGN, dict(v=_rows(p=8))),
    (SHAPE, dict(k=_rows(stride_token=(1 << 23) + 8)))])
def test_prefill_sinks_refusals(status, kw):
    assert _prefill(**kw) == status


def _tree(cfg=None, sinks=0, q=None, cache=None, table=16, width=4, lens=16, masks=16, out=None, lse=None, ws=256,
          ws_bytes=1 << 40):
    return lib.moe_attn_tree(ref(cfg or _cfg(q_len=3, tokens=12)), sinks, ref(q or _rows()), ref(cache or _cache()),
                             table, width, lens, masks, ref(out or _rows()), lse, ws, ws_bytes, None)


@pytest.mark.parametrize("status,kw", [(SHAPE, dict(cfg=_cfg(**c))) for c in BAD_CFG] + COMMON + [
    (SHAPE, dict(cfg=_cfg(q_len=0))), (SHAPE, dict(cfg=_cfg(q_len=65, tokens=260))),
    (SHAPE, dict(cfg=_cfg(q_len=3, tokens=8))), (NULL, dict(masks=None)), (ALIGN, dict(masks=20)),
    (UNSUPPORTED, dict(cfg=_cfg(q_len=3, tokens=12, window=2)))])
def test_tree_refusals(status, kw):
    assert _tree(**kw) == status


def test_tree_workspace_size():
    a = lib.moe_attn_tree_workspace_size(ref(_cfg(q_len=64, tokens=256)))
    assert a > 0 and a % 256 == 0
    assert lib.moe_attn_tree_workspace_size(ref(_cfg(q_len=65, tokens=260))) == 0
    assert lib.moe_attn_tree_workspace_size(None) == 0
    assert lib.moe_attn_workspace_size(ref(_cfg(q_len=64, tokens=256))) == 0


@pytest.mark.parametrize("status,args", [
    (SHAPE, (-1, 4, 16, 16, None)), (SHAPE, (70000, 4, 16, 16, None)), (SHAPE, (2, 0, 16, 16, None)),
    (SHAPE, (2, 65, 16, 16, None)), (NULL, (2, 4, None, 16, None)), (NULL, (2, 4, 16, None, None)),
    (ALIGN, (2, 4, 18, 16, None)), (ALIGN, (2, 4, 16, 20, None)), (ALIGN, (2, 4, 16, 16, 18))])
def test_tree_masks_refusals(status, args):
    assert lib.moe_tree_masks(*args, None) == status


def _compact(cache=None, batch=4, nodes=7, table=16, width=4, lens=16, path=16, counts=16):
    return lib.moe_kv_compact(ref(cache or _cache()), batch, nodes, table, width, lens, path, counts, None)


@pytest.mark.parametrize("status,kw", [
    (SHAPE, dict(cache=_cache(head_dim=96))), (NULL, dict(cache=_cache(v=None))), (SHAPE, dict(batch=-1)),
    (SHAPE, dict(batch=65537)), (SHAPE, dict(nodes=0)), (SHAPE, dict(nodes=65)), (SHAPE, dict(width=-1)),
    (SHAPE, dict(width=1 << 27)), (NULL, dict(table=None)), (NULL, dict(lens=None)), (NULL, dict(path=None)),
    (NULL, dict(counts=None)), (ALIGN, dict(table=18)), (ALIGN, dict(lens=18)), (ALIGN, dict(path=18)),
    (ALIGN, dict(counts=18))])
def test_compact_refusals(status, kw):
    assert _compact(**kw) == status


@pytest.mark.parametrize("status,kw", [
    (SHAPE, dict(cache=_cache(page_size=24))), (SHAPE, dict(n=-1)), (SHAPE, dict(n=1 << 31)), (NULL, dict(src=None)),
    (NULL, dict(dst=None)), (ALIGN, dict(src=18)), (ALIGN, dict(dst=18))])
def test_copy_pages_refusals(status, kw):
    a = {**dict(cache=_cache(), n=3, src=16, dst=16), **kw}
    assert lib.moe_kv_copy_pages(ref(a["cache"]), a["n"], a["src"], a["dst"], None) == status


BAD_POOL = [(SHAPE, dict(pages=-1)), (SHAPE, dict(pages=(1 << 28) + 1)), (SHAPE, dict(batch=-1)),
            (SHAPE, dict(batch=65537)), (SHAPE, dict(width=0)), (SHAPE, dict(width=(1 << 26) + 1)),
            (SHAPE, dict(page_size=8)), (SHAPE, dict(page_size=24)), (SHAPE, dict(page_size=8192)),
            (SHAPE, dict(width=1 << 20, page_size=4096)), (SHAPE, dict(batch=40000, width=1 << 16)),
            (NULL, dict(refs=None)), (NULL, dict(table=None)), (NULL, dict(lens=None)), (ALIGN, dict(refs=24)),
            (ALIGN, dict(table=18)), (ALIGN, dict(lens=18))]


def _grow(pool=None, tokens=5, cu=16, slots=16, positions=16, src=16, dst=16, missing=16, ws=256, ws_bytes=1 << 40):
    return lib.moe_pool_grow(ref(pool or _pool()), tokens, cu, slots, positions, src, dst, missing, ws, ws_bytes, None)


@pytest.mark.parametrize("status,kw", [(s, dict(pool=_pool(**p))) for s, p in BAD_POOL] + [
    (SHAPE, dict(tokens=-1)), (SHAPE, dict(tokens=1 << 31)), (NULL, dict(cu=None)), (NULL, dict(slots=None)),
    (NULL, dict(positions=None)), (NULL, dict(src=None)), (NULL, dict(dst=None)), (NULL, dict(missing=None)),
    (ALIGN, dict(cu=18)), (ALIGN, dict(slots=20)), (ALIGN, dict(positions=18)), (ALIGN, dict(src=18)),
    (ALIGN, dict(missing=18)), (SMALL, dict(ws_bytes=100)), (NULL, dict(ws=None)), (ALIGN, dict(ws=24))])
def test_grow_refusals(status, kw):
    assert _grow(**kw) == status


@pytest.mark.parametrize("status,pool", BAD_POOL)
def test_fork_and_trim_refuse_the_same_pools(status, pool):
    assert lib.moe_pool_fork(ref(_pool(**pool)), 16, None) == status
    assert lib.moe_pool_trim(ref(_pool(**pool)), None, 0, 0, None) == status


def test_fork_and_trim_refusals():
    assert lib.moe_pool_fork(ref(_pool()), None, None) == NULL
    assert lib.moe_pool_fork(ref(_pool()), 18, None) == ALIGN
    assert lib.moe_pool_fork(None, 16, None) == NULL
    assert lib.moe_pool_trim(ref(_pool()), 18, 0, 0, None) == ALIGN
    assert lib.moe_pool_trim(ref(_pool()), None, -1, 0, None) == SHAPE
    assert lib.moe_pool_trim(ref(_pool()), None, 0, -1, None) == SHAPE
    assert lib.moe_pool_trim(ref(_pool()), None, (1 << 30) + 1, 0, None) == SHAPE


def test_pool_workspace_size():
    a = lib.moe_pool_workspace_size(ref(_pool()))
    assert a > 0 and a % 256 == 0
    assert lib.moe_pool_workspace_size(ref(_pool(pages=1 << 20))) >= 4 << 20
    assert lib.moe_pool_workspace_size(ref(_pool(width=0))) == 0
    assert lib.moe_pool_workspace_size(None) == 0


def test_calls_of_nothing_are_no_ops():
    none = _rows(p=None)
    assert _decode(cfg=_cfg(batch=0, tokens=0, window=8), q=none, out=none, table=None, lens=None) == 0
    assert _prefill(cfg=_cfg(tokens=0, tokens_kv=0, window=8), q=none, k=none, v=none, out=none, cu_q=None) == 0
    assert _tree(cfg=_cfg(batch=0, tokens=0, q_len=3), q=none, out=none, table=None, lens=None, masks=None) == 0
    assert lib.moe_tree_masks(0, 4, None, None, None, None) == 0
    assert _compact(batch=0, table=None, lens=None, path=None, counts=None) == 0
    assert lib.moe_kv_copy_pages(ref(_cache()), 0, None, None, None) == 0
    empty = _pool(batch=0, table=None, lens=None)
    assert lib.moe_pool_fork(ref(empty), None, None) == 0
    assert lib.moe_pool_trim(ref(empty), None, 0, 0, None) == 0
