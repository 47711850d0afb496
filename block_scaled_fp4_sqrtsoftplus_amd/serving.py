"""Binding of what a serving loop needs around the paged cache (include/moe_serving.h):
attention for a tree of drafted tokens, the rows of an accepted path moved to
their places, copies of pages, and a pool from which sequences fork, grow and
free pages.

One step of speculative decoding, for every sequence of a pool:

    before = pool.lens.clone()
    masks, depths = tree_masks(parents)
    slots, _, src, dst = pool.grow(cu, tokens)              # room for the drafted tokens
    masks = masks * (slots >= 0).view_as(masks)             # a node without a place is an empty one
    kv_copy_pages(cache, src, dst)                          # ... in every layer's cache
    positions = (before[:, None] + depths).flatten()
    q = kv_append(cache, k, v, slots, positions, rope, q)
    out = attend(q, pool.table, before, masks)              # a TreeAttention
    kv_compact(cache, pool.table, before, path, counts)     # the accepted ones move up
    pool.trim(before + counts)                              # the others' pages are free again

`path` and `counts` are chosen among the nodes whose mask is not 0.  Where the pool runs out of pages
(`pool.missing`), the nodes without a slot then are seen by none and accepted by none, and trim leaves
the length right; nothing of the step has to wait for the host.  A loop without a tree looks at
`missing`, or at the slots, before it goes on: tokens without a slot are stored nowhere, and
pool.trim(before), after the copies, takes the call back.

Like the other attention operators these have no backward pass.
"""

import ctypes

import torch

from . import STATUS_NAMES, MoeError, _i32, _i64, _sz, _vp, lib
from . import _attn_binding as _native
from .attention import (DecodeAttention, KVCache, MoeAttnConfigC, MoeKvCacheC, MoeRowsC, _byref, _check_fit, _P,
                        _raw_stream)


class MoePagePoolC(ctypes.Structure):
    _fields_ = [("refs", _vp), ("table", _vp), ("lens", _vp), ("pages", _i64), ("batch", _i32), ("width", _i32),
                ("page_size", _i32), ("reserved", _i32)]


lib.moe_attn_decode_sinks.restype = ctypes.c_int
lib.moe_attn_decode_sinks.argtypes = [_P(MoeAttnConfigC), _i32, _P(MoeRowsC), _P(MoeKvCacheC), _vp, _i32, _vp,
                                      _P(MoeRowsC), _vp, _vp, _sz, _vp]
lib.moe_attn_prefill_sinks.restype = ctypes.c_int
lib.moe_attn_prefill_sinks.argtypes = [_P(MoeAttnConfigC), _i32, _P(MoeRowsC), _P(MoeRowsC), _P(MoeRowsC), _vp, _vp,
                                       _P(MoeRowsC), _vp, _vp]
lib.moe_tree_masks.restype = ctypes.c_int
lib.moe_tree_masks.argtypes = [_i32, _i32, _vp, _vp, _vp, _vp]
lib.moe_attn_tree_workspace_size.restype = _sz
lib.moe_attn_tree_workspace_size.argtypes = [_P(MoeAttnConfigC)]
lib.moe_attn_tree.restype = ctypes.c_int
lib.moe_attn_tree.argtypes = [_P(MoeAttnConfigC), _i32, _P(MoeRowsC), _P(MoeKvCacheC), _vp, _i32, _vp, _vp,
                              _P(MoeRowsC), _vp, _vp, _sz, _vp]
lib.moe_kv_compact.restype = ctypes.c_int
lib.moe_kv_compact.argtypes = [_P(MoeKvCacheC), _i32, _i32, _vp, _i32, _vp, _vp, _vp, _vp]
lib.moe_kv_copy_pages.restype = ctypes.c_int
lib.moe_kv_copy_pages.argtypes = [_P(MoeKvCacheC), _i64, _vp, _vp, _vp]
lib.moe_pool_workspace_size.restype = _sz
lib.moe_pool_workspace_size.argtypes = [_P(MoePagePoolC)]
lib.moe_pool_grow.restype = ctypes.c_int
lib.moe_pool_grow.argtypes = [_P(MoePagePoolC), _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
lib.moe_pool_fork.restype = ctypes.c_int
lib.moe_pool_fork.argtypes = [_P(MoePagePoolC), _vp, _vp]
lib.moe_pool_trim.restype = ctypes.c_int
lib.moe_pool_trim.argtypes = [_P(MoePagePoolC), _vp, _i32, _i32, _vp]


def tree_masks(parents):
    """parents [batch, nodes] int32 (moe_tree_masks: -1 hangs a node on the sequence's last token, -2 leaves its place
    empty) -> masks [batch, nodes] int64, whose bits are the node and those above it, and depths [batch, nodes] int32."""
    if not parents.is_cuda:
        raise ValueError("tensors passed to the HIP library must be on the GPU")
    index = parents.get_device()
    return _native.tree_masks(index, _raw_stream(index), parents)


class TreeAttention(DecodeAttention):
    """Holds the sizes, the cache and the workspace of moe_attn_tree and runs it on the current stream:
    attention of every sequence's `nodes` drafted tokens, which the cache holds already behind the context.
    What DecodeAttention says of streams, graphs and calls that overlap holds here too."""

    _workspace_size = staticmethod(lib.moe_attn_tree_workspace_size)

    def __init__(self, cache: KVCache, batch, heads_q, nodes, window=0, scale=None, sinks=0):
        super().__init__(cache, batch, heads_q, nodes, window, scale, sinks)
        self.nodes = nodes

    def __call__(self, q, block_table, context_lens, masks, out=None, want_lse=False):
        """q [batch * nodes, heads_q, head_dim] bf16, block_table [batch, width] int32 contiguous, context_lens [batch]
        int32 (drafted tokens not included: node i is row context_lens + i of the cache), masks [batch, nodes] int64:
        out like q, and with want_lse also lse [batch * nodes, heads_q] fp32."""
        return _native.attn_tree(self._at, self.cache._at, self._index, self._on_stream(), self._ws, self.ws_bytes, q,
                                 block_table, context_lens, out, want_lse, self.sinks, masks)


def attn_tree(q, cache: KVCache, block_table, context_lens, masks, window=0, scale=None, out=None, want_lse=False,
              sinks=0):
    """One call of TreeAttention."""
    a = TreeAttention(cache, masks.shape[0], q.shape[1], masks.shape[1], window, scale, sinks)
    return a(q, block_table, context_lens, masks, out, want_lse)


def kv_compact(cache: KVCache, block_table, context_lens, path, counts):
    """Moves rows context_lens[b] + path[b, i] of every sequence's keys and values to context_lens[b] + i, for
    i < counts[b] (moe_kv_compact); block_table [batch, width], context_lens [batch], path [batch, nodes] and counts
    [batch] are int32."""
    index = cache._index
    _native.kv_compact(cache._at, index, _raw_stream(index), block_table, context_lens, path, counts)


def kv_copy_pages(cache: KVCache, src, dst):
    """Copies pages src to pages dst, int32 [pairs] (moe_kv_copy_pages); pairs outside the cache copy nothing."""
    index = cache._index
    _native.kv_copy_pages(cache._at, index, _raw_stream(index), src, dst)


class PagePool:
    """Handle on the tensors of a pool of cache pages (moe_page_pool), all int32 on one GPU and updated in place:
    refs [pages], table [batch, width], lens [batch].  One pool serves the caches of all layers.  Calls go to the
    current stream, one after another; a graph that recorded one needs the object as long as it is replayed."""

    def __init__(self, refs, table, lens, page_size):
        if not refs.is_cuda:
            raise ValueError("tensors passed to the HIP library must be on the GPU")
        if refs.dim() != 1 or table.dim() != 2 or lens.shape != table.shape[:1]:
            raise ValueError("a pool has refs [pages], table [batch, width] and lens [batch]")
        for t, name in ((refs, "refs"), (table, "table"), (lens, "lens")):
            if t.dtype is not torch.int32 or t.device != refs.device or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous int32 on {refs.device}")
        self.refs, self.table, self.lens, self.page_size = refs, table, lens, page_size
        self.pages, (self.batch, self.width) = refs.shape[0], table.shape
        _check_fit(self.batch, self.width, page_size)
        self.device, self._index = refs.device, refs.device.index
        self.c = MoePagePoolC(refs.data_ptr() or None, table.data_ptr() or None, lens.data_ptr() or None, self.pages,
                              self.batch, self.width, page_size, 0)
        self._at = ctypes.addressof(self.c)
        self.ws_bytes = lib.moe_pool_workspace_size(_byref(self.c))
        if self.ws_bytes == 0:
            raise MoeError(STATUS_NAMES.index("MOE_ERR_BAD_SHAPE"))
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        self.missing = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._streams = {_raw_stream(self._index)}   # those the allocator knows the tensors to be used on

    @classmethod
    def empty(cls, pages, page_size, batch, width, device="cuda"):
        """A pool of new tensors: all pages free, all sequences empty."""
        return cls(torch.zeros(pages, dtype=torch.int32, device=device),
                   torch.full((batch, width), -1, dtype=torch.int32, device=device),
                   torch.zeros(batch, dtype=torch.int32, device=device), page_size)

    def _on_stream(self):
        stream = _raw_stream(self._index)
        if stream not in self._streams:
            current = torch.cuda.current_stream(self._index)
            for t in (self.refs, self.table, self.lens, self.ws, self.missing):
                t.record_stream(current)
            self._streams.add(stream)
        return stream

    def grow(self, cu, tokens):
        """Adds cu[b + 1] - cu[b] tokens to every sequence b, `tokens` in all (moe_pool_grow); cu [batch + 1] int32.
        Returns slots [tokens] int64 and positions [tokens] int32 of the new tokens, and the pages to copy before
        their rows are stored, src and dst [batch] int32.  `missing` then holds how many pages were not to be had: one
        tensor, like the pool's others, which the next call writes again."""
        return _native.pool_grow(self._at, self._index, self._on_stream(), self.ws.data_ptr(), self.ws_bytes, cu,
                                 tokens, self.missing.data_ptr())

    def fork(self, parents):
        """Makes every sequence b a fork of sequence parents[b], int32 [batch]; -1 leaves it empty (moe_pool_fork)."""
        _native.pool_fork(self._at, self._index, self._on_stream(), parents)

    def trim(self, lens=None, window=0, sinks=0):
        """Cuts sequences to lens, int32 [batch], and frees the pages that no token from now on sees
        (moe_pool_trim)."""
        _native.pool_trim(self._at, self._index, self._on_stream(), lens, window, sinks)
