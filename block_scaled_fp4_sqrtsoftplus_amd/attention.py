"""Binding of the attention operators (include/moe_attn.h): the paged
key-value cache's append with the position rotation, attention of new tokens
over the cache, and attention over packed prompts.

Rows are bf16 tensors [tokens, heads, head_dim] whose last index is
contiguous; the other strides are free (multiples of 8 elements), so slices of
a fused projection's output are taken as they are.  Tensors are checked, and
outputs made, by the binding's native half (csrc/attn_binding.cpp).  There is no
backward pass: rows that require a gradient are refused unless gradients are off.
"""

import ctypes

import torch

from . import STATUS_NAMES, MoeError, _i32, _i64, _ptr, _sz, _vp, lib
from . import _attn_binding as _native

KV_BF16, KV_FP8 = 0, 1


class MoeRowsC(ctypes.Structure):
    _fields_ = [("p", _vp), ("stride_token", _i64), ("stride_head", _i64)]


class MoeKvCacheC(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("pages", _i64),
                ("stride_page", _i64), ("stride_head", _i64), ("stride_token", _i64),
                ("page_size", _i32), ("heads", _i32), ("head_dim", _i32), ("format", _i32)]


class MoeRopeC(ctypes.Structure):
    _fields_ = [("cos_sin", _vp), ("positions", _i64), ("rot_dim", _i32), ("rot_offset", _i32),
                ("interleaved", _i32), ("reserved", _i32)]


class MoeAttnConfigC(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("tokens_kv", _i64), ("batch", _i32), ("q_len", _i32), ("heads_q", _i32),
                ("heads_kv", _i32), ("head_dim", _i32), ("causal", _i32), ("window", _i32),
                ("scale", ctypes.c_float)]


_P = ctypes.POINTER
lib.moe_kv_append.restype = ctypes.c_int
lib.moe_kv_append.argtypes = [_P(MoeKvCacheC), _P(MoeRopeC), _i64, _vp, _vp, _P(MoeRowsC), _P(MoeRowsC), _i32,
                              _P(MoeRowsC), _P(MoeRowsC), _P(MoeRowsC), _vp]
lib.moe_attn_workspace_size.restype = _sz
lib.moe_attn_workspace_size.argtypes = [_P(MoeAttnConfigC)]
lib.moe_attn_decode.restype = ctypes.c_int
lib.moe_attn_decode.argtypes = [_P(MoeAttnConfigC), _P(MoeRowsC), _P(MoeKvCacheC), _vp, _i32, _vp, _P(MoeRowsC),
                                _vp, _vp, _sz, _vp]
lib.moe_attn_prefill.restype = ctypes.c_int
lib.moe_attn_prefill.argtypes = [_P(MoeAttnConfigC), _P(MoeRowsC), _P(MoeRowsC), _P(MoeRowsC), _vp, _vp,
                                 _P(MoeRowsC), _vp, _vp]

_byref = ctypes.byref
_raw_stream = torch._C._cuda_getCurrentRawStream


_native.set_error(MoeError)


def _fit(*sizes):
    """Whether the C structs' 32-bit fields hold these: ctypes would drop their upper bits."""
    return all(-(1 << 31) <= n < 1 << 31 for n in sizes)


def _check_fit(*sizes):
    if not _fit(*sizes):
        raise MoeError(STATUS_NAMES.index("MOE_ERR_BAD_SHAPE"))


def _bytes_at(t, shape, device, name):
    """The address of a contiguous uint8 tensor on `device`."""
    if t.dtype is not torch.uint8 or t.shape != shape or t.device != device:
        raise ValueError(f"{name} must be uint8 {tuple(shape)} on {device}")
    return _ptr(t)


class KVCache:
    """Handle on a paged cache's tensors (moe_kv_cache).

    k, v [pages, heads, page_size, head_dim]: bf16, or FP8 (uint8 E4M3 codes or
    float8_e4m3fn) with k_scale, v_scale [pages, heads, page_size,
    max(1, head_dim // 128)] uint8 E8M0 bytes.  v None or k itself (or its very
    elements): one tensor serves as keys and values, under the keys' scales unless v_scale
    is given too.  Any strides over the first three indices that
    k and v share, such as those of [pages, page_size, heads, head_dim]
    transposed."""

    def __init__(self, k, v=None, k_scale=None, v_scale=None):
        if v is None:
            v = k
        codes = (torch.uint8, torch.float8_e4m3fn)
        if k.dim() != 4 or v.shape != k.shape or v.device != k.device or \
                v.dtype != k.dtype and not (k.dtype in codes and v.dtype in codes):
            raise ValueError("k and v must be alike, [pages, heads, page_size, head_dim]")
        if not k.is_cuda:
            raise ValueError("tensors passed to the HIP library must be on the GPU")
        if k.dtype is torch.bfloat16:
            self.format = KV_BF16
            if k_scale is not None or v_scale is not None:
                raise ValueError("a bf16 cache has no scales")
        elif k.dtype in codes:
            self.format = KV_FP8
        else:
            raise ValueError("a cache is bfloat16, or uint8 / float8_e4m3fn with scales")
        if any(n > 1 and a != b for n, a, b in zip(k.shape, k.stride(), v.stride())) or k.stride(3) != 1:
            raise ValueError("k and v must share their strides and be contiguous in the last index")
        # one tensor, if not one object: the same elements (an empty tensor has no address)
        self.shared = v is k or (k.numel() > 0 and v.data_ptr() == k.data_ptr())
        if self.shared:
            v, v_scale = k, k_scale if v_scale is None else v_scale
        self.pages, self.heads, self.page_size, self.head_dim = k.shape
        _check_fit(self.heads, self.page_size, self.head_dim)
        self.device = k.device
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        ks = vs = None
        if self.format == KV_FP8:
            shape = (*k.shape[:3], max(1, self.head_dim // 128))
            if k_scale is None or v_scale is None:
                raise ValueError("an FP8 cache needs k_scale and v_scale")
            ks = _bytes_at(k_scale, shape, self.device, "k_scale")
            vs = _bytes_at(v_scale, shape, self.device, "v_scale")
        st = k.stride()
        self.c = MoeKvCacheC(k.data_ptr() or None, v.data_ptr() or None, ks, vs, self.pages, st[0], st[1], st[2],
                             self.page_size, self.heads, self.head_dim, self.format)
        self._at, self._index = ctypes.addressof(self.c), self.device.index

    @classmethod
    def empty(cls, pages, page_size, heads, head_dim, format=KV_BF16, shared=False, device="cuda"):
        """A cache of new zeroed tensors."""
        shape = (pages, heads, page_size, head_dim)

        def one():
            if format == KV_BF16:
                return torch.zeros(shape, dtype=torch.bfloat16, device=device), None
            return (torch.zeros(shape, dtype=torch.uint8, device=device),
                    torch.zeros((*shape[:3], max(1, head_dim // 128)), dtype=torch.uint8, device=device))

        k, ks = one()
        return cls(k, None, ks) if shared else cls(k, *(lambda v, vs: (v, ks, vs))(*one()))


class Rope:
    """Handle on a rotation table (moe_rope): cos_sin [positions, rot_dim] fp32, rot_dim / 2
    cosines and then the sines of each position."""

    def __init__(self, cos_sin, rot_offset=0, interleaved=False):
        if cos_sin.dtype is not torch.float32 or cos_sin.dim() != 2:
            raise ValueError("cos_sin must be float32 [positions, rot_dim]")
        _check_fit(cos_sin.shape[1], rot_offset)
        self.cos_sin, self.device = cos_sin, cos_sin.device
        self.c = MoeRopeC(_ptr(cos_sin), cos_sin.shape[0], cos_sin.shape[1], rot_offset, int(interleaved), 0)
        self._at, self._index = ctypes.addressof(self.c), self.device.index

    @classmethod
    def of(cls, positions, rot_dim, base=10000.0, rot_offset=0, interleaved=False, device="cuda"):
        """The table of angles position * base ** (-2 i / rot_dim)."""
        half = rot_dim // 2
        a = torch.arange(positions, dtype=torch.float64)[:, None] \
            * base ** (-torch.arange(half, dtype=torch.float64) / half)
        return cls(torch.cat([a.cos(), a.sin()], -1).float().to(device), rot_offset, interleaved)


def kv_append(cache: KVCache, k, v, slots, positions=None, rope: Rope = None, q=None, q_out=None, k_out=None):
    """Rotate q and k, store k and v at `slots` of the cache (moe_kv_append);
    returns q_out (a new tensor if q is given without one; None without q).
    v is None exactly when the cache has one tensor for keys and values."""
    index = cache._index
    at = 0
    if rope is not None:
        if rope._index != index:
            raise ValueError("rope is on another device than the cache")
        at = rope._at
    return _native.kv_append(cache._at, at, index, _raw_stream(index), k, v, slots, positions, q, q_out, k_out)


def attn_workspace_size(batch, heads_q, heads_kv, head_dim, q_len=1):
    """Bytes of workspace moe_attn_decode needs (0 for an invalid configuration)."""
    if not _fit(batch, q_len, heads_q, heads_kv, head_dim):
        return 0
    c = MoeAttnConfigC(batch * q_len, 0, batch, q_len, heads_q, heads_kv, head_dim, 1, 0, 1.0)
    return lib.moe_attn_workspace_size(_byref(c))


class DecodeAttention:
    """Holds the sizes, the cache and the workspace of moe_attn_decode and runs
    it on the current stream: attention of every sequence's newest q_len tokens
    over the cache, which holds them already.  Calls that may overlap, on other
    streams, need an object each: they would share the workspace.  The object may go
    while calls are still running; a graph that recorded one needs it as long as it is replayed."""

    def __init__(self, cache: KVCache, batch, heads_q, q_len=1, window=0, scale=None):
        _check_fit(batch, q_len, heads_q, window)
        self.cache, self.batch, self.heads_q, self.q_len = cache, batch, heads_q, q_len
        self.tokens = batch * q_len
        scale = cache.head_dim ** -0.5 if scale is None else scale
        self.c = MoeAttnConfigC(self.tokens, 0, batch, q_len, heads_q, cache.heads, cache.head_dim, 1, window, scale)
        self._at, self._index = ctypes.addressof(self.c), cache._index
        self.ws_bytes = lib.moe_attn_workspace_size(_byref(self.c))
        self.ws = torch.empty(max(self.ws_bytes, 1), dtype=torch.uint8, device=cache.device)
        self._ws = self.ws.data_ptr()
        self._streams = {_raw_stream(self._index)}   # those the allocator knows the workspace to be used on

    def __call__(self, q, block_table, seq_lens, out=None, want_lse=False):
        """q [batch * q_len, heads_q, head_dim] bf16, block_table [batch, width]
        int32 contiguous, seq_lens [batch] int32 (new tokens included): out like q, and
        with want_lse also lse [batch * q_len, heads_q] fp32."""
        index = self._index
        stream = _raw_stream(index)
        if stream not in self._streams:
            self.ws.record_stream(torch.cuda.current_stream(index))
            self._streams.add(stream)
        return _native.attn_decode(self._at, self.cache._at, index, stream, self._ws, self.ws_bytes, q,
                                   block_table, seq_lens, out, want_lse)


def attn_decode(q, cache: KVCache, block_table, seq_lens, q_len=1, window=0, scale=None, out=None, want_lse=False):
    """One call of DecodeAttention."""
    a = DecodeAttention(cache, seq_lens.shape[0], q.shape[1], q_len, window, scale)
    return a(q, block_table, seq_lens, out, want_lse)


def attn_prefill(q, k, v, cu_q, cu_k=None, causal=True, window=0, scale=None, out=None, want_lse=False):
    """Attention over packed prompts (moe_attn_prefill): q [tokens, heads_q, head_dim], k and v [tokens_kv, heads_kv,
    head_dim] bf16, cu_q and cu_k [sequences + 1] int32; returns out like q, and with want_lse also lse
    [tokens, heads_q] fp32."""
    if not q.is_cuda:
        raise ValueError("tensors passed to the HIP library must be on the GPU")
    index = q.get_device()
    return _native.attn_prefill(index, _raw_stream(index), q, k, v, cu_q, cu_k, causal, window, scale, out, want_lse)
