"""Binding of the attention operators (include/moe_attn.h): the paged
key-value cache's append with the position rotation, attention of new tokens
over the cache, and attention over packed prompts.

Rows are bf16 tensors [tokens, heads, head_dim] whose last index is
contiguous; the other strides are free (multiples of 8 elements), so slices of
a fused projection's output are taken as they are.
"""

import ctypes

import torch

from . import _check, _i32, _i64, _ptr, _sz, _vp, lib

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


def _stream(device):
    return _raw_stream(device.index)


_bf16, _int32, _int64 = torch.bfloat16, torch.int32, torch.int64


def _refuse(t, dtype, shape, device, name):
    """Raises for what is wrong with an argument."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_cuda:
        raise ValueError("tensors passed to the HIP library must be on the GPU")
    raise ValueError(f"{name} is on {t.device}, the call's other tensors are on {device}")


# The checks below run on every call of a decode step, where the host's time
# is what a small call costs: one test for all that is usual, the reasons apart.


def _rows(t, tokens, heads, dim, device, name):
    """MoeRowsC of a [tokens, heads, dim] bf16 tensor on the GPU `device`."""
    if t.dtype is not _bf16 or t.shape != (tokens, heads, dim) or t.device != device:
        _refuse(t, _bf16, (tokens, heads, dim), device, name)
    st, sh, se = t.stride()
    if se != 1:
        raise ValueError(f"{name}: the last index must be contiguous")
    # strides over indices of one value are free
    return MoeRowsC(t.data_ptr() or None, st if tokens > 1 else 0, sh if heads > 1 else 0)


def _new_rows(tokens, heads, dim, device):
    """A new [tokens, heads, dim] bf16 tensor and its MoeRowsC."""
    t = torch.empty((tokens, heads, dim), dtype=_bf16, device=device)
    return t, MoeRowsC(t.data_ptr() or None, heads * dim, dim)


def _ints(t, dtype, shape, device, name):
    """The address of a contiguous tensor on the GPU `device`."""
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        _refuse(t, dtype, shape, device, name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr() or _ptr(t)


class KVCache:
    """Handle on a paged cache's tensors (moe_kv_cache).

    k, v [pages, heads, page_size, head_dim]: bf16, or FP8 (uint8 E4M3 codes or
    float8_e4m3fn) with k_scale, v_scale [pages, heads, page_size,
    max(1, head_dim // 128)] uint8 E8M0 bytes.  v None or k itself: one tensor
    serves as keys and values.  Any strides over the first three indices that
    k and v share, such as those of [pages, page_size, heads, head_dim]
    transposed."""

    def __init__(self, k, v=None, k_scale=None, v_scale=None):
        self.shared = v is None or v is k or v.data_ptr() == k.data_ptr()
        if self.shared:
            v, v_scale = k, k_scale
        if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype or v.device != k.device:
            raise ValueError("k and v must be alike, [pages, heads, page_size, head_dim]")
        if not k.is_cuda:
            raise ValueError("tensors passed to the HIP library must be on the GPU")
        if k.dtype is torch.bfloat16:
            self.format = KV_BF16
            if k_scale is not None:
                raise ValueError("a bf16 cache has no scales")
        elif k.dtype in (torch.uint8, torch.float8_e4m3fn):
            self.format = KV_FP8
        else:
            raise ValueError("a cache is bfloat16, or uint8 / float8_e4m3fn with scales")
        if k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError("k and v must share their strides and be contiguous in the last index")
        self.pages, self.heads, self.page_size, self.head_dim = k.shape
        self.device = k.device
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        ks = vs = None
        if self.format == KV_FP8:
            shape = (*k.shape[:3], max(1, self.head_dim // 128))
            if k_scale is None or v_scale is None:
                raise ValueError("an FP8 cache needs k_scale and v_scale")
            ks = _ints(k_scale, torch.uint8, shape, self.device, "k_scale")
            vs = _ints(v_scale, torch.uint8, shape, self.device, "v_scale")
        st = k.stride()
        self.c = MoeKvCacheC(k.data_ptr() or None, v.data_ptr() or None, ks, vs, self.pages, st[0], st[1], st[2],
                             self.page_size, self.heads, self.head_dim, self.format)
        self._ref = _byref(self.c)

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
        self.cos_sin, self.device = cos_sin, cos_sin.device
        self.c = MoeRopeC(_ptr(cos_sin), cos_sin.shape[0], cos_sin.shape[1], rot_offset, int(interleaved), 0)
        self._ref = _byref(self.c)

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
    if k.dim() != 3:
        raise ValueError("k must be [tokens, heads, head_dim]")
    tokens, heads, dim, dev = k.shape[0], cache.heads, cache.head_dim, cache.device
    kc = _rows(k, tokens, heads, dim, dev, "k")
    vc = _byref(_rows(v, tokens, heads, dim, dev, "v")) if v is not None else None
    sl = _ints(slots, _int64, (tokens,), dev, "slots")
    ps = _ints(positions, _int32, (tokens,), dev, "positions") if positions is not None else None
    if rope is not None and rope.device != dev:
        raise ValueError("rope is on another device than the cache")
    qc = oc = None
    hq = 0
    if q is not None:
        hq = q.shape[1]
        qc = _byref(_rows(q, tokens, hq, dim, dev, "q"))
        if q_out is None:
            q_out, oc = _new_rows(tokens, hq, dim, dev)
        else:
            oc = _rows(q_out, tokens, hq, dim, dev, "q_out")
        oc = _byref(oc)
    elif q_out is not None:
        raise ValueError("q_out without q")
    ko = _byref(_rows(k_out, tokens, heads, dim, dev, "k_out")) if k_out is not None else None
    _check(lib.moe_kv_append(cache._ref, rope._ref if rope is not None else None, tokens, sl, ps, _byref(kc), vc,
                             hq, qc, oc, ko, _stream(dev)))
    return q_out


def attn_workspace_size(batch, heads_q, heads_kv, head_dim, q_len=1):
    """Bytes of workspace moe_attn_decode needs (0 for an invalid configuration)."""
    c = MoeAttnConfigC(batch * q_len, 0, batch, q_len, heads_q, heads_kv, head_dim, 1, 0, 1.0)
    return lib.moe_attn_workspace_size(_byref(c))


class DecodeAttention:
    """Holds the sizes, the cache and the workspace of moe_attn_decode and runs
    it on the current stream: attention of every sequence's newest q_len tokens
    over the cache, which holds them already."""

    def __init__(self, cache: KVCache, batch, heads_q, q_len=1, window=0, scale=None):
        self.cache, self.batch, self.heads_q, self.q_len = cache, batch, heads_q, q_len
        self.tokens = batch * q_len
        scale = cache.head_dim ** -0.5 if scale is None else scale
        self.c = MoeAttnConfigC(self.tokens, 0, batch, q_len, heads_q, cache.heads, cache.head_dim, 1, window, scale)
        self._ref = _byref(self.c)
        self.ws_bytes = lib.moe_attn_workspace_size(self._ref)
        self.ws = torch.empty(max(self.ws_bytes, 1), dtype=torch.uint8, device=cache.device)
        self._ws = self.ws.data_ptr()

    def __call__(self, q, block_table, seq_lens, out=None, want_lse=False):
        """q [batch * q_len, heads_q, head_dim] bf16, block_table [batch, width]
        int32, seq_lens [batch] int32 (new tokens included): out like q, and
        with want_lse also lse [batch * q_len, heads_q] fp32."""
        cache, n, dev = self.cache, self.tokens, self.cache.device
        qc = _rows(q, n, self.heads_q, cache.head_dim, dev, "q")
        if out is None:
            out, oc = _new_rows(n, self.heads_q, cache.head_dim, dev)
        else:
            oc = _rows(out, n, self.heads_q, cache.head_dim, dev, "out")
        if block_table.dim() != 2:
            raise ValueError("block_table must be [batch, width]")
        width = block_table.shape[1]
        bt = _ints(block_table, _int32, (self.batch, width), dev, "block_table")
        sl = _ints(seq_lens, _int32, (self.batch,), dev, "seq_lens")
        lse = torch.empty((n, self.heads_q), dtype=torch.float32, device=dev) if want_lse else None
        _check(lib.moe_attn_decode(self._ref, _byref(qc), cache._ref, bt, width, sl, _byref(oc),
                                   lse.data_ptr() if want_lse else None, self._ws, self.ws_bytes, _stream(dev)))
        return (out, lse) if want_lse else out


def attn_decode(q, cache: KVCache, block_table, seq_lens, q_len=1, window=0, scale=None, out=None, want_lse=False):
    """One call of DecodeAttention."""
    a = DecodeAttention(cache, seq_lens.shape[0], q.shape[1], q_len, window, scale)
    return a(q, block_table, seq_lens, out, want_lse)


def attn_prefill(q, k, v, cu_q, cu_k=None, causal=True, window=0, scale=None, out=None, want_lse=False):
    """Attention over packed prompts (moe_attn_prefill): q [tokens, heads_q, head_dim], k and v [tokens_kv, heads_kv,
    head_dim] bf16, cu_q and cu_k [sequences + 1] int32; returns out like q, and with want_lse also lse
    [tokens, heads_q] fp32."""
    if q.dim() != 3 or k.dim() != 3 or cu_q.dim() != 1:
        raise ValueError("q, k and v must be [tokens, heads, head_dim], cu_q [sequences + 1]")
    if not q.is_cuda:
        raise ValueError("tensors passed to the HIP library must be on the GPU")
    (tokens, hq, dim), (keys, hkv, _), dev = q.shape, k.shape, q.device
    if cu_q.shape[0] < 1:
        raise ValueError("cu_q has sequences + 1 entries")
    if cu_k is None and keys != tokens:
        raise ValueError("without cu_k, k has as many rows as q")
    qc, kc = _rows(q, tokens, hq, dim, dev, "q"), _rows(k, keys, hkv, dim, dev, "k")
    vc = kc if v is k else _rows(v, keys, hkv, dim, dev, "v")
    batch = cu_q.shape[0] - 1
    cq = _ints(cu_q, _int32, (batch + 1,), dev, "cu_q")
    ck = _ints(cu_k, _int32, (batch + 1,), dev, "cu_k") if cu_k is not None else None
    if out is None:
        out, oc = _new_rows(tokens, hq, dim, dev)
    else:
        oc = _rows(out, tokens, hq, dim, dev, "out")
    lse = torch.empty((tokens, hq), dtype=torch.float32, device=dev) if want_lse else None
    c = MoeAttnConfigC(tokens, keys, batch, 1, hq, hkv, dim, int(causal), window,
                       dim ** -0.5 if scale is None else scale)
    _check(lib.moe_attn_prefill(_byref(c), _byref(qc), _byref(kc), _byref(vc), cq, ck, _byref(oc),
                                lse.data_ptr() if want_lse else None, _stream(dev)))
    return (out, lse) if want_lse else out
