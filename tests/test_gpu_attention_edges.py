"""Edges of the attention operators' contract (include/moe_attn.h): what lies in
places that no row keeps, caches of one tensor, streams, and sizes at the ends of the declared
ranges.  Bounds are those of test_gpu_attention."""

import numpy as np
import pytest
import torch

from gpu_util import dev, dev_bf16
from oracle import attention
from test_gpu_attention import _Paged, _check, _cu, _f, _vals
from test_gpu_attention_paths import splits_of

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("block_scaled_fp4_sqrtsoftplus_amd")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,dim,shared", [
    (4, 2, 64, False), (6, 2, 128, False), (4, 2, 256, False), (3, 1, 512, False), (8, 1, 512, True)])
def test_prefill_does_not_read_keys_before_every_window(hq, hkv, dim, shared, causal):
    # a window over a context: the keys before the first row's window (91, 102 and 14 of them, inside the tile that
    # the first kept key lies in) hold NaN and infinities
    rng = np.random.default_rng(dim + hq + causal)
    q_lens, k_lens, window = [40, 129, 7], [200, 300, 90], 70
    q, k = _vals(rng, sum(q_lens), hq, dim), _vals(rng, sum(k_lens), hkv, dim)
    v = k if shared else _vals(rng, sum(k_lens), hkv, dim)
    cq, ck = _cu(q_lens), _cu(k_lens)
    for b, (n, m) in enumerate(zip(q_lens, k_lens)):
        before = m - n + 1 - window
        assert 0 < before < m and before % 32
        for x in (k, v):
            x[ck[b]:ck[b] + before] = 0x7FC0                 # NaN
            x[ck[b]:ck[b] + before:3] = 0x7F80               # infinity
            x[ck[b] + 1:ck[b] + before:3] = 0xFF80
    kd = dev_bf16(k)
    out, lse = moe.attn_prefill(dev_bf16(q), kd, kd if shared else dev_bf16(v), dev(cq), dev(ck), causal, window,
                                want_lse=True)
    torch.cuda.synchronize()
    parts = []
    for b in range(3):
        rows = [_f(x[ck[b]:ck[b + 1]]).swapaxes(0, 1) for x in (k, v)]
        with np.errstate(invalid="ignore"):
            parts.append(attention.attend(_f(q[cq[b]:cq[b + 1]]), *rows, k_lens[b] - q_lens[b], dim ** -0.5, causal,
                                          window))
    _check(out, lse, tuple(np.concatenate(x) for x in zip(*parts)), dim)



@pytest.mark.parametrize("hq,dim,page,q_len,fp8", [
    (4, 128, 16, 2, False), (4, 64, 64, 1, True), (24, 128, 16, 2, False), (24, 256, 32, 1, True), (64, 512, 16, 3, False)])
def test_decode_does_not_read_keys_before_every_window(hq, dim, page, q_len, fp8):
    rng = np.random.default_rng(dim + hq)
    lens, window = [500, 77, 2000], 45
    p = _Paged(rng, lens, 1, dim, page, fp8)
    for b, n in enumerate(lens):
        at = np.arange(n - q_len + 1 - window)
        pages, rows = (dev(x.astype(np.int64)) for x in (p.table[b, at // page], at % page))
        for x, scale in ((p.cache.k, p.cache.k_scale), (p.cache.v, p.cache.v_scale)):
            x[pages, :, rows] = 0x7F if fp8 else float("nan")
            x[pages[::3], :, rows[::3]] = 0x7F if fp8 else float("inf")
            if fp8:
                scale[pages, :, rows] = 255
    q = _vals(rng, len(lens) * q_len, hq, dim)
    out, lse = moe.attn_decode(dev_bf16(q), p.cache, dev(p.table), dev(p.lens), q_len, window, want_lse=True)
    torch.cuda.synchronize()
    _check(out, lse, p.reference(q, q_len, dim ** -0.5, window), dim)


# ----------------------------------------------------------------------------
# Caches of one tensor
# ----------------------------------------------------------------------------


def test_append_writes_both_scales_of_one_tensor():
    # one tensor of codes under two arrays of scales: a new row's scales go into both, so that its values are its keys
    rng = np.random.default_rng(71)
    n, dim, page = 40, 256, 16
    cache = moe.KVCache.empty(4, page, 1, dim, moe.KV_FP8, shared=True)
    values = torch.full_like(cache.k_scale, 9)
    cache.c.v_scale = values.data_ptr()
    slots = rng.permutation(4 * page)[:n].astype(np.int64)
    slots[5] = -1
    moe.kv_append(cache, dev_bf16(_vals(rng, n, 1, dim, scale=30.0)), None, dev(slots))
    torch.cuda.synchronize()
    stored = dev(slots[slots >= 0])
    keys, values = (t.permute(0, 2, 1, 3).reshape(4 * page, -1) for t in (cache.k_scale, values))
    assert (keys[stored] > 100).all() and torch.equal(values[stored], keys[stored])
    others = torch.ones(4 * page, dtype=torch.bool, device="cuda")
    others[stored] = False
    assert (values[others] == 9).all() and (keys[others] == 0).all()


def test_cache_keeps_what_it_is_given():
    u8 = dict(dtype=torch.uint8, device="cuda")
    k = torch.zeros((4, 2, 16, 128), **u8)
    ks, vs = torch.zeros((4, 2, 16, 1), **u8), torch.ones((4, 2, 16, 1), **u8)
    for v in (None, k, k.view(4, 2, 16, 128), k.view(torch.float8_e4m3fn)):
        c = moe.KVCache(k, v, ks, vs)
        assert c.shared and c.v is c.k
        assert (c.c.k_scale, c.c.v_scale) == (ks.data_ptr(), vs.data_ptr()) and c.v_scale is vs
        c = moe.KVCache(k, v, ks)
        assert c.shared and (c.c.k_scale, c.c.v_scale) == (ks.data_ptr(), ks.data_ptr())
    # values that lie at the keys' address in another layout are not the keys
    for v in (k[:2], k[..., :64], k.view(4, 16, 2, 128).transpose(1, 2), k.view(torch.bfloat16)):
        assert v.data_ptr() == k.data_ptr()
        with pytest.raises(ValueError, match="k and v"):
            moe.KVCache(k, v, ks, vs)
    with pytest.raises(ValueError, match="scale"):
        moe.KVCache(k, None, ks, vs[:2])
    with pytest.raises(ValueError, match="scale"):
        moe.KVCache(k, torch.zeros_like(k), ks)
    b = torch.zeros((4, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
    for scales in (dict(k_scale=ks), dict(v_scale=vs)):
        with pytest.raises(ValueError, match="scales"):
            moe.KVCache(b, **scales)
    # strides over indices of one value are free, and empty tensors share no address
    one = torch.zeros((1, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
    moe.KVCache(one, torch.zeros((2, 2, 16, 128), dtype=torch.bfloat16, device="cuda")[1:])
    assert not moe.KVCache.empty(0, 16, 2, 64).shared


@pytest.mark.parametrize("hq,dim", [(8, 128), (64, 512)])
def test_values_under_their_own_scales(hq, dim):
    # the values are the keys' codes, four times as large
    rng = np.random.default_rng(hq)
    lens = [400, 33, 0]
    p = _Paged(rng, lens, 1, dim, 16, fp8=True, shared=True)
    scales = p.cache.k_scale.clone()
    scales[scales != 255] += 2
    cache = moe.KVCache(p.cache.k, None, p.cache.k_scale, scales)
    p.v = p.v * 4
    q = _vals(rng, 3, hq, dim)
    out, lse = moe.attn_decode(dev_bf16(q), cache, dev(p.table), dev(p.lens), want_lse=True)
    torch.cuda.synchronize()
    _check(out, lse, p.reference(q, 1, dim ** -0.5), dim)


# ----------------------------------------------------------------------------
# Streams
# ----------------------------------------------------------------------------


def test_workspace_is_kept_for_the_stream_it_is_used_on():
    # the object goes while its call still waits on a side stream: its workspace must not be given away
    rng = np.random.default_rng(73)
    p = _Paged(rng, [900, 5000], 2, 128, 16)
    q, table, lens = dev_bf16(_vals(rng, 2, 4, 128)), dev(p.table), dev(p.lens)
    a = moe.DecodeAttention(p.cache, 2, 4)
    want = a(q, table, lens)
    size, at = a.ws.numel(), a.ws.data_ptr()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)       # some ms in which the host goes on
        got = a(q, table, lens)
    del a
    other = torch.empty(size, dtype=torch.uint8, device="cuda")
    given_away = other.data_ptr() == at
    if not given_away:
        other.fill_(0xFF)
    torch.cuda.synchronize()
    assert not given_away and torch.equal(got, want)


# ----------------------------------------------------------------------------
# Refusals
# ----------------------------------------------------------------------------


def test_sizes_past_32_bits_are_refused():
    # they must not lose their upper bits on the way into the C structs
    cache = moe.KVCache.empty(2, 16, 2, 64)
    far = 1 << 32
    for kw in (dict(window=far + 5), dict(window=-far), dict(q_len=far + 1), dict(batch=far + 1),
               dict(heads_q=far + 2)):
        with pytest.raises(moe.MoeError, match="SHAPE"):
            moe.DecodeAttention(cache, **{**dict(batch=1, heads_q=2), **kw})
    table = torch.zeros((10, 64), device="cuda")
    with pytest.raises(moe.MoeError, match="SHAPE"):
        moe.Rope(table, rot_offset=far)
    wide = torch.zeros((1, 1, 16, 64), dtype=torch.bfloat16, device="cuda").expand(1, far + 1, 16, 64)
    with pytest.raises(moe.MoeError, match="SHAPE"):
        moe.KVCache(wide)
    none = torch.zeros((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.MoeError, match="SHAPE"):
        moe.kv_append(cache, none.expand(0, 2, 64), none.expand(0, 2, 64),
                      torch.zeros(0, dtype=torch.int64, device="cuda"), q=none.expand(0, far + 1, 64))


# ----------------------------------------------------------------------------
# Grids past 2^32 work-items
# ----------------------------------------------------------------------------


def _spread(x):
    """Bits of a tensor's rows summed per row, to compare many rows of the same inputs cheaply."""
    return x.view(torch.int16).flatten(1).long().sum(1)


def test_append_of_more_tokens_than_a_launch_takes():
    # 2^26 tokens and some, one wave each; all but the first and last three are padding
    n, dim = (1 << 26) + 5, 64
    cache = moe.KVCache.empty(1, 16, 1, dim, shared=True)
    k = torch.arange(dim, device="cuda").bfloat16().view(1, 1, dim).expand(n, 1, dim)
    slots = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    slots[:3], slots[-3:] = torch.arange(3), torch.arange(5, 8)
    moe.kv_append(cache, k, None, slots)
    torch.cuda.synchronize()
    rows = cache.k[0, 0]
    for i in range(16):
        assert torch.equal(rows[i], k[0, 0] if i in (0, 1, 2, 5, 6, 7) else torch.zeros_like(rows[i])), i


@pytest.mark.parametrize("batch,q_len,hq,hkv,width", [
    (65536, 16, 16, 16, 160),      # the join of cut sequences: a workgroup per row, 2^24 of them
    (16384, 1, 1024, 1024, 2),     # a workgroup per sequence and head, 2^24 of them
])
def test_decode_of_more_rows_than_a_launch_takes(batch, q_len, hq, hkv, width):
    # every sequence has the same keys and the same queries, but for its length: 3, 40 or 19
    rng = np.random.default_rng(75)
    dim, page = 64, 16
    p = _Paged(rng, [48], hkv, dim, page)
    q = dev_bf16(_vals(rng, q_len, hq, dim))
    lens = torch.tensor([3, 40, 19], dtype=torch.int32, device="cuda").repeat(batch // 3 + 1)[:batch].contiguous()
    lens[0], lens[-1] = 19, 40
    if width > 3:
        lens[2030:2060] = width * page                      # most of it on no page; some are cut
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    wide = min(width, p.table.shape[1])
    table[:, :wide] = dev(p.table)[:, :wide]
    lens.clamp_(max=width * page)
    many = q.repeat(batch, 1, 1)
    a = moe.DecodeAttention(p.cache, batch, hq, q_len)
    out = a(many, table, lens)
    torch.cuda.synchronize()
    assert (splits_of(a)[1] > 1).any() == (width > 3)
    sums = _spread(out).view(batch, q_len)
    del many, a
    for n in lens.unique().tolist():
        which = (lens == n).nonzero().flatten()
        b = int(which[0])
        one = moe.attn_decode(q, p.cache, table[b:b + 1].contiguous(), lens[b:b + 1].contiguous(), q_len)
        if n > 64:      # the order of its sums depends on where it is cut: both round weights and outputs to bf16
            got = out.view(batch, q_len, hq, dim)[which].float()
            assert (got - one.float()).abs().max() <= 4 * 2.0 ** -8 * 1.01 * np.nanmax(np.abs(p.v))
        else:
            assert torch.equal(sums[which], _spread(one).expand(len(which), q_len)), n
    del out
    torch.cuda.empty_cache()


def test_prefill_of_more_tiles_than_a_launch_takes():
    # 16384 prompts of one token, 1024 heads: each output is its value
    n, heads, dim = 16384, 1024, 64
    x = torch.randn((n, heads, dim), device="cuda", dtype=torch.bfloat16)
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    out = moe.attn_prefill(x, x, x, cu)
    torch.cuda.synchronize()
    assert torch.equal(out, x)
    del out, x
    torch.cuda.empty_cache()


def test_rows_of_nan_are_not_empty_rows():
    # lse is -inf for a row that keeps nothing, and NaN like the output for one whose query is NaN
    rng = np.random.default_rng(74)
    nan = float("nan")
    for lens, hq, dim in (([40, 0, 300], 3, 128), ([9000, 0, 8000], 3, 64), ([700, 0, 70], 20, 128),
                          ([3000, 0, 70], 64, 512)):       # whole, joined, many rows, many rows joined
        p = _Paged(rng, lens, 1, dim, 16)
        q = dev_bf16(_vals(rng, 3, hq, dim))
        want, want_lse = moe.attn_decode(q, p.cache, dev(p.table), dev(p.lens), want_lse=True)
        q[:2, 1] = nan
        out, lse = moe.attn_decode(q, p.cache, dev(p.table), dev(p.lens), want_lse=True)
        assert out[0, 1].isnan().all() and lse[0, 1].isnan()
        assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
        keep = [h for h in range(hq) if h != 1]
        assert torch.equal(out[0, keep], want[0, keep]) and torch.equal(lse[0, keep], want_lse[0, keep])
        assert torch.equal(out[2], want[2])
    for dim in (64, 128, 256, 512):
        q, k = dev_bf16(_vals(rng, 90, 2, dim)), dev_bf16(_vals(rng, 60, 1, dim))
        cu_q, cu_k = dev(_cu([40, 50])), dev(_cu([40, 20]))
        q[[7, 45], 1] = nan                                 # a row with keys, and one without
        out, lse = moe.attn_prefill(q, k, k, cu_q, cu_k, want_lse=True)
        assert out[7, 1].isnan().all() and lse[7, 1].isnan()
        assert (out[40:70] == 0).all() and torch.isneginf(lse[40:70]).all()
        assert lse.isnan().sum() == 1 and out.isnan().sum() == dim


def test_inputs_that_require_gradients_are_refused():
    # there is no backward pass: outputs without a graph would lose the gradient silently
    cache = moe.KVCache.empty(2, 16, 2, 64)
    i32 = dict(dtype=torch.int32, device="cuda")
    x = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    y = x.clone().requires_grad_()
    slots, table, ones, cu = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros((1, 1), **i32), \
        torch.ones(1, **i32), torch.tensor([0, 1], **i32)
    calls = [lambda t: moe.kv_append(cache, t, x, slots), lambda t: moe.kv_append(cache, x, t, slots),
             lambda t: moe.kv_append(cache, x, x, slots, q=t), lambda t: moe.attn_decode(t, cache, table, ones),
             lambda t: moe.attn_decode(x, cache, table, ones, out=t), lambda t: moe.attn_prefill(t, x, x, cu),
             lambda t: moe.attn_prefill(x, t, t, cu), lambda t: moe.attn_prefill(x, x, t, cu)]
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call(y)
        call(x)
        with torch.no_grad():
            call(y)
    torch.cuda.synchronize()


def test_flags_without_a_truth_value_are_refused():
    i32 = dict(dtype=torch.int32, device="cuda")
    cache, x = moe.KVCache.empty(2, 16, 2, 64), torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    table, ones, cu, two = torch.zeros((1, 1), **i32), torch.ones(1, **i32), torch.tensor([0, 1], **i32), \
        torch.tensor([1, 0])
    for call in (lambda: moe.attn_decode(x, cache, table, ones, want_lse=two),
                 lambda: moe.attn_prefill(x, x, x, cu, want_lse=two), lambda: moe.attn_prefill(x, x, x, cu, causal=two)):
        with pytest.raises(RuntimeError, match="ambiguous"):
            call()
