"""The attention operators (include/moe_attn.h) against the oracle: kv_append bit by
bit, attn_decode and attn_prefill within bounds derived from their roundings.

Bounds.  With u = 2^-8 (bf16's unit roundoff) an output is a sum of weights
rounded to bf16 times v, rounded to bf16 once more: u (|out| + sum p |v|).
Scores are fp32 sums of D products in any order, off by at most
e = D 2^-23 max_j scale sum_d |q_d k_jd|, which moves every weight by at most
2 e relatively; exponentials, sums and joins in fp32 are within 2^-14 of
sum p |v| together.  lse is off by e and the fp32 arithmetic's 2^-20."""

import math

import numpy as np
import pytest
import torch

from gpu_util import dev, dev_bf16, host
from oracle import attention, formats, quant

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("block_scaled_fp4_sqrtsoftplus_amd")


def _vals(rng, *shape, scale=1.0):
    """bf16 bit patterns of normal values."""
    return formats.bf16_encode((rng.standard_normal(shape) * scale).astype(np.float32))


def _f(bits):
    return formats.bf16_decode(bits).astype(np.float32)


def _check(out, lse, ref, dim):
    want, want_lse, absv, size = ref
    got = formats.bf16_decode(host(out)).astype(np.float64)
    e = dim * 2.0 ** -23 * size
    tol = 2.0 ** -8 * (np.abs(want) + absv) * 1.01 + absv * (2.0 ** -14 + 2 * e[..., None])
    assert np.isfinite(got).all()
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])
    if lse is not None:
        g = lse.cpu().numpy().astype(np.float64)
        empty = np.isneginf(want_lse)
        assert np.array_equal(empty, np.isneginf(g))
        w = np.where(empty, 0, want_lse)
        assert (np.abs(np.where(empty, 0, g) - w) <= e + 2.0 ** -20 * (8 + np.abs(w))).all()


# ----------------------------------------------------------------------------
# kv_append
# ----------------------------------------------------------------------------


def _quant_rows(x):
    """act_quant per 128 elements, or per row of a 64-element head."""
    if x.shape[-1] >= 128:
        q, s = quant.act_quant(x.reshape(-1, x.shape[-1]))
    else:  # a row of 64 padded with zeros has the same scale
        q, s = quant.act_quant(np.concatenate([x.reshape(-1, 64), np.zeros((x.size // 64, 64), x.dtype)], -1))
        q = q[:, :64]
    return q.reshape(x.shape), s.reshape(*x.shape[:-1], -1)


def _table(n, rot):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    return np.concatenate([np.cos(a), np.sin(a)], -1).astype(np.float32)


@pytest.mark.parametrize("tokens,hq,hkv,dim,fp8,rot,offset,inter,page,by_token", [
    (1, 32, 8, 128, False, 128, 0, False, 16, False),
    (1, 5, 1, 64, True, 64, 0, True, 32, False),
    (7, 4, 2, 64, False, 32, 16, False, 16, True),
    (33, 64, 1, 512, True, 64, 448, True, 64, False),
    (50, 3, 3, 256, True, 256, 0, False, 128, True),
    (50, 16, 4, 256, False, 16, 8, True, 16, False),
    (64, 28, 4, 128, True, 96, 32, False, 16, True),
    (5000, 2, 1, 64, False, 64, 0, False, 16, False),      # more tokens than waves that share a token
    (4100, 1, 1, 128, True, 128, 0, True, 256, False),
    (12, 0, 2, 128, False, 0, 0, False, 16, False),        # no q, no rotation
    (19000, 24, 2, 64, False, 64, 0, False, 16, False),    # rows read past the caches
    (19000, 24, 2, 64, True, 32, 32, True, 64, False),
])
def test_kv_append_bits(tokens, hq, hkv, dim, fp8, rot, offset, inter, page, by_token):
    rng = np.random.default_rng(tokens * 7 + dim)
    pages = -(-tokens // page) + 3
    n_pos = 90
    qkv = _vals(rng, tokens, hq + 2 * hkv, dim, scale=3.0)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    positions = rng.integers(0, n_pos, tokens).astype(np.int32)
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    if tokens > 3:
        positions[1], positions[2] = n_pos, -1           # outside the table: NaN
        slots[0], slots[3] = -1, pages * page            # stored nowhere
    g = dev_bf16(qkv)
    groups = max(1, dim // 128)

    def pages_of(fill, dtype, last):
        shape = (pages, page, hkv, last) if by_token else (pages, hkv, page, last)
        t = torch.full(shape, fill, dtype=dtype, device="cuda")
        return t.transpose(1, 2) if by_token else t

    kc, vc = (pages_of(77, torch.uint8, dim) if fp8 else pages_of(-2.5, torch.bfloat16, dim) for _ in range(2))
    ks, vs = (torch.full((pages, hkv, page, groups), 9, dtype=torch.uint8, device="cuda") if fp8 else None
              for _ in range(2))
    cache = moe.KVCache(kc, vc, ks, vs)
    rope = moe.Rope(dev(_table(n_pos, rot)), offset, inter) if rot else None
    k_out = torch.zeros((tokens, hkv, dim), dtype=torch.bfloat16, device="cuda")
    q_out = moe.kv_append(cache, g[:, hq:hq + hkv], g[:, hq + hkv:], dev(slots), dev(positions) if rot else None,
                          rope, g[:, :hq] if hq else None, None, k_out)
    torch.cuda.synchronize()

    def turned(x):
        return attention.rotate(_f(x), _table(n_pos, rot), positions, offset, inter) if rot else _f(x)

    def same(got, want):
        got = formats.bf16_decode(host(got.contiguous())).astype(np.float32)
        assert np.array_equal(got, want, equal_nan=True)

    if hq:
        same(q_out, turned(q))
    else:
        assert q_out is None
    same(k_out, turned(k))
    stored = (slots >= 0) & (slots < pages * page)
    for got, sc, rows in ((kc, ks, turned(k)), (vc, vs, _f(v))):
        nan = np.isnan(rows).any(-1)
        if fp8:
            code, scale = np.full((pages * page, hkv, dim), 77, np.uint8), np.full((pages * page, hkv, groups), 9)
            c, s = _quant_rows(np.where(np.isnan(rows), 0, rows))
            code[slots[stored]], scale[slots[stored]] = c[stored], s[stored]
            gc = got.permute(0, 2, 1, 3).reshape(-1, hkv, dim).cpu().numpy()
            gs = sc.permute(0, 2, 1, 3).reshape(-1, hkv, groups).cpu().numpy()
            fine = np.ones((pages * page, hkv), bool)
            fine[slots[stored]] = ~nan[stored]
            assert np.array_equal(gc[fine], code[fine]) and np.array_equal(gs[fine], scale[fine])
        else:
            want = np.full((pages * page, hkv, dim), -2.5, np.float32)
            want[slots[stored]] = rows[stored]
            same(got.permute(0, 2, 1, 3).reshape(-1, hkv, dim), want)


def test_kv_append_in_place_and_one_tensor_cache():
    rng = np.random.default_rng(5)
    T, hq, dim = 37, 6, 512
    q, k = _vals(rng, T, hq, dim), _vals(rng, T, 1, dim)
    positions = np.arange(T, dtype=np.int32)
    table = _table(64, 64)
    cache = moe.KVCache.empty(4, 16, 1, dim, shared=True)
    assert cache.shared and cache.k is cache.v
    qd, kd = dev_bf16(q), dev_bf16(k)
    got = moe.kv_append(cache, kd, None, dev(np.arange(T, dtype=np.int64)), dev(positions),
                        moe.Rope(dev(table), dim - 64), qd, q_out=qd, k_out=kd)
    assert got is qd
    want_q = attention.rotate(_f(q), table, positions, dim - 64)
    want_k = attention.rotate(_f(k), table, positions, dim - 64)
    assert np.array_equal(_f(host(qd)), want_q) and np.array_equal(_f(host(kd)), want_k)
    rows = cache.k.permute(0, 2, 1, 3).reshape(-1, 1, dim)
    assert np.array_equal(_f(host(rows[:T].contiguous())), want_k)
    assert (rows[T:] == 0).all()


def test_rope_table_helper():
    r = moe.Rope.of(100, 32, base=500.0)
    a = np.arange(100)[:, None] * 500.0 ** (-2.0 * np.arange(16) / 32)
    # fp32 rounding of values at most 1
    assert np.abs(r.cos_sin.cpu().numpy() - np.concatenate([np.cos(a), np.sin(a)], -1)).max() <= 2.0 ** -24


# ----------------------------------------------------------------------------
# attn_decode
# ----------------------------------------------------------------------------


class _Paged:
    """Random sequences in a paged cache whose unused rows hold NaN."""

    def __init__(self, rng, lens, hkv, dim, page, fp8=False, shared=False, by_token=False, width=None, kv_scale=1.0):
        counts = [-(-n // page) for n in lens]
        pages = max(1, sum(counts)) + 2
        order = rng.permutation(pages)
        width = max(max(counts), 1) if width is None else width
        self.table = np.full((len(lens), width), -1, np.int32)
        self.lens, self.page = np.asarray(lens, np.int32), page
        at = 0
        for b, n in enumerate(counts):
            self.table[b, :n] = order[at:at + n]
            at += n
        groups = max(1, dim // 128)
        used = np.zeros((pages, page), bool)
        for b, n in enumerate(lens):
            for i, pg in enumerate(self.table[b, :counts[b]]):
                used[pg, :min(page, n - i * page)] = True
        used = np.broadcast_to(used[:, None, :], (pages, hkv, page))

        def one():
            x = _vals(rng, pages, hkv, page, dim, scale=kv_scale)
            if not fp8:
                x[~used] = 0x7FC0
                return x, None, _f(x).astype(np.float64)
            c, s = _quant_rows(_f(x))
            c[~used], s[~used] = 0x7F, 255
            return c, s.astype(np.uint8), attention.fp8_values(c, np.where(s == 255, 127, s))

        k, ks, self.k = one()
        v, vs, self.v = (k, ks, self.k) if shared else one()

        def up(x):
            t = dev(x) if fp8 else dev_bf16(x)
            return t.transpose(1, 2).contiguous().transpose(1, 2) if by_token else t

        kd = up(k)
        vd = None if shared else up(v)
        self.cache = moe.KVCache(kd, vd, dev(ks) if fp8 else None, dev(vs) if fp8 and not shared else None)

    def reference(self, q, q_len, scale, window=0, hidden=None):
        parts = []
        for b, n in enumerate(self.lens):
            n = int(n)
            rows = [attention.cache_rows(x, self.table[b], n) for x in (self.k, self.v)]
            parts.append(attention.attend(_f(q[b * q_len:(b + 1) * q_len]), *rows, n - q_len, scale, True, window,
                                          None if hidden is None else hidden[b]))
        return tuple(np.concatenate(x) for x in zip(*parts))


LENS = [1, 0, 16, 17, 31, 33, 128, 129, 700, 2]


@pytest.mark.parametrize("hq,hkv,dim,page,q_len,window,fp8,shared,by_token", [
    (8, 8, 128, 16, 1, 0, False, False, False),
    (32, 8, 128, 16, 1, 0, False, False, True),
    (10, 2, 64, 16, 1, 0, False, False, False),
    (10, 2, 64, 64, 3, 0, True, False, False),
    (32, 8, 128, 32, 4, 0, True, False, True),
    (28, 4, 128, 16, 1, 40, False, False, False),
    (16, 4, 256, 16, 2, 1, False, False, False),
    (16, 4, 256, 128, 1, 130, True, False, True),
    (24, 1, 64, 16, 1, 0, False, False, False),        # two row tiles
    (20, 1, 128, 32, 3, 100, True, False, False),      # four row tiles, the last partly filled
    (64, 1, 512, 64, 1, 0, False, True, False),
    (64, 1, 512, 16, 2, 33, True, True, False),        # two row groups
    (5, 1, 512, 16, 16, 0, False, False, False),       # more new tokens than some sequences hold
    (8, 1, 512, 32, 1, 0, True, False, True),
])
def test_attn_decode(hq, hkv, dim, page, q_len, window, fp8, shared, by_token):
    rng = np.random.default_rng(hq + dim + page)
    p = _Paged(rng, LENS, hkv, dim, page, fp8, shared, by_token, width=-(-700 // page) + 2)
    q = _vals(rng, len(LENS) * q_len, hq, dim)
    scale = dim ** -0.5 * 1.5
    out, lse = moe.attn_decode(dev_bf16(q), p.cache, dev(p.table), dev(p.lens), q_len, window, scale, want_lse=True)
    torch.cuda.synchronize()
    _check(out, lse, p.reference(q, q_len, scale, window), dim)


@pytest.mark.parametrize("lens,hq,hkv,dim,fp8", [
    ([5000], 4, 1, 64, False),                 # one sequence over all splits
    ([9001, 3, 0, 130], 8, 2, 128, True),      # one long among short ones
    ([300] * 130, 2, 2, 64, False),            # more sequences than lanes of a wave
    ([1] * 700, 1, 1, 64, False),
])
def test_attn_decode_splits(lens, hq, hkv, dim, fp8):
    rng = np.random.default_rng(len(lens))
    p = _Paged(rng, lens, hkv, dim, 16, fp8)
    q = _vals(rng, len(lens), hq, dim)
    a = moe.DecodeAttention(p.cache, len(lens), hq)
    a.ws.fill_(0xFF)                           # the workspace need not be cleared
    out, lse = a(dev_bf16(q), dev(p.table), dev(p.lens), want_lse=True)
    torch.cuda.synchronize()
    _check(out, lse, p.reference(q, 1, dim ** -0.5), dim)
    again, _ = a(dev_bf16(q), dev(p.table), dev(p.lens), want_lse=True)
    assert torch.equal(out, again)             # equal calls give equal bits


@pytest.mark.parametrize("hq,hkv,dim,q_len,fp8,shared", [
    (24, 1, 256, 1, False, False),     # 17 to 32 rows of 256 elements: four row tiles
    (16, 2, 256, 3, True, False),
    (12, 1, 256, 2, False, True),
    (40, 1, 256, 1, True, True),
])
def test_attn_decode_rows_of_large_heads(hq, hkv, dim, q_len, fp8, shared):
    rng = np.random.default_rng(hq + q_len)
    p = _Paged(rng, LENS, hkv, dim, 32, fp8, shared)
    q = _vals(rng, len(LENS) * q_len, hq, dim)
    out, lse = moe.attn_decode(dev_bf16(q), p.cache, dev(p.table), dev(p.lens), q_len, want_lse=True)
    torch.cuda.synchronize()
    _check(out, lse, p.reference(q, q_len, dim ** -0.5), dim)


@pytest.mark.parametrize("hq,dim", [(8, 128), (24, 128), (40, 256), (64, 512)])
def test_attn_decode_one_tensor_with_two_sets_of_scales(hq, dim):
    # keys and values of the same codes, the values four times as large
    rng = np.random.default_rng(hq)
    p = _Paged(rng, [400, 33, 0], 1, dim, 16, fp8=True, shared=True)
    scales = p.cache.k_scale.clone()
    scales[scales != 255] += 2
    p.cache.c.v_scale = scales.data_ptr()
    p.v = p.v * 4
    q = _vals(rng, 3, hq, dim)
    out, lse = moe.attn_decode(dev_bf16(q), p.cache, dev(p.table), dev(p.lens), want_lse=True)
    torch.cuda.synchronize()
    _check(out, lse, p.reference(q, 1, dim ** -0.5), dim)


def test_attn_decode_window_leaves_freed_pages_unread():
    # pages before every row's window are gone from the table
    rng = np.random.default_rng(9)
    p = _Paged(rng, [500, 77], 2, 128, 16)
    table = p.table.copy()
    table[0, :(500 - 1 - 64) // 16] = -1
    table[0, 0] = 1 << 30
    q = _vals(rng, 4, 4, 128)
    out, lse = moe.attn_decode(dev_bf16(q), p.cache, dev(table), dev(p.lens), 2, 64, want_lse=True)
    torch.cuda.synchronize()
    _check(out, lse, p.reference(q, 2, 128 ** -0.5, 64), 128)


def test_attn_decode_values_out_of_range():
    rng = np.random.default_rng(10)
    p = _Paged(rng, [64, 40, 64], 1, 64, 16)
    q = _vals(rng, 3, 2, 64)
    table, lens = p.table.copy(), p.lens.copy()
    hidden = [np.zeros(64, bool), np.zeros(40, bool), np.zeros(64, bool)]
    table[0, 1], hidden[0][16:32] = 99999, True     # a page past the cache, its keys left out
    table[0, 3], hidden[0][48:64] = -5, True
    lens[2] = 1000                                  # longer than the table: what the table holds
    out, lse = moe.attn_decode(dev_bf16(q), p.cache, dev(table), dev(lens), want_lse=True)
    torch.cuda.synchronize()
    _check(out, lse, p.reference(q, 1, 64 ** -0.5, hidden=hidden), 64)
    lens[:] = -3
    out, lse = moe.attn_decode(dev_bf16(q), p.cache, dev(table), dev(lens), want_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_attn_decode_peaked_and_negative_scale():
    # scores far apart: the running maximum rises late and by a lot
    rng = np.random.default_rng(11)
    p = _Paged(rng, [400, 33], 1, 128, 32, kv_scale=4.0)
    q = _vals(rng, 2, 8, 128, scale=4.0)
    for scale in (1.0, -1.0):
        out, lse = moe.attn_decode(dev_bf16(q), p.cache, dev(p.table), dev(p.lens), scale=scale, want_lse=True)
        torch.cuda.synchronize()
        _check(out, lse, p.reference(q, 1, scale), 128)


# ----------------------------------------------------------------------------
# attn_prefill
# ----------------------------------------------------------------------------


def _cu(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


@pytest.mark.parametrize("hq,hkv,dim,q_lens,k_lens,causal,window,shared", [
    (2, 2, 64, [1], None, True, 0, False),
    (2, 1, 64, [0, 130, 1, 0, 33], None, True, 0, False),
    (8, 2, 128, [65, 7, 200], None, True, 0, False),
    (8, 8, 128, [300, 64], None, True, 50, False),        # key-value heads dealt to the XCDs
    (5, 1, 64, [77, 140], None, False, 0, False),
    (6, 2, 128, [40, 129], [200, 129], True, 0, False),   # a context before the prompt
    (6, 2, 128, [40, 129], [200, 150], True, 70, False),
    (4, 4, 64, [50, 20, 5], [20, 20, 0], True, 0, False),  # fewer keys: rows that keep nothing
    (4, 4, 64, [50, 20, 5], [20, 20, 0], False, 0, False),
    (3, 1, 128, [90], [200], False, 30, False),           # a window alone
    (4, 2, 256, [100, 31], None, True, 0, False),
    (4, 2, 256, [70, 31], [90, 131], True, 20, False),
    (64, 1, 512, [5, 40], None, True, 0, True),
    (3, 1, 512, [150, 1], [150, 70], True, 0, False),
    (2, 1, 512, [70, 9], [100, 33], False, 0, False),
])
def test_attn_prefill(hq, hkv, dim, q_lens, k_lens, causal, window, shared):
    rng = np.random.default_rng(hq * 3 + dim + sum(q_lens))
    T, kl = sum(q_lens), q_lens if k_lens is None else k_lens
    K = sum(kl)
    # rows inside wider ones, with NaN beside them
    kinds = 1 if shared else 2
    wide_q, wide_k = _vals(rng, T + 1, hq + 1, dim), _vals(rng, K + 1, kinds * hkv + 1, dim)
    wide_q[T], wide_q[:, hq], wide_k[K], wide_k[:, kinds * hkv] = 0x7FC0, 0x7FC0, 0x7FC0, 0x7FC0
    qd, kvd = dev_bf16(wide_q)[:T, :hq], dev_bf16(wide_k)[:K]
    kd = kvd[:, :hkv]
    vd = kd if shared else kvd[:, hkv:2 * hkv]
    scale = dim ** -0.5 * 1.3
    back = torch.full((T + 1, hq, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    out, lse = moe.attn_prefill(qd, kd, vd, dev(_cu(q_lens)), None if k_lens is None else dev(_cu(k_lens)), causal,
                                window, scale, out=back[:T], want_lse=True)
    torch.cuda.synchronize()
    parts, cq, ck = [], _cu(q_lens), _cu(kl)
    for b in range(len(q_lens)):
        k = _f(wide_k[ck[b]:ck[b + 1], :hkv]).swapaxes(0, 1)
        v = k if shared else _f(wide_k[ck[b]:ck[b + 1], hkv:2 * hkv]).swapaxes(0, 1)
        parts.append(attention.attend(_f(wide_q[cq[b]:cq[b + 1], :hq]), k, v, kl[b] - q_lens[b], scale, causal,
                                      window))
    _check(out, lse, tuple(np.concatenate(x) for x in zip(*parts)), dim)
    assert (back[T] == 7.0).all()


def test_attn_prefill_peaked_scores_and_negative_scale():
    rng = np.random.default_rng(21)
    q, k, v = _vals(rng, 150, 2, 128, scale=4.0), _vals(rng, 150, 1, 128, scale=4.0), _vals(rng, 150, 1, 128)
    for scale in (1.0, -1.0):
        out, lse = moe.attn_prefill(dev_bf16(q), dev_bf16(k), dev_bf16(v), dev(_cu([150])), scale=scale, want_lse=True)
        torch.cuda.synchronize()
        _check(out, lse, attention.attend(_f(q), _f(k).swapaxes(0, 1), _f(v).swapaxes(0, 1), 0, scale), 128)


def test_attn_prefill_offsets_out_of_range_stay_in_bounds():
    # offsets past the rows are clamped, falling ones make empty sequences; rows of no sequence are left alone
    rng = np.random.default_rng(22)
    q, k, v = _vals(rng, 40, 2, 64), _vals(rng, 40, 2, 64), _vals(rng, 40, 2, 64)
    back = torch.full((40, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    cu = np.array([5, 20, 12, 9999], np.int32)
    moe.attn_prefill(dev_bf16(q), dev_bf16(k), dev_bf16(v), dev(cu), out=back)
    torch.cuda.synchronize()
    assert (back[:5] == 7.0).all() and torch.isfinite(back.float()).all()
    ref = attention.attend(_f(q[5:12]), _f(k[5:20]).swapaxes(0, 1), _f(v[5:20]).swapaxes(0, 1), 0, 64 ** -0.5)
    _check(back[5:12], None, ref, 64)      # rows of one sequence alone


# ----------------------------------------------------------------------------
# Offsets past 32 bits
# ----------------------------------------------------------------------------


@pytest.mark.parametrize("fp8,hq,dim", [(False, 8, 128), (True, 8, 128), (False, 40, 128)])
def test_far_pages_of_a_large_cache(fp8, hq, dim):
    # 4.9 GiB (bf16) or 2.4 GiB (FP8, past 2^31 bytes); the sequence's pages are the last ones
    rng = np.random.default_rng(50 + hq)
    hkv, page, n = 2, 64, 150
    pages = int((5.2e9 if not fp8 else 2.6e9) / (hkv * page * dim * (1 if fp8 else 2)))
    cache = moe.KVCache.empty(pages, page, hkv, dim, moe.KV_FP8 if fp8 else moe.KV_BF16, shared=True)
    table = np.array([[pages - 1, pages - 3, pages - 2]], np.int32)
    at = np.arange(n)
    slots = table[0, at // page].astype(np.int64) * page + at % page
    k, q = _vals(rng, n, hkv, dim), _vals(rng, 1, hq, dim)
    moe.kv_append(cache, dev_bf16(k), None, dev(slots))
    out, lse = moe.attn_decode(dev_bf16(q), cache, dev(table), dev(np.array([n], np.int32)), want_lse=True)
    torch.cuda.synchronize()
    rows = _f(k)
    if fp8:
        rows = attention.fp8_values(*_quant_rows(rows))
    rows = rows.swapaxes(0, 1)
    _check(out, lse, attention.attend(_f(q), rows, rows, n - 1, dim ** -0.5), dim)
    del cache
    torch.cuda.empty_cache()


def test_prefill_rows_far_apart():
    # a token stride of 2^22 elements: the last rows lie past 2^32 bytes
    rng = np.random.default_rng(60)
    n, dim, step = 600, 64, 1 << 22
    q, k = _vals(rng, n, 2, dim), _vals(rng, n, 1, dim)
    wide = torch.zeros(n * step, dtype=torch.bfloat16, device="cuda").view(n, step)
    wide[:, :2 * dim] = dev_bf16(q).view(n, -1)
    wide[:, 1024:1024 + dim] = dev_bf16(k).view(n, -1)
    qd = wide[:, :2 * dim].unflatten(1, (2, dim))
    kd = wide[:, 1024:1024 + dim].unflatten(1, (1, dim))
    out, lse = moe.attn_prefill(qd, kd, kd, dev(_cu([n])), want_lse=True)
    torch.cuda.synchronize()
    rows = _f(k).swapaxes(0, 1)
    _check(out, lse, attention.attend(_f(q), rows, rows, 0, dim ** -0.5), dim)
    del wide, qd, kd
    torch.cuda.empty_cache()


# ----------------------------------------------------------------------------
# Streams, graphs, refusals
# ----------------------------------------------------------------------------


def test_attention_calls_on_a_side_stream_and_in_a_graph():
    rng = np.random.default_rng(31)
    lens = [70, 5]
    p = _Paged(rng, lens, 2, 128, 16)
    q = _vals(rng, 2, 4, 128)
    qd, table, ln = dev_bf16(q), dev(p.table), dev(p.lens)
    a = moe.DecodeAttention(p.cache, 2, 4)
    eager = a(qd, table, ln).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = a(qd, table, ln)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(eager, on_side)
    out = torch.zeros_like(eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a(qd, table, ln, out=out)
    for i in range(4):
        qd.copy_(dev_bf16(_vals(np.random.default_rng(40 + i), 2, 4, 128)))
        ln.copy_(dev(np.array([70 - 9 * i, 5 - i], np.int32)))
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, a(qd, table, ln)), i


def test_empty_calls():
    cache = moe.KVCache.empty(2, 16, 2, 64)
    z = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    got = moe.kv_append(cache, z, z, torch.zeros(0, dtype=torch.int64, device="cuda"), None, None, z)
    assert got.shape == (0, 2, 64)
    assert moe.attn_decode(z, cache, torch.zeros((0, 3), **i32), torch.zeros(0, **i32)).shape == (0, 2, 64)
    assert moe.attn_prefill(z, z, z, torch.zeros(1, **i32)).shape == (0, 2, 64)
    # a cache of no pages: every row keeps nothing
    none = moe.KVCache.empty(0, 16, 2, 64)
    q = torch.ones((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = moe.attn_decode(q, none, torch.zeros((3, 2), **i32), torch.full((3,), 9, **i32), want_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_binding_refuses():
    cache = moe.KVCache.empty(4, 16, 2, 64)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    x = torch.zeros((3, 2, 64), **bf)
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="bfloat16"):
        moe.kv_append(cache, x.float(), x, slots)
    with pytest.raises(ValueError, match="shape"):
        moe.kv_append(cache, x, x[:2], slots)
    with pytest.raises(ValueError, match="slots"):
        moe.kv_append(cache, x, x, slots.int())
    with pytest.raises(ValueError, match="last index"):
        moe.kv_append(cache, torch.zeros((3, 64, 2), **bf).transpose(1, 2), x, slots)
    with pytest.raises(moe.MoeError, match="NULL"):
        moe.kv_append(cache, x, None, slots)               # two tensors take v
    with pytest.raises(moe.MoeError, match="NULL"):
        moe.kv_append(cache, x, x, slots, None, moe.Rope.of(4, 64))   # a rotation needs positions
    with pytest.raises(moe.MoeError, match="MISALIGNED"):
        moe.kv_append(cache, torch.zeros(3 * 128 + 1, **bf)[1:].view(3, 2, 64), x, slots)
    with pytest.raises(moe.MoeError, match="SHAPE"):
        moe.kv_append(cache, x, x, slots, torch.zeros(3, **i32), moe.Rope.of(4, 24))
    with pytest.raises(ValueError, match="GPU"):
        moe.KVCache(torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="scale"):
        moe.KVCache(torch.zeros((2, 2, 16, 64), dtype=torch.uint8, device="cuda"))
    q = torch.zeros((3, 4, 64), **bf)
    table, lens = torch.zeros((3, 2), **i32), torch.ones(3, **i32)
    with pytest.raises(ValueError, match="shape"):
        moe.attn_decode(q, cache, table[:2], lens)
    with pytest.raises(moe.MoeError, match="SHAPE"):
        moe.attn_decode(torch.zeros((3, 3, 64), **bf), cache, table, lens)   # 3 heads over 2
    with pytest.raises(moe.MoeError, match="SHAPE"):
        moe.attn_decode(q, cache, table, lens, scale=math.inf)
    with pytest.raises(ValueError, match="cu_k"):
        moe.attn_prefill(q, x[:2], x[:2], torch.tensor([0, 3], **i32))
    with pytest.raises(moe.MoeError, match="SHAPE"):
        moe.attn_prefill(q, x, x, torch.tensor([0, 3], **i32), window=-1)
    with pytest.raises(moe.MoeError, match="SHAPE"):
        y = torch.zeros((3, 2, 32), **bf)
        moe.attn_prefill(y, y, y, torch.tensor([0, 3], **i32))
