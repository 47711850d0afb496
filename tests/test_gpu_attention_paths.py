"""Attention over lengths that take the kernels' loops round many times, against the oracle:
decode work cut into pieces of many steps that cross the ends of sequences, read
from far more pages than a wave holds at once, and prompts whose tiles of K and V
go round the LDS several times.  What a decode call was cut into is read from the
workspace it leaves, so that a test which no longer reaches its path fails.

Bounds are those of test_gpu_attention."""

import numpy as np
import pytest
import torch

from gpu_util import dev, dev_bf16
from oracle import attention
from test_gpu_attention import _Paged, _check, _cu, _f, _vals

pytestmark = pytest.mark.gpu

moe = pytest.importorskip("block_scaled_fp4_sqrtsoftplus_amd")


def splits_of(a):
    """(first slot, splits) of every sequence, which a call of DecodeAttention leaves in the last
    ceil(batch * 8 / 256) * 256 bytes of its workspace."""
    n = -(-a.batch * 8 // 256) * 256
    m = a.ws[a.ws_bytes - n:][:a.batch * 8].view(torch.int32).view(-1, 2).cpu().numpy().astype(np.int64)
    return m[:, 0], m[:, 1]


def _lens(rng, count, most, empty=True):
    """Ragged lengths up to `most`, with 0, 1 and `most` among them."""
    lens = rng.integers(2, most, count)
    lens[0], lens[count // 2] = most, 1
    if empty:
        lens[[3, count - 1]] = 0
    return [int(n) for n in lens]


def _run(p, hq, q_len=1, window=0):
    """A call on workspace bytes of 0xFF against the oracle; its equal bits; (slots, splits)."""
    dim, batch = p.cache.head_dim, len(p.lens)
    q = _vals(np.random.default_rng(batch + hq), batch * q_len, hq, dim)
    a = moe.DecodeAttention(p.cache, batch, hq, q_len, window)
    a.ws.fill_(0xFF)
    qd, table, lens = dev_bf16(q), dev(p.table), dev(p.lens)
    out, lse = a(qd, table, lens, want_lse=True)
    torch.cuda.synchronize()
    _check(out, lse, p.reference(q, q_len, dim ** -0.5, window), dim)
    again, lse2 = a(qd, table, lens, want_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    return splits_of(a)


def _tiles(lens, size, q_len=1, window=0):
    lo = [max(0, n - q_len + 1 - window) & ~31 if window else 0 for n in lens]
    return np.array([max(1, -(-(n - a) // size)) for n, a in zip(lens, lo)])


# Up to 16 rows a head: pieces of 128-key tiles, equal over all sequences, four waves a tile.
# Sequence b's part of piece w has slot w + b.
@pytest.mark.parametrize("count,most,hq,hkv,dim,page,width,q_len,window,fp8,shared", [
    (130, 1500, 16, 8, 128, 16, 0, 1, 0, False, False),      # more sequences than lanes of a wave
    (130, 1500, 16, 8, 128, 16, 140, 1, 0, True, False),
    (130, 1500, 16, 8, 128, 32, 0, 2, 300, False, False),
    (70, 1300, 24, 24, 64, 64, 60, 1, 0, False, False),
    (70, 1300, 10, 2, 64, 16, 500, 3, 0, True, True),
    (20, 4000, 16, 4, 256, 16, 0, 1, 0, False, False),
    (20, 4000, 16, 4, 256, 128, 0, 2, 1000, True, False),
])
def test_decode_pieces_across_sequences(count, most, hq, hkv, dim, page, width, q_len, window, fp8, shared):
    rng = np.random.default_rng(count + dim + page)
    lens = _lens(rng, count, most)
    p = _Paged(rng, lens, hkv, dim, page, fp8, shared, width=width or None)
    slots, splits = _run(p, hq, q_len, window)
    tiles = _tiles(lens, 128, q_len, window)
    first = slots - np.arange(count)                         # piece of each sequence's first tile
    last = first + splits - 1
    assert (splits > 1).any()                                # cut,
    assert (last[:-1] == first[1:]).any()                    # in pieces that cross the end of a sequence
    assert tiles.sum() / (last[-1] + 1) > 1                  # and take more than a tile


# The page ids of 1024 consecutive keys are in the lanes of a wave: parts of more keys take the next ones.
@pytest.mark.parametrize("lens,hq,hkv,dim,page,fp8", [
    ([20011, 9000, 3000, 15000], 16, 16, 64, 16, False),
    ([20011, 9000, 3000, 15000], 16, 16, 64, 128, True),
    ([9000, 8011], 320, 16, 64, 16, False),                  # 20 rows a head: the kernel that shares K and V
    ([9000, 8011], 640, 16, 64, 32, True),                   # 40
])
def test_decode_parts_of_many_pages(lens, hq, hkv, dim, page, fp8):
    p = _Paged(np.random.default_rng(hq + page), lens, hkv, dim, page, fp8)
    _, splits = _run(p, hq)
    keys = max(n / s for n, s in zip(lens, splits))
    assert keys > 1024 + 64 and (splits > 1).any()


# More rows a head: each sequence cut by itself in pieces of 64-key tiles, which are one or two steps.
@pytest.mark.parametrize("lens,hq,hkv,dim,page,q_len,window,fp8,shared", [
    ("70 of 1500", 64, 1, 512, 64, 1, 0, False, True),       # one tensor, 64 keys a step
    ("70 of 1500", 64, 1, 512, 16, 1, 0, True, True),
    ("70 of 1500", 24, 1, 512, 16, 1, 0, False, False),      # two tensors, 32 keys a step
    ("9 of 5000", 64, 1, 512, 16, 4, 0, False, True),        # four row groups
    ("70 of 1500", 16, 2, 512, 32, 3, 700, True, True),
    ("70 of 1500", 20, 1, 128, 16, 1, 0, False, False),      # two row tiles, two waves a tile
    ("12 of 4000", 80, 4, 128, 16, 1, 0, True, False),
    ("12 of 4000", 80, 4, 64, 64, 1, 0, False, True),
    ("12 of 4000", 40, 4, 128, 16, 4, 900, False, False),    # 40 rows: four row tiles
    ("12 of 4000", 160, 4, 64, 16, 1, 0, True, True),
    ("12 of 4000", 80, 4, 256, 16, 1, 0, False, False),
    ("12 of 4000", 80, 4, 256, 128, 2, 0, True, True),
])
def test_decode_many_rows_over_many_steps(lens, hq, hkv, dim, page, q_len, window, fp8, shared):
    rng = np.random.default_rng(hq + dim + page)
    count, most = (int(x) for x in lens.split(" of "))
    lens = _lens(rng, count, most)
    p = _Paged(rng, lens, hkv, dim, page, fp8, shared)
    _, splits = _run(p, hq, q_len, window)
    tiles = _tiles(lens, 64, q_len, window)
    per = -(-tiles // splits)
    assert (splits > 1).any() and per.max() >= 3, (splits.max(), per.max())


# Prompts.  128- and 256-element heads run a step whose keys all rows keep, with the next tiles on their way, in a
# form of its own from four steps (of 64 and 32 keys) on; 512-element heads of one tensor turn three tiles.
@pytest.mark.parametrize("dim", [64, 128, 256, 512])
@pytest.mark.parametrize("q_lens,k_lens,causal,window", [
    ([733], None, True, 0),
    ([611, 900], None, True, 0),
    ([333, 801], None, False, 0),
    ([130, 47], [901, 633], True, 0),                        # a context
    ([300, 610], [811, 610], True, 450),                     # a window that keeps whole tiles
    ([410], [700], False, 333),
])
def test_prefill_of_many_steps(dim, q_lens, k_lens, causal, window):
    rng = np.random.default_rng(dim + sum(q_lens))
    hq, hkv, shared = (3, 1, True) if dim == 512 else (4, 2, False)
    kl = q_lens if k_lens is None else k_lens
    q, k = _vals(rng, sum(q_lens), hq, dim), _vals(rng, sum(kl), hkv, dim)
    v = k if shared else _vals(rng, sum(kl), hkv, dim)
    qd, kd, cq, ck = dev_bf16(q), dev_bf16(k), _cu(q_lens), _cu(kl)
    args = (qd, kd, kd if shared else dev_bf16(v), dev(cq), None if k_lens is None else dev(ck), causal, window)
    out, lse = moe.attn_prefill(*args, want_lse=True)
    torch.cuda.synchronize()
    parts = []
    for b in range(len(q_lens)):
        rows = [_f(x[ck[b]:ck[b + 1]]).swapaxes(0, 1) for x in (k, v)]
        parts.append(attention.attend(_f(q[cq[b]:cq[b + 1]]), *rows, kl[b] - q_lens[b], dim ** -0.5, causal, window))
    _check(out, lse, tuple(np.concatenate(x) for x in zip(*parts)), dim)
    again, lse2 = moe.attn_prefill(*args, want_lse=True)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("q_lens,k_lens,causal,window", [([333, 300], None, True, 0), ([200], [450], True, 170)])
def test_prefill_of_many_steps_on_two_tensors_of_512(q_lens, k_lens, causal, window):
    rng = np.random.default_rng(sum(q_lens))
    kl = q_lens if k_lens is None else k_lens
    q, k, v = _vals(rng, sum(q_lens), 2, 512), _vals(rng, sum(kl), 1, 512), _vals(rng, sum(kl), 1, 512)
    cq, ck = _cu(q_lens), _cu(kl)
    out, lse = moe.attn_prefill(dev_bf16(q), dev_bf16(k), dev_bf16(v), dev(cq), dev(ck), causal, window, want_lse=True)
    torch.cuda.synchronize()
    parts = [attention.attend(_f(q[cq[b]:cq[b + 1]]), _f(k[ck[b]:ck[b + 1]]).swapaxes(0, 1),
                              _f(v[ck[b]:ck[b + 1]]).swapaxes(0, 1), kl[b] - q_lens[b], 512 ** -0.5, causal, window)
             for b in range(len(q_lens))]
    _check(out, lse, tuple(np.concatenate(x) for x in zip(*parts)), 512)
