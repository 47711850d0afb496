"""Pins of the attention oracle: closed forms, the group property of rotations,
and the softmax identities."""

import numpy as np
import pytest

from oracle import attention, formats


def _bf16(x):
    return formats.bf16_decode(formats.bf16_encode(np.asarray(x, np.float32))).astype(np.float32)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_by_quarter_turns(interleaved):
    # cos = 0, sin = 1: (a, b) -> (-b, a), exactly; two of them negate
    x = _bf16(np.random.default_rng(1).standard_normal((3, 2, 64)))
    table = np.concatenate([np.zeros((4, 16)), np.ones((4, 16))], -1).astype(np.float32)
    pos = np.array([0, 1, 3])
    y = attention.rotate(x, table, pos, 32, interleaved)
    assert np.array_equal(y[..., :32], x[..., :32])
    p, r = x[..., 32:], y[..., 32:]
    if interleaved:
        assert np.array_equal(r[..., 0::2], -p[..., 1::2]) and np.array_equal(r[..., 1::2], p[..., 0::2])
    else:
        assert np.array_equal(r[..., :16], -p[..., 16:]) and np.array_equal(r[..., 16:], p[..., :16])
    z = attention.rotate(y, table, pos, 32, interleaved)
    assert np.array_equal(z[..., 32:], -p)


def test_rotation_keeps_relative_scores_and_marks_unknown_positions():
    # <R(p) q, R(p') k> depends on p - p' alone
    rng = np.random.default_rng(2)
    half = 32
    ang = np.arange(50)[:, None] * 10000.0 ** (-np.arange(half) / half)
    table = np.concatenate([np.cos(ang), np.sin(ang)], -1).astype(np.float32)
    q, k = (_bf16(rng.standard_normal((1, 1, 64))) for _ in range(2))
    dots = [float(np.sum(attention.rotate(q, table, [a]) * attention.rotate(k, table, [a - 7]), dtype=np.float64))
            for a in (7, 20, 49)]
    # 64 products of values near 1, each factor rounded to bf16
    assert np.ptp(dots) < 64 * 4 * 2.0 ** -8
    y = attention.rotate(q, table, [50])
    assert np.isnan(y).all()


def test_attention_closed_forms():
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((2, 9, 16)), rng.standard_normal((2, 9, 16))
    # zero queries: the mean of the kept values, lse = ln of their number
    out, lse, _, _ = attention.attend(np.zeros((4, 4, 16)), k, v, 5, 0.25)
    for i in range(4):
        assert np.allclose(out[i, 3], v[1, :6 + i].mean(0)) and np.isclose(lse[i, 0], np.log(6 + i))
    # one kept key: that value
    out, lse, _, _ = attention.attend(rng.standard_normal((1, 2, 16)), k, v, 6, 1.0, window=1)
    assert np.allclose(out[0, 0], v[0, 6])
    # nothing kept
    out, lse, _, _ = attention.attend(rng.standard_normal((2, 2, 16)), k, v, -1, 1.0)
    assert (out[0] == 0).all() and np.isneginf(lse[0]).all() and np.isfinite(lse[1]).all()


def test_attention_joins_over_parts():
    # softmax over all keys = the lse-weighted join of two halves
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((3, 2, 16)), rng.standard_normal((1, 40, 16)), rng.standard_normal((1, 40, 16))
    whole = attention.attend(q, k, v, 40, 0.3, causal=False)
    a = attention.attend(q, k[:, :13], v[:, :13], 40, 0.3, causal=False)
    b = attention.attend(q, k[:, 13:], v[:, 13:], 40, 0.3, causal=False)
    lse = np.logaddexp(a[1], b[1])
    out = np.exp(a[1] - lse)[..., None] * a[0] + np.exp(b[1] - lse)[..., None] * b[0]
    assert np.allclose(lse, whole[1]) and np.allclose(out, whole[0])


def test_cache_rows_follow_the_table():
    pages = np.arange(5 * 2 * 16 * 3).reshape(5, 2, 16, 3)
    rows = attention.cache_rows(pages, [3, 0, 4, -1], 37)
    assert rows.shape == (2, 37, 3)
    assert np.array_equal(rows[1, 20], pages[0, 1, 4]) and np.array_equal(rows[0, 36], pages[4, 0, 4])
