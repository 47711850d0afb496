"""Pins of the serving oracle: known small cases, and the pool's bookkeeping against its own table."""

import random

import numpy as np
import pytest

from oracle import attention, serving


def test_tree_masks_by_hand():
    #      -1      -1
    #      0       3
    #     1 2      4      5: empty, 6: under the empty one, 7: no parent before it
    masks, depths = serving.tree_masks([[-1, 0, 0, -1, 3, -2, 5, 7]])
    assert masks == [[0b1, 0b11, 0b101, 0b1000, 0b11000, 0, 0, 0]]
    assert depths.tolist() == [[0, 1, 1, 0, 1, -1, -1, -1]]


def test_tree_keep_is_causal_for_a_chain():
    rng = np.random.default_rng(0)
    n, context = 5, 9
    q, k, v = rng.standard_normal((n, 2, 8)), rng.standard_normal((1, 14, 8)), rng.standard_normal((1, 14, 8))
    masks, _ = serving.tree_masks([[i - 1 for i in range(n)]])
    for window in (0, 6):
        got = serving.attend(q, k, v, serving.tree_keep(masks[0], context, n, window), 0.3)
        want = attention.attend(q, k, v, context, 0.3, True, window)
        for a, b in zip(got, want):
            assert np.allclose(a, b, rtol=1e-12, atol=0)


def test_window_keep_with_first_keys():
    keep = serving.window_keep(2, 10, 3, 2)
    assert np.flatnonzero(keep[0]).tolist() == [0, 1, 6, 7, 8]
    assert np.flatnonzero(keep[1]).tolist() == [0, 1, 7, 8, 9]
    assert serving.window_keep(2, 1, 3, 2).tolist() == [[False], [True]]    # the first row stands before the keys


def test_pool_by_hand():
    p = serving.Pool(6, 16, 3, 4)
    slots, positions, pairs, missing = p.grow([20, 0, 0])
    assert slots == list(range(20)) and positions == list(range(20)) and missing == 0
    p.fork([0, 0, -1])
    assert p.table[1][:2] == [0, 1] and p.refs == [2, 2, 0, 0, 0, 0] and p.lens == [20, 20, 0]
    # both grow on page 1: the first keeps it
    slots, _, pairs, _ = p.grow([1, 1, 17])
    assert pairs == [(-1, -1), (1, 2), (-1, -1)] and slots[:2] == [1 * 16 + 4, 2 * 16 + 4]
    assert p.table[2][:2] == [3, 4] and p.refs == [2, 1, 1, 1, 1, 0]
    p.trim([20, 3, 0])
    assert p.lens == [20, 3, 0] and p.refs == [2, 1, 0, 0, 0, 0]
    # sequence 1 now grows on page 0, which sequence 0 holds and does not grow on
    _, _, pairs, _ = p.grow([0, 1, 0])
    assert pairs[1] == (0, 2) and p.refs == [1, 1, 1, 0, 0, 0]


@pytest.mark.parametrize("seed", range(6))
def test_pool_counts_are_those_of_its_table(seed):
    rng = random.Random(seed)
    p = serving.Pool(30, 16, 5, 6)
    rows = {}                                             # what every slot holds: the sequence's history
    story = [[] for _ in range(5)]
    for turn in range(60):
        act = rng.choice(["grow", "fork", "trim", "window"])
        if act == "grow":
            counts = [rng.choice([0, 1, 5, 30]) for _ in range(5)]
            before = list(p.lens)
            slots, _, pairs, missing = p.grow(counts)
            for a, z in pairs:
                for r in range(16):
                    if a >= 0:
                        rows[z * 16 + r] = rows.get(a * 16 + r)
            at = 0
            for b, c in enumerate(counts):
                for i in range(c):
                    token = (turn, b, i)
                    if slots[at] >= 0:
                        rows[slots[at]] = token
                    if before[b] + i < p.lens[b]:
                        story[b].append(token if slots[at] >= 0 else None)
                    at += 1
        elif act == "fork":
            parents = [rng.randint(-1, 4) for _ in range(5)]
            p.fork(parents)
            story = [list(story[x]) if x >= 0 else [] for x in parents]
        else:
            lens = [rng.randint(0, 90) for _ in range(5)]
            window = act == "window"
            p.trim(lens, 20 if window else 0, 3)
            story = [s[:n] for s, n in zip(story, lens)]
            if window:
                story = [[t if j < 16 or j // 16 >= (len(s) - 19) // 16 else None for j, t in enumerate(s)]
                         for s in story]
        held = [page for r in p.table for page in r if page >= 0]
        assert p.refs == [held.count(i) for i in range(30)]
        for b, s in enumerate(story):
            assert len(s) == p.lens[b]
            for j, token in enumerate(s):
                page = p.table[b][j // 16]
                if token is not None and page >= 0:
                    assert rows[page * 16 + j % 16] == token


def test_a_shared_page_stays_with_its_longest_holder():
    p = serving.Pool(2, 16, 2, 4)
    p.grow([25, 0])
    p.fork([0, 0])
    p.trim([18, 25])
    # no page is left, and rows 2 to 8 of the shared one are positions 18 to 24 of sequence 1
    slots, _, pairs, missing = p.grow([3, 3])
    assert slots == [-1, -1, -1, 25, 26, 27] and pairs == [(-1, -1)] * 2 and missing == 1


@pytest.mark.parametrize("pages", [10, 14])
@pytest.mark.parametrize("seed", range(8))
def test_pool_short_of_pages_keeps_what_sequences_hold(seed, pages):
    """Forks cut to different lengths inside a page, then grown until pages run out: no slot that is given out is a
    row that another sequence holds."""
    rng = random.Random(100 * pages + seed)
    p = serving.Pool(pages, 16, 5, 6)
    rows, story, short = {}, [[] for _ in range(5)], 0
    for turn in range(80):
        act = rng.choice(["grow", "grow", "fork", "cut"])
        if act == "grow":
            counts = [rng.choice([1, 2, 5, 20])] * 5 if rng.random() < 0.7 else [rng.choice([0, 1, 20]) for _ in range(5)]
            before, tables = list(p.lens), [list(r) for r in p.table]
            slots, _, pairs, missing = p.grow(counts)
            short += missing
            for a, z in pairs:
                for r in range(16):
                    if a >= 0:
                        rows[z * 16 + r] = rows.get(a * 16 + r)
            at = 0
            for b, c in enumerate(counts):
                for i in range(c):
                    if slots[at] >= 0:
                        page, row = divmod(slots[at], 16)
                        for o in range(5):              # the other sequences as they are after the call
                            held = [col for col, x in enumerate(p.table[o]) if x == page and tables[o][col] == page]
                            assert all(o == b or col * 16 + row >= before[o] for col in held)
                        rows[slots[at]] = (turn, b, i)
                    if before[b] + i < p.lens[b]:
                        story[b].append((turn, b, i) if slots[at] >= 0 else None)
                    at += 1
        elif act == "fork":
            parents = [rng.choice([b, rng.randint(-1, 4)]) for b in range(5)]
            p.fork(parents)
            story = [list(story[x]) if x >= 0 else [] for x in parents]
        else:
            lens = [max(0, n - rng.choice([0, 0, 1, 3, 7, 12, 40])) for n in p.lens]
            p.trim(lens)
            story = [s[:n] for s, n in zip(story, lens)]
        for b, s in enumerate(story):
            assert len(s) == p.lens[b]
            for j, token in enumerate(s):
                page = p.table[b][j // 16]
                if token is not None and page >= 0:
                    assert rows[page * 16 + j % 16] == token
    assert short > 0


def test_a_sequence_whose_copy_is_refused_stays_as_it_is():
    p = serving.Pool(4, 16, 2, 4)
    p.refs[2:] = [1, 1]                                   # pages of somebody else
    p.grow([20, 0])
    p.fork([0, 0])
    slots, _, pairs, missing = p.grow([1, 30])
    assert slots == [20] + [-1] * 30 and pairs == [(-1, -1)] * 2 and missing == 3
    assert p.lens == [21, 20] and p.table == [[0, 1, -1, -1]] * 2 and p.refs == [2, 2, 1, 1]
    p.refs[3] = 0
    slots, _, pairs, missing = p.grow([0, 1])             # now there is a page for its copy
    assert slots == [3 * 16 + 4] and pairs == [(-1, -1), (1, 3)] and missing == 0 and p.lens == [21, 21]


@pytest.mark.parametrize("pages", [10, 14])
@pytest.mark.parametrize("seed", range(8))
def test_sequences_see_no_rows_but_their_own(seed, pages):
    """While pages run out: a token in a sequence's length is on no page, or on one whose row holds it."""
    rng = random.Random(7000 + 100 * pages + seed)
    p = serving.Pool(pages, 16, 5, 6)
    rows, story = {}, [[] for _ in range(5)]
    for turn in range(80):
        act = rng.choice(["grow", "grow", "fork", "cut"])
        if act == "grow":
            counts = [rng.choice([1, 2, 5, 20])] * 5 if rng.random() < 0.7 else [rng.choice([0, 1, 20]) for _ in range(5)]
            before = list(p.lens)
            slots, _, pairs, _ = p.grow(counts)
            for a, z in pairs:
                for r in range(16):
                    if a >= 0:
                        rows[z * 16 + r] = rows.get(a * 16 + r)
            at = 0
            for b, c in enumerate(counts):
                for i in range(c):
                    if slots[at] >= 0:
                        rows[slots[at]] = (turn, b, i)
                    at += 1
                story[b] += [(turn, b, i) for i in range(p.lens[b] - before[b])]
        elif act == "fork":
            parents = [rng.choice([b, rng.randint(-1, 4)]) for b in range(5)]
            p.fork(parents)
            story = [list(story[x]) if x >= 0 else [] for x in parents]
        else:
            lens = [max(0, n - rng.choice([0, 0, 1, 3, 7, 12, 40])) for n in p.lens]
            p.trim(lens)
            story = [s[:n] for s, n in zip(story, lens)]
        for b, s in enumerate(story):
            assert len(s) == p.lens[b]
            for j, token in enumerate(s):
                page = p.table[b][j // 16]
                assert page < 0 or rows[page * 16 + j % 16] == token
