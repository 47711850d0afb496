"""What a serving loop does around the paged cache (oracle; test infrastructure only): masked attention with any
mask, drafted trees, and the page pool, from their definitions."""

import numpy as np


def tree_masks(parents):
    """parents [batch, nodes] -> masks (Python ints) and depths, node by node."""
    masks, depths = [], []
    for row in parents:
        m, d = [], []
        for i, p in enumerate(row):
            up = 0 if p == -1 else m[p] if 0 <= p < i else None
            m.append(0 if up is None or (p >= 0 and up == 0) else up | 1 << i)
            d.append(bin(m[-1]).count("1") - 1)
        masks.append(m)
        depths.append(d)
    return masks, np.array(depths, np.int32).reshape(np.shape(parents))


def tree_keep(masks, context, nodes, window=0, sinks=0, capacity=None):
    """Which of context + nodes keys each row of a drafted tree keeps: [nodes, context + nodes]."""
    keep = np.zeros((nodes, context + nodes), bool)
    for i, m in enumerate(masks):
        m &= (1 << nodes) - 1
        if m == 0:
            continue
        position = context + bin(m).count("1") - 1
        for j in range(context):
            keep[i, j] = not window or j > position - window or j < sinks
        for n in range(nodes):
            keep[i, context + n] = m >> n & 1
    if capacity is not None:
        keep[:, capacity:] = False
    return keep


def window_keep(rows, keys, window, sinks, causal=True):
    """Rows at the last positions of `keys` keys: a window behind which the first keys stay visible."""
    p = keys - rows + np.arange(rows)[:, None]
    j = np.arange(keys)[None, :]
    keep = (j > p - window) | (j < sinks)
    return keep & (j <= p) if causal else keep


def attend(q, k, v, keep, scale):
    """One sequence.  q [rows, heads, dim], k and v [kv_heads, keys, dim], keep [rows, keys].  Returns out, lse, the
    sums sum_j p_j |v_j| and max_j scale sum_d |q_d k_jd| over kept j (for error bounds)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    rows, heads, _ = q.shape
    group = heads // k.shape[0]
    out, absv = np.zeros(q.shape), np.zeros(q.shape)
    lse, size = np.full((rows, heads), -np.inf), np.zeros((rows, heads))
    some = keep.any(1)
    for h in range(heads):
        kh, vh = k[h // group], v[h // group]
        s = np.where(keep, scale * (q[:, h] @ kh.T), -np.inf)
        m = np.where(some, s.max(1, initial=-np.inf), 0.0)
        e = np.exp(s - m[:, None])
        t = np.where(some, e.sum(1), 1.0)
        p = e / t[:, None]
        lse[some, h] = (m + np.log(t))[some]
        out[:, h], absv[:, h] = p @ vh, p @ np.abs(vh)
        size[:, h] = np.where(keep, abs(scale) * (np.abs(q[:, h]) @ np.abs(kh).T), 0.0).max(1, initial=0.0)
    return out, lse, absv, size


class Pool:
    """The page pool, one entry after another."""

    def __init__(self, pages, page_size, batch, width):
        self.refs, self.table, self.lens = [0] * pages, [[-1] * width for _ in range(batch)], [0] * batch
        self.page_size, self.width = page_size, width

    def _release(self, page):
        if 0 <= page < len(self.refs):
            self.refs[page] -= 1

    def grow(self, counts):
        """Returns slots, positions, (src, dst) of each sequence, and how many pages were missing.  Where all holders of
        a partly filled page grow, the one with the most tokens on it keeps it (of equals the first): what it writes
        there is behind the others' tokens, whether their copies are to be had or not.  A sequence whose copy is not to
        be had does not grow: its new rows would have to lie among the keeper's."""
        size, cap = self.page_size, self.width * self.page_size
        free = iter([p for p, n in enumerate(self.refs) if n == 0])
        longer = [min(n + c, cap) for n, c in zip(self.lens, counts)]
        held = [row[n // size] if n % size and m > n else -1 for row, n, m in zip(self.table, self.lens, longer)]
        refs = list(self.refs)
        growers = {}
        for b, page in enumerate(held):
            growers.setdefault(page, []).append(b)
        keeper = {page: max(bs, key=lambda b: (self.lens[b] % size, -b)) for page, bs in growers.items()}
        slots, positions, pairs, missing = [], [], [], 0
        for b, (n, m) in enumerate(zip(self.lens, longer)):
            pair, lost = (-1, -1), False
            mine = growers[held[b]]
            if 0 <= held[b] < len(refs) and refs[held[b]] > 1 and not (len(mine) == refs[held[b]] and keeper[held[b]] == b):
                page = next(free, -1)
                if page < 0:
                    missing, lost = missing + 1, True
                else:
                    pair = (held[b], page)
                    self.table[b][n // size] = page
                    self.refs[page] = 1
                    self.refs[held[b]] -= 1
            pairs.append(pair)
            for c in range(-(-n // size), -(-m // size)):
                page = next(free, -1)
                missing += page < 0
                self.table[b][c] = page
                if page >= 0:
                    self.refs[page] = 1
            for i in range(counts[b]):
                pos = n + i
                page = self.table[b][pos // size] if pos < cap else -1
                if lost and pos // size == n // size:
                    page = -1
                slots.append(page * size + pos % size if 0 <= page < len(self.refs) else -1)
                positions.append(pos)
            self.lens[b] = n if lost else m
        return slots, positions, pairs, missing

    def fork(self, parents):
        table, lens = [list(r) for r in self.table], list(self.lens)
        for b, p in enumerate(parents):
            if p == b:
                continue
            there = 0 <= p < len(lens)
            for page in table[b]:
                self._release(page)
            self.table[b] = list(table[p]) if there else [-1] * self.width
            for page in self.table[b]:
                if 0 <= page < len(self.refs):
                    self.refs[page] += 1
            self.lens[b] = lens[p] if there else 0

    def trim(self, lens=None, window=0, sinks=0):
        for b, row in enumerate(self.table):
            n = max(self.lens[b], 0) if lens is None else min(max(self.lens[b], 0), max(lens[b], 0))
            self.lens[b] = n
            for c in range(self.width):
                keys = range(c * self.page_size, (c + 1) * self.page_size)
                # the next token stands at position n
                if not any(j < n and (not window or j > n - window or j < sinks) for j in keys) and \
                        not (window and keys[0] < n and any(j > n - window or j < sinks for j in keys)):
                    self._release(row[c])
                    row[c] = -1
