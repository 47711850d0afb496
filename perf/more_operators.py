"""Measured cases of the operators that a serving loop adds to the paged cache and its attentions: attention for a
tree of drafted tokens (tree_masks, attn_tree), windowed attention whose first tokens stay visible (attn_decode and
attn_prefill with sinks), the rows of a tree's accepted path moved to its front (kv_compact), and a pool of pages
that sequences fork, grow and free (PagePool, kv_copy_pages).

With `own` false, run() computes them in plain torch operations in 32 bits; with `own` true it calls the package.
listed() and draw() give the cases, prepare() their inputs, work() what one pass has to move and compute, and
exact() the results from the definitions in 64 bits (of what is moved, the values in their new places).

Head layouts (query heads / key-value heads x head size): 32/8 x 128 is the usual grouped layout, 64/1 x 512 the
decoder around this layer (64 heads on one shared 512-element key-value head), the others are generic."""

import math
import random

import torch

own = False

DEVICE = "cuda"


# ------------------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------------------


def _named(name, c):
    return dict(c, name=name) if name else c


def _tree(name, batch, longest, shortest, nodes, heads, kv_heads, dim, fmt="bf16", page=16, window=0, sinks=0,
          shared=False, mix=0):
    """Sequences of `shortest` to `longest` tokens in the cache and up to `nodes` drafted ones each."""
    return _named(name, dict(op="tree", batch=batch, longest=longest, shortest=shortest, nodes=nodes, heads=heads,
                             kv_heads=kv_heads, dim=dim, fmt=fmt, page=page, window=window, sinks=sinks, shared=shared,
                             mix=mix))


def _decode(name, batch, longest, shortest, window, sinks, heads, kv_heads, dim, fmt="bf16", page=16, q_len=1,
            shared=False, mix=0):
    """New tokens of streams that are `shortest` to `longest` tokens long."""
    return _named(name, dict(op="decode", batch=batch, longest=longest, shortest=shortest, window=window, sinks=sinks,
                             heads=heads, kv_heads=kv_heads, dim=dim, fmt=fmt, page=page, q_len=q_len, shared=shared,
                             mix=mix))


def _prefill(name, batch, longest, shortest, window, sinks, heads, kv_heads, dim, context=0, causal=True, shared=False,
             mix=0):
    return _named(name, dict(op="prefill", batch=batch, longest=longest, shortest=shortest, window=window, sinks=sinks,
                             heads=heads, kv_heads=kv_heads, dim=dim, context=context, causal=causal, shared=shared,
                             mix=mix))


def _compact(name, batch, longest, shortest, nodes, kv_heads, dim, fmt="bf16", page=16, shared=False, mix=0):
    """The rows of up to nodes / 2 accepted tokens of each sequence's `nodes` drafted ones."""
    return _named(name, dict(op="compact", batch=batch, longest=longest, shortest=shortest, nodes=nodes,
                             kv_heads=kv_heads, dim=dim, fmt=fmt, page=page, shared=shared, mix=mix))


def _pool(name, prompts, samples, longest, shortest, grown, pages, kv_heads, dim, fmt="bf16", page=16, shared=False,
          mix=0):
    """`prompts` sequences in a pool of `pages` pages, each sampled `samples` times by up to `grown` tokens."""
    return _named(name, dict(op="pool", prompts=prompts, samples=samples, longest=longest, shortest=shortest,
                             grown=grown, pages=pages, kv_heads=kv_heads, dim=dim, fmt=fmt, page=page, shared=shared,
                             mix=mix))


def listed():
    return [
        # one short conversation and a small draft: latency
        _tree("tree 1x300 8 nodes", 1, 300, 300, 8, 32, 8, 128),
        # drafts of up to 26 tokens checked for 32 sequences of different lengths
        _tree("tree 32x4096 26 nodes", 32, 4096, 700, 26, 32, 8, 128, mix=1),
        # the widest drafts over an FP8 cache: the matrix rate beside the reads
        _tree("tree 8x8192 64 nodes fp8", 8, 8192, 3000, 64, 32, 8, 128, "fp8", 64, mix=2),
        # the shared 512-element head under 64 query heads: the matrix rate
        _tree("tree 16x4096 16 nodes mqa512", 16, 4096, 2048, 16, 64, 1, 512, "bf16", 64, shared=True, mix=3),
        # one stream past its window, one new token: latency
        _decode("sinks decode 1x9000", 1, 9000, 9000, 512, 4, 32, 8, 128),
        # long streams in FP8 pages, of which only those of the window and the first tokens are still held: bandwidth
        _decode("sinks decode 64x500000 fp8", 64, 500000, 5000, 4096, 64, 32, 8, 128, "fp8", 64, mix=4),
        # packed prompts around the window's length
        _prefill("sinks prefill 5 packed", 5, 1500, 90, 256, 5, 28, 4, 128, mix=5),
        # one long prompt: the matrix rate
        _prefill("sinks prefill 1x8192", 1, 8192, 8192, 1024, 16, 32, 8, 128),
        # the accepted tokens of a few sequences: latency
        _compact("compact 3x500", 3, 500, 20, 7, 8, 128, mix=6),
        # a large batch with wide drafts, FP8 pages: scattered rows
        _compact("compact 512x2000 64 nodes fp8", 512, 2000, 100, 64, 8, 128, "fp8", 32, mix=7),
        # one prompt and five samples of it, a token each, in a pool of small pages: latency
        _pool("pool 1x5", 1, 5, 470, 470, 1, 4000, 1, 64, mix=8),
        # 16 prompts with 16 samples each, which grow by a few tokens: the copies of partly filled pages
        _pool("pool 16x16", 16, 16, 4000, 300, 9, 2560, 8, 128, "bf16", 64, mix=9),
    ]


#: (query heads, key-value heads, head size)
HEADS = [(32, 8, 128), (16, 2, 64), (64, 1, 512), (24, 24, 64), (28, 4, 128), (16, 4, 256), (8, 8, 128), (5, 1, 64)]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    heads, kv_heads, dim = rng.choice(HEADS)
    page = rng.choice([16, 32, 64, 128])
    fmt = rng.choice(["bf16", "fp8"])
    mix = rng.randrange(1 << 30)
    shared = dim == 512 and rng.random() < 0.5
    op = rng.choice(["tree", "decode", "prefill", "compact", "pool"])
    if op == "tree":
        batch, nodes = _spread(rng, 1, 64), _spread(rng, 1, 64)
        most = min(1.3e8 / (kv_heads * dim), 3.4e10 / (heads * dim * nodes)) / batch
        longest = _spread(rng, 1, min(65536, max(1, int(most))))
        window, sinks = rng.choice([(0, 0), (0, 0), (200, 0), (1000, 8)])
        return _tree(None, batch, longest, rng.randint(0, longest), nodes, heads, kv_heads, dim, fmt, page, window,
                     sinks, shared, mix)
    if op == "decode":
        batch, q_len = _spread(rng, 1, 96), rng.choice([1, 1, 1, 2, 5])
        most = min(2.5e8 / (kv_heads * dim), 3e9 / (heads * dim * q_len)) / batch
        window = _spread(rng, 32, min(8192, max(33, int(most))))
        longest = _spread(rng, 64, 500000)
        return _decode(None, batch, longest, rng.randint(0, longest), window, _spread(rng, 1, 130), heads, kv_heads,
                       dim, fmt, page, q_len, shared, mix)
    if op == "prefill":
        batch = _spread(rng, 1, 16)
        most = min(math.sqrt(8192 * 8192 * 32 * 128 / (batch * heads * dim * 2)), 6e7 / (batch * heads * dim))
        longest = _spread(rng, 1, min(8192, int(most)))
        return _prefill(None, batch, longest, rng.randint(1, longest), _spread(rng, 16, 2048), _spread(rng, 1, 130),
                        heads, kv_heads, dim, rng.choice([0, 0, rng.randint(1, longest)]), rng.random() < 0.8, shared,
                        mix)
    if op == "compact":
        batch, nodes = _spread(rng, 1, 512), _spread(rng, 2, 64)
        most = 4e8 / (kv_heads * dim * batch)
        longest = _spread(rng, 1, min(4096, max(1, int(most))))
        return _compact(None, batch, longest, rng.randint(0, longest), nodes, kv_heads, dim, fmt, page, shared, mix)
    prompts, samples, grown = _spread(rng, 1, 16), _spread(rng, 1, 16), _spread(rng, 1, 200)
    most = 3e8 / (kv_heads * dim)                          # rows of the cache
    longest = _spread(rng, 1, 4000)
    least = prompts * (longest // page + 1) + prompts * samples * (grown // page + 2)
    return _pool(None, prompts, samples, longest, rng.randint(1, longest), grown,
                 _spread(rng, least, max(least + 1, min(60000, int(most / page)))), kv_heads, dim, fmt, page, shared,
                 mix)


def _lengths(case, count):
    """`count` lengths between shortest and longest, the longest among them; the case alone decides."""
    rng = random.Random(case["mix"])
    lens = [rng.randint(case["shortest"], case["longest"]) for _ in range(count)]
    lens[rng.randrange(count)] = case["longest"]
    return lens


def _parents(case):
    """The drafted trees: each node's parent (-1: the sequence's last token), -2 for places that a smaller tree
    leaves empty."""
    rng = random.Random(case["mix"] + 1)
    n, trees = case["nodes"], []
    for b in range(case["batch"]):
        used = n if b == 0 else rng.randint(max(1, n // 2), n)
        # a parent is drawn from the nodes of late: trees of some depth
        trees.append([max(-1, i - 1 - int(rng.expovariate(0.4))) if i < used else -2 for i in range(n)])
    return trees


def _paths(parents):
    """For each node the nodes from the root to itself; none for an empty place."""
    paths = []
    for i, p in enumerate(parents):
        paths.append([] if p < -1 else (paths[p] if p >= 0 else []) + [i])
    return paths


def _accepted(case):
    """Each sequence's accepted nodes, in order: the first may stay, the others lie behind the places they go to."""
    rng = random.Random(case["mix"] + 1)
    paths = []
    for _ in range(case["batch"]):
        m = rng.randint(0, case["nodes"] // 2)
        path = sorted(rng.sample(range(m, case["nodes"]), m))
        if m and rng.random() < 0.5:
            path[0] = 0
        paths.append(path)
    return paths


def _grown(case):
    """How many tokens each sequence of a pool grows by: all by one at least, so that a prompt keeps its own pages."""
    rng = random.Random(case["mix"] + 1)
    return [rng.randint(1, case["grown"]) for _ in range(case["prompts"] * case["samples"])]


def _kept(case, q_len, kv_len):
    """How many (query, key) pairs the window and the first tokens keep, for one head."""
    total = 0
    for i in range(q_len):
        end = kv_len - q_len + i + 1
        high = min(kv_len, max(0, end)) if case.get("causal", True) else kv_len
        low = max(0, end - case["window"]) if case["window"] else 0
        total += max(0, high - low) + min(case["sinks"], low, high)
    return total


def _row_bytes(case):
    return case["dim"] * 2 if case["fmt"] == "bf16" else case["dim"] + max(1, case["dim"] // 128)


def work(case):
    kv_heads, dim = case["kv_heads"], case["dim"]
    kinds = 1 if case["shared"] else 2
    if case["op"] == "tree":
        heads, n = case["heads"], case["nodes"]
        keys = pairs = 0
        for length, parents in zip(_lengths(case, case["batch"]), _parents(case)):
            live = [p for p in _paths(parents) if p]
            seen = [max(0, length + len(p) - case["window"]) if case["window"] else 0 for p in live]   # windows' starts
            pairs += sum(max(0, length - s) + min(case["sinks"], s, length) + len(p) for s, p in zip(seen, live))
            keys += max(0, length - min(seen)) + min(case["sinks"], min(seen), length) + len(live)
        rows = case["batch"] * n
        return {"bytes": keys * kv_heads * _row_bytes(case) * kinds + rows * heads * (dim * 4 + 4)
                + rows * 8 + keys // case["page"] * 4, "flops": pairs * heads * 4 * dim}
    if case["op"] == "decode":
        q_len = case["q_len"]
        seen = [min(n, case["window"] + q_len - 1) + min(case["sinks"], max(0, n - case["window"] - q_len + 1))
                for n in _lengths(case, case["batch"])]
        rows = case["batch"] * q_len * case["heads"]
        pairs = sum(_kept(case, q_len, n) for n in _lengths(case, case["batch"])) * case["heads"]
        return {"bytes": sum(seen) * kv_heads * _row_bytes(case) * kinds + rows * (dim * 4 + 4)
                + sum(seen) // case["page"] * 4, "flops": pairs * 4 * dim}
    if case["op"] == "prefill":
        lens, heads = _lengths(case, case["batch"]), case["heads"]
        tokens, keys = sum(lens), sum(n + case["context"] for n in lens)
        pairs = sum(_kept(case, n, n + case["context"]) for n in lens) * heads
        return {"bytes": tokens * heads * (dim * 4 + 4) + keys * kv_heads * dim * 2 * kinds, "flops": pairs * 4 * dim}
    if case["op"] == "compact":
        moved = sum(sum(i != p for i, p in enumerate(path)) for path in _accepted(case))
        return {"bytes": moved * kv_heads * _row_bytes(case) * kinds * 2 + case["batch"] * (case["nodes"] * 4 + 8),
                "flops": 0}
    page, samples = case["page"], case["samples"]
    lens, more = _lengths(case, case["prompts"]), _grown(case)
    held = sum(-(-n // page) for n in lens) * samples + sum(more) // page      # entries while the samples live
    copied = sum(samples - 1 for n in lens if n % page)         # one of those on a partly filled page keeps it
    return {"bytes": copied * page * kv_heads * _row_bytes(case) * kinds * 2 + case["pages"] * 4 + held * 16
            + sum(more) * 12, "flops": 0}


# ------------------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------------------


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEVICE)


def _quantized(x):
    """FP8 codes and power-of-two scale bytes (biased by 127) of rows, one scale for 128 elements (or the row,
    where it is shorter): the smallest scale with which nothing passes 448."""
    size = min(128, x.shape[-1])
    g = x.float().unflatten(-1, (-1, size))
    m, e = torch.frexp(g.abs().amax(-1))  # amax = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-127, 127)
    codes = torch.ldexp(g, -e.unsqueeze(-1)).flatten(-2).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), (e + 127).to(torch.uint8)


def _pages(case, gen, pages):
    """Filled pages [pages, kv_heads, page, dim] of the case's format, and their scales."""
    x = _normal(gen, pages, case["kv_heads"], case["page"], case["dim"])
    return _quantized(x.bfloat16()) if case["fmt"] == "fp8" else (x.bfloat16(), None)


def _cache(case, gen, pages):
    k, ks = _pages(case, gen, pages)
    v, vs = (k, ks) if case["shared"] else _pages(case, gen, pages)
    return {"k": k, "v": v, "k_scale": ks, "v_scale": vs}


def _table(gen, held):
    """Block table whose entries that `held` [sequences, width] marks are pages in random order, -1 elsewhere; and
    how many pages that is."""
    count = int(held.sum())
    order = torch.randperm(max(1, count), generator=gen, device=DEVICE, dtype=torch.int32)
    rank = (held.flatten().cumsum(0) - 1).clamp(min=0).view(held.shape)
    return torch.where(held, order[rank], -1).int().contiguous(), max(1, count)


def _columns(lens, page, width=None):
    """Which entries of a block table hold tokens of sequences that are `lens` long."""
    width = max(1, -(-max(lens) // page)) if width is None else width
    return torch.arange(width, device=DEVICE) * page < _ints(lens)[:, None]


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    op, kv_heads, dim, page = case["op"], case["kv_heads"], case["dim"], case.get("page")
    s = {"case": case}
    if op == "tree":
        lens, n = _lengths(case, case["batch"]), case["nodes"]
        s["table"], total = _table(gen, _columns([x + n for x in lens], page))
        s["lens"], s["parents"] = _ints(lens), _ints(_parents(case))
        s["cache"] = _cache(case, gen, total)
        s["q"] = _normal(gen, case["batch"] * n, case["heads"], dim).bfloat16()
    elif op == "decode":
        lens = _lengths(case, case["batch"])
        held = _columns(lens, page)
        first = torch.arange(held.shape[1], device=DEVICE) * page
        seen = _ints(lens)[:, None] - case["q_len"] - case["window"] + 1     # the first row's window starts there
        held &= (first < case["sinks"]) | (first + page > seen)              # the other pages are given back
        s["table"], total = _table(gen, held)
        s["lens"] = _ints(lens)
        s["cache"] = _cache(case, gen, total)
        s["q"] = _normal(gen, case["batch"] * case["q_len"], case["heads"], dim).bfloat16()
    elif op == "prefill":
        lens = _lengths(case, case["batch"])
        keys = [n + case["context"] for n in lens]
        s["cu_q"] = _ints([sum(lens[:i]) for i in range(len(lens) + 1)])
        s["cu_k"] = _ints([sum(keys[:i]) for i in range(len(lens) + 1)])
        s["q"] = _normal(gen, sum(lens), case["heads"], dim).bfloat16()
        # keys and values lie side by side in one row, as a fused projection leaves them
        kv = _normal(gen, sum(keys), (1 if case["shared"] else 2) * kv_heads, dim).bfloat16()
        s["k"], s["v"] = kv[:, :kv_heads], kv[:, -kv_heads:]
    elif op == "compact":
        lens, n = _lengths(case, case["batch"]), case["nodes"]
        s["table"], total = _table(gen, _columns([x + n for x in lens], page))
        paths = _accepted(case)
        s["lens"] = _ints(lens)
        s["path"] = _ints([p + [-1] * (n - len(p)) for p in paths])
        s["counts"] = _ints([len(p) for p in paths])
        s["cache"] = _cache(case, gen, total)
    else:
        prompts, samples = case["prompts"], case["samples"]
        lens, grown = _lengths(case, prompts), _grown(case)
        batch = prompts * samples
        # the prompts stand in rows 0, samples, 2 samples ..; the rows between are free for their samples
        rows = [lens[b // samples] if b % samples == 0 else 0 for b in range(batch)]
        width = (max(lens) + case["grown"]) // page + 2
        table, total = _table(gen, _columns(rows, page, width))
        where = torch.randperm(case["pages"], generator=gen, device=DEVICE, dtype=torch.int32)[:total]
        s["table"] = torch.where(table >= 0, where[table.clamp(min=0).long()], -1)
        s["lens"] = _ints(rows)
        s["refs"] = torch.zeros(case["pages"] + 1, dtype=torch.int32, device=DEVICE)
        s["refs"].index_fill_(0, torch.where(s["table"] >= 0, s["table"], case["pages"]).flatten().long(), 1)
        s["refs"] = s["refs"][:-1].contiguous()
        s["parents"] = _ints([b // samples * samples for b in range(batch)])
        s["first"] = s["lens"].clone()
        s["cu"] = _ints([sum(grown[:i]) for i in range(batch + 1)])
        s["tokens"] = sum(grown)
        s["cache"] = _cache(case, gen, case["pages"])
    return s


# ------------------------------------------------------------------------------------------------------------
# The plain forms, in 32 bits
# ------------------------------------------------------------------------------------------------------------


def _values(case, cache, name, *at):
    """Rows cache[at] as 32-bit numbers."""
    x = cache[name][at]
    if case["fmt"] == "fp8":
        scale = torch.exp2(cache[name + "_scale"][at].float() - 127.0)
        x = (x.view(torch.float8_e4m3fn).float().unflatten(-1, (scale.shape[-1], -1)) * scale.unsqueeze(-1)).flatten(-2)
    return x.float()


def _softmax(scores, keep):
    """Weights, and the log of their sum before division, of scores whose kept places `keep` marks; a row that
    keeps nothing has weights of zero and minus infinity."""
    scores = torch.where(keep, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(torch.isfinite(top), top, 0.0))
    total = e.sum(-1, keepdim=True)
    lse = torch.log(total) + top
    return e / torch.where(total > 0, total, 1.0), lse.squeeze(-1)


def _attended(case, q, k, v, keep, n):
    """q [batch * n, heads, dim] over k, v [batch, kv_heads, keys, dim], masked by keep [batch, n, keys]."""
    heads, kv_heads, dim, batch = case["heads"], case["kv_heads"], case["dim"], case["batch"]
    group = heads // kv_heads
    q = q.float().view(batch, n, kv_heads, group, dim).permute(0, 2, 1, 3, 4).flatten(2, 3)
    scores = torch.matmul(q, k.transpose(-1, -2)) * dim ** -0.5
    keep = keep[:, None, :, None].expand(batch, 1, n, group, -1).flatten(2, 3)
    p, lse = _softmax(scores, keep)
    o = torch.matmul(p, v).unflatten(2, (n, group)).permute(0, 2, 1, 3, 4).reshape(batch * n, heads, dim)
    return o.bfloat16(), lse.unflatten(2, (n, group)).permute(0, 2, 1, 3).reshape(batch * n, heads)


def _plain_tree(s):
    case, cache, n, parents = s["case"], s["cache"], s["case"]["nodes"], s["parents"]
    node = torch.arange(n, device=DEVICE)
    # (1 + A)^64 > 0, with A the step from a node to its parent: the node and what is above it
    step = (parents[..., None] == node).float() + torch.eye(n, device=DEVICE)
    above = (torch.linalg.matrix_power(step, 64) > 0) & (parents >= -1)[..., None]
    masks = (above.long() << node).sum(-1)
    depths = above.sum(-1, dtype=torch.int32) - 1
    table = s["table"].clamp(min=0).long()
    k = _values(case, cache, "k", table).transpose(1, 2).flatten(2, 3)
    v = k if case["shared"] else _values(case, cache, "v", table).transpose(1, 2).flatten(2, 3)
    pos, lens = torch.arange(k.shape[2], device=DEVICE), s["lens"].long()[:, None, None]
    keep = pos < lens
    if case["window"]:
        keep = keep & ((pos > lens + depths[..., None] - case["window"]) | (pos < case["sinks"]))
    at = (pos - lens).expand(-1, n, -1)
    tree = above.gather(2, at.clamp(0, n - 1)) & (at >= 0) & (at < n)
    keep = (keep & (parents >= -1)[..., None]) | tree
    out, lse = _attended(case, s["q"], k, v, keep, n)
    return {"masks": masks, "depths": depths, "out": out, "lse": lse}


def _plain_decode(s):
    case, cache, n = s["case"], s["cache"], s["case"]["q_len"]
    lens, window, sinks, page = s["lens"].long()[:, None], case["window"], case["sinks"], case["page"]
    # the positions that the first tokens and the rows' windows span, and no others, are gathered
    near = lens - (window + n - 1) + torch.arange(window + n - 1, device=DEVICE)
    near = torch.where(near >= sinks, near, -1)
    far = torch.arange(sinks, device=DEVICE).expand(len(lens), -1)
    pos = torch.cat([torch.where(far < lens, far, -1), near], 1)
    col = (pos.clamp(min=0) // page).clamp(max=s["table"].shape[1] - 1)
    at, row = s["table"].gather(1, col).clamp(min=0).long(), pos.clamp(min=0) % page
    head = torch.arange(case["kv_heads"], device=DEVICE)[:, None]
    k = _values(case, cache, "k", at[:, None], head, row[:, None])
    v = k if case["shared"] else _values(case, cache, "v", at[:, None], head, row[:, None])
    mine = (lens - n + torch.arange(n, device=DEVICE))[..., None]           # the rows' positions
    pos = pos[:, None]
    keep = (pos >= 0) & (pos <= mine) & ((pos > mine - window) | (pos < sinks))
    out, lse = _attended(case, s["q"], k, v, keep, n)
    return {"out": out, "lse": lse}


def _plain_prefill(s):
    case = s["case"]
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    group, tokens = heads // kv_heads, s["q"].shape[0]
    longest = case["longest"]
    q_len, k_len = s["cu_q"].diff(), s["cu_k"].diff()
    row, col = torch.arange(longest, device=DEVICE), torch.arange(longest + case["context"], device=DEVICE)
    # packed rows spread over [batch, longest]; places past a sequence's end take some row of it
    at_q = (s["cu_q"][:-1, None] + torch.minimum(row, q_len[:, None] - 1)).long()
    at_k = (s["cu_k"][:-1, None] + torch.minimum(col, k_len[:, None] - 1)).long()
    k = s["k"][at_k].float().permute(0, 2, 1, 3)
    v = s["v"][at_k].float().permute(0, 2, 1, 3)
    end = ((k_len - q_len)[:, None] + row + 1)[..., None]
    keep = (col < k_len[:, None, None]) & ((col >= end - case["window"]) | (col < case["sinks"]))
    if case["causal"]:
        keep = keep & (col < end)
    keep = keep[:, None, None].expand(-1, 1, 1, longest, -1)
    batch = case["batch"]
    q = s["q"][at_q].float().unflatten(2, (kv_heads, group)).permute(0, 2, 3, 1, 4)
    scores = torch.matmul(q.reshape(batch, kv_heads, group * longest, dim), k.transpose(-1, -2))
    p, lse = _softmax(scores.unflatten(2, (group, longest)) * dim ** -0.5, keep)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (group, longest))
    o = o.permute(0, 3, 1, 2, 4).reshape(batch * longest, heads, dim)
    lse = lse.permute(0, 3, 1, 2).reshape(batch * longest, heads)
    # back to the packed rows
    t = torch.arange(tokens, device=DEVICE)
    seq = torch.searchsorted(s["cu_q"][1:].long(), t, right=True)
    back = seq * longest + t - s["cu_q"][seq]
    return {"out": o[back].bfloat16(), "lse": lse[back]}


def _plain_compact(s):
    case, cache, table, page = s["case"], s["cache"], s["table"].long(), s["case"]["page"]
    i = torch.arange(case["nodes"], device=DEVICE)
    to = s["lens"].long()[:, None] + i
    # a place past the accepted ones keeps what it has
    source = torch.where(i < s["counts"][:, None], s["lens"].long()[:, None] + s["path"], to)
    p, r = table.gather(1, source // page), source % page
    p2, r2 = table.gather(1, to // page), to % page
    rows = {name: x[p, :, r] for name, x in cache.items() if x is not None}
    cache["k"][p2, :, r2] = rows["k"]
    if not case["shared"]:
        cache["v"][p2, :, r2] = rows["v"]
    if case["fmt"] == "fp8":
        cache["k_scale"][p2, :, r2] = rows["k_scale"]
        if not case["shared"]:
            cache["v_scale"][p2, :, r2] = rows["v_scale"]


def _plain_pool(s):
    case, cache, page, refs = s["case"], s["cache"], s["case"]["page"], s["refs"]
    pages, batch = case["pages"], len(s["lens"])
    width = s["table"].shape[1]
    seq, col = torch.arange(batch, device=DEVICE), torch.arange(width, device=DEVICE)

    def count(entries, by):
        """refs of the pages among `entries` changed by `by` for each."""
        return refs.add_(by * torch.zeros(pages + 1, dtype=torch.int32, device=DEVICE).scatter_add_(
            0, torch.where(entries >= 0, entries, pages).flatten().long(),
            torch.ones(entries.numel(), dtype=torch.int32, device=DEVICE))[:-1])

    # fork: every row becomes its parent's
    up = s["parents"].long()
    table, old = torch.where(up[:, None] >= 0, s["table"][up.clamp(min=0)], -1), s["table"]
    lens = torch.where(up >= 0, s["lens"][up.clamp(min=0)], 0)
    count(table, 1)
    count(old, -1)
    # grow: new tokens, fresh pages for those that start one, and for partly filled pages that others hold
    n = s["cu"].diff()
    longer = torch.minimum(lens + n, torch.full_like(lens, width * page))
    c0, c1 = (lens + page - 1) // page, (longer + page - 1) // page
    part = table.gather(1, (lens // page).clamp(max=width - 1).long()[:, None])[:, 0]
    part = torch.where((n > 0) & (lens % page > 0), part, -1)
    others = torch.where(part >= 0, refs[part.clamp(min=0).long()], 0) > 1
    where = torch.where(others, part, pages).long()
    growers = torch.zeros(pages + 1, dtype=torch.int32, device=DEVICE).scatter_add_(0, where, torch.ones_like(lens))
    lowest = torch.full((pages + 1,), batch, device=DEVICE).scatter_reduce_(0, where, seq, "amin")
    stays = (growers[where] == refs[part.clamp(min=0).long()]) & (lowest[where] == seq)
    fork = others & ~stays
    need = fork.int() + (c1 - c0)
    base = (need.cumsum(0) - need).long()
    free = refs == 0
    at = torch.where(free, free.cumsum(0) - 1, pages)
    fresh = torch.full((pages + batch * width + 1,), -1, dtype=torch.int32, device=DEVICE)
    fresh.scatter_(0, at, torch.arange(pages, dtype=torch.int32, device=DEVICE))
    fresh[pages] = -1
    short = (need.sum() - free.sum()).clamp(min=0).int()
    dst = torch.where(fork, fresh[base], -1)
    src = torch.where(dst >= 0, part, -1)
    new = (col >= c0[:, None]) & (col < c1[:, None])
    here = (dst >= 0)[:, None] & (col == (lens // page)[:, None])
    grown = torch.where(new, fresh[(base + fork)[:, None] + (col - c0[:, None]).clamp(min=0)], table)
    grown = torch.where(here, dst[:, None], grown)
    count(torch.where(new | here, grown, -1), 1)
    count(src, -1)
    t = torch.arange(s["tokens"], device=DEVICE)
    b = torch.searchsorted(s["cu"][1:].contiguous(), t.int(), right=True)
    pos = lens[b] + (t - s["cu"][b]).int()
    on = grown[b, (pos // page).clamp(max=width - 1).long()].long()
    lost = (fork & (dst < 0))[b] & (pos // page == lens[b] // page)       # its shared page could not be copied
    slots = torch.where((on >= 0) & (pos < width * page) & ~lost, on * page + pos % page, -1)
    # the copies
    pair = src >= 0
    a, z = src[pair].long(), dst[pair].long()
    for_all = [x for name, x in cache.items() if x is not None and not (case["shared"] and name[0] == "v")]
    [x.index_copy_(0, z, x[a]) for x in for_all]
    # the samples end: back to the lengths from before
    lens = torch.minimum(longer, s["first"])
    keep = col * page < lens[:, None]
    count(torch.where(keep, -1, grown), -1)
    s["table"].copy_(torch.where(keep, grown, -1))
    s["lens"].copy_(lens)
    return {"slots": slots, "positions": pos, "src": src, "dst": dst, "missing": short}


# ------------------------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------------------------


def _handle(s, moe):
    """The package's handle on the state's cache, which a program makes once."""
    if "handle" not in s:
        c = s["cache"]
        s["handle"] = moe.KVCache(c["k"], None if s["case"]["shared"] else c["v"], c["k_scale"],
                                  None if s["case"]["shared"] else c["v_scale"])
    return s["handle"]


def _held(case, cache):
    """The cache's contents, codes as the values they stand for."""
    out = {}
    for name in ("k",) if case["shared"] else ("k", "v"):
        if case["fmt"] == "fp8":
            out[name] = cache[name].view(torch.float8_e4m3fn)
            out[name + "_scale"] = cache[name + "_scale"].view(torch.float8_e8m0fnu)
        else:
            out[name] = cache[name]
    return out


def run(s):
    case, op = s["case"], s["case"]["op"]
    if not own:
        if op == "tree":
            return _plain_tree(s)
        if op == "decode":
            return _plain_decode(s)
        if op == "prefill":
            return _plain_prefill(s)
        if op == "compact":
            _plain_compact(s)
            return _held(case, s["cache"])
        out = _plain_pool(s)
        return {**out, "table": s["table"], "lens": s["lens"], "refs": s["refs"], **_held(case, s["cache"])}
    import block_scaled_fp4_sqrtsoftplus_amd as moe
    if op == "tree":
        if "attend" not in s:
            s["attend"] = moe.TreeAttention(_handle(s, moe), case["batch"], case["heads"], case["nodes"],
                                            window=case["window"], sinks=case["sinks"])
        masks, depths = moe.tree_masks(s["parents"])
        out, lse = s["attend"](s["q"], s["table"], s["lens"], masks, want_lse=True)
        return {"masks": masks, "depths": depths, "out": out, "lse": lse}
    if op == "decode":
        if "attend" not in s:
            s["attend"] = moe.DecodeAttention(_handle(s, moe), case["batch"], case["heads"], case["q_len"],
                                              window=case["window"], sinks=case["sinks"])
        out, lse = s["attend"](s["q"], s["table"], s["lens"], want_lse=True)
        return {"out": out, "lse": lse}
    if op == "prefill":
        out, lse = moe.attn_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=case["causal"],
                                    window=case["window"], sinks=case["sinks"], want_lse=True)
        return {"out": out, "lse": lse}
    if op == "compact":
        moe.kv_compact(_handle(s, moe), s["table"], s["lens"], s["path"], s["counts"])
        return _held(case, s["cache"])
    if "pool" not in s:
        s["pool"] = moe.PagePool(s["refs"], s["table"], s["lens"], case["page"])
    pool = s["pool"]
    pool.fork(s["parents"])
    slots, positions, src, dst = pool.grow(s["cu"], s["tokens"])
    moe.kv_copy_pages(_handle(s, moe), src, dst)
    pool.trim(s["first"])
    return {"slots": slots, "positions": positions, "src": src, "dst": dst, "missing": pool.missing[0],
            "table": s["table"], "lens": s["lens"], "refs": s["refs"], **_held(case, s["cache"])}


# ------------------------------------------------------------------------------------------------------------
# The definitions, in 64 bits
# ------------------------------------------------------------------------------------------------------------


def _attend64(q, k, v, keep):
    """softmax(q k^T / sqrt(dim)) v of one sequence and one key-value head over the keys that keep(a, b), for the
    rows a .. b, marks: q [rows, group, dim]; k, v [keys, dim]."""
    rows, group, dim = q.shape
    out, lse = torch.zeros_like(q), torch.full((rows, group), -math.inf, dtype=q.dtype, device=q.device)
    step = max(1, (1 << 27) // max(1, group * len(k)))
    for a in range(0, rows, step):
        b = min(rows, a + step)
        if not len(k):
            break
        x = torch.matmul(q[a:b].reshape(-1, dim), k.t()).view(b - a, group, -1) / math.sqrt(dim)
        x = x.masked_fill(~keep(a, b)[:, None], -math.inf)
        lse[a:b] = torch.logsumexp(x, -1)
        out[a:b] = torch.matmul(torch.nan_to_num(torch.exp(x - lse[a:b, :, None]), nan=0.0), v)
    return out, lse


def _moved64(case, cache, moves):
    """The cache's contents after rows [page, row] went to others, by `moves` of (from page, row, to page, row)."""
    out = {}
    at = torch.tensor(moves, dtype=torch.long).view(-1, 4).t().to(DEVICE)
    for name in ("k",) if case["shared"] else ("k", "v"):
        for part, kind in (("", torch.float8_e4m3fn), ("_scale", torch.float8_e8m0fnu))[:1 + (case["fmt"] == "fp8")]:
            x = cache[name + part]
            x = x.view(kind).float().double() if case["fmt"] == "fp8" else x.double()
            x[at[2], :, at[3]] = x[at[0], :, at[1]]
            out[name + part] = x
    return out


def _pool64(case, s):
    """Which pages the copies of a pool's pass go from and to, sequence by sequence, page by page."""
    page, samples = case["page"], case["samples"]
    table, lens, cu = s["table"].tolist(), s["lens"].tolist(), s["cu"].tolist()
    holders = {}
    for b in range(len(lens)):                           # every sample stands on its prompt's pages
        for p in table[b // samples * samples]:
            if p >= 0:
                holders.setdefault(p, []).append(b)
    free = iter(p for p in range(case["pages"]) if p not in holders)
    pairs = []
    for b in range(len(lens)):
        n, more = lens[b // samples * samples], cu[b + 1] - cu[b]
        p = table[b // samples * samples][n // page] if n % page else -1
        growers = [x for x in holders.get(p, []) if cu[x + 1] > cu[x]]
        if more and len(holders.get(p, [])) > 1 and not (growers == holders[p] and b == growers[0]):
            to = next(free, -1)
            if to >= 0:
                pairs.append((p, to))
        for _ in range(-(-n // page), -(-(n + more) // page)):
            next(free, -1)
    return pairs


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "compact":
        moves, table = [], s["table"].tolist()
        for at, start, path in zip(table, s["lens"].tolist(), _accepted(case)):
            for i, node in enumerate(path):
                moves.append([x for y in (start + node, start + i) for x in (at[y // case["page"]], y % case["page"])])
        return _moved64(case, s["cache"], moves)
    if op == "pool":
        moves = [(a, r, z, r) for a, z in _pool64(case, s) for r in range(case["page"])]
        return {**dict.fromkeys(("slots", "positions", "src", "dst", "missing", "table", "lens", "refs")),
                **_moved64(case, s["cache"], moves)}
    kv_heads, group = case["kv_heads"], case["heads"] // case["kv_heads"]
    q = s["q"].double()
    out = torch.zeros_like(q)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    window, sinks = case["window"], case["sinks"]

    def rows_of(name, b, pos):
        """The cache's rows at a sequence's positions, [kv_heads, positions, dim]."""
        page = s["table"][b].long()[pos // case["page"]]
        x = s["cache"][name][page, :, pos % case["page"]]
        if case["fmt"] == "fp8":
            e = s["cache"][name + "_scale"][page, :, pos % case["page"]].double() - 127.0
            x = (x.view(torch.float8_e4m3fn).double().unflatten(-1, (e.shape[-1], -1)) * torch.exp2(e)[..., None]).flatten(-2)
        return x.double().transpose(0, 1)

    for b in range(case["batch"]):
        if op == "tree":
            n, length = case["nodes"], int(s["lens"][b])
            lo, hi = b * n, (b + 1) * n
            paths = _paths(s["parents"][b].tolist())
            kept = torch.zeros(n, length + n, dtype=torch.bool)
            for i, path in enumerate(paths):
                if path:
                    first = length + len(path) - window if window else 0     # position - window + 1
                    kept[i, max(0, first):length] = True
                    kept[i, :min(sinks, length)] = True
                    kept[i, [length + j for j in path]] = True
            kept = kept.to(q.device)
            pos = torch.arange(length + n, device=q.device)
            keep = lambda a, z, kept=kept: kept[a:z]  # noqa: E731
            k, v = rows_of("k", b, pos), rows_of("k" if case["shared"] else "v", b, pos)
        else:
            if op == "decode":
                n, length = case["q_len"], int(s["lens"][b])
                lo, hi = b * n, (b + 1) * n
                seen = max(0, length - n + 1 - window)       # keys between the first tokens and it are in no window
                pos = torch.cat([torch.arange(min(sinks, seen)), torch.arange(seen, length)]).to(q.device)
                k, v = rows_of("k", b, pos), rows_of("k" if case["shared"] else "v", b, pos)
            else:
                lo, hi = int(s["cu_q"][b]), int(s["cu_q"][b + 1])
                a, z = int(s["cu_k"][b]), int(s["cu_k"][b + 1])
                length = z - a
                pos = torch.arange(length, device=q.device)
                k, v = s["k"][a:z].double().transpose(0, 1), s["v"][a:z].double().transpose(0, 1)
            causal = case.get("causal", True)

            def keep(a, z, start=length - (hi - lo), pos=pos, causal=causal):
                mine = start + torch.arange(a, z, device=q.device)[:, None]
                near = (pos > mine - window) | (pos < sinks)
                return near & (pos <= mine) if causal else near
        for h in range(kv_heads):
            part = slice(h * group, (h + 1) * group)
            out[lo:hi, part], lse[lo:hi, part] = _attend64(q[lo:hi, part], k[h], v[h], keep)
    if op == "tree":
        return {"masks": None, "depths": None, "out": out, "lse": lse}
    return {"out": out, "lse": lse}
