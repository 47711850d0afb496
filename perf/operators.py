"""Measured cases of the attention operators: the paged key-value cache's append with the position rotation
(kv_append), attention of new tokens over the paged cache (attn_decode) and attention over packed prompts
(attn_prefill).

With `own` false, run() computes them in plain torch operations in 32 bits; with `own` true it calls the package.
listed() and draw() give the cases, prepare() their inputs, work() what one pass has to move and compute, and
exact() the results from the definitions in 64 bits.

Head layouts (query heads / key-value heads x head size): 32/8 x 128 is the usual grouped layout, 64/1 x 512 the
decoder around this layer (64 heads on one shared 512-element key-value head, its last 64 elements rotated,
hidden 4096), the others are generic."""

import math
import random

import torch

own = False

DEVICE = "cuda"


# ------------------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------------------


def _append(name, tokens, heads, kv_heads, dim, fmt="bf16", page=16, rot=None, interleaved=False, shared=False,
            sequences=1, mix=0):
    c = dict(op="append", tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, fmt=fmt, page=page,
             rot=dim if rot is None else rot, interleaved=interleaved, shared=shared, sequences=sequences, mix=mix)
    return dict(c, name=name) if name else c


def _decode(name, batch, longest, shortest, heads, kv_heads, dim, fmt="bf16", page=16, q_len=1, window=0,
            shared=False, mix=0):
    c = dict(op="decode", batch=batch, longest=longest, shortest=shortest, heads=heads, kv_heads=kv_heads, dim=dim,
             fmt=fmt, page=page, q_len=q_len, window=window, shared=shared, mix=mix)
    return dict(c, name=name) if name else c


def _prefill(name, batch, longest, shortest, heads, kv_heads, dim, context=0, window=0, causal=True, shared=False,
             mix=0):
    c = dict(op="prefill", batch=batch, longest=longest, shortest=shortest, heads=heads, kv_heads=kv_heads, dim=dim,
             context=context, window=window, causal=causal, shared=shared, mix=mix)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one sequence's new token, the least a decode step appends: latency
        _append("append 1 token", 1, 32, 8, 128),
        # the decode step of 64 sequences on the shared 512-element head, into an FP8 cache
        _append("append 64 fp8 mqa512", 64, 64, 1, 512, "fp8", 64, rot=64, interleaved=True, shared=True,
                sequences=64),
        # packed prompts of an odd total length
        _append("append 4099 packed", 4099, 32, 8, 128, "bf16", 16, sequences=5, mix=1),
        # long prompts into an FP8 cache: bandwidth
        _append("append 16384 fp8", 16384, 32, 8, 128, "fp8", 32, sequences=2, mix=2),
        # a short conversation, one sequence: latency
        _decode("decode 1x300", 1, 300, 300, 32, 8, 128),
        # a decode step of 64 sequences of different lengths up to 4096
        _decode("decode 64x4096 ragged", 64, 4096, 700, 32, 8, 128, mix=3),
        # one long document in an FP8 cache: the split over the length
        _decode("decode 1x131071 fp8", 1, 131071, 131071, 32, 8, 128, "fp8", 64),
        # the shared 512-element head under 64 query heads, at the context of 4096
        _decode("decode 32x4096 mqa512", 32, 4096, 2048, 64, 1, 512, "bf16", 64, shared=True, mix=4),
        # small heads, one short prompt: latency
        _prefill("prefill 1x200 d64", 1, 200, 200, 16, 2, 64),
        # packed prompts of different lengths, 4096-token class
        _prefill("prefill 6 packed", 6, 1500, 100, 32, 8, 128, mix=5),
        # one long prompt: the matrix rate
        _prefill("prefill 1x8192", 1, 8192, 8192, 32, 8, 128),
        # the shared 512-element head under 64 query heads
        _prefill("prefill 2048 mqa512", 1, 2048, 2048, 64, 1, 512, shared=True),
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
    op = rng.choice(["append", "decode", "prefill"])
    if op == "append":
        most = max(1, 16384 * 48 * 128 // ((heads + 2 * kv_heads) * dim))
        tokens = _spread(rng, 1, min(16384, most))
        rot = rng.choice([dim, dim // 2 if dim < 512 else 64])
        return _append(None, tokens, heads, kv_heads, dim, fmt, page, rot, rng.random() < 0.5, shared,
                       _spread(rng, 1, min(64, tokens)), mix)
    if op == "decode":
        batch = _spread(rng, 1, 128)
        q_len = rng.choice([1, 1, 1, 2, 4])
        most = min(1.5e8 / (kv_heads * dim), 3e9 / (heads * dim * q_len)) / batch
        longest = _spread(rng, 1, min(131072, max(1, int(most))))
        return _decode(None, batch, longest, rng.randint(0, longest), heads, kv_heads, dim, fmt, page,
                       q_len, rng.choice([0, 0, 0, 128, 1000]), shared, mix)
    batch = _spread(rng, 1, 16)
    most = min(math.sqrt(8192 * 8192 * 32 * 128 / (batch * heads * dim * 2)), 6e7 / (batch * heads * dim))
    longest = _spread(rng, 1, min(8192, int(most)))
    return _prefill(None, batch, longest, rng.randint(1, longest), heads, kv_heads, dim,
                    rng.choice([0, 0, 0, rng.randint(1, longest)]), rng.choice([0, 0, 0, 128, 1000]),
                    rng.random() < 0.8, shared, mix)


def _lengths(case, count):
    """`count` lengths between shortest and longest, the longest among them; the case alone decides."""
    rng = random.Random(case["mix"])
    lens = [rng.randint(case["shortest"], case["longest"]) for _ in range(count)]
    lens[rng.randrange(count)] = case["longest"]
    return lens


def _parts(case):
    """An append's tokens dealt to its sequences, at least one each."""
    rng = random.Random(case["mix"])
    cuts = sorted(rng.sample(range(1, case["tokens"]), case["sequences"] - 1)) if case["sequences"] > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [case["tokens"]])]


def _kept(case, q_len, kv_len):
    """How many (query, key) pairs the mask keeps, for one head."""
    total = 0
    for i in range(q_len):
        high = min(kv_len, max(0, kv_len - q_len + i + 1)) if case.get("causal", True) else kv_len
        low = max(0, kv_len - q_len + i + 1 - case["window"]) if case["window"] else 0
        total += max(0, high - low)
    return total


def work(case):
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    kinds = 1 if case["shared"] else 2
    if case["op"] == "append":
        groups = max(1, dim // 128)
        tokens = case["tokens"]
        row = dim * 2 if case["fmt"] == "bf16" else dim + groups
        read = tokens * (heads + kinds * kv_heads) * dim * 2 + tokens * (8 + 4 + case["rot"] * 4)
        write = tokens * heads * dim * 2 + tokens * kinds * kv_heads * row
        return {"bytes": read + write, "flops": tokens * (heads + kv_heads) * case["rot"] * 3}
    if case["op"] == "decode":
        lens = _lengths(case, case["batch"])
        q_len = case["q_len"]
        row = dim * 2 if case["fmt"] == "bf16" else dim + max(1, dim // 128)
        seen = [min(n, case["window"] + q_len - 1) if case["window"] else n for n in lens]
        rows = case["batch"] * q_len * heads
        pairs = sum(_kept(case, q_len, n) for n in lens) * heads
        return {"bytes": sum(seen) * kv_heads * row * kinds + rows * (dim * 4 + 4)
                + sum(-(-n // case["page"]) for n in seen) * 4, "flops": pairs * 4 * dim}
    lens = _lengths(case, case["batch"])
    tokens, keys = sum(lens), sum(n + case["context"] for n in lens)
    pairs = sum(_kept(case, n, n + case["context"]) for n in lens) * heads
    return {"bytes": tokens * heads * (dim * 4 + 4) + keys * kv_heads * dim * 2 * kinds, "flops": pairs * 4 * dim}


# ------------------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------------------


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32)


def _quantized(x):
    """FP8 codes and power-of-two scale bytes (biased by 127) of rows, one scale for 128 elements (or the row,
    where it is shorter): the smallest scale with which nothing passes 448."""
    size = min(128, x.shape[-1])
    g = x.float().unflatten(-1, (-1, size))
    m, e = torch.frexp(g.abs().amax(-1))  # amax = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-127, 127)
    e = torch.where(m > 0, e, torch.full_like(e, -127))
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


def _table(gen, counts):
    """Block table [sequences, widest]: pages in random order, -1 past a sequence's last one; and the page count."""
    total, width = sum(counts), max(counts)
    order = torch.randperm(total, generator=gen, device=DEVICE, dtype=torch.int32)
    ends = torch.tensor([sum(counts[:i]) for i in range(len(counts))], device=DEVICE)
    col = torch.arange(width, device=DEVICE)
    at = (ends[:, None] + col).clamp(max=total - 1)
    return torch.where(col < torch.tensor(counts, device=DEVICE)[:, None], order[at], -1).contiguous(), total


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    s = {"case": case}
    # q, k and v lie side by side in one row, as a fused projection leaves them
    def projected(tokens):
        kinds = 1 if case["shared"] else 2
        qkv = _normal(gen, tokens, heads + kinds * kv_heads, dim).bfloat16()
        k = qkv[:, heads:heads + kv_heads]
        return qkv[:, :heads], k, k if case["shared"] else qkv[:, heads + kv_heads:]

    if case["op"] == "append":
        # a prompt's tokens from its start, or one new token each somewhere in its sequence
        parts = _parts(case)
        rng = random.Random(case["mix"] + 1)
        first = [rng.randrange(4096) if n == 1 else 0 for n in parts]
        counts = [-(-(f % case["page"] + n) // case["page"]) for f, n in zip(first, parts)]
        table, total = _table(gen, counts)
        pos = torch.cat([torch.arange(f, f + n, dtype=torch.int32) for f, n in zip(first, parts)]).to(DEVICE)
        seq = torch.repeat_interleave(torch.arange(len(parts)), torch.tensor(parts)).to(DEVICE)
        start = torch.tensor([f - f % case["page"] for f in first], device=DEVICE)[seq]
        local = pos - start
        s["slots"] = table[seq, local // case["page"]].long() * case["page"] + local % case["page"]
        s["positions"] = pos
        s["cache"] = _cache(case, gen, total)
        s["q"], s["k"], s["v"] = projected(case["tokens"])
        half = case["rot"] // 2
        angle = torch.arange(int(pos.max()) + 1, dtype=torch.float64)[:, None] \
            * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], -1).float().to(DEVICE)
    elif case["op"] == "decode":
        lens = _lengths(case, case["batch"])
        s["table"], total = _table(gen, [-(-n // case["page"]) for n in lens])
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEVICE)
        s["cache"] = _cache(case, gen, total)
        s["q"] = _normal(gen, case["batch"] * case["q_len"], heads, dim).bfloat16()
    else:
        lens = _lengths(case, case["batch"])
        cu = lambda v: torch.tensor([0] + [sum(v[:i + 1]) for i in range(len(v))], dtype=torch.int32,  # noqa: E731
                                    device=DEVICE)
        s["cu_q"] = cu(lens)
        s["cu_k"] = cu([n + case["context"] for n in lens])
        if case["context"]:
            keys = sum(lens) + case["context"] * len(lens)
            s["q"] = projected(sum(lens))[0]
            _, s["k"], s["v"] = projected(keys)
        else:
            s["q"], s["k"], s["v"] = projected(sum(lens))
    return s


# ------------------------------------------------------------------------------------------------------------
# The plain forms, in 32 bits
# ------------------------------------------------------------------------------------------------------------


def _rotated(x, cos, sin, offset, rot, interleaved):
    """x [tokens, heads, dim] with its elements offset .. offset + rot rotated in pairs, rounded to bf16."""
    x = x.float()
    part = x[..., offset:offset + rot]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
    c, n = cos[:, None], sin[:, None]
    u, w = a * c - b * n, b * c + a * n
    part = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([x[..., :offset], part, x[..., offset + rot:]], -1).bfloat16()


def _plain_append(s):
    case, cache = s["case"], s["cache"]
    rot, offset = case["rot"], case["dim"] - case["rot"]
    cs = s["cos_sin"][s["positions"].long()]
    cos, sin = cs[:, :rot // 2], cs[:, rot // 2:]
    q = _rotated(s["q"], cos, sin, offset, rot, case["interleaved"])
    k = _rotated(s["k"], cos, sin, offset, rot, case["interleaved"])
    page, row = s["slots"] // case["page"], s["slots"] % case["page"]

    def put(name, x):
        if case["fmt"] == "fp8":
            x, scale = _quantized(x)
            cache[name + "_scale"][page, :, row] = scale
        cache[name][page, :, row] = x

    put("k", k)
    if not case["shared"]:
        put("v", s["v"])
    return q


def _softmax(scores, keep):
    """Weights, and the log of their sum before division, of scores whose kept places `keep` marks; a row that
    keeps nothing has weights of zero and minus infinity."""
    scores = torch.where(keep, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(torch.isfinite(top), top, 0.0))
    total = e.sum(-1, keepdim=True)
    lse = torch.log(total) + top
    return e / torch.where(total > 0, total, 1.0), lse.squeeze(-1)


def _plain_decode(s):
    case, cache = s["case"], s["cache"]
    heads, kv_heads, dim, n = case["heads"], case["kv_heads"], case["dim"], case["q_len"]
    batch, group = case["batch"], heads // kv_heads
    table = s["table"].clamp(min=0).long()

    def gathered(name):
        x = cache[name][table]  # [batch, width, kv_heads, page, dim]
        if case["fmt"] == "fp8":
            scale = torch.exp2(cache[name + "_scale"][table].float() - 127.0)
            x = (x.view(torch.float8_e4m3fn).float().unflatten(-1, (scale.shape[-1], -1)) * scale.unsqueeze(-1)).flatten(-2)
        return x.float().transpose(1, 2).flatten(2, 3)  # [batch, kv_heads, keys, dim]

    k = gathered("k")
    v = k if case["shared"] else gathered("v")
    q = s["q"].float().view(batch, n, kv_heads, group, dim).permute(0, 2, 1, 3, 4).flatten(2, 3)
    scores = torch.matmul(q, k.transpose(-1, -2)) * dim ** -0.5
    pos = torch.arange(k.shape[2], device=DEVICE)
    end = s["seq_lens"][:, None] - n + 1 + torch.arange(n, device=DEVICE)  # keys before it are seen
    keep = pos < end[..., None]
    if case["window"]:
        keep &= pos >= end[..., None] - case["window"]
    keep = keep[:, None, :, None].expand(batch, 1, n, group, -1).flatten(2, 3)
    p, lse = _softmax(scores, keep)
    o = torch.matmul(p, v).unflatten(2, (n, group)).permute(0, 2, 1, 3, 4).reshape(batch * n, heads, dim)
    return o.bfloat16(), lse.unflatten(2, (n, group)).permute(0, 2, 1, 3).reshape(batch * n, heads)


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
    q = s["q"][at_q].float().unflatten(2, (kv_heads, group)).permute(0, 2, 3, 1, 4)
    k = s["k"][at_k].float().permute(0, 2, 1, 3).unsqueeze(2)
    v = s["v"][at_k].float().permute(0, 2, 1, 3).unsqueeze(2)
    end = (k_len - q_len)[:, None] + row + 1
    keep = col < k_len[:, None, None]
    if case["causal"]:
        keep = keep & (col < end[..., None])
    if case["window"]:
        keep = keep & (col >= end[..., None] - case["window"])
    keep = keep[:, None, None].expand(-1, 1, 1, longest, -1)
    batch = case["batch"]
    scores = torch.matmul(q.reshape(batch, kv_heads, group * longest, dim), k.squeeze(2).transpose(-1, -2))
    p, lse = _softmax(scores.unflatten(2, (group, longest)) * dim ** -0.5, keep)
    o = torch.matmul(p.flatten(2, 3), v.squeeze(2)).unflatten(2, (group, longest))
    o = o.permute(0, 3, 1, 2, 4).reshape(batch * longest, heads, dim)
    lse = lse.permute(0, 3, 1, 2).reshape(batch * longest, heads)
    # back to the packed rows
    t = torch.arange(tokens, device=DEVICE)
    seq = torch.searchsorted(s["cu_q"][1:].long(), t, right=True)
    back = seq * longest + t - s["cu_q"][seq]
    return o[back].bfloat16(), lse[back]


# ------------------------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------------------------


def _handle(s, moe):
    """The package's handle on the state's cache, which a program makes once."""
    if "handle" not in s:
        c = s["cache"]
        s["handle"] = moe.KVCache(c["k"], c["v"], c["k_scale"], c["v_scale"])
    return s["handle"]


def run(s):
    case, cache = s["case"], s.get("cache")
    if own:
        import block_scaled_fp4_sqrtsoftplus_amd as moe
    if case["op"] == "append":
        if own:
            if "rope" not in s:
                s["rope"] = moe.Rope(s["cos_sin"], case["dim"] - case["rot"], case["interleaved"])
            q = moe.kv_append(_handle(s, moe), s["k"], None if case["shared"] else s["v"], s["slots"],
                              s["positions"], s["rope"], s["q"])
        else:
            q = _plain_append(s)
        out = {"q": q}
        for name in ("k",) if case["shared"] else ("k", "v"):
            if case["fmt"] == "fp8":
                out[name] = cache[name].view(torch.float8_e4m3fn)
                out[name + "_scale"] = cache[name + "_scale"].view(torch.float8_e8m0fnu)
            else:
                out[name] = cache[name]
        return out
    if case["op"] == "decode":
        if own:
            if "attend" not in s:
                s["attend"] = moe.DecodeAttention(_handle(s, moe), case["batch"], case["heads"], case["q_len"],
                                                  window=case["window"])
            out, lse = s["attend"](s["q"], s["table"], s["seq_lens"], want_lse=True)
        else:
            out, lse = _plain_decode(s)
        return {"out": out, "lse": lse}
    if own:
        out, lse = moe.attn_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=case["causal"],
                                    window=case["window"], want_lse=True)
    else:
        out, lse = _plain_prefill(s)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------------------------------------------------
# The definitions, in 64 bits
# ------------------------------------------------------------------------------------------------------------


def _attend64(q, k, v, first, causal, window):
    """softmax(q k^T / sqrt(dim)) v of one sequence and one key-value head: q [rows, group, dim], whose row i
    stands at position first + i; k, v [keys, dim]."""
    rows, group, dim = q.shape
    out, lse = torch.zeros_like(q), torch.full((rows, group), -math.inf, dtype=q.dtype, device=q.device)
    step = max(1, (1 << 27) // max(1, group * len(k)))
    for a in range(0, rows, step):
        b = min(rows, a + step)
        x = torch.einsum("rgd,kd->rgk", q[a:b], k) / math.sqrt(dim)
        i = first + torch.arange(a, b, device=q.device)[:, None, None]
        j = torch.arange(len(k), device=q.device)
        if causal:
            x = x.masked_fill(j > i, -math.inf)
        if window:
            x = x.masked_fill(j <= i - window, -math.inf)
        if len(k):
            lse[a:b] = torch.logsumexp(x, -1)
        w = torch.exp(x - lse[a:b, :, None])
        out[a:b] = torch.nan_to_num(w, nan=0.0) @ v
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    group = heads // kv_heads
    if case["op"] == "append":
        rot, half = case["rot"], case["rot"] // 2
        lo = dim - rot
        cs = s["cos_sin"].double()[s["positions"].long()]
        turn = torch.complex(cs[:, :half], cs[:, half:])[:, None]

        def turned(x):
            x = x.double().clone()
            z = x[..., lo:]
            first = slice(0, None, 2) if case["interleaved"] else slice(0, half)
            second = slice(1, None, 2) if case["interleaved"] else slice(half, None)
            y = torch.complex(z[..., first].contiguous(), z[..., second].contiguous()) * turn
            z[..., first], z[..., second] = y.real.clone(), y.imag.clone()
            return x

        out = {"q": turned(s["q"])}
        for name in ("k",) if case["shared"] else ("k", "v"):
            x = turned(s["k"]) if name == "k" else s["v"].double()
            page, row = s["slots"] // case["page"], s["slots"] % case["page"]
            if case["fmt"] == "fp8":
                size = min(dim, 128)
                g = x.unflatten(-1, (-1, size))
                # the scale is that of the row as bf16 holds it
                e = torch.ceil(torch.log2(g.bfloat16().double().abs().amax(-1).clamp(min=2.0 ** -100) / 448.0))
                held = s["cache"][name].view(torch.float8_e4m3fn).double()
                held[page, :, row] = (g * torch.exp2(-e).unsqueeze(-1)).flatten(-2)
                scale = torch.exp2(s["cache"][name + "_scale"].double() - 127.0)
                scale[page, :, row] = torch.exp2(e)
                out[name], out[name + "_scale"] = held, scale
            else:
                held = s["cache"][name].double()
                held[page, :, row] = x
                out[name] = held
        return out
    q = s["q"].double()
    out = torch.zeros_like(q)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    for b in range(case["batch"]):
        if case["op"] == "decode":
            n, length = case["q_len"], int(s["seq_lens"][b])
            at = s["table"][b, :-(-length // case["page"])].long()

            def row(name):
                x = s["cache"][name][at]
                if case["fmt"] == "fp8":
                    e = s["cache"][name + "_scale"][at].double() - 127.0
                    x = x.view(torch.float8_e4m3fn).double().unflatten(-1, (e.shape[-1], -1)) * torch.exp2(e)[..., None]
                    x = x.flatten(-2)
                return x.double().transpose(0, 1).flatten(1, 2)[:, :length]

            k, v = row("k"), row("v")
            lo, hi, causal = b * n, (b + 1) * n, True
        else:
            lo, hi = int(s["cu_q"][b]), int(s["cu_q"][b + 1])
            a, z = int(s["cu_k"][b]), int(s["cu_k"][b + 1])
            k, v = s["k"][a:z].double().transpose(0, 1), s["v"][a:z].double().transpose(0, 1)
            length, causal = z - a, case["causal"]
        for h in range(kv_heads):
            part = slice(h * group, (h + 1) * group)
            out[lo:hi, part], lse[lo:hi, part] = _attend64(q[lo:hi, part], k[h], v[h], length - (hi - lo), causal,
                                                           case["window"])
    return {"out": out, "lse": lse}
