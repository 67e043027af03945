"""What stands around attention in a decoder's step, measured: rotary positions with several axes, norms of queries and
keys with the rotation in the same pass (both forward and backward), the tables of a paged cache built from request
lengths, and attention over the cache for sequences that share long prefixes.

`run` computes each in elementary torch operations in 32 bits (angles and long sums in 64), or, where `own` is true, through
the package's own entry points.  `exact` computes the same from the definitions in 64 bits.
"""
import functools
import math
import random

import torch

own = False

EPS = 1e-6


# --------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token for each of 48 sequences that began with images: three axes, latency counts
        dict(name="axes_single_tokens", op="rotary", batch=0, tokens=48, heads=32, heads_k=8, dim=128, sections="16,24,24", order="blocks",
             interleaved=False, dtype="bf16", train=False, places="tokens"),
        # patches of several images packed for an image encoder: row and column, each with frequencies of its own
        dict(name="axes_patches", op="rotary", batch=0, tokens=12987, heads=16, heads_k=16, dim=64, sections="16,16", order="blocks",
             interleaved=False, dtype="fp16", train=False, places="patches"),
        # a training step over text with images between, the axes taking turns over the pairs
        dict(name="axes_train", op="rotary", batch=2, tokens=16384, heads=16, heads_k=4, dim=128, sections="24,20,20", order="turns",
             interleaved=False, dtype="bf16", train=True, places="mixed"),
        # single tokens of a serving batch: norm and rotation
        dict(name="norm_single_tokens", op="norm", batch=0, tokens=32, heads=32, heads_k=8, dim=128, sections="64", order="blocks",
             interleaved=False, dtype="bf16", train=False, places="tokens"),
        # a packed ragged prompt, pairs side by side
        dict(name="norm_prompt", op="norm", batch=0, tokens=5003, heads=32, heads_k=8, dim=128, sections="64", order="blocks",
             interleaved=True, dtype="fp16", train=False, places="text"),
        # the training step of the benchmark's workload (B1 H8 N65536 D128): queries, keys and both weights, forward and backward
        dict(name="norm_train", op="norm", batch=1, tokens=65536, heads=8, heads_k=8, dim=128, sections="64", order="blocks",
             interleaved=False, dtype="bf16", train=True, places="text"),
        # small heads in 32 bits, half of each rotated along three axes, odd lengths
        dict(name="norm_axes_train", op="norm", batch=4, tokens=2039, heads=12, heads_k=4, dim=64, sections="8,4,4", order="blocks",
             interleaved=False, dtype="fp32", train=True, places="mixed"),
        # the tables of one step of generation: one token each for 64 sequences
        dict(name="tables_single_tokens", op="tables", batch=64, new_lo=1, new_hi=1, ctx_lo=128, ctx_hi=16000, page=64),
        # ragged prompts taken into a cache of small pages
        dict(name="tables_prompts", op="tables", batch=48, new_lo=300, new_hi=8192, ctx_lo=0, ctx_hi=0, page=16),
        # generation under one long system prompt: 64 sequences, each with its own shorter context behind it
        dict(name="shared_prompt", op="shared", groups=1, members=64, new_lo=1, new_hi=1, prefix_lo=16000, prefix_hi=16000, own_lo=16, own_hi=2000,
             heads=32, heads_k=8, dim=128, page=64, cache="bf16", dtype="bf16"),
        # several answers sampled to each of 8 prompts of different lengths, 8-bit cache
        dict(name="shared_samples_e4m3", op="shared", groups=8, members=16, new_lo=1, new_hi=1, prefix_lo=1000, prefix_hi=8000, own_lo=1,
             own_hi=1500, heads=32, heads_k=8, dim=128, page=16, cache="e4m3", dtype="bf16"),
        # a few drafted tokens for each of 24 sequences under one prompt, small heads, three to a key head
        dict(name="shared_drafts", op="shared", groups=1, members=24, new_lo=2, new_hi=9, prefix_lo=6000, prefix_hi=6000, own_lo=1, own_hi=700,
             heads=12, heads_k=4, dim=64, page=32, cache="fp16", dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    top = max(_cost(c) for c in listed())
    while True:
        c = _draw(rng)
        if _cost(c) <= top and _plain_bytes(c) <= 12e9:
            return c


def _draw(rng):
    op = rng.choice(["rotary", "norm", "norm", "tables", "shared", "shared"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    dim = rng.choice([64, 128, 128])
    heads_k = rng.choice([1, 2, 3, 4, 8, 8, 16])
    if op in ("rotary", "norm"):
        pairs = rng.choice([dim, dim, dim // 2]) // 2
        axes = rng.choice([2, 3, 3, 4]) if op == "rotary" else rng.choice([1, 1, 2, 3])
        cuts = sorted(rng.sample(range(1, pairs), axes - 1))
        sections = ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [pairs]))
        return dict(op=op, batch=rng.choice([0, 0, 1, 2, 3]), tokens=_log(rng, 1, 20000), heads=heads_k * rng.choice([1, 2, 4, 5, 8]),
                    heads_k=heads_k, dim=dim, sections=sections, order=rng.choice(["blocks", "turns"]), interleaved=rng.random() < 0.4,
                    dtype=rng.choice([dtype, dtype, "fp32"]), train=rng.random() < 0.5,
                    places="text" if axes == 1 else "patches" if axes == 2 else "mixed")
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "tables":
        new = rng.choice([1, 1, _log(rng, 2, 8000)])
        return dict(op=op, batch=_log(rng, 1, 1000 if new < 100 else 40), new_lo=1 if new == 1 else rng.randint(0, 1) + new // 5, new_hi=new, ctx_lo=0,
                    ctx_hi=rng.choice([0, 300, 20000]), page=page)
    groups = rng.choice([1, 1, 2, _log(rng, 3, 12)])
    new = rng.choice([1, 1, rng.randint(2, 24)])
    prefix, own_keys = _log(rng, 300, 30000), _log(rng, 1, 3000)
    return dict(op=op, groups=groups, members=_log(rng, 1, max(2, 128 // groups)), new_lo=max(1, new // 3), new_hi=new, prefix_lo=prefix // 3,
                prefix_hi=prefix, own_lo=max(1, own_keys // 8), own_hi=own_keys, heads=heads_k * rng.choice([1, 2, 3, 4, 5, 8]), heads_k=heads_k, dim=dim,
                page=page, cache=rng.choice(["e4m3", dtype]), dtype=dtype)


# ------------------------------------------------------------------------------------------------ lengths and work
def _lens(key, n, lo, hi):
    rng = random.Random(key)
    return [hi if lo == hi else 0 if hi == 0 else lo if lo == 0 and rng.random() < 0.2 else _log(rng, max(1, lo), hi) for _ in range(n)]


@functools.lru_cache(maxsize=256)
def _lengths_of(*v):
    return [_lens(f"{i} {v}", n, lo, hi) for i, (n, lo, hi) in enumerate(zip(v[::3], v[1::3], v[2::3]))]


def _lengths(c):
    """By the case alone: the new tokens of each sequence and what its cache held before them (tables); the new tokens of
    each sequence, its own keys before them, and each group's shared pages (shared)."""
    if c["op"] == "tables":
        return _lengths_of(c["batch"], c["new_lo"], c["new_hi"], c["batch"], c["ctx_lo"], c["ctx_hi"])
    batch = c["groups"] * c["members"]
    new, own_keys, prefix = _lengths_of(batch, c["new_lo"], c["new_hi"], batch, c["own_lo"], c["own_hi"], c["groups"], c["prefix_lo"], c["prefix_hi"])
    return new, own_keys, [p // c["page"] for p in prefix]


def _size(name):
    return {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}[name]


def work(case):
    c = case
    if c["op"] in ("rotary", "norm"):
        rows = max(1, c["batch"]) * c["tokens"] * (c["heads"] + c["heads_k"])
        axes, rotary = c["sections"].count(",") + 1, 2 * sum(map(int, c["sections"].split(",")))
        moved = 2 + (0 if not c["train"] else 2 if c["op"] == "rotary" else 3)  # a norm's gradient reads its input again
        flops = (2 if c["train"] else 1) * 3 * rotary
        if c["op"] == "norm":
            flops += (14 if c["train"] else 4) * c["dim"]
        return {"bytes": moved * rows * c["dim"] * _size(c["dtype"]) + 4 * axes * c["tokens"], "flops": rows * flops}
    if c["op"] == "tables":
        new, ctx = _lengths(c)
        pages = sum(-(-(a + b) // c["page"]) - -(-b // c["page"]) for a, b in zip(new, ctx))
        return {"bytes": 12 * sum(new) + 20 * c["batch"] + 8 * pages, "flops": 4 * sum(new)}
    new, own_keys, shared = _lengths(c)
    row = 2 * c["heads_k"] * c["dim"] * _size(c["cache"]) + (2 * c["heads_k"] if c["cache"] == "e4m3" else 0)
    pairs = sum(n * (shared[b // c["members"]] * c["page"] + k) + n * (n + 1) // 2 for b, (n, k) in enumerate(zip(new, own_keys)))
    keys = sum(shared) * c["page"] + sum(new) + sum(own_keys)
    q = sum(new) * c["heads"] * c["dim"] * _size(c["dtype"])
    return {"bytes": 2 * q + 4 * sum(new) * c["heads"] + keys * row, "flops": 4 * pairs * c["heads"] * c["dim"]}


def _cost(c):
    w = work(c)
    return max(w["bytes"] / 6.7e12, w["flops"] / 1.9e15)


def _plain_bytes(c):
    if c["op"] != "shared":
        return 0
    new, own_keys, shared = _lengths(c)
    end, batch = max(a + b for a, b in zip(new, own_keys)), c["groups"] * c["members"]
    first = 8 * max(shared) * c["page"] * c["heads_k"] * c["dim"] + 4 * c["members"] * max(new) * max(shared) * c["page"] * c["heads"]
    return first + 8 * batch * end * c["heads_k"] * c["dim"] + 4 * batch * max(new) * end * c["heads"]


# --------------------------------------------------------------------------------------------------------- inputs
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}


def _rows(g, n, heads, dim, dtype):
    """Rows as projections give them: normal, each with its own magnitude, one channel in 32 larger."""
    x = torch.randn(n, heads, dim, generator=g, device="cuda")
    x *= torch.exp2(torch.randn(n, heads, 1, generator=g, device="cuda") * 0.5)
    x[..., ::32] *= 4
    return x.to(dtype)


def _places(c, seed):
    """Positions (axes, tokens): of text on every axis alike; of images, one time and a place in the grid."""
    axes, n, rng = c["sections"].count(",") + 1, c["tokens"], random.Random(seed)
    if c["places"] == "tokens":  # single tokens of separate sequences
        return torch.tensor([[rng.randrange(131072) for _ in range(n)]], dtype=torch.int32).expand(axes, n).contiguous()
    parts, at, filled = [], rng.randrange(1000), 0
    while filled < n:
        if c["places"] == "text" or (c["places"] == "mixed" and len(parts) % 2 == 0):
            k = n if c["places"] == "text" else _log(rng, 20, 500)
            parts.append((at + torch.arange(k)).expand(axes, k))
            at += k
        else:
            t, h, w = rng.choice([1, 1, 1, 4]) if axes > 2 else 1, rng.randint(8, 64), rng.randint(8, 64)
            first = 0 if c["places"] == "patches" else at
            grid = torch.stack(torch.meshgrid(torch.arange(t), torch.arange(h), torch.arange(w), indexing="ij")).reshape(3, -1)
            grid = grid[1:] if axes == 2 else torch.cat((grid, grid[:1].expand(axes - 3, -1)))
            parts.append(first + grid)
            at += max(t, h, w)
        filled += parts[-1].shape[1]
    return torch.cat(parts, 1)[:, :n].to(torch.int32).contiguous()


def _frequencies(c):
    """Per pair: image patches have a spectrum of frequencies on each axis, everything else one over all pairs."""
    sections = [int(x) for x in c["sections"].split(",")]
    if c["places"] == "patches" and c["order"] == "blocks":
        return torch.cat([100.0 ** -(torch.arange(s, dtype=torch.float64) / s) for s in sections]).cuda()
    n = sum(sections)
    return 10000.0 ** -(torch.arange(n, dtype=torch.float64, device="cuda") / n)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 2 + 1)
    s = {"case": c}
    if c["op"] in ("rotary", "norm"):
        dtype = _TYPES[c["dtype"]]
        lead = (c["batch"], c["tokens"]) if c["batch"] else (c["tokens"],)
        count = max(1, c["batch"]) * c["tokens"]
        for name, heads in (("q", c["heads"]), ("k", c["heads_k"])):
            s[name] = _rows(g, count, heads, c["dim"], dtype).view(*lead, heads, c["dim"])
            if c["train"]:
                s["d" + name] = torch.randn(*lead, heads, c["dim"], generator=g, device="cuda").to(dtype)
                s[name].requires_grad_()
            if c["op"] == "norm":
                s[name + "_weight"] = (1 + 0.2 * torch.randn(c["dim"], generator=g, device="cuda")).to(dtype).requires_grad_(c["train"])
        s["positions"] = _places(c, seed).cuda()
        s["freq"] = _frequencies(c)
        s["sections"] = tuple(int(x) for x in c["sections"].split(","))
        return s
    page = c["page"]
    if c["op"] == "tables":
        new, ctx = _lengths(c)
        held = [-(-b // page) for b in ctx]
        need = [-(-(a + b) // page) for a, b in zip(new, ctx)]
        pages, spare = sum(need) + 70, 37
        width = max(need) + 3
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        s["table"] = _table(order, held, width)
        s["free"] = order[sum(held):].contiguous()
        s["count"] = torch.tensor([sum(need) - sum(held) + spare], dtype=torch.int32, device="cuda")
        s["new"] = torch.tensor(new, dtype=torch.int32, device="cuda")
        s["before"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        s["total"] = sum(new)
        return s
    new, own_keys, shared = _lengths(c)
    dtype, heads, dim, members = _TYPES[c["dtype"]], c["heads_k"], c["dim"], c["members"]
    own_need = [-(-(a + b) // page) for a, b in zip(new, own_keys)]
    pages = sum(own_need) + sum(shared) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    width = max(shared[b // members] + n for b, n in enumerate(own_need))
    prefix = _table(order, shared, max(1, max(shared)))
    mine = _table(order[sum(shared):], own_need, max(own_need))
    s["table"] = torch.zeros(len(new), width, dtype=torch.int32, device="cuda")
    for i, p in enumerate(shared):
        rows = slice(i * members, (i + 1) * members)
        s["table"][rows, :p] = prefix[i, :p]
        n = min(width - p, mine.shape[1])
        s["table"][rows, p: p + n] = mine[rows, :n]
    s["cu"] = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
    s["lens"] = torch.tensor([shared[b // members] * page + a + k for b, (a, k) in enumerate(zip(new, own_keys))], dtype=torch.int32, device="cuda")
    s["cu_groups"] = torch.arange(0, len(new) + 1, members, dtype=torch.int32, device="cuda")
    s["shared"] = torch.tensor(shared, dtype=torch.int32, device="cuda")
    s["total"], s["max_new"] = sum(new), max(new)
    s["max_own"] = max(a + b for a, b in zip(new, own_keys))
    for name in ("k", "v"):
        x = _rows(g, pages * page, heads, dim, dtype)
        s[name + "_exp"] = None
        if c["cache"] == "e4m3":
            code, exp = _quantise(x)
            s[name + "_pages"] = code.view(pages, page, heads, dim)
            s[name + "_exp"] = exp.view(pages, page, heads).transpose(1, 2).contiguous()
        else:
            s[name + "_pages"] = x.view(pages, page, heads, dim)
    s["q"] = torch.randn(s["total"], c["heads"], dim, generator=g, device="cuda").to(dtype)
    return s


def _table(order, need, width):
    """Rows of a block table: the pages of `order`, need[b] of them for row b, zeros behind."""
    table = torch.zeros(len(need), width, dtype=torch.int32, device="cuda")
    at = torch.tensor([0] + need, device="cuda").cumsum(0)
    col = torch.arange(width, device="cuda")
    held = col[None, :] < torch.tensor(need, device="cuda")[:, None]
    table[held] = order[(at[:-1, None] + col[None, :])[held]]
    return table


def _quantise(x):
    """Rows of e4m3 codes and for each row the exponent byte e of its scale 2^(e - 127): the smallest power of two
    with which the largest magnitude is at most 448; a row of zeros has e = 0."""
    top = x.abs().amax(-1).float()
    m, e = torch.frexp(top)
    e = (e - 9 + (m > 0.875)).clamp(-126, 127)
    code = torch.ldexp(x.float(), -e[..., None]).to(torch.float8_e4m3fn)
    return code, torch.where(top > 0, e + 127, 0).to(torch.uint8)


# ------------------------------------------------------------------------------------------- the plain forms
def _axis_of_pair(sections, order):
    """The axis that each pair takes its position from: the axes one after the other, or dealing pairs out in turns, those
    axes left out that have all of theirs."""
    if order == "blocks":
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while len(out) < sum(sections):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def _turn(y, cos, sin, interleaved, rotary):
    """One rotation of the first `rotary` elements of each head, in 32 bits; cos and sin: (..., rotary / 2)."""
    a, b = (y[..., 0:rotary:2], y[..., 1:rotary:2]) if interleaved else (y[..., :rotary // 2], y[..., rotary // 2:rotary])
    cos, sin = cos[..., None, :], sin[..., None, :]
    u, w = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((turned, y[..., rotary:]), -1)


def _turns(s, c):
    axis = torch.tensor(_axis_of_pair(s["sections"], c["order"]), device="cuda")
    angle = s["positions"][axis].t().double() * s["freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    return lambda y, sign: _turn(y, cos, sign * sin, c["interleaved"], 2 * len(axis))


def _normed(s, c, name, turn):
    x, w = s[name].float(), s[name + "_weight"].float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    out = {name: turn(x * r * w, 1).to(s[name].dtype)}
    if c["train"]:
        g = turn(s["d" + name].float(), -1)
        x = x * r
        gw = g * w
        out["d" + name] = (r * (gw - x * (gw * x).mean(-1, keepdim=True))).to(s[name].dtype)
        out["d" + name + "_weight"] = (g * x).flatten(0, -2).sum(0, dtype=torch.float64).to(w.dtype).to(s[name + "_weight"].dtype)
    return out


def _plan(s, c):
    page, before, new, width = c["page"], s["before"], s["new"], s["table"].shape[1]
    after = before + new
    held, need = (before + page - 1) // page, (after + page - 1) // page
    cu = torch.cat((torch.zeros_like(new[:1]), new.cumsum(0, dtype=torch.int32)))
    first = (need - held).cumsum(0, dtype=torch.int32) - (need - held)  # pages taken by the sequences before
    col = torch.arange(width, device="cuda", dtype=torch.int32)[None, :]
    take = (s["count"] - 1 - first)[:, None] - (col - held[:, None])
    fresh = (col >= held[:, None]) & (col < need[:, None])
    s["table"].copy_(torch.where(fresh, s["free"][take.clamp(0, s["free"].shape[0] - 1)], s["table"]))
    row = torch.arange(s["total"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(cu[1:].contiguous(), row, right=True)
    position = before[b] + row - cu[b]
    slot = s["table"][b, position // page].long() * page + position % page
    return {"cu_seqlens": cu, "seqlens": after, "positions": position, "slots": slot, "table": s["table"], "free_count": s["count"] - (need - held).sum(),
            "missing": torch.zeros_like(s["count"])}


def _held(s, name, at, off):
    """The values of some slots of the cache, in 32 bits."""
    if s["case"]["cache"] == "e4m3":
        code = s[name + "_pages"].view(torch.uint8)[at, off].view(torch.float8_e4m3fn).float()
        return torch.ldexp(code, s[name + "_exp"].transpose(1, 2)[at, off].int()[..., None] - 127)
    return s[name + "_pages"][at, off].float()


def _part(q, k, v, hidden):
    """Maximum, sum and weighted values of scores q k, all but the hidden ones; (..., rows, dim) and (..., keys, dim)."""
    z = q @ k.transpose(-1, -2)
    if hidden is not None:
        z.masked_fill_(hidden, -math.inf)
    top = z.amax(-1, keepdim=True)
    z.sub_(top).exp_()
    return top, z.sum(-1, keepdim=True), z @ v


def _attend(s, c):
    page, heads, kv, dim, members = c["page"], c["heads"], c["heads_k"], c["dim"], c["members"]
    group, batch, n, end, total = heads // kv, c["groups"] * c["members"], s["max_new"], s["max_own"], s["total"]
    new, _, shared = _lengths(c)
    scaled = s["q"].float() * dim ** -0.5
    top, count, o = scaled.new_empty(total, heads, 1), scaled.new_empty(total, heads, 1), torch.empty_like(scaled)
    # the shared part, once for all rows of a group
    row = 0
    for i, pages in enumerate(shared):
        rows = sum(new[i * members: (i + 1) * members])
        at = slice(row, row + rows)
        row += rows
        if pages == 0:
            top[at], count[at], o[at] = -math.inf, 0, 0
            continue
        j = torch.arange(pages * page, device="cuda")
        where = s["table"][i * members, j // page].long(), j % page
        q = scaled[at].view(rows, kv, group, dim).permute(1, 2, 0, 3).reshape(kv, group * rows, dim)
        got = _part(q, _held(s, "k", *where).transpose(0, 1), _held(s, "v", *where).transpose(0, 1), None)
        for x, y in zip((top, count, o), got):
            x[at] = y.view(kv, group, rows, -1).permute(2, 0, 1, 3).reshape(rows, heads, -1)
    # each sequence's own keys, padded to the longest
    i, j = torch.arange(n, device="cuda"), torch.arange(end, device="cuda")
    first = s["shared"].repeat_interleave(members, output_size=batch)
    lens, rows = s["lens"] - first * page, s["cu"][1:] - s["cu"][:-1]
    real = i[None, :] < rows[:, None]
    q = scaled[(s["cu"][:-1, None] + i[None, :]).clamp(max=total - 1)].view(batch, n, kv, group, dim).permute(0, 2, 3, 1, 4)
    where = s["table"].gather(1, (first[:, None] + j[None, :] // page).clamp(max=s["table"].shape[1] - 1).long()).long(), (j % page)[None, :].expand(batch, end)
    hidden = j[None, None, :] > ((lens - rows)[:, None] + i[None, :])[:, :, None]
    got = _part(q.reshape(batch, kv, group * n, dim), _held(s, "k", *where).transpose(1, 2), _held(s, "v", *where).transpose(1, 2),
                hidden[:, None, None].expand(batch, 1, group, n, end).reshape(batch, 1, group * n, end))
    top2, count2, o2 = (x.view(batch, kv, group, n, -1).permute(0, 3, 1, 2, 4).reshape(batch, n, heads, -1)[real] for x in got)
    both = torch.maximum(top, top2)
    a, b = torch.exp(top - both), torch.exp(top2 - both)
    count = a * count + b * count2
    return ((a * o + b * o2) / count).to(s["q"].dtype), (both + count.log())[..., 0].t().contiguous()


def _ordered(out):
    return {name: out[name] for name in ("q", "k", "dq", "dk", "dq_weight", "dk_weight") if name in out}


def run(state):
    s = state
    c = s["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "tables":
        return _plan(s, c)
    if c["op"] == "shared":
        o, lse = _attend(s, c)
        return {"o": o, "lse": lse}
    with torch.no_grad():
        turn = _turns(s, c)
        if c["op"] == "norm":
            return _ordered(_normed(s, c, "q", turn) | _normed(s, c, "k", turn))
        out = {name: turn(s[name].float(), 1).to(s[name].dtype) for name in ("q", "k")}
        if c["train"]:  # a rotation's transpose is the rotation back
            out |= {"d" + name: turn(s["d" + name].float(), -1).to(s[name].dtype) for name in ("q", "k")}
        return out


# ------------------------------------------------------------------------------------------- the package's calls
def _run_own(s, c):
    from exact_attention_93_gb300 import attention, kvcache, rotary
    if c["op"] == "rotary":
        q, k = rotary.rotary_func(s["q"], s["k"], s["freq"], positions=s["positions"], interleaved=c["interleaved"], sections=s["sections"],
                                  section_order=c["order"])
        out = {"q": q, "k": k}
        if c["train"]:
            out["dq"], out["dk"] = torch.autograd.grad((q, k), (s["q"], s["k"]), (s["dq"], s["dk"]))
        return out
    if c["op"] == "norm":
        several = len(s["sections"]) > 1
        q, k = rotary.qk_norm_rotary_func(s["q"], s["k"], s["q_weight"], s["k_weight"], s["freq"],
                                          positions=s["positions"] if several else s["positions"][0], eps=EPS, interleaved=c["interleaved"],
                                          sections=s["sections"] if several else None, section_order=c["order"])
        out = {"q": q, "k": k}
        if c["train"]:
            leaves = ("q", "k", "q_weight", "k_weight")
            out |= zip(("d" + x for x in leaves), torch.autograd.grad((q, k), [s[x] for x in leaves], (s["dq"], s["dk"])))
        return out
    if c["op"] == "tables":
        step = kvcache.kv_cache_reserve(s["new"], s["before"], s["table"], s["free"], s["count"], c["page"], s["total"])
        return {"cu_seqlens": step.cu_seqlens, "seqlens": step.seqlens, "positions": step.positions, "slots": step.slots, "table": s["table"],
                "free_count": step.free_count, "missing": step.missing}
    o, lse = attention.flash_attn_paged_func(s["q"], s["k_pages"], s["v_pages"], s["table"], s["cu"], s["lens"], k_exp=s["k_exp"], v_exp=s["v_exp"],
                                             return_lse=True, cu_groups=s["cu_groups"], shared_pages=s["shared"])
    return {"o": o, "lse": lse}


# ------------------------------------------------------------------------------------------- definitions, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "tables":
        return _exact_plan(s, c)
    if c["op"] == "shared":
        return _exact_attention(s, c)
    if c["tokens"] * max(1, c["batch"]) * (c["heads"] + c["heads_k"]) * c["dim"] > 3e8:
        return None
    left = list(s["sections"])  # pairs that each axis still gets, one at a time
    axis = []
    for i in range(sum(left)):
        now = next(a for a, n in enumerate(left) if n) if c["order"] == "blocks" else (axis[-1] + 1) % len(left) if axis else 0
        while not left[now]:
            now = (now + 1) % len(left)
        left[now] -= 1
        axis.append(now)
    pos = torch.stack([s["positions"][a] for a in axis], 1).double()
    turn = torch.polar(torch.ones_like(pos), pos * s["freq"])[:, None]  # pair (a, b) as a + ib, turned by e^(i angle)
    r = 2 * len(axis)
    lo, hi = (slice(0, r, 2), slice(1, r, 2)) if c["interleaved"] else (slice(0, r // 2), slice(r // 2, r))

    def turned(x, t):
        y = x.clone()
        z = torch.complex(x[..., lo], x[..., hi]) * t
        y[..., lo], y[..., hi] = z.real, z.imag
        return y

    out = {}
    with torch.no_grad():
        for name in ("q", "k"):
            x = s[name].double()
            if c["op"] == "norm":
                w = s[name + "_weight"].double()
                size = torch.sqrt(x.square().sum(-1, keepdim=True) / c["dim"] + EPS)
                out[name] = turned(x / size * w, turn)
            else:
                out[name] = turned(x, turn)
            if not c["train"]:
                continue
            g = turned(s["d" + name].double(), turn.conj())
            if c["op"] == "norm":
                out["d" + name + "_weight"] = (g * x / size).sum(tuple(range(g.dim() - 1)))
                g = g * w
                g = g / size - x * (g * x).sum(-1, keepdim=True) / (c["dim"] * size ** 3)
            out["d" + name] = g
    return _ordered(out)


def _exact_plan(s, c):
    new, ctx = _lengths(c)
    page, table, free = c["page"], s["table"].tolist(), s["free"].tolist()
    count = int(s["count"])
    cu, after, positions, slots = [0], [], [], []
    for b, (n, held) in enumerate(zip(new, ctx)):
        for p in range(held, held + n):
            if p % page == 0:
                count -= 1
                table[b][p // page] = free[count]
            positions.append(p)
            slots.append(table[b][p // page] * page + p % page)
        cu.append(cu[-1] + n)
        after.append(held + n)
    whole = lambda x, t=torch.int32: torch.tensor(x, dtype=t, device="cuda")  # noqa: E731
    return {"cu_seqlens": whole(cu), "seqlens": whole(after), "positions": whole(positions), "slots": whole(slots, torch.int64), "table": whole(table),
            "free_count": whole([count]), "missing": whole([0])}


def _exact_attention(s, c):
    if work(c)["flops"] > 3e12:
        return None
    new, own_keys, shared = _lengths(c)
    o, lse, row, group, page = [], [], 0, c["heads"] // c["heads_k"], c["page"]
    for b, n in enumerate(new):
        end = shared[b // c["members"]] * page + own_keys[b] + n
        pages = s["table"][b, : -(-end // page)].long()
        k, v = (s[x + "_pages"].view(torch.uint8)[pages].view(s[x + "_pages"].dtype).double() for x in ("k", "v"))
        if c["cache"] == "e4m3":
            k, v = (x * torch.exp2(s[y][pages].double() - 127).permute(0, 2, 1)[..., None] for x, y in ((k, "k_exp"), (v, "v_exp")))
        k, v = (x.flatten(0, 1)[:end].repeat_interleave(group, 1) for x in (k, v))
        z = torch.einsum("nhd,jhd->hnj", s["q"][row: row + n].double(), k) / math.sqrt(c["dim"])
        row += n
        z += torch.full((n, end), -math.inf, dtype=torch.float64, device="cuda").triu(end - n + 1)
        lse.append(torch.logsumexp(z, 2))
        o.append(torch.einsum("hnj,jhd->nhd", torch.exp(z - lse[-1][..., None]), v))
    return {"o": torch.cat(o), "lse": torch.cat(lse, 1)}
