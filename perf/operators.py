"""What a decoder needs beside exact attention, measured: rotary positions (forward and backward), writing keys
and values into a paged cache and reading them back, and attention of new tokens over that cache.

`run` computes each in elementary torch operations in 32 bits (angles in 64), or, where `own` is true, through the
package's own entry points.  `exact` computes the same from the definitions in 64 bits.
"""
import functools
import math
import random

import torch

own = False

E4M3_MAX = 448.0


# --------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token for each of 32 sequences of a serving batch, far into their contexts: latency counts
        dict(name="rotary_single_tokens", op="rotary", batch=0, tokens=32, heads=32, heads_k=8, dim=128, rotary=128, interleaved=False,
             dtype="bf16", scaling="by_parts", factor=32.0, train=False, max_pos=131072),
        # a ragged packed prompt, half of each head rotated, pairs side by side, positions interpolated
        dict(name="rotary_prompt_interleaved", op="rotary", batch=0, tokens=5003, heads=32, heads_k=8, dim=128, rotary=64,
             interleaved=True, dtype="fp16", scaling="linear", factor=4.0, train=False, max_pos=32768),
        # the training step of the benchmark's workload (B1 H8 N65536 D128): queries and keys, forward and backward
        dict(name="rotary_train", op="rotary", batch=1, tokens=65536, heads=8, heads_k=8, dim=128, rotary=128, interleaved=False,
             dtype="bf16", scaling="none", factor=1.0, train=True, max_pos=65536),
        # one token for each of 64 sequences written into an 8-bit cache, and the new rows as the cache then holds them
        dict(name="cache_single_tokens", op="cache", batch=64, new_lo=1, new_hi=1, ctx_lo=128, ctx_hi=2048, heads_k=8, dim=128, page=64,
             cache="e4m3", dtype="bf16", back="new"),
        # ragged prompts written into an 8-bit cache of small pages and read back whole
        dict(name="cache_prompts", op="cache", batch=12, new_lo=300, new_hi=4096, ctx_lo=0, ctx_hi=0, heads_k=8, dim=128, page=16,
             cache="e4m3", dtype="bf16", back="new"),
        # long contexts of a serving batch read back in 16 bits (moved elsewhere, or into a training step)
        dict(name="cache_read", op="read", batch=16, new_lo=1, new_hi=1, ctx_lo=500, ctx_hi=12000, heads_k=8, dim=128, page=64, cache="e4m3",
             dtype="bf16"),
        # one sequence being generated: the smallest call, all latency
        dict(name="decode_one", op="attention", batch=1, new_lo=1, new_hi=1, ctx_lo=1000, ctx_hi=1000, heads=32, heads_k=8, dim=128, page=16,
             cache="bf16", dtype="bf16", causal=True, window=-1, alibi=False),
        # generation for a serving batch of mixed context lengths, 16-bit cache
        dict(name="decode_batch", op="attention", batch=64, new_lo=1, new_hi=1, ctx_lo=256, ctx_hi=16000, heads=32, heads_k=8, dim=128,
             page=64, cache="bf16", dtype="bf16", causal=True, window=-1, alibi=False),
        # the same with eight query heads to a key head and an 8-bit cache
        dict(name="decode_batch_e4m3", op="attention", batch=128, new_lo=1, new_hi=1, ctx_lo=256, ctx_hi=8000, heads=64, heads_k=8, dim=128,
             page=128, cache="e4m3", dtype="bf16", causal=True, window=-1, alibi=False),
        # chunks of prompts being read in over long contexts already in an 8-bit cache
        dict(name="chunk_e4m3", op="attention", batch=4, new_lo=61, new_hi=256, ctx_lo=6000, ctx_hi=30000, heads=32, heads_k=8, dim=128,
             page=32, cache="e4m3", dtype="bf16", causal=True, window=-1, alibi=False),
        # small heads, three to a key head, sliding window and linear biases, chunks of all lengths
        dict(name="chunk_window_alibi", op="attention", batch=9, new_lo=1, new_hi=500, ctx_lo=100, ctx_hi=6000, heads=12, heads_k=4, dim=64,
             page=16, cache="fp16", dtype="fp16", causal=True, window=1000, alibi=True),
        # whole prompts, packed, each its own length
        dict(name="prompts", op="attention", batch=4, new_lo=900, new_hi=5000, ctx_lo=0, ctx_hi=0, heads=32, heads_k=8, dim=128, page=64,
             cache="bf16", dtype="bf16", causal=True, window=-1, alibi=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    top = max(_cost(c) for c in listed())
    while True:
        c = _draw(rng)
        if _cost(c) <= top and _plain_bytes(c) <= 20e9:
            return c


def _draw(rng):
    op = rng.choice(["rotary", "cache", "read", "attention", "attention", "attention"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    dim = rng.choice([64, 128, 128])
    heads_k = rng.choice([1, 2, 3, 4, 8, 8, 16])
    if op == "rotary":
        scaling = rng.choice(["none", "linear", "ntk", "by_parts"])
        return dict(op=op, batch=rng.choice([0, 0, 1, 2, 3]), tokens=_log(rng, 1, 20000), heads=heads_k * rng.choice([1, 2, 4, 8]),
                    heads_k=heads_k, dim=dim, rotary=rng.choice([dim, dim, dim // 2, dim // 4]), interleaved=rng.random() < 0.5,
                    dtype=rng.choice([dtype, dtype, "fp32"]), scaling=scaling, factor=1.0 if scaling == "none" else float(rng.choice([2, 4, 8, 40])),
                    train=rng.random() < 0.5, max_pos=_log(rng, 100, 1000000))
    page = rng.choice([16, 32, 64, 128, 256])
    cache = rng.choice(["e4m3", dtype])
    if op == "cache":
        new = _log(rng, 1, 4000)
        return dict(op=op, batch=_log(rng, 1, 100), new_lo=max(1, new // 4), new_hi=new, ctx_lo=0, ctx_hi=rng.choice([0, 300, 3000]),
                    heads_k=heads_k, dim=dim, page=page, cache=cache, dtype=dtype, back="new")
    if op == "read":
        ctx = _log(rng, 2, 16000)
        return dict(op=op, batch=_log(rng, 1, 60), new_lo=1, new_hi=1, ctx_lo=max(1, ctx // 5), ctx_hi=ctx, heads_k=heads_k, dim=dim, page=page,
                    cache=cache, dtype=dtype)
    kind = rng.choice(["tokens", "few", "chunk", "prompt"])
    batch = _log(rng, 1, 100 if kind == "tokens" else 30 if kind == "few" else 8)
    new = {"tokens": 1, "few": rng.randint(2, 16), "chunk": _log(rng, 17, 600), "prompt": _log(rng, 50, 3000)}[kind]
    ctx = 0 if kind == "prompt" else _log(rng, 20, 20000)
    return dict(op=op, batch=batch, new_lo=max(1, new // 4) if kind != "tokens" else 1, new_hi=new, ctx_lo=ctx // 4, ctx_hi=ctx,
                heads=heads_k * rng.choice([1, 2, 3, 4, 5, 8]), heads_k=heads_k, dim=dim, page=page, cache=cache, dtype=dtype,
                causal=rng.random() < 0.85, window=rng.choice([-1, -1, -1, _log(rng, 1, 4000)]), alibi=rng.random() < 0.25)


# ------------------------------------------------------------------------------------------------ lengths and work
@functools.lru_cache(maxsize=256)
def _lengths_of(batch, new_lo, new_hi, ctx_lo, ctx_hi):
    rng = random.Random(f"{batch} {new_lo} {new_hi} {ctx_lo} {ctx_hi}")
    new = [_log(rng, new_lo, new_hi) for _ in range(batch)]
    ctx = [0 if ctx_hi == 0 else _log(rng, max(1, ctx_lo), ctx_hi) for _ in range(batch)]
    return new, ctx


def _lengths(c):
    """The new tokens of each sequence and what its cache held before them: by the case alone."""
    return _lengths_of(c["batch"], c["new_lo"], c["new_hi"], c["ctx_lo"], c["ctx_hi"])


def _size(name):
    return {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}[name]


def _pairs(c):
    """Pairs (query, key) that attention weighs, and for each sequence the keys that any of its queries sees."""
    pairs, keys = 0, 0
    for n, ctx in zip(*_lengths(c)):
        end, w = ctx + n, c["window"]
        for_all = lambda last: last * (last + 1) // 2  # noqa: E731  1 + 2 + ... + last
        if c["causal"]:
            if w < 0:
                pairs += for_all(end) - for_all(ctx)
            else:  # query at p sees min(p + 1, w + 1) keys
                few = max(0, min(end, w + 1) - ctx)
                pairs += for_all(ctx + few) - for_all(ctx) + (n - few) * (w + 1)
        else:
            pairs += sum(end - max(0, p - w) for p in range(ctx, end)) if w >= 0 else n * end
        keys += end - (max(0, ctx - w) if w >= 0 else 0)
    return pairs, keys


def work(case):
    c = case
    if c["op"] == "rotary":
        rows = max(1, c["batch"]) * c["tokens"] * (c["heads"] + c["heads_k"])
        ways = 2 if c["train"] else 1
        return {"bytes": ways * 2 * rows * c["dim"] * _size(c["dtype"]) + 4 * c["tokens"], "flops": ways * 3 * rows * c["rotary"]}
    new, ctx = _lengths(c)
    row = 2 * c["heads_k"] * c["dim"] * _size(c["cache"]) + (2 * c["heads_k"] if c["cache"] == "e4m3" else 0)
    wide = 2 * c["heads_k"] * c["dim"] * _size(c["dtype"])
    if c["op"] == "cache":
        return {"bytes": sum(new) * (2 * wide + 2 * row), "flops": sum(new) * wide}
    if c["op"] == "read":
        return {"bytes": (sum(new) + sum(ctx)) * (wide + row), "flops": (sum(new) + sum(ctx)) * wide / 2}
    pairs, keys = _pairs(c)
    q = sum(new) * c["heads"] * c["dim"] * _size(c["dtype"])
    return {"bytes": 2 * q + 4 * sum(new) * c["heads"] + keys * row, "flops": 4 * pairs * c["heads"] * c["dim"]}


def _cost(c):
    w = work(c)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def _plain_bytes(c):
    if c["op"] == "rotary":
        return 0
    new, ctx = _lengths(c)
    end = max(a + b for a, b in zip(new, ctx))
    kv = 8 * c["batch"] * end * c["heads_k"] * c["dim"]
    return kv + (4 * c["batch"] * max(new) * end * c["heads"] if c["op"] == "attention" else 0)


# --------------------------------------------------------------------------------------------------------- inputs
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}


def _rows(g, n, heads, dim, dtype):
    """Keys or values as projections give them: normal, each row with its own magnitude, one channel in 32 larger."""
    x = torch.randn(n, heads, dim, generator=g, device="cuda")
    x *= torch.exp2(torch.randn(n, heads, 1, generator=g, device="cuda") * 0.5)
    x[..., ::32] *= 4
    return x.to(dtype)


def _frequencies(c):
    """The angle of pair i at position p is p * f[i]; values are also scaled by the second result."""
    r = c["rotary"]
    i = torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r
    base, s = 10000.0, c["factor"]
    if c["scaling"] == "ntk":
        base = base * s ** (r / (r - 2))
    f = base ** -i
    if c["scaling"] == "linear":
        f = f / s
    if c["scaling"] == "by_parts":  # pairs that turn often within 4096 positions stay, slow ones are interpolated
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = f * keep + f / s * (1 - keep)
    return f, 0.1 * math.log(s) + 1.0 if c["scaling"] == "by_parts" else 1.0


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 2 + 1)
    s = {"case": c}
    dtype = _TYPES[c["dtype"]]
    if c["op"] == "rotary":
        lead = (c["batch"], c["tokens"]) if c["batch"] else (c["tokens"],)
        draw_rows = lambda h: torch.randn(*lead, h, c["dim"], generator=g, device="cuda").to(dtype)  # noqa: E731
        s["q"], s["k"] = draw_rows(c["heads"]), draw_rows(c["heads_k"])
        if c["train"]:
            s["dq"], s["dk"] = draw_rows(c["heads"]), draw_rows(c["heads_k"])
            s["q"].requires_grad_()
            s["k"].requires_grad_()
        first = torch.randint(0, max(1, c["max_pos"] - c["tokens"] + 1), (1,), generator=g, device="cuda")
        s["positions"] = (first + torch.arange(c["tokens"], device="cuda")).to(torch.int32)
        if c["tokens"] <= 256 and not c["batch"]:  # single tokens of separate sequences
            s["positions"] = torch.randint(0, c["max_pos"], (c["tokens"],), generator=g, device="cuda", dtype=torch.int32)
        s["freq"], s["magnitude"] = _frequencies(c)
        return s
    new, ctx = _lengths(c)
    page, heads, dim = c["page"], c["heads_k"], c["dim"]
    ends = [a + b for a, b in zip(new, ctx)]
    need = [-(-e // page) for e in ends]
    pages = sum(need) + 3  # a pool with a few pages that no sequence holds
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(new), max(need), dtype=torch.int32, device="cuda")
    at = torch.tensor([0] + need, device="cuda").cumsum(0)
    col = torch.arange(max(need), device="cuda")
    held = col[None, :] < torch.tensor(need, device="cuda")[:, None]
    table[held] = order[(at[:-1, None] + col[None, :])[held]]
    s["table"] = table
    s["cu"] = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
    s["lens"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    s["starts"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    s["zeros"] = torch.zeros(len(new), dtype=torch.int32, device="cuda")
    s["cu_ends"] = torch.tensor([0] + ends, device="cuda").cumsum(0).to(torch.int32)
    s["total"], s["total_ends"], s["max_new"], s["max_end"] = sum(new), sum(ends), max(new), max(ends)
    for name in ("k", "v"):
        s[name + "_exp"] = None
        if c["op"] == "cache":  # a cache that is being filled
            s[name] = _rows(g, s["total"], heads, dim, dtype)
            s[name + "_pages"] = torch.zeros(pages, page, heads, dim, device="cuda", dtype=torch.uint8 if c["cache"] == "e4m3" else dtype)
            if c["cache"] == "e4m3":
                s[name + "_pages"] = s[name + "_pages"].view(torch.float8_e4m3fn)
                s[name + "_exp"] = torch.zeros(pages, heads, page, dtype=torch.uint8, device="cuda")
        else:
            x = _rows(g, pages * page, heads, dim, dtype)
            if c["cache"] == "e4m3":
                code, exp = _quantise(x)
                s[name + "_pages"] = code.view(pages, page, heads, dim)
                s[name + "_exp"] = exp.view(pages, page, heads).transpose(1, 2).contiguous()
            else:
                s[name + "_pages"] = x.view(pages, page, heads, dim)
    if c["op"] == "attention":
        s["q"] = torch.randn(s["total"], c["heads"], dim, generator=g, device="cuda").to(dtype)
        s["slopes"] = None
        if c["alibi"]:
            s["slopes"] = torch.exp2(-8.0 * torch.arange(1, c["heads"] + 1, device="cuda") / c["heads"]).float()
    return s


# ------------------------------------------------------------------------------------------- the plain forms
def _turn(x, cos, sin, interleaved, rotary):
    """One rotation of the first `rotary` elements of each head; cos and sin: (..., rotary / 2)."""
    y = x.float()
    a, b = (y[..., 0:rotary:2], y[..., 1:rotary:2]) if interleaved else (y[..., :rotary // 2], y[..., rotary // 2:rotary])
    cos, sin = cos[..., None, :], sin[..., None, :]
    u, w = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((turned, y[..., rotary:]), -1).to(x.dtype)


def _quantise(x):
    """Rows of e4m3 codes and for each row the exponent byte e of its scale 2^(e - 127): the smallest power of two
    with which the largest magnitude is at most 448; a row of zeros has e = 0."""
    top = x.abs().amax(-1).float()
    m, e = torch.frexp(top)
    e = (e - 9 + (m > 0.875)).clamp(-126, 127)
    code = torch.ldexp(x.float(), -e[..., None]).to(torch.float8_e4m3fn)
    return code, torch.where(top > 0, e + 127, 0).to(torch.uint8)


def _row_of(s, cu, first, total):
    """For each of `total` packed rows its sequence and its position, `first` being its sequence's first one."""
    i = torch.arange(total, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(cu, i, right=True) - 1
    return b, first[b] + i - cu[b]


def _slots(s, cu, first, total):
    b, pos = _row_of(s, cu, first, total)
    page = s["case"]["page"]
    return s["table"][b, pos // page].long(), (pos % page).long()


def _append(s, name):
    at, off = _slots(s, s["cu"], s["starts"], s["total"])
    if s["case"]["cache"] == "e4m3":
        code, exp = _quantise(s[name])
        s[name + "_pages"].view(torch.uint8)[at, off] = code.view(torch.uint8)
        s[name + "_exp"].transpose(1, 2)[at, off] = exp
    else:
        s[name + "_pages"][at, off] = s[name]


def _held(s, name, at, off):
    """The values of some slots of the cache, in 32 bits."""
    if s["case"]["cache"] == "e4m3":
        code = s[name + "_pages"].view(torch.uint8)[at, off].view(torch.float8_e4m3fn).float()
        return torch.ldexp(code, s[name + "_exp"].transpose(1, 2)[at, off].int()[..., None] - 127)
    return s[name + "_pages"][at, off].float()


def _attend(s):
    c = s["case"]
    heads, kv, dim, group = c["heads"], c["heads_k"], c["dim"], c["heads"] // c["heads_k"]
    batch, n, end = c["batch"], s["max_new"], s["max_end"]
    # queries and keys, padded to the longest sequence
    i, j = torch.arange(n, device="cuda"), torch.arange(end, device="cuda")
    count, lens = s["cu"][1:] - s["cu"][:-1], s["lens"]
    real = i[None, :] < count[:, None]
    row = (s["cu"][:-1, None] + i[None, :]).clamp(max=s["total"] - 1)
    q = s["q"][row].float().view(batch, n, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(batch, kv, group * n, dim)
    at, off = s["table"][:, j // c["page"]].long(), (j % c["page"])[None, :].expand(batch, end)
    k = _held(s, "k", at, off).permute(0, 2, 3, 1)
    v = _held(s, "v", at, off).permute(0, 2, 1, 3)
    pos = (lens - count)[:, None] + i[None, :]
    apart = j[None, None, :] - pos[:, :, None]
    seen = (j[None, :] < lens[:, None])[:, None, :].expand(batch, n, end)
    if c["causal"]:
        seen = seen & (apart <= 0)
    if c["window"] >= 0:
        seen = seen & (apart >= -c["window"])
    z = (q @ k).mul_(dim ** -0.5).view(batch, kv, group, n, end)
    if s["slopes"] is not None:
        z -= s["slopes"].view(1, kv, group, 1, 1) * apart.abs()[:, None, None]
    z.masked_fill_(~seen[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    z.sub_(top).exp_()
    total = z.sum(-1)
    o = (z.view(batch, kv, group * n, end) @ v.contiguous()).view(batch, kv, group, n, dim) / total[..., None]
    lse = top[..., 0] + total.log()
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, n, heads, dim)[real]
    return o.to(s["q"].dtype), lse.permute(0, 3, 1, 2).reshape(batch, n, heads)[real].t().contiguous()


def run(state):
    s = state
    c = s["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "rotary":
        angle = s["positions"].double()[:, None] * s["freq"]
        cos, sin = (torch.cos(angle) * s["magnitude"]).float(), (torch.sin(angle) * s["magnitude"]).float()
        turn = lambda x, sign: _turn(x, cos, sign * sin, c["interleaved"], c["rotary"])  # noqa: E731
        with torch.no_grad():
            out = {"q": turn(s["q"], 1), "k": turn(s["k"], 1)}
            if c["train"]:  # a rotation's transpose is the rotation back, with the same magnitude
                out |= {"dq": turn(s["dq"], -1), "dk": turn(s["dk"], -1)}
        return out
    if c["op"] == "cache":
        _append(s, "k")
        _append(s, "v")
        if c["cache"] != "e4m3":
            return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        at, off = _slots(s, s["cu"], s["starts"], s["total"])
        return {"k": _held(s, "k", at, off).to(s["k"].dtype), "v": _held(s, "v", at, off).to(s["v"].dtype), "k_exp": s["k_exp"], "v_exp": s["v_exp"]}
    if c["op"] == "read":
        at, off = _slots(s, s["cu_ends"], s["zeros"], s["total_ends"])
        return {name: _held(s, name, at, off).to(_TYPES[c["dtype"]]) for name in ("k", "v")}
    o, lse = _attend(s)
    return {"o": o, "lse": lse}


# ------------------------------------------------------------------------------------------- the package's calls
def _run_own(s, c):
    from exact_attention_93_gb300 import attention, kvcache, rotary
    if c["op"] == "rotary":
        q, k = rotary.rotary_func(s["q"], s["k"], s["freq"], positions=s["positions"], interleaved=c["interleaved"], magnitude=s["magnitude"])
        out = {"q": q, "k": k}
        if c["train"]:
            out["dq"], out["dk"] = torch.autograd.grad((q, k), (s["q"], s["k"]), (s["dq"], s["dk"]))
        return out
    if c["op"] == "cache":
        kvcache.kv_cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["cu"], s["lens"], k_exp=s["k_exp"], v_exp=s["v_exp"])
        if c["cache"] != "e4m3":
            return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        k, v = kvcache.kv_cache_read(s["k_pages"], s["v_pages"], s["table"], s["cu"], s["total"], starts=s["starts"], k_exp=s["k_exp"], v_exp=s["v_exp"],
                                     dtype=_TYPES[c["dtype"]])
        return {"k": k, "v": v, "k_exp": s["k_exp"], "v_exp": s["v_exp"]}
    if c["op"] == "read":
        k, v = kvcache.kv_cache_read(s["k_pages"], s["v_pages"], s["table"], s["cu_ends"], s["total_ends"], k_exp=s["k_exp"], v_exp=s["v_exp"],
                                     dtype=_TYPES[c["dtype"]])
        return {"k": k, "v": v}
    o, lse = attention.flash_attn_paged_func(s["q"], s["k_pages"], s["v_pages"], s["table"], s["cu"], s["lens"], causal=c["causal"],
                                             window_size=(c["window"], -1), alibi_slopes=s["slopes"], k_exp=s["k_exp"], v_exp=s["v_exp"], return_lse=True)
    return {"o": o, "lse": lse}


# ------------------------------------------------------------------------------------------- definitions, 64 bits
def _to_e4m3(x):
    """Each row of x, in 64 bits, as the 8-bit cache holds it."""
    top = x.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-300) / E4M3_MAX)).clamp(-126, 127))
    y = x / scale
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * scale


def _cached(s, name, b, n):
    """The first n keys or values of sequence b, in 64 bits."""
    c = s["case"]
    pages = s["table"][b, : -(-n // c["page"])].long()
    x = s[name + "_pages"].view(torch.uint8)[pages].view(s[name + "_pages"].dtype).double()
    if c["cache"] == "e4m3":
        x = x * torch.exp2(s[name + "_exp"][pages].double() - 127).permute(0, 2, 1)[..., None]
    return x.flatten(0, 1)[:n]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rotary":
        if c["tokens"] * max(1, c["batch"]) * (c["heads"] + c["heads_k"]) * c["dim"] > 3e8:
            return None
        with torch.no_grad():
            # pair (a, b) as the complex number a + ib, turned by e^(i angle)
            turn = torch.polar(torch.full((), s["magnitude"], dtype=torch.float64, device="cuda"), s["positions"].double()[:, None] * s["freq"])[:, None]

            def turned(x, t):
                y, r = x.double().clone(), c["rotary"]
                a, b = (slice(0, r, 2), slice(1, r, 2)) if c["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
                z = torch.complex(y[..., a], y[..., b]) * t
                y[..., a], y[..., b] = z.real, z.imag
                return y

            out = {"q": turned(s["q"], turn), "k": turned(s["k"], turn)}
            if c["train"]:
                out |= {"dq": turned(s["dq"], turn.conj()), "dk": turned(s["dk"], turn.conj())}
        return out
    new, ctx = _lengths(c)
    if c["op"] == "cache":
        if c["cache"] == "e4m3":
            return {"k": _to_e4m3(s["k"].double()), "v": _to_e4m3(s["v"].double()), "k_exp": None, "v_exp": None}
        out = {}
        for name in ("k", "v"):
            x = s[name + "_pages"].double()
            row = 0
            for b in range(c["batch"]):
                p = torch.arange(ctx[b], ctx[b] + new[b], device="cuda")
                x[s["table"][b, p // c["page"]].long(), p % c["page"]] = s[name][row: row + new[b]].double()
                row += new[b]
            out[name + "_pages"] = x
        return out
    if c["op"] == "read":
        return {name: torch.cat([_cached(s, name, b, new[b] + ctx[b]) for b in range(c["batch"])]) for name in ("k", "v")}
    if 4 * _pairs(c)[0] * c["heads"] * c["dim"] > 3e12:
        return None
    o, lse, row, group = [], [], 0, c["heads"] // c["heads_k"]
    for b in range(c["batch"]):
        n, end = new[b], new[b] + ctx[b]
        k, v = _cached(s, "k", b, end), _cached(s, "v", b, end)
        q = s["q"][row: row + n].double()
        row += n
        d = torch.arange(end, device="cuda")[None, :] - torch.arange(ctx[b], end, device="cuda")[:, None]
        hidden = ((d > 0) if c["causal"] else torch.zeros_like(d, dtype=torch.bool)) | ((d < -c["window"]) if c["window"] >= 0 else False)
        ob, lb = [], []
        for h in range(c["heads"]):
            z = q[:, h] @ k[:, h // group].t() / math.sqrt(c["dim"])
            if s["slopes"] is not None:
                z = z - s["slopes"][h].double() * d.abs()
            z = z.masked_fill(hidden, -math.inf)
            lb.append(torch.logsumexp(z, 1))
            ob.append(torch.exp(z - lb[-1][:, None]) @ v[:, h // group])
        o.append(torch.stack(ob, 1))
        lse.append(torch.stack(lb, 0))
    return {"o": torch.cat(o), "lse": torch.cat(lse, 1)}
