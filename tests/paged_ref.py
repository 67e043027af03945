"""Plain 64-bit forms of rotary positions, the paged cache and attention over
it, on the CPU, ragged batches to test with, and the C structs of
include/fattn_cache.h."""
import ctypes
import math

import torch

from exact_attention_93_gb300 import fattn

EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
E4M3 = torch.float8_e4m3fn


# the structs of include/fattn_cache.h
class KvPages(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_exp", "v_exp")] + [
        (n, ctypes.c_longlong) for n in ("k_page", "k_token", "k_head", "v_page", "v_token",
                                         "v_head")] + [
        (n, ctypes.c_int) for n in ("pages", "page_size", "heads", "head_dim", "type")]


class Ragged(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_longlong),
                ("max_pages", ctypes.c_int), ("cu_seqlens", ctypes.c_void_p),
                ("seqlens", ctypes.c_void_p), ("batch", ctypes.c_int), ("total", ctypes.c_int)]


class RotaryOperand(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("heads", ctypes.c_int),
                ("xs", fattn.FaStrides), ("ys", fattn.FaStrides)]


def rotary(x, pos, inv_freq, interleaved=False, magnitude=1.0, inverse=False):
    """x: (batch, n, heads, D) in any type; pos: (batch, n); fp64 out."""
    y = x.double().clone()
    r = 2 * inv_freq.numel()
    a, b = ((slice(0, r, 2), slice(1, r, 2)) if interleaved
            else (slice(0, r // 2), slice(r // 2, r)))
    angle = (pos.double()[..., None] * inv_freq.double()) * (-1 if inverse else 1)
    c, s = (magnitude * t(angle)[:, :, None] for t in (torch.cos, torch.sin))
    u, v = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = u * c - v * s, u * s + v * c
    return y


def quantise(x):
    """(values, exponent bytes) of rows x (..., D) as an e4m3 cache holds them."""
    x = x.double()
    finite = torch.where(torch.isfinite(x), x.abs(), 0.0)
    top = finite.amax(-1)
    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)).clamp(-126, 127)
    scale = torch.exp2(e)[..., None]
    y = (x / scale).clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    vals = torch.round(y / step) * step * scale
    odd = ~torch.isfinite(x).all(-1)
    return vals, torch.where((top > 0) | odd, e + 127, 0.0).to(torch.uint8)


class Batch:
    """Sequences with `rows` new tokens each, `ctx` cached before them (a
    negative ctx: the cache is shorter than the rows), in scattered pages.  The
    cache's other bytes are NaN, unused table entries are out of range."""

    def __init__(self, rows, ctx, heads_k, D, page, dtype, fp8, seed=0, tail=0, poison=True,
                 spare_cols=2):
        g = torch.Generator().manual_seed(seed)
        self.rows, self.heads_k, self.D, self.page = list(rows), heads_k, D, page
        self.dtype, self.fp8 = dtype, fp8
        self.lens = [max(0, r + c) for r, c in zip(rows, ctx)]
        n = len(self.rows)
        need = [-(-x // page) for x in self.lens]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=g).tolist()
        table = torch.full((n, max(need + [1]) + spare_cols), 1 << 30, dtype=torch.int32)
        table[:, -1] = -7
        pool = torch.full((2, pages, page, heads_k, D), math.nan if poison else 0.0)
        self.exp = torch.full((2, pages, heads_k, page), 200 if poison else 0, dtype=torch.uint8)
        self.k, self.v = [], []  # what each sequence's cache holds, fp64
        for b in range(n):
            mine = [order.pop() for _ in range(need[b])]
            table[b, :need[b]] = torch.tensor(mine, dtype=torch.int32)
            for w, to in ((0, self.k), (1, self.v)):
                x = torch.randn(self.lens[b], heads_k, D, generator=g)
                x *= torch.exp2(torch.randn(self.lens[b], heads_k, 1, generator=g))
                x = x.to(dtype)
                vals, exps = quantise(x) if fp8 else (x.double(), None)
                to.append(vals)
                for j in range(self.lens[b]):
                    at = (mine[j // page], j % page)
                    if fp8:
                        pool[w, at[0], at[1]] = torch.ldexp(
                            vals[j], 127 - exps[j].int()[:, None]).float()
                        self.exp[w, at[0], :, at[1]] = exps[j]
                    else:
                        pool[w, at[0], at[1]] = vals[j].float()
        self.pool = pool.to(E4M3 if fp8 else dtype)
        self.table = table
        self.total = sum(self.rows) + tail
        self.cu = torch.tensor([0] + self.rows).cumsum(0).to(torch.int32)
        self.len_t = torch.tensor(self.lens, dtype=torch.int32)

    def gpu(self):
        d = lambda t: t.cuda()  # noqa: E731
        kw = dict(k_exp=d(self.exp[0]), v_exp=d(self.exp[1])) if self.fp8 else {}
        pool = self.pool.view(torch.uint8).cuda().view(self.pool.dtype) if self.fp8 else self.pool.cuda()
        return pool[0], pool[1], d(self.table), d(self.cu), d(self.len_t), kw


def attention(batch, q, scale, causal=True, window=(-1, -1), slopes=None):
    """For packed q (total, H, D) in fp64: o (rows, H, D), lse (H, rows), A =
    sum_j P |v| + 2^-20 sum_j |v| over the keys a row sees (16-bit weights are
    rounded relatively down to 2^-20 of the largest at least, and by a share of
    that below), S = the largest sum_d |scale q_d k_d| + |bias| of a row."""
    H, G = q.shape[1], q.shape[1] // batch.heads_k
    os_, ls, As, Ss, at = [], [], [], [], 0
    for b, n in enumerate(batch.rows):
        L = batch.lens[b]
        x = q[at:at + n].double()
        at += n
        k, v = batch.k[b].repeat_interleave(G, 1), batch.v[b].repeat_interleave(G, 1)
        pos = L - n + torch.arange(n)
        d = torch.arange(L)[None, :] - pos[:, None]
        z = torch.einsum("ihd,jhd->hij", x, k) * scale
        mag = torch.einsum("ihd,jhd->hij", x.abs(), k.abs()) * abs(scale)
        if slopes is not None:
            sl = (slopes if slopes.dim() == 1 else slopes[b]).double()
            z = z - sl[:, None, None] * d.abs()
            mag = mag + sl.abs()[:, None, None] * d.abs()
        seen = torch.ones_like(d, dtype=torch.bool)
        if causal:
            seen &= d <= 0
        if window[0] >= 0:
            seen &= d >= -window[0]
        if window[1] >= 0:
            seen &= d <= window[1]
        z = z.masked_fill(~seen, -math.inf)
        lse = torch.logsumexp(z, -1) if L else torch.full((H, n), -math.inf, dtype=torch.float64)
        p = torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)[..., None])
        os_.append(torch.einsum("hij,jhd->ihd", p, v))
        weak = p + 2.0 ** -20 * seen * (lse > -math.inf)[..., None]
        As.append(torch.einsum("hij,jhd->ihd", weak, v.abs()))
        Ss.append(mag.masked_fill(~seen, 0.0).amax(-1) if L else torch.zeros(H, n).double())
        ls.append(lse)
    return torch.cat(os_), torch.cat(ls, 1), torch.cat(As), torch.cat(Ss, 1)


def attention_bounds(o, lse, A, S, dtype, p_eps, D):
    """How far o and lse may be off.  Scores: fp32 sums of D products and the
    scaling, each off by (D + 8) 2^-24 of the magnitudes at most, S; a weight
    then moves by that much relatively, and by 2^-21 for the exponential.  o is
    off by twice that (weights and their sum) and by the weights' rounding to
    16 bits (p_eps), both times A = sum P |v|, and by its own rounding; joining
    pieces adds 2^-20."""
    u = EPS[dtype]
    ds = (D + 8) * 2.0 ** -24 * S + 2.0 ** -21
    per = ds.t()[..., None]
    tol_o = u * o.abs() * 1.01 + (1.01 * p_eps + 2 * per + 2.0 ** -20) * A + 1e-30
    tol_l = ds + 2.0 ** -20 + 2.0 ** -22 * torch.where(torch.isfinite(lse), lse.abs(), 0.0)
    if dtype == torch.float16:
        tol_o = tol_o + 2.0 ** -25  # subnormal results
    return tol_o, tol_l
