"""The serving calls at the ends of their ranges, on the GPU: gradients and
tangents as autograd hands them over, rows marked as zeros, the smallest and
most different row scales of an e4m3 cache, rows without keys, scales of zero
and below, many query heads to a key head, infinities and NaN in visible places."""
import math

import pytest
import torch

import paged_ref as R
from exact_attention_93_gb300 import attention, fattn, kvcache, rotary

pytestmark = pytest.mark.gpu
BF, HF, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def slot(b, s, j):
    """Where key j of sequence s of a batch lives."""
    return int(b.table[s, j // b.page]), j % b.page


def refresh(b):
    """The batch's 64-bit keys and values, read anew from an e4m3 cache's bytes."""
    for w, to in ((0, b.k), (1, b.v)):
        for s, n in enumerate(b.lens):
            pages = b.table[s, :-(-n // b.page)].long()
            e = b.exp[w][pages].permute(0, 2, 1).flatten(0, 1)[:n, :, None]
            code = b.pool[w].view(torch.uint8)[pages].view(E4).float().double().flatten(0, 1)[:n]
            to[s] = torch.where(e > 0, torch.ldexp(code, e.int() - 127), 0.0)


def shift_exponents(b, w, s, by):
    """Adds by (keys,) to the exponent bytes of the keys' (w = 0) or values' (w = 1) rows."""
    for j in range(b.lens[s]):
        pg, off = slot(b, s, j)
        e = b.exp[w, pg, :, off].int()
        b.exp[w, pg, :, off] = torch.where(e > 0, (e + int(by[j])).clamp(1, 248), 0).to(torch.uint8)


def queries(b, H, seed=5, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(b.total, H, b.D, generator=g) * scale).to(b.dtype)


def attend(b, q, *, scale=None, causal=True, window=(-1, -1), slopes=None, error=fattn.FA_OK):
    k, v, table, cu, lens, kw = b.gpu()
    o, lse = attention.flash_attn_paged_func(q.cuda(), k, v, table, cu, lens, softmax_scale=scale,
                                             causal=causal, window_size=window, alibi_slopes=slopes,
                                             return_lse=True, **kw)
    torch.cuda.synchronize()
    assert fattn.fa_device_error() == error
    return o.cpu(), lse.cpu()


def reference(b, q, scale, causal=True, window=(-1, -1), without=None):
    """o, lse in 64 bits, and how far each may be off; without: a (sequence, key, key
    head) left out.

    Scores are fp32 sums of D products, scaled: off by (D + 8) 2^-24 of S, the
    largest sum of magnitudes, and the exponential by 2^-21; o takes that twice
    (weights and their sum) times A = sum P |v|.  Weights in bf16 are off by 2^-8
    of themselves; in fp16 by 2^-11, and below 2^-18 of the largest by 2^-29 of it
    at most.  Joining, and the sums, 2^-20.  Over an e4m3 cache, R being a
    sequence's largest exponent byte:
      few rows: weight * 2^(e - R) below 2^-29 is off by 2^-40 at most, that is
        by 448 * 2^(R - 127) * 2^-40 of a value;
      many rows: keys and values below 2^(R - 22) are off by 2^-32 * 2^(R - 127),
        those of 2^(R - 32) and below are zeros."""
    H, G = q.shape[1], q.shape[1] // b.heads_k
    few = b.total * G <= 16 * len(b.rows)
    fp16 = b.fp8 or b.dtype == HF
    os_, ls, tos, tls, at = [], [], [], [], 0
    for s, n in enumerate(b.rows):
        L = b.lens[s]
        x = q[at:at + n].double()
        at += n
        k, v = b.k[s].repeat_interleave(G, 1), b.v[s].repeat_interleave(G, 1)
        left_out = torch.zeros(H, 1, L, dtype=torch.bool)
        if without and without[0] == s:
            left_out[without[2] * G:(without[2] + 1) * G, :, without[1]] = True
            k = k.masked_fill(left_out[:, 0].t()[..., None], 0.0)
        d = torch.arange(L)[None, :] - (L - n + torch.arange(n))[:, None]
        seen = torch.ones_like(d, dtype=torch.bool)
        if causal:
            seen &= d <= 0
        if window[0] >= 0:
            seen &= d >= -window[0]
        if window[1] >= 0:
            seen &= d <= window[1]
        z = (torch.einsum("ihd,jhd->hij", x, k) * scale).masked_fill(~seen | left_out, -math.inf)
        lse = torch.logsumexp(z, -1) if L else torch.full((H, n), -math.inf, dtype=torch.float64)
        p = torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)[..., None])
        o = torch.einsum("hij,jhd->ihd", p, v)
        ev, ek = torch.zeros_like(v), torch.zeros_like(k)  # errors of the operands
        flat = 0.0                                         # of each value that is seen
        if b.fp8 and L:
            e = [torch.stack([b.exp[w, slot(b, s, j)[0], :, slot(b, s, j)[1]] for j in range(L)])
                 .int().repeat_interleave(G, 1)[..., None] for w in (0, 1)]
            top = [int(t.max()) for t in e]
            if few:
                flat = 448 * 2.0 ** (top[1] - 127 - 40)
            else:
                for t, err, val, R_ in zip(e, (ek, ev), (k, v), top):
                    low = torch.where(t <= R_ - 22, 2.0 ** (R_ - 127 - 32), 0.0)
                    err += torch.where(t <= R_ - 32, val.abs(), low)
        mag = torch.einsum("ihd,jhd->hij", x.abs(), k.abs()) * abs(scale)
        off = torch.einsum("ihd,jhd->hij", x.abs(), ek) * abs(scale)
        S, dk = (t.masked_fill(~seen, 0.0).amax(-1) if L else torch.zeros(H, n).double()
                 for t in (mag, off))
        ds = (b.D + 8) * 2.0 ** -24 * S + 2.0 ** -21 + dk
        A = torch.einsum("hij,jhd->ihd", p, v.abs())
        some = torch.einsum("hij,jhd->ihd", seen.double().expand_as(p), v.abs())
        count = seen.sum(-1).double()[:, None, None]
        u, p_eps = R.EPS[b.dtype], 2.0 ** -11 if fp16 else 2.0 ** -8
        tos.append(1.01 * u * o.abs() + (1.01 * p_eps + 2 * ds.t()[..., None] + 2.0 ** -20) * A
                   + (2.0 ** -29 if fp16 else 0.0) * some + count * flat
                   + torch.einsum("hij,jhd->ihd", p, ev)
                   + (2.0 ** -133 if b.dtype == BF else 2.0 ** -24))
        tls.append(ds + 2.0 ** -20 + 2.0 ** -22 * torch.where(torch.isfinite(lse), lse.abs(), 0.0))
        os_.append(o)
        ls.append(lse)
    return torch.cat(os_), torch.cat(ls, 1), torch.cat(tos), torch.cat(tls, 1)


def compare(b, q, o, lse, scale=None, **kw):
    ro, rl, to, tl = reference(b, q[:sum(b.rows)], b.D ** -0.5 if scale is None else scale, **kw)
    n = sum(b.rows)
    o, lse = o[:n].double(), lse[:, :n].double()
    assert torch.equal(lse == -math.inf, rl == -math.inf)
    fin = torch.isfinite(rl)
    assert ((lse - rl).abs()[fin] <= tl[fin]).all(), (lse - rl).abs()[fin].max()
    bad = ~((o - ro).abs() <= to)
    assert not bad.any(), (bad.nonzero()[:5], ((o - ro).abs() / to).nan_to_num(9e9).max())


# ---- tangents and gradients

def test_forward_mode_is_refused():
    """A tangent is never dropped: each call that has none to give refuses its input."""
    freq, _ = rotary.rotary_frequencies(64)
    x, t = torch.randn(2, 3, 9, 2, 64, device="cuda").to(BF)
    b = R.Batch([3, 2], [5, 0], 2, 64, 16, BF, False)
    k, v, table, cu, lens, _ = b.gpu()
    q = queries(b, 4).cuda()
    new = torch.randn(5, 2, 64, device="cuda").to(BF)
    keep = k.clone()
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual
        for grad in (torch.enable_grad(), torch.no_grad()):
            with grad:
                for call in (
                        lambda: rotary.rotary_func(dual(x, t), None, freq),
                        lambda: rotary.rotary_func(x, dual(x, t), freq),
                        lambda: rotary.rotary_func(dual(x, t), None, freq, inplace=True),
                        lambda: rotary.rotary_func(x, None, dual(freq, freq)),
                        lambda: attention.flash_attn_paged_func(dual(q, q), k, v, table, cu, lens),
                        lambda: attention.flash_attn_paged_func(q, dual(k, k), v, table, cu, lens),
                        lambda: kvcache.kv_cache_append(dual(new, new), new, k, v, table, cu, lens),
                        lambda: kvcache.kv_cache_append(new, new, k, dual(v, v), table, cu, lens),
                        lambda: kvcache.kv_cache_read(dual(k, k), v, table, cu, 5)):
                    with pytest.raises(NotImplementedError):
                        call()
    assert torch.equal(k.view(torch.int16), keep.view(torch.int16))
    rotary.rotary_func(x, x, freq)  # and without tangents it runs
    # a gradient that carries a tangent
    y = rotary.rotary_func(x.requires_grad_(), None, freq)
    with torch.autograd.forward_ad.dual_level():
        for create in (False, True):
            with pytest.raises(NotImplementedError):
                torch.autograd.grad(y, (x,), (dual(t, t),), create_graph=create, retain_graph=True)


# ---- rows marked as zeros

@pytest.mark.parametrize("D,H,Hk,dtype", [(128, 8, 2, BF), (64, 6, 6, HF), (64, 16, 2, BF)])
@pytest.mark.parametrize("rows,spare", [([1, 1, 1], 2), ([1, 2, 2], 200), ([40, 3, 140], 2),
                                        ([40, 3, 140], 200)])
def test_rows_marked_as_zeros(D, H, Hk, dtype, rows, spare):
    """e = 0 makes a row of zeros, whatever codes lie under it."""
    b = R.Batch(rows, [300, 20, 1000], Hk, D, 16, dtype, True, seed=D + H, spare_cols=spare)
    g = torch.Generator().manual_seed(1)
    for w in range(2):
        for s, n in enumerate(b.lens):
            for j in range(n):
                pg, off = slot(b, s, j)
                none = torch.rand(Hk, generator=g) < (1.0 if s == 1 else 0.2)
                b.exp[w, pg, none, off] = 0
                b.pool[w].view(torch.uint8)[pg, off, none] = 0x7f  # NaN
    refresh(b)
    q = queries(b, H)
    o, lse = attend(b, q)
    compare(b, q, o, lse)
    assert (o[rows[0]:rows[0] + rows[1]] == 0).all()


# ---- the smallest row scales

@pytest.mark.parametrize("top", [1, 9, 15, 30])
@pytest.mark.parametrize("D,H,Hk", [(128, 8, 2), (64, 6, 6)])
@pytest.mark.parametrize("rows,spare", [([1, 1, 1], 2), ([1, 2, 2], 200), ([40, 3, 140], 2),
                                        ([40, 3, 140], 200)])
def test_smallest_value_scales(top, D, H, Hk, rows, spare):
    """Values near 2^-117 and up come out as such, not as zeros."""
    b = R.Batch(rows, [300, 20, 1000], Hk, D, 32, BF, True, seed=D, spare_cols=spare)
    for s, n in enumerate(b.lens):
        most = max(int(b.exp[1, slot(b, s, j)[0], :, slot(b, s, j)[1]].max()) for j in range(n))
        shift_exponents(b, 1, s, [top - most] * n)
    refresh(b)
    q = queries(b, H)
    o, lse = attend(b, q)
    compare(b, q, o, lse)
    assert (o != 0).any()


@pytest.mark.parametrize("top", [4, 20])
@pytest.mark.parametrize("rows,spare", [([1, 2, 2], 2), ([40, 3, 140], 200)])
@pytest.mark.parametrize("D,H,Hk", [(128, 8, 2), (64, 6, 6)])
def test_smallest_key_scales_under_the_largest_queries(top, D, H, Hk, rows, spare):
    b = R.Batch(rows, [300, 20, 1000], Hk, D, 32, BF, True, seed=D, spare_cols=spare)
    for s, n in enumerate(b.lens):
        most = max(int(b.exp[0, slot(b, s, j)[0], :, slot(b, s, j)[1]].max()) for j in range(n))
        shift_exponents(b, 0, s, [top - most] * n)
    refresh(b)
    q = queries(b, H, scale=2.0 ** (119 - top))  # scores of a few units
    o, lse = attend(b, q)
    compare(b, q, o, lse)


# ---- rows without keys

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,rows,spare", [(64, [3, 1], 2), (128, [2, 1], 200), (64, [90, 40], 2),
                                          (128, [90, 40], 200)])
def test_rows_without_keys_beside_values_that_are_not_finite(fp8, D, rows, spare):
    """A row that sees no key gets zeros, also where rows of its block see a NaN."""
    b = R.Batch(rows, [-1, 40], 2, D, 16, BF, fp8, spare_cols=spare)
    pg, off = slot(b, 0, 0)
    if fp8:
        b.pool[1].view(torch.uint8)[pg, off] = 0x7f
    else:
        b.pool[1, pg, off] = math.nan
    o, lse = attend(b, queries(b, 4))
    assert (o[0] == 0).all() and (lse[:, 0] == -math.inf).all()
    assert torch.isnan(o[1:rows[0]]).all() and torch.isfinite(lse[:, 1:]).all()
    assert torch.isfinite(o[rows[0]:]).all()


# ---- gradients at addresses that are no multiple of 16

def misaligned(shape, dtype):
    n = math.prod(shape)
    t = torch.randn(n + 1, device="cuda").to(dtype)[1:].view(shape)
    assert t.is_contiguous() and t.data_ptr() % 16
    return t


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_misaligned_gradient_of_rotary(dtype):
    freq, _ = rotary.rotary_frequencies(64)
    x, z = (torch.randn(2, 9, h, 64, device="cuda").to(dtype).requires_grad_() for h in (3, 1))
    y, u = rotary.rotary_func(x, z, freq)
    dy, du = misaligned(y.shape, dtype), misaligned(u.shape, dtype)
    want = torch.autograd.grad((y, u), (x, z), (dy.clone(), du.clone()), retain_graph=True)
    got = torch.autograd.grad((y, u), (x, z), (dy, du), retain_graph=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # as a join behind an odd offset leaves it
    one = torch.ones(1, device="cuda", dtype=dtype)
    w = torch.randn(1 + y.numel(), device="cuda").to(dtype)
    gx, = torch.autograd.grad((torch.cat((one, y.flatten())) * w).sum(), (x,), retain_graph=True)
    wx, = torch.autograd.grad(y, (x,), (w[1:].clone().view_as(y),))
    assert torch.equal(gx, wx)


def test_misaligned_gradient_of_dense_attention():
    q, k, v = (torch.randn(1, 200, 2, 64, device="cuda").to(BF).requires_grad_() for _ in range(3))
    o = attention.flash_attn_func(q, k, v, causal=True, deterministic=True)
    do = misaligned(o.shape, BF)
    want = torch.autograd.grad(o, (q, k, v), (do.clone(),), retain_graph=True)
    got = torch.autograd.grad(o, (q, k, v), (do,))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# ---- no tokens

@pytest.mark.parametrize("shape,pos", [((2, 0, 4, 64), (0,)), ((2, 0, 4, 64), (2, 0)),
                                       ((0, 5, 4, 64), (0, 5)), ((0, 4, 64), (0,))])
@pytest.mark.parametrize("bits", [torch.int32, torch.int64])
def test_rotary_of_no_tokens_with_positions(shape, pos, bits):
    freq, _ = rotary.rotary_frequencies(64)
    x = torch.zeros(shape, device="cuda", requires_grad=True)
    p = torch.zeros(pos, dtype=bits, device="cuda")
    y = rotary.rotary_func(x, None, freq, positions=p)
    assert y.shape == x.shape
    gx, = torch.autograd.grad(y.sum(), (x,))
    assert gx.shape == x.shape
    with torch.no_grad():
        assert rotary.rotary_func(x, x, freq, positions=p)[1].shape == x.shape


# ---- row scales that differ

def climbs(n, kind):
    """Exponents added to the rows of n keys, tile by tile of 128."""
    tile = torch.arange(n) // 128
    if kind == "up 5":
        return tile * 5
    if kind == "up 12":
        return (tile * 12).clamp(max=60)
    if kind == "up 20":
        return (tile * 20).clamp(max=80)
    if kind == "down":
        return 60 - (tile * 12).clamp(max=60)
    if kind == "last":
        return torch.where(torch.arange(n) == n - 1, 25, 0)
    return (tile * 7) % 40  # up and down


@pytest.mark.parametrize("kind", ["up 5", "up 12", "up 20", "down", "last", "both ways"])
@pytest.mark.parametrize("D,H,Hk,dtype", [(128, 8, 2, BF), (64, 6, 6, BF), (128, 4, 4, HF)])
@pytest.mark.parametrize("rows,spare", [([1, 1, 1], 2), ([1, 2, 2], 200), ([40, 3, 140], 2),
                                        ([40, 3, 140], 200)])
def test_value_scales_that_climb_and_fall(kind, D, H, Hk, dtype, rows, spare):
    b = R.Batch(rows, [900, 20, 1300], Hk, D, 64, dtype, True, seed=D, spare_cols=spare)
    for s, n in enumerate(b.lens):
        shift_exponents(b, 1, s, climbs(n, kind) - 70 * (dtype == HF))
    refresh(b)
    q = queries(b, H)
    compare(b, q, *attend(b, q))
    window = (300, 0)  # the largest rows are hidden from some queries
    compare(b, q, *attend(b, q, causal=False, window=window), causal=False, window=window)


@pytest.mark.parametrize("kind", ["up 5", "down", "last", "both ways"])
@pytest.mark.parametrize("D,H,Hk", [(128, 8, 2), (64, 6, 6)])
@pytest.mark.parametrize("rows,spare", [([1, 2, 2], 2), ([40, 3, 140], 200)])
def test_key_scales_that_climb_and_fall(kind, D, H, Hk, rows, spare):
    b = R.Batch(rows, [900, 20, 1300], Hk, D, 64, BF, True, seed=D, spare_cols=spare)
    for s, n in enumerate(b.lens):
        shift_exponents(b, 0, s, climbs(n, kind))
    refresh(b)
    q = queries(b, H)
    scale = D ** -0.5 * 2.0 ** -int(climbs(max(b.lens), kind).max())
    compare(b, q, *attend(b, q, scale=scale), scale=scale)


@pytest.mark.parametrize("below", [15, 22, 27, 31, 32, 40])
@pytest.mark.parametrize("D,H,Hk", [(128, 8, 2), (64, 6, 6)])
@pytest.mark.parametrize("rows", [[1, 2, 2], [40, 3, 140]])
def test_one_row_far_above_the_others(below, D, H, Hk, rows):
    """Keys and values 2^below under one row, which has next to no weight."""
    b = R.Batch(rows, [300, 20, 1000], Hk, D, 64, BF, True, seed=D)
    q = queries(b, H)
    for s, n in enumerate(b.lens):
        by = torch.full((n,), -below)
        by[0] = 0
        shift_exponents(b, 1, s, by)
        pg, off = slot(b, s, 0)  # key 0: -112 in column 0, where the queries hold 4
        b.pool[0].view(torch.uint8)[pg, off, :, 0] = 0xfe
        b.exp[0, pg, :, off] = 125
    q[:, :, 0] = 4
    refresh(b)
    compare(b, q, *attend(b, q))


@pytest.mark.parametrize("first", [1, 128, 200])
@pytest.mark.parametrize("rows,spare", [([1, 2, 2], 200), ([40, 3, 140], 2), ([40, 3, 140], 200)])
@pytest.mark.parametrize("D,H,Hk", [(128, 8, 2), (64, 6, 6)])
def test_zeros_first(first, rows, spare, D, H, Hk):
    b = R.Batch(rows, [900, 200, 1300], Hk, D, 16, BF, True, seed=D, spare_cols=spare)
    for w in range(2):
        for s in range(3):
            for j in range(min(first, b.lens[s])):
                pg, off = slot(b, s, j)
                b.exp[w, pg, :, off] = 0
                b.pool[w].view(torch.uint8)[pg, off] = 0
    refresh(b)
    q = queries(b, H)
    compare(b, q, *attend(b, q))


# ---- weights over an e4m3 cache are fp16 for any number of rows

@pytest.mark.parametrize("rows,ctx,H,Hk,D", [([33, 1, 64], [5, 900, 64], 3, 1, 128),
                                             ([300, 5, 129], [1000, 150, 0], 8, 2, 64),
                                             ([700, 300], [0, 650], 16, 4, 128)])
def test_weights_of_many_rows_over_e4m3(rows, ctx, H, Hk, D):
    b = R.Batch(rows, ctx, Hk, D, 32, BF, True, seed=4)
    q = queries(b, H)
    compare(b, q, *attend(b, q))


# ---- scales, heads, pages

@pytest.mark.parametrize("scale", [0.0, -0.0, -0.2, 1.5])
@pytest.mark.parametrize("fp8,D,dtype", [(False, 128, BF), (True, 64, BF), (False, 64, HF),
                                         (True, 128, HF)])
@pytest.mark.parametrize("rows,spare", [([1, 2, 1], 200), ([60, 1, 200], 2), ([60, 1, 200], 200)])
def test_softmax_scales(scale, fp8, D, dtype, rows, spare):
    b = R.Batch(rows, [900, 0, 300], 2, D, 32, dtype, fp8, seed=3, spare_cols=spare)
    q = queries(b, 8)
    compare(b, q, *attend(b, q, scale=scale), scale=scale)
    window = (150, 3)
    compare(b, q, *attend(b, q, scale=scale, causal=False, window=window), scale=scale,
            causal=False, window=window)


@pytest.mark.parametrize("group", [17, 24, 40, 64, 65, 100, 127, 128])
@pytest.mark.parametrize("fp8,D,Hk", [(False, 128, 1), (True, 64, 2), (False, 64, 2),
                                      (True, 128, 1)])
@pytest.mark.parametrize("rows,spare", [([1, 1, 1], 2), ([1, 0, 2], 200), ([9, 40, 1], 200)])
def test_many_heads_to_a_key_head(group, fp8, D, Hk, rows, spare):
    b = R.Batch(rows, [700, 0, 130], Hk, D, 16, BF, fp8, seed=group, tail=2, spare_cols=spare)
    q = queries(b, group * Hk)
    compare(b, q, *attend(b, q))
    window = (50, -1)
    compare(b, q, *attend(b, q, window=window), window=window)


def test_sequences_that_share_pages():
    """A common beginning lies in the cache once; single tokens and chunks read it."""
    for rows in ([1, 1, 1], [70, 3, 30]):
        b = R.Batch(rows, [400, 400, 400], 2, 64, 16, BF, False, seed=2)
        shared = 320  # keys
        for s in (1, 2):
            b.table[s, :shared // 16] = b.table[0, :shared // 16]
            b.k[s][:shared], b.v[s][:shared] = b.k[0][:shared], b.v[0][:shared]
        q = queries(b, 8)
        compare(b, q, *attend(b, q))


@pytest.mark.parametrize("dtype", [BF, E4])
def test_offsets_beyond_32_bits(dtype):
    """A cache of more than 2^32 elements: its last pages are written, read and attended to."""
    Hk, D, page = 8, 128, 256
    pages = (1 << 32) // (Hk * D * page) + 40
    cache = kvcache.alloc_kv_cache(pages, page, Hk, D, dtype)
    kp, vp, ke, ve = cache
    kw = dict(k_exp=ke, v_exp=ve)
    b = R.Batch([300, 1, 2], [0, 600, 20], Hk, D, page, BF, False, seed=1, poison=False)
    table = (pages - 1 - b.table.clamp(0, 30)).cuda()
    cu = torch.tensor([0] + b.lens).cumsum(0).to(torch.int32).cuda()
    lens = b.len_t.cuda()
    k, v = (torch.cat(t).to(BF).cuda() for t in (b.k, b.v))
    kvcache.kv_cache_append(k, v, kp, vp, table, cu, lens, **kw)
    kr, vr = kvcache.kv_cache_read(kp, vp, table, cu, sum(b.lens), **kw)
    want = [R.quantise(t.cpu())[0].to(BF) if dtype == E4 else t.cpu() for t in (k, v)]
    assert torch.equal(kr.cpu(), want[0]) and torch.equal(vr.cpu(), want[1])
    b.k, b.v = (list(t.double().split(b.lens)) for t in want)
    for rows in ([300, 1, 2], [1, 1, 1]):
        b.rows, b.total = rows, sum(rows)
        q = queries(b, 16)
        o = attention.flash_attn_paged_func(q.cuda(), kp, vp, table, torch.tensor(
            [0] + rows).cumsum(0).to(torch.int32).cuda(), lens, **kw).cpu()
        ref, lse, A, S = R.attention(b, q, D ** -0.5)
        tol, _ = R.attention_bounds(ref, lse, A, S, BF, R.EPS[BF], D)
        assert ((o.double() - ref).abs() <= tol).all()
    assert fattn.fa_device_error() == fattn.FA_OK


# ---- infinities and NaN that are visible

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,rows,spare", [(128, [1, 1, 2], 2), (64, [1, 1, 2], 200),
                                          (128, [70, 3, 200], 2), (64, [70, 3, 200], 200)])
def test_values_that_are_not_finite(fp8, D, rows, spare):
    b = R.Batch(rows, [300, 20, 1000], 2, D, 16, BF, fp8, seed=6, spare_cols=spare)
    q = queries(b, 8)
    clean, clean_lse = attend(b, q)
    # NaN in column 5 of key 250 of sequence 0, key head 1; infinity in column 9
    pg, off = slot(b, 0, 250)
    if fp8:
        b.pool[1].view(torch.uint8)[pg, off, 1, 5] = 0x7f
    else:
        b.pool[1, pg, off, 1, 5] = math.nan
        b.pool[1, pg, off, 1, 9] = -math.inf
    o, lse = attend(b, q)
    n = rows[0]
    assert torch.equal(lse, clean_lse)
    assert torch.isnan(o[:n, 4:, 5]).all()
    if not fp8:
        assert (o[:n, 4:, 9] == -math.inf).all()
    o[:n, 4:, 5], o[:n, 4:, 9] = clean[:n, 4:, 5], clean[:n, 4:, 9]
    assert torch.equal(o, clean)


@pytest.mark.parametrize("what", ["nan", "inf"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,rows,spare", [(128, [3, 1, 2], 2), (64, [3, 1, 1], 200),
                                          (128, [70, 3, 200], 2), (64, [70, 3, 200], 200)])
def test_keys_that_are_not_finite(what, fp8, D, rows, spare):
    if fp8 and what == "inf":
        return  # e4m3 has none
    b = R.Batch(rows, [300, 20, 1000], 2, D, 16, BF, fp8, seed=6, spare_cols=spare)
    q = queries(b, 8)
    clean, clean_lse = attend(b, q)
    n, at = rows[0], b.lens[0] - rows[0] + rows[0] // 2  # visible to the last rows alone
    pg, off = slot(b, 0, at)
    if fp8:
        b.pool[0].view(torch.uint8)[pg, off, 1, 5] = 0x7f
    else:
        b.pool[0, pg, off, 1, 5] = math.nan if what == "nan" else math.inf
    o, lse = attend(b, q)
    see = torch.zeros(b.total, 8, dtype=torch.bool)
    see[rows[0] // 2:n, 4:] = True
    if what == "inf":  # a score of -inf is a weight of zero, one of +inf makes NaN
        up = q[:, :, 5] > 0
        ro, rl, to, tl = reference(b, q, D ** -0.5, without=(0, at, 1))
        low = see & ~up
        assert ((o.double() - ro).abs() <= to)[low].all()
        assert ((lse.double() - rl).abs() <= tl)[low.t()].all()
        see_nan = see & up
    else:
        see_nan = see
        assert torch.isnan(lse[see.t()]).all()
    assert torch.isnan(o[see_nan]).all()
    assert torch.equal(o[~see], clean[~see]) and torch.equal(lse[~see.t()], clean_lse[~see.t()])


@pytest.mark.parametrize("fp8,D", [(False, 128), (True, 64), (True, 128)])
@pytest.mark.parametrize("rows,spare", [([3, 1, 2], 200), ([70, 3, 200], 2)])
def test_queries_that_are_not_finite(fp8, D, rows, spare):
    b = R.Batch(rows, [300, 20, 1000], 2, D, 16, BF, fp8, seed=6, spare_cols=spare)
    q = queries(b, 8)
    clean, clean_lse = attend(b, q)
    bad = torch.zeros(b.total, 8, dtype=torch.bool)
    for token, head, value in ((0, 0, math.nan), (1, 5, math.inf), (rows[0], 7, -math.inf)):
        q[token, head, 3] = value
        bad[token, head] = True
    o, lse = attend(b, q)
    assert torch.isnan(o[bad]).all()
    assert torch.equal(o[~bad], clean[~bad]) and torch.equal(lse[~bad.t()], clean_lse[~bad.t()])
