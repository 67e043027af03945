"""Attention for sequences that share their first pages against 64 bits, on the GPU."""
import ctypes
import math

import pytest
import torch

import paged_ref as R
from exact_attention_93_gb300 import attention, fattn

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def shared_batch(rows, ctx, groups, Hk, D, page, dtype, fp8, **kw):
    """groups: (first sequence, end, pages in common)."""
    b = R.Batch(rows, ctx, Hk, D, page, dtype, fp8, **kw)
    for lo, hi, pages in groups:
        for i in range(lo + 1, hi):
            b.table[i, :pages] = b.table[lo, :pages]
            n = pages * page
            for x in (b.k, b.v):
                x[i] = torch.cat((x[lo][:n], x[i][n:]))
    return b


def columns(b):
    """Spare columns for a table so wide that keys are walked once for a group: by the width the
    call judges what sharing saves."""
    return (1 << 24) // (len(b.rows) * b.heads_k * b.page)


def widen(b):
    table = torch.full((len(b.rows), b.table.shape[1] + columns(b)), 1 << 30, dtype=torch.int32)
    table[:, :b.table.shape[1]] = b.table
    b.table = table
    return b


def divided(b, H, groups=(0,)):
    """Whether the call walks shared keys once for a group: then it needs room for two parts."""
    n, m, lib = ctypes.c_size_t(), ctypes.c_size_t(), fattn.load()
    args = (len(b.rows), b.total, H, b.heads_k, b.D, b.table.shape[1] * b.page)
    assert lib.fa_fwd_paged_workspace_size(*args, ctypes.byref(n)) == 0
    assert lib.fa_fwd_paged_shared_workspace_size(*args, len(groups), ctypes.byref(m)) == 0
    return m.value > n.value


def tensors(groups):
    cu = [groups[0][0]] + [hi for _, hi, _ in groups] if groups else [0]
    return (torch.tensor(cu, dtype=torch.int32, device="cuda"),
            torch.tensor([p for _, _, p in groups], dtype=torch.int32, device="cuda"))


def queries(b, H, seed=5):
    return torch.randn(b.total, H, b.D, generator=torch.Generator().manual_seed(seed)).to(b.dtype)


def run(b, H, groups, q=None, scale=None):
    q = queries(b, H) if q is None else q
    k, v, table, cu, lens, kw = b.gpu()
    cu_groups, shared = tensors(groups)
    o, lse = attention.flash_attn_paged_func(q.cuda(), k, v, table, cu, lens, softmax_scale=scale,
                                             return_lse=True, cu_groups=cu_groups,
                                             shared_pages=shared, **kw)
    torch.cuda.synchronize()
    return q, o.cpu(), lse.cpu()


def check(b, H, q, o, lse, scale=None):
    n = sum(b.rows)
    ro, rl, A, S = R.attention(b, q[:n], b.D ** -0.5 if scale is None else scale)
    # Weights are 16-bit numbers, fp16 over an e4m3 cache, where those below 2^-18 of the
    # largest are off by 2^-29 of it at most.  Joining the two parts is one more step like
    # the joining of pieces, which the bounds have room for: 2^-20 of A, where two
    # exponentials, a sum and a quotient take 2^-21.
    p_eps = R.EPS[HF if b.fp8 else b.dtype]
    tol_o, tol_l = R.attention_bounds(ro, rl, A, S, b.dtype, p_eps, b.D)
    if b.fp8:
        G = H // b.heads_k
        most = torch.cat([v.abs().sum(0).repeat_interleave(G, 0).expand(r, H, b.D)
                          for v, r in zip(b.v, b.rows)])
        tol_o = tol_o + 2.0 ** -28 * most
    got, gl = o[:n].double(), lse[:, :n].double()
    assert torch.equal(gl == -math.inf, rl == -math.inf)
    fin = torch.isfinite(rl)
    assert ((gl - rl).abs()[fin] <= tol_l[fin]).all(), (gl - rl).abs()[fin].max()
    bad = ~((got - ro).abs() <= tol_o)
    assert not bad.any(), (bad.nonzero()[:5], (got - ro).abs().max())


CASES = [
    # rows, ctx, groups (first, end, pages), heads, heads_k, D, page, dtype, fp8
    ([1, 1], [32, 40], [(0, 2, 2)], 1, 1, 64, 16, BF, False),
    ([1] * 5, [640, 700, 641, 1200, 655], [(0, 5, 40)], 32, 8, 128, 16, BF, False),
    ([1] * 5, [640, 700, 641, 1200, 655], [(0, 5, 40)], 32, 8, 128, 16, BF, True),
    ([1] * 9, [300] * 9, [(1, 4, 9), (4, 8, 4)], 12, 4, 64, 32, HF, False),
    ([1] * 9, [300] * 9, [(1, 4, 9), (4, 8, 4)], 12, 4, 64, 32, HF, True),
    ([3, 0, 9, 1, 5, 2], [520, 600, 530, 512, 900, 513], [(0, 6, 8)], 6, 2, 128, 64, HF, False),
    ([3, 0, 9, 1, 5, 2], [520, 600, 530, 512, 900, 513], [(0, 6, 8)], 6, 2, 128, 64, BF, True),
    ([1] * 40, [2100 + 3 * i for i in range(40)], [(0, 40, 16)], 10, 2, 128, 128, BF, False),
    ([2] * 20, [1030] * 20, [(0, 3, 60), (3, 4, 50), (4, 20, 64)], 8, 8, 64, 16, BF, True),
    ([1, 1, 1, 1], [256, 512, 256, 300], [(0, 1, 1), (1, 4, 1)], 64, 1, 64, 256, HF, False),
    ([1] * 6, [256, 512, 256, 300, 700, 1000], [(0, 6, 1)], 64, 1, 64, 256, HF, False),
    ([1] * 6, [256, 512, 256, 300, 700, 1000], [(0, 6, 1)], 64, 1, 128, 128, BF, True),
    ([17, 30, 8], [400, 401, 402], [(0, 3, 25)], 4, 1, 128, 16, BF, False),
    ([17, 30, 8], [400, 401, 402], [(0, 3, 25)], 4, 1, 128, 16, HF, True),
    ([90, 200, 60], [200, 201, 202], [(0, 3, 12)], 4, 2, 64, 16, BF, False),  # too many rows
]


@pytest.mark.parametrize("wide", [False, True])  # wide tables: shared keys are walked once
@pytest.mark.parametrize("rows,ctx,groups,H,Hk,D,page,dtype,fp8", CASES)
def test_groups(rows, ctx, groups, H, Hk, D, page, dtype, fp8, wide):
    b = shared_batch(rows, ctx, groups, Hk, D, page, dtype, fp8, seed=len(rows) + H)
    if wide:
        widen(b)
    few = sum(rows) * (H // Hk) / len(rows) <= 64
    if not wide or not few or 2 * len(groups) < len(rows):  # (else it pays hardly or not)
        assert divided(b, H, groups) == (wide and few)
    q, o, lse = run(b, H, groups)
    assert fattn.fa_device_error() == fattn.FA_OK
    check(b, H, q, o, lse)
    q, again, lse2 = run(b, H, groups)  # the same bits
    n = sum(rows)
    assert torch.equal(o[:n], again[:n]) and torch.equal(lse[:, :n], lse2[:, :n])


@pytest.mark.parametrize("fp8", [False, True])
def test_long_prefix(fp8):
    b = widen(shared_batch([1] * 12, [20000 + 50 * i for i in range(12)], [(0, 12, 312)], 2, 128, 64,
                           BF, fp8, seed=2))
    assert divided(b, 8)
    q, o, lse = run(b, 8, [(0, 12, 312)])
    check(b, 8, q, o, lse)
    q, o, lse = run(b, 8, [(0, 12, 312)], scale=-0.3)
    check(b, 8, q, o, lse, scale=-0.3)
    q, o, lse = run(b, 8, [(0, 12, 312)], scale=0.0)
    check(b, 8, q, o, lse, scale=0.0)


@pytest.mark.parametrize("fp8", [False, True])
def test_many_sequences_and_short_tables(fp8):
    # units are not cut below 1536 keys, and sharing pays all the same for 1100 of them
    n = 140
    groups = [(0, 100, 60), (100, n, 50)]
    b = shared_batch([1] * n, [960 + i for i in range(n)], groups, 8, 128, 16, BF, fp8, seed=5)
    b.table = b.table[:, :95].contiguous()
    assert divided(b, 16, groups) and b.table.shape[1] * 16 <= 1536
    q, o, lse = run(b, 16, groups)
    check(b, 16, q, o, lse)


def test_no_more_is_shared_than_lies_before_every_new_token():
    # the second sequence's new tokens begin in page 3, whatever is claimed; the third is
    # shorter than its rows; the fourth has no rows and does not count
    b = widen(shared_batch([1, 4, 3, 0], [200, 60, -1, 0], [(0, 2, 3)], 2, 64, 16, BF, False, seed=3))
    assert divided(b, 4)
    for claim in (4, 12, 1 << 20):
        for end in (2, 3, 4):
            q, o, lse = run(b, 4, [(0, end, min(claim, b.table.shape[1]))])
            assert fattn.fa_device_error() == fattn.FA_OK
            check(b, 4, q, o, lse)
    run(b, 4, [(0, 2, 1 << 20)])  # beyond the table: clamped all the same, and recorded
    assert fattn.fa_device_error() == fattn.FA_ERR_INVALID_ARG


def test_groups_of_nothing():
    b = widen(shared_batch([1, 1, 2], [64, 80, 5], [(0, 2, 4)], 2, 64, 16, HF, False, seed=3))
    want = run(b, 4, [])
    check(b, 4, *want)
    for groups in ([(0, 0, 0)], [(3, 3, 4)], [(0, 3, 0)], [(1, 1, 2), (1, 2, 3)], [(0, 1, 4), (1, 3, 0)]):
        q, o, lse = run(b, 4, groups)
        check(b, 4, q, o, lse)
    assert fattn.fa_device_error() == fattn.FA_OK


def call_c(q, o, lse, b, groups):
    lib, total, H, D = fattn.load(), *q.shape
    k, v, table, cu, lens, kw = b.gpu()
    cu_groups, shared = tensors(groups)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    code = {BF: 0, HF: 1, R.E4M3: 3}
    c = R.KvPages(ptr(k), ptr(v), ptr(kw.get("k_exp")), ptr(kw.get("v_exp")), *k.stride()[:3],
                  *v.stride()[:3], *k.shape, code[k.dtype])
    r = R.Ragged(ptr(table), table.stride(0), table.shape[1], ptr(cu), ptr(lens), len(lens), total)
    n = ctypes.c_size_t()
    assert lib.fa_fwd_paged_shared_workspace_size(len(lens), total, H, k.shape[2], D,
                                                  table.shape[1] * k.shape[1], len(groups),
                                                  ctypes.byref(n)) == 0
    ws = torch.full((n.value,), 255, dtype=torch.uint8, device="cuda")
    args = lambda w, size: (ptr(q), *q.stride()[:2], ptr(o), *o.stride()[:2], ptr(lse),  # noqa: E731
                            ctypes.addressof(c), ctypes.addressof(r), ptr(cu_groups), ptr(shared),
                            len(groups), H, D ** -0.5, code[q.dtype], w, size,
                            torch.cuda.current_stream().cuda_stream)
    if n.value:
        assert lib.fa_fwd_paged_shared(*args(ptr(ws), n.value // 2)) == fattn.FA_ERR_INVALID_ARG
        assert lib.fa_fwd_paged_shared(*args(ptr(ws) + 16, n.value)) == fattn.FA_ERR_INVALID_ARG
    assert lib.fa_fwd_paged_shared(*args(ptr(ws) if n.value else None, n.value)) == fattn.FA_OK
    torch.cuda.synchronize()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("wide", [False, True])
def test_rows_behind_the_last_sequence_and_rows_without_keys(fp8, wide):
    groups = [(0, 3, 2), (3, 5, 0)]
    b = shared_batch([1, 1, 2, 4, 1], [40, 33, 32, -2, 0], groups, 2, 128, 16, BF, fp8, seed=2, tail=5)
    if wide:
        widen(b)
    assert divided(b, 4, groups) == wide
    q = queries(b, 4)
    o = torch.full((b.total, 2, 4, 128), 7.0, dtype=BF, device="cuda")[:, 1]  # strided results
    lse = torch.full((4, b.total), 7.0, device="cuda")
    call_c(q.cuda(), o, lse, b, groups)
    assert fattn.fa_device_error() == fattn.FA_OK
    check(b, 4, q, o.cpu(), lse.cpu())
    n = sum(b.rows)
    assert (o[n:] == 7).all() and (lse[:, n:] == 7).all()
    assert (lse[:, 4] == -math.inf).all() and (o[4] == 0).all()


def test_values_that_are_not_finite():
    # a NaN value in the shared part reaches the group and nobody else
    groups = [(0, 2, 2), (2, 4, 2)]
    b = widen(shared_batch([1] * 4, [40] * 4, groups, 1, 64, 16, BF, False, seed=2))
    assert divided(b, 2, groups)
    first = int(b.table[0, 1])
    b.pool[1, first, 3, 0, 5] = math.nan
    q, o, lse = run(b, 2, groups)
    assert torch.isnan(o[:2, :, 5]).all() and not torch.isnan(o[2:]).any()
    assert not torch.isnan(o[:2, :, :5]).any() and torch.isfinite(lse).all()


@pytest.mark.parametrize("bad", ["order", "beyond", "negative", "pages", "table", "length"])
def test_bad_groups_and_tables_are_contained(bad):
    groups = [(0, 2, 3), (2, 4, 3)]
    b = widen(shared_batch([1] * 4, [100] * 4, groups, 2, 64, 16, BF, False, seed=6))
    assert divided(b, 4, groups)
    k, v, table, cu, lens, _ = b.gpu()
    q = queries(b, 4).cuda()
    c, p = tensors(groups)
    call = lambda: attention.flash_attn_paged_func(q, k, v, table, cu, lens, cu_groups=c, shared_pages=p)  # noqa: E731
    good = call()
    if bad == "order":
        c[1] = 4
        c[2] = 3
    elif bad == "beyond":
        c[2] = 1 << 30
    elif bad == "negative":
        c[0] = -1 << 30
    elif bad == "pages":
        p[1] = -1
    elif bad == "table":
        table[2, 1] = k.shape[0]
    else:
        lens[3] = -5
    got = call()
    torch.cuda.synchronize()
    assert fattn.fa_device_error() == fattn.FA_ERR_INVALID_ARG
    if bad in ("table", "length"):
        assert torch.equal(got[:2], good[:2])  # the other group is unharmed
    assert fattn.fa_device_error() == fattn.FA_OK


def test_streams_and_graphs():
    groups = [(0, 6, 20)]
    b = widen(shared_batch([1] * 6, [900, 320, 330, 500, 321, 2500], groups, 4, 128, 16, BF, False, seed=8))
    assert divided(b, 16, groups)
    k, v, table, cu, lens, _ = b.gpu()
    c, p = tensors(groups)
    qs = [queries(b, 16, seed=i).cuda() for i in range(3)]
    call = lambda q: attention.flash_attn_paged_func(q, k, v, table, cu, lens, return_lse=True,  # noqa: E731
                                                     cu_groups=c, shared_pages=p)
    want = [call(q) for q in qs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in qs], []
    for q, st in zip(qs, streams):
        with torch.cuda.stream(st):
            got.append(call(q))
    torch.cuda.synchronize()
    for w, x in zip(want, got):
        assert torch.equal(w[0], x[0]) and torch.equal(w[1], x[1])
    q, graphs = qs[0].clone(), []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = call(q)
        graphs.append((gr, out))
    p.fill_(11)  # less in common than the graphs were captured with
    lens.sub_(torch.tensor([70, 0, 9, 100, 0, 1], device="cuda", dtype=torch.int32))
    for i in (1, 2):
        q.copy_(qs[i])
        for gr, _ in graphs:
            gr.replay()
        fresh = call(q)
        torch.cuda.synchronize()
        for _, out in graphs:
            assert torch.equal(out[0], fresh[0]) and torch.equal(out[1], fresh[1])
    b.lens = lens.tolist()
    b.k, b.v = ([x[:n] for x, n in zip(t, b.lens)] for t in (b.k, b.v))
    check(b, 16, q.cpu(), fresh[0].cpu(), fresh[1].cpu())


def test_refusals():
    groups = [(0, 2, 1)]
    b = shared_batch([1, 1], [40, 50], groups, 2, 64, 16, BF, False)
    k, v, table, cu, lens, _ = b.gpu()
    q = queries(b, 4).cuda()
    c, p = tensors(groups)
    call = lambda **kw: attention.flash_attn_paged_func(q, k, v, table, cu, lens,  # noqa: E731
                                                        **{**dict(cu_groups=c, shared_pages=p), **kw})
    slopes = torch.ones(4, device="cuda")
    for kw in (dict(causal=False), dict(window_size=(5, -1)), dict(window_size=(-1, 0)),
               dict(alibi_slopes=slopes), dict(cu_groups=None), dict(shared_pages=None),
               dict(cu_groups=c.long()), dict(shared_pages=p.long()), dict(cu_groups=c[:1]),
               dict(cu_groups=torch.zeros(4, dtype=torch.int32, device="cuda"),
                    shared_pages=torch.zeros(3, dtype=torch.int32, device="cuda")),
               dict(shared_pages=p.cpu())):
        with pytest.raises(ValueError):
            call(**kw)
