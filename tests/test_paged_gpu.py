"""Attention of new tokens over a paged cache against 64 bits, on the GPU."""
import ctypes
import math

import pytest
import torch

import paged_ref as R
from exact_attention_93_gb300 import attention, fattn

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def run(batch, H, *, causal=True, window=(-1, -1), slopes=None, seed=5, scale=None):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(batch.total, H, batch.D, generator=g).to(batch.dtype)
    k, v, table, cu, lens, kw = batch.gpu()
    o, lse = attention.flash_attn_paged_func(
        q.cuda(), k, v, table, cu, lens, causal=causal, window_size=window, softmax_scale=scale,
        alibi_slopes=None if slopes is None else slopes.cuda(), return_lse=True, **kw)
    torch.cuda.synchronize()
    assert fattn_error() == fattn.FA_OK
    return q, o.cpu(), lse.cpu()


def fattn_error():
    return fattn.fa_device_error()


def check(batch, H, q, o, lse, *, causal=True, window=(-1, -1), slopes=None, scale=None):
    scale = batch.D ** -0.5 if scale is None else scale
    n = sum(batch.rows)
    ro, rl, A, S = R.attention(batch, q[:n], scale, causal, window, slopes)
    # 16-bit weights: fp16 under an e4m3 cache, else the type of q
    p_eps = R.EPS[HF if batch.fp8 and n * H // batch.heads_k <= 32 * len(batch.rows)
                  else batch.dtype]
    tol_o, tol_l = R.attention_bounds(ro, rl, A, S, batch.dtype, p_eps, batch.D)
    got, gl = o[:n].double(), lse[:, :n].double()
    assert torch.equal(gl == -math.inf, rl == -math.inf)
    fin = torch.isfinite(rl)
    assert ((gl - rl).abs()[fin] <= tol_l[fin]).all(), (gl - rl).abs()[fin].max()
    bad = ~((got - ro).abs() <= tol_o)
    assert not bad.any(), (bad.nonzero()[:5], (got - ro).abs().max())


CASES = [
    # rows, ctx, heads, heads_k, D, page, dtype, fp8
    ([1], [0], 1, 1, 64, 16, BF, False),
    ([1], [999], 32, 8, 128, 16, BF, False),
    ([1, 1, 1], [0, 127, 128], 8, 8, 128, 32, HF, False),
    ([1] * 7, [5, 300, 1, 0, 2000, 128, 63], 16, 2, 128, 64, BF, True),
    ([1] * 5, [700, 31, 32, 33, 1500], 12, 4, 64, 128, HF, True),
    ([1, 1], [4000, 77], 5, 1, 64, 256, BF, False),
    ([2, 5, 0, 3], [100, 0, 50, 1000], 8, 2, 128, 16, HF, False),
    ([4, 1, 7], [260, 511, 13], 16, 4, 64, 16, BF, True),
    ([8, 16], [130, 0], 6, 2, 128, 256, BF, False),
    ([33, 1, 64], [5, 900, 64], 3, 1, 128, 32, BF, True),
    ([130, 3], [0, 400], 4, 2, 64, 64, HF, False),
    ([1], [20000], 16, 1, 128, 128, BF, True),
    ([1], [20000], 8, 1, 64, 64, HF, False),
    ([257, 100], [300, 0], 8, 1, 128, 16, HF, True),
]


@pytest.mark.parametrize("wide", [False, True])  # wide tables: work may be cut and joined
@pytest.mark.parametrize("rows,ctx,H,Hk,D,page,dtype,fp8", CASES)
def test_causal(rows, ctx, H, Hk, D, page, dtype, fp8, wide):
    b = R.Batch(rows, ctx, Hk, D, page, dtype, fp8, seed=len(rows) + H,
                spare_cols=200 if wide else 2)
    q, o, lse = run(b, H)
    check(b, H, q, o, lse)


@pytest.mark.parametrize("causal,window", [(False, (-1, -1)), (True, (0, -1)), (True, (40, 7)),
                                           (False, (100, 3)), (False, (-1, 20)), (True, (2000, 0))])
@pytest.mark.parametrize("fp8,D", [(False, 128), (True, 64)])
@pytest.mark.parametrize("rows,spare", [([1, 1, 1], 2), ([1, 1, 1], 90), ([3, 90, 17], 90),
                                        ([300, 5, 129], 2)])
def test_windows(causal, window, fp8, D, rows, spare):
    b = R.Batch(rows, [1000, 150, 0], 2, D, 32, BF, fp8, seed=3, spare_cols=spare)
    q, o, lse = run(b, 8, causal=causal, window=window)
    check(b, 8, q, o, lse, causal=causal, window=window)


@pytest.mark.parametrize("per_batch", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [[1, 1], [20, 150]])
def test_alibi(per_batch, fp8, rows):
    b = R.Batch(rows, [700, 33], 4, 64, 16, HF, fp8, seed=9)
    slopes = torch.exp2(-torch.arange(1, 13) * 0.6).float()
    if per_batch:
        slopes = torch.stack([slopes, slopes * 0.5])
    q, o, lse = run(b, 12, slopes=slopes)
    check(b, 12, q, o, lse, slopes=slopes)


@pytest.mark.parametrize("rows", [[1, 1, 2, 1], [40, 3, 200, 1]])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("spare", [1, 200])
def test_rows_without_keys_and_rows_behind_the_last_sequence(rows, fp8, spare):
    # sequences shorter than their rows: the first rows sit before key 0
    b = R.Batch(rows, [-1, -3, -1, 0], 2, 128, 16, BF, fp8, seed=2, tail=5, spare_cols=spare)
    H = 4
    g = torch.Generator().manual_seed(1)
    q = torch.randn(b.total, H, 128, generator=g).to(BF)
    k, v, table, cu, lens, kw = b.gpu()
    o = torch.full((b.total, H, 128), 7.0, dtype=BF, device="cuda")
    lse = torch.full((H, b.total), 7.0, device="cuda")
    call_c(q.cuda(), o, lse, k, v, table, cu, lens, **kw)
    torch.cuda.synchronize()
    assert fattn_error() == fattn.FA_OK
    check(b, H, q, o.cpu(), lse.cpu())
    n = sum(rows)
    assert (o[n:] == 7).all() and (lse[:, n:] == 7).all()
    assert (o[0] == 0).all() and (lse[:, 0] == -math.inf).all()


def call_c(q, o, lse, k, v, table, cu, lens, k_exp=None, v_exp=None):
    """fa_fwd_paged itself, on results of the caller's."""
    lib, total, H, D = fattn.load(), *q.shape
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    code = {BF: 0, HF: 1, R.E4M3: 3}
    c = R.KvPages(ptr(k), ptr(v), ptr(k_exp), ptr(v_exp), *k.stride()[:3], *v.stride()[:3],
                  *k.shape, code[k.dtype])
    r = R.Ragged(ptr(table), table.stride(0), table.shape[1], ptr(cu), ptr(lens), len(lens), total)
    n = ctypes.c_size_t()
    assert lib.fa_fwd_paged_workspace_size(len(lens), total, H, k.shape[2], D,
                                           table.shape[1] * k.shape[1], ctypes.byref(n)) == 0
    ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")
    st = lib.fa_fwd_paged(ptr(q), *q.stride()[:2], ptr(o), *o.stride()[:2], ptr(lse),
                          ctypes.addressof(c), ctypes.addressof(r), H, None, D ** -0.5, 1,
                          code[q.dtype], ptr(ws) if n.value else None, n.value,
                          torch.cuda.current_stream().cuda_stream)
    assert st == fattn.FA_OK


def test_strided_operands_and_other_page_orders():
    b = R.Batch([1, 30], [200, 90], 2, 64, 16, BF, False, seed=4)
    k, v, table, cu, lens, _ = b.gpu()
    q = torch.randn(b.total, 8, 64, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    want, wl = attention.flash_attn_paged_func(q, k, v, table, cu, lens, return_lse=True)
    # heads before tokens inside a page, keys and values side by side, a wide table, a cut q
    kv = torch.stack([k, v], 1).permute(0, 1, 3, 2, 4).contiguous()  # (pages, 2, heads, page, D)
    wide = torch.full((2, table.shape[1] + 9), 5, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    big = torch.zeros(b.total, 8, 3, 64, dtype=BF, device="cuda")
    big[:, :, 1] = q
    got, gl = attention.flash_attn_paged_func(
        big[:, :, 1], kv[:, 0].transpose(1, 2), kv[:, 1].transpose(1, 2),
        wide[:, :table.shape[1]], cu, lens, return_lse=True)
    assert torch.equal(got, want) and torch.equal(gl, wl)


@pytest.mark.parametrize("rows", [[1, 1, 1], [50, 1, 130]])
def test_bad_tables_and_lengths_are_contained(rows):
    b = R.Batch(rows, [100, 200, 0], 2, 64, 16, BF, False, seed=6)
    k, v, table, cu, lens, _ = b.gpu()
    q = torch.randn(b.total, 4, 64, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    good = attention.flash_attn_paged_func(q, k, v, table, cu, lens)
    for fix in ("page", "negative", "long", "negative length", "cu"):
        t, c, n = table.clone(), cu.clone(), lens.clone()
        if fix == "page":
            t[1, 2] = k.shape[0]
        elif fix == "negative":
            t[1, 0] = -1
        elif fix == "long":
            n[1] = 1 << 30
            t[1] = t[0, 0]
        elif fix == "negative length":
            n[1] = -5
        else:
            c[3] = 1 << 28
        got = attention.flash_attn_paged_func(q, k, v, t, c, n)
        torch.cuda.synchronize()
        assert fattn_error() == fattn.FA_ERR_INVALID_ARG, fix
        assert torch.equal(got[:rows[0]], good[:rows[0]])  # the other sequences are unharmed
    assert fattn_error() == fattn.FA_OK


@pytest.mark.parametrize("rows", [[1] * 6, [70, 1, 128, 5, 0, 9]])
def test_same_bits_twice_on_streams_and_in_graphs(rows):
    b = R.Batch(rows, [900, 5, 300, 0, 64, 2500], 4, 128, 64, BF, False, seed=8)
    k, v, table, cu, lens, _ = b.gpu()
    qs = [torch.randn(b.total, 16, 128, generator=torch.Generator().manual_seed(i)).to(BF).cuda()
          for i in range(3)]
    call = lambda q: attention.flash_attn_paged_func(q, k, v, table, cu, lens, return_lse=True)  # noqa: E731
    want = [call(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = []
    for q, st in zip(qs, streams):
        with torch.cuda.stream(st):
            got.append(call(q))
    torch.cuda.synchronize()
    for w, x in zip(want, got):
        assert torch.equal(w[0], x[0]) and torch.equal(w[1], x[1])
    # two captured graphs, replayed with new queries and lengths in place
    q = qs[0].clone()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = call(q)
        graphs.append((gr, out))
    for i in (1, 2):
        q.copy_(qs[i])
        for gr, out in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert torch.equal(out[0], want[i][0]) and torch.equal(out[1], want[i][1])


@pytest.mark.parametrize("spare", [2, 200])  # units whole, and cut and joined
@pytest.mark.parametrize("fp8,D,H,Hk,dtype", [(False, 128, 8, 2, BF), (True, 128, 8, 2, BF),
                                              (True, 64, 6, 6, HF), (False, 64, 16, 1, HF)])
def test_single_tokens_beside_a_chunk(fp8, D, H, Hk, dtype, spare):
    rows = [1] * 11 + [790] + [0, 1, 2, 4, 5, 16, 17] + [1] * 130 + [3]
    ctx = [(i * 97) % 700 for i in range(len(rows))]
    b = R.Batch(rows, ctx, Hk, D, 16, dtype, fp8, seed=4, spare_cols=spare)
    q, o, lse = run(b, H)
    check(b, H, q, o, lse)
    q, o, lse = run(b, H, causal=False, window=(60, 5))
    check(b, H, q, o, lse, causal=False, window=(60, 5))
    q, again, lse2 = run(b, H, causal=False, window=(60, 5))
    n = sum(b.rows)
    assert torch.equal(o[:n], again[:n]) and torch.equal(lse[:, :n], lse2[:, :n])


def test_many_short_sequences():
    n = 700
    lens = [(i * 37) % 90 for i in range(n)]
    rows = [(i * 7) % 3 for i in range(n)]
    b = R.Batch(rows, [x - r if x >= r else 0 for x, r in zip(lens, rows)], 1, 64, 16, BF, False,
                seed=1)
    q, o, lse = run(b, 2)
    check(b, 2, q, o, lse)


@pytest.mark.parametrize("fp8,D,H,Hk,dtype", [(False, 128, 16, 4, BF), (True, 128, 16, 4, BF),
                                              (False, 64, 24, 8, HF), (True, 64, 15, 5, HF)])
def test_several_long_units_per_cta(fp8, D, H, Hk, dtype):
    b = R.Batch([1900, 1, 700, 0, 1333], [0, 900, 650, 10, 3], Hk, D, 64, dtype, fp8, seed=12)
    q, o, lse = run(b, H)
    check(b, H, q, o, lse)
    b = R.Batch([1900, 700, 1333], [0, 650, 3], Hk, D, 32, dtype, fp8, seed=13)
    q, o, lse = run(b, H, window=(500, 0))
    check(b, H, q, o, lse, window=(500, 0))
