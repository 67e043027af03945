"""Attention over shared prefixes at the ends of its ranges: scores far from zero, sequences in no
group."""
import ctypes
import math

import pytest
import torch

import paged_ref as R
import test_shared_prefix_gpu as P
from exact_attention_93_gb300 import fattn

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def shares(b, H, groups):
    """Whether this call, of this type, walks shared keys once for a group: the workspace of the
    ordinary call is then refused."""
    n, lib = ctypes.c_size_t(), fattn.load()
    k, v, table, cu, lens, kw = b.gpu()
    assert lib.fa_fwd_paged_workspace_size(len(lens), b.total, H, b.heads_k, b.D,
                                           table.shape[1] * b.page, ctypes.byref(n)) == 0
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    code = {BF: 0, HF: 1, R.E4M3: 3}
    q = torch.zeros(b.total, H, b.D, dtype=b.dtype, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(H, b.total, device="cuda")
    ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")
    c = R.KvPages(ptr(k), ptr(v), ptr(kw.get("k_exp")), ptr(kw.get("v_exp")), *k.stride()[:3],
                  *v.stride()[:3], *k.shape, code[k.dtype])
    r = R.Ragged(ptr(table), table.stride(0), table.shape[1], ptr(cu), ptr(lens), len(lens), b.total)
    cu_groups, shared = P.tensors(groups)
    st = lib.fa_fwd_paged_shared(ptr(q), *q.stride()[:2], ptr(o), *o.stride()[:2], ptr(lse),
                                 ctypes.addressof(c), ctypes.addressof(r), ptr(cu_groups), ptr(shared),
                                 len(groups), H, b.D ** -0.5, code[b.dtype], ptr(ws), n.value,
                                 torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st in (fattn.FA_OK, fattn.FA_ERR_INVALID_ARG)
    return st == fattn.FA_ERR_INVALID_ARG


def hold(b, i, w, x):
    """Makes x the keys (w = 0) or the values of sequence i."""
    vals, exps = R.quantise(x) if b.fp8 else (x.double(), None)
    (b.k, b.v)[w][i] = vals
    for j in range(len(x)):
        page, off = int(b.table[i, j // b.page]), j % b.page
        if b.fp8:
            codes = torch.ldexp(vals[j], 127 - exps[j].int()[:, None]).float().to(R.E4M3)
            b.pool[w].view(torch.uint8)[page, off] = codes.view(torch.uint8)
            b.exp[w][page, :, off] = exps[j]
        else:
            b.pool[w][page, off] = vals[j].to(b.dtype)


@pytest.mark.parametrize("dtype,fp8", [(BF, False), (HF, False), (BF, True), (HF, True)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tokens", [1, 4, 8])  # the own part: eight rows, 16, many
def test_scores_far_from_zero(tokens, D, dtype, fp8):
    # Scores are 65536 less 0, 1 or 2 in log2 units, all of them and the weights exact (sums of
    # two products of whole numbers, a scale of one, powers of two), so what the parts' joining
    # does to the result is all that is off but for its own rounding: two exponentials, a sum
    # and a quotient, 2^-21 of the weights' sum, one, in which 2^-20 leaves room.
    n, page, batch = 256, 16, 8
    scale = math.log(2.0)
    assert float(torch.tensor(scale, dtype=torch.float32) *
                 torch.tensor(1.4426950408889634, dtype=torch.float32)) == 1.0
    groups = [(0, batch, n // page)]
    b = P.shared_batch([tokens] * batch, [n + 250 + i for i in range(batch)], groups, 2, D, page, dtype,
                       fp8, seed=D)
    g = torch.Generator().manual_seed(1)
    low = lambda k: -torch.randint(0, 3, (k, 2), generator=g).double()  # noqa: E731
    first = low(n)
    for i in range(batch):
        own = b.lens[i] - n
        k = torch.zeros(b.lens[i], 2, D, dtype=torch.float64)
        k[..., 0] = 256
        k[..., 1] = torch.cat((first, low(own)))
        v = torch.ones(b.lens[i], 2, D, dtype=torch.float64)
        v[n:] = -1
        hold(b, i, 0, k)
        hold(b, i, 1, v)
    P.widen(b)
    assert shares(b, 8, groups)
    q = torch.zeros(b.total, 8, D)
    q[..., 0], q[..., 1] = 256, 1
    q = q.to(dtype)
    ro, rl, _, _ = R.attention(b, q, scale)
    _, o, lse = P.run(b, 8, groups, q=q, scale=scale)
    tol = R.EPS[dtype] * 1.01 * ro.abs() + 2.0 ** -20 + 2.0 ** -25
    off = (o.double() - ro).abs()
    assert (off <= tol).all(), (off.max(), float((off / tol).max()))
    assert ((lse.double() - rl).abs() <= 2.0 ** -22 * rl.abs()).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tokens", [1, 3, 9])  # the own part: eight rows, 16, many
@pytest.mark.parametrize("groups", [[(3, 5, 4)], [(0, 2, 4)], [(5, 7, 4)], [(2, 4, 2), (4, 6, 6)]])
def test_sequences_in_no_group(groups, tokens, fp8):
    # before the groups and behind them; what the workspace holds there is NaN
    rows = [tokens, 2 * tokens, 0, tokens, tokens, 1, tokens] + [tokens] * 7
    ctx = [100, 120, 110, 130, 140, 99, 300] + [20 * i for i in range(7)]
    b = P.widen(P.shared_batch(rows, ctx, groups, 2, 64, 16, BF, fp8, seed=3, tail=4))
    assert shares(b, 8, groups)
    q = P.queries(b, 8)
    o = torch.full((b.total, 8, 64), 7.0, dtype=BF, device="cuda")
    lse = torch.full((8, b.total), 7.0, device="cuda")
    P.call_c(q.cuda(), o, lse, b, groups)
    assert fattn.fa_device_error() == fattn.FA_OK
    P.check(b, 8, q, o.cpu(), lse.cpu())
    n = sum(rows)
    assert (o[n:] == 7).all() and (lse[:, n:] == 7).all()
