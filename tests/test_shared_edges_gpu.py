"""Attention over shared prefixes at the ends of its ranges: sequences in no group."""
import ctypes

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
