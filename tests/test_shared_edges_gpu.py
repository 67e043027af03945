"""Attention over shared prefixes at the ends of its ranges: scores far from zero, sequences in no
group, several tokens a sequence, single tokens beside a prompt's chunk, and the step around it."""
import ctypes
import math

import pytest
import torch

import paged_ref as R
import test_decoder_step_gpu as step
import test_shared_prefix_gpu as P
from exact_attention_93_gb300 import fattn, kvcache

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
I32 = torch.int32


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


SEVERAL = [
    # rows, ctx, groups, heads, heads_k, D, page, dtype, fp8
    ([8] * 12, [310 + 7 * i for i in range(12)], [(0, 12, 19)], 8, 2, 128, 16, BF, False),
    ([8] * 12, [310 + 7 * i for i in range(12)], [(0, 12, 19)], 8, 2, 128, 16, HF, True),
    ([5, 9, 0, 16, 7, 12], [400, 257, 256, 300, 1000, 290], [(0, 6, 8)], 12, 3, 128, 32, HF, False),
    ([5, 9, 0, 16, 7, 12], [400, 257, 256, 300, 1000, 290], [(0, 6, 8)], 12, 3, 64, 32, BF, True),
    ([4] * 7, [513 + i for i in range(7)], [(1, 4, 2), (4, 7, 1)], 32, 2, 64, 256, HF, False),
    ([60, 70, 62, 64], [1700, 1600, 1610, 1650], [(0, 4, 25)], 2, 2, 128, 64, BF, False),
    # single tokens beside a chunk of a prompt: either kernel takes its own sequences
    ([1] * 129 + [200], [40 + i % 9 for i in range(130)], [(0, 130, 2)], 8, 2, 64, 16, HF, False),
    ([1] * 20 + [100] + [1] * 19, [70 + i % 5 for i in range(40)], [(0, 15, 3), (15, 30, 4)], 8, 2, 128,
     16, BF, True),
    ([1] * 71 + [400], [40 + i % 9 for i in range(72)], [(i, i + 2, 2) for i in range(0, 72, 2)], 4, 4,
     64, 16, BF, True),  # (in both parts)
]


@pytest.mark.parametrize("rows,ctx,groups,H,Hk,D,page,dtype,fp8", SEVERAL)
def test_several_tokens_a_sequence(rows, ctx, groups, H, Hk, D, page, dtype, fp8):
    b = P.widen(P.shared_batch(rows, ctx, groups, Hk, D, page, dtype, fp8, seed=len(rows) + H))
    assert shares(b, H, groups)
    q, o, lse = P.run(b, H, groups)
    assert fattn.fa_device_error() == fattn.FA_OK
    P.check(b, H, q, o, lse)
    _, again, lse2 = P.run(b, H, groups)
    assert torch.equal(o, again) and torch.equal(lse, lse2)


# ---- the step around it

class Wide(step.Decoder):
    """With a table so wide that its calls walk shared keys once."""

    def __init__(self, batch, pages, heads, heads_k, D, *rest):
        super().__init__(batch, pages, heads, heads_k, D, *rest)
        self.table = torch.zeros(batch, (1 << 24) // (batch * heads_k * 16), dtype=I32, device="cuda")
        n, m, lib = ctypes.c_size_t(), ctypes.c_size_t(), fattn.load()
        args = (batch, 2 * batch, heads, heads_k, D, self.table.shape[1] * 16)
        assert lib.fa_fwd_paged_workspace_size(*args, ctypes.byref(n)) == 0
        assert lib.fa_fwd_paged_shared_workspace_size(*args, 1, ctypes.byref(m)) == 0
        assert m.value > n.value


@pytest.mark.parametrize("dtype,cache,by_slots", [(BF, BF, True), (HF, HF, False)])
def test_step(monkeypatch, dtype, cache, by_slots):
    monkeypatch.setattr(step, "Decoder", Wide)
    step.test_prompt_then_tokens(dtype, cache, by_slots)


def test_step_in_one_graph():
    heads, heads_k, D, batch, prompt, steps = 16, 4, 128, 5, 100, 20
    gen = torch.Generator(device="cuda").manual_seed(3)
    draw = lambda n, h: torch.randn(n, h, D, device="cuda", generator=gen).to(BF)  # noqa: E731
    start = draw(prompt, heads), draw(prompt, heads_k), draw(prompt, heads_k)
    data = [(draw(batch, heads), draw(batch, heads_k), draw(batch, heads_k)) for _ in range(steps)]
    new = torch.ones(batch, dtype=I32, device="cuda")
    shared = prompt // 16
    groups = dict(cu_groups=torch.tensor([0, batch], dtype=I32, device="cuda"),
                  shared_pages=torch.tensor([shared], dtype=I32, device="cuda"))

    def prompted():
        dec = Wide(batch, 30, heads, heads_k, D, BF, BF, True)
        dec.step(*start, torch.tensor([prompt] + [0] * (batch - 1), dtype=I32, device="cuda"))
        dec.table[1:, :shared] = dec.table[0, :shared]
        dec.lens[1:] = shared * 16
        return dec

    eager = prompted()
    want = [eager.step(*x, new, **groups)[0] for x in data]
    dec = prompted()
    q, k, v = (torch.zeros_like(t) for t in data[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, _ = dec.step(q, k, v, new, **groups)
    for x, w in zip(data, want):
        for a, y in zip((q, k, v), x):
            a.copy_(y)
        graph.replay()
        assert torch.equal(o, w)
    assert torch.equal(dec.lens, eager.lens) and fattn.fa_device_error() == fattn.FA_OK
    # without pages nothing happens, and the groups have no rows
    held = [t.clone() for t in dec.pages[:2]] + [dec.lens.clone()]
    dec.count.zero_()
    _, s = dec.step(draw(16 * batch, heads), draw(16 * batch, heads_k), draw(16 * batch, heads_k), 16 * new,
                    **groups)
    assert int(s.missing) > 0 and s.cu_seqlens.tolist() == [0] * (batch + 1)
    for a, y in zip(held, [*dec.pages[:2], dec.lens]):
        assert torch.equal(a, y)
    assert fattn.fa_device_error() == fattn.FA_OK


@pytest.mark.parametrize("tokens", [1, 8])
def test_no_sequence_has_rows(tokens):
    # what attention gets after a reservation that failed
    groups = [(0, 3, 2), (3, 5, 3)]
    b = P.widen(P.shared_batch([tokens] * 5, [60] * 5, groups, 2, 64, 16, BF, False, seed=2))
    assert shares(b, 8, groups)
    b.cu = torch.zeros(6, dtype=I32)
    o = torch.full((b.total, 8, 64), 7.0, dtype=BF, device="cuda")
    lse = torch.full((8, b.total), 7.0, device="cuda")
    P.call_c(P.queries(b, 8).cuda(), o, lse, b, groups)
    assert (o == 7).all() and (lse == 7).all() and fattn.fa_device_error() == fattn.FA_OK


def test_pages_are_given_back_after_a_shared_prompt():
    # the prompt's whole pages once, by the sequence that brought them
    batch, heads, heads_k, D, prompt = 3, 4, 2, 64, 50
    dec = Wide(batch, 20, heads, heads_k, D, HF, HF, True)
    x = lambda n, h: torch.ones(n, h, D, device="cuda", dtype=HF)  # noqa: E731
    one = torch.ones(batch, dtype=I32, device="cuda")
    dec.step(x(prompt, heads), x(prompt, heads_k), x(prompt, heads_k),
             torch.tensor([prompt, 0, 0], dtype=I32, device="cuda"))
    dec.table[1:, :3] = dec.table[0, :3]
    dec.lens[1:] = 48
    dec.step(x(batch, heads), x(batch, heads_k), x(batch, heads_k), one,
             cu_groups=torch.tensor([0, batch], dtype=I32, device="cuda"),
             shared_pages=torch.tensor([3], dtype=I32, device="cuda"))
    assert dec.count.tolist() == [20 - 4 - 2]
    kvcache.kv_cache_release(torch.ones(batch, dtype=torch.bool, device="cuda"), dec.lens, dec.table,
                             dec.free, dec.count, 16,
                             keep_pages=torch.tensor([0, 3, 3], dtype=I32, device="cuda"))
    assert dec.count.tolist() == [20] and sorted(dec.free.tolist()) == list(range(20))
    assert fattn.fa_device_error() == fattn.FA_OK
