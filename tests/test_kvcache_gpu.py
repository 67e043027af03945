"""Writing the paged cache and reading it back, on the GPU."""
import math

import pytest
import torch

import paged_ref as R
from exact_attention_93_gb300 import attention, fattn, kvcache, rotary

pytestmark = pytest.mark.gpu
BF, HF, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def bytes_of(t):
    return t.contiguous().view(torch.uint8)


def setup(rows, ctx, heads, D, page, cache_dtype, dtype, seed=0, tail=0):
    """An empty cache over scattered pages, and packed rows."""
    b = R.Batch(rows, ctx, heads, D, page, BF, False, seed=seed, tail=tail)
    cache = kvcache.alloc_kv_cache(b.pool.shape[1], page, heads, D, cache_dtype)
    g = torch.Generator().manual_seed(seed + 1)
    k, v = (torch.randn(b.total, heads, D, generator=g) *
            torch.exp2(3 * torch.randn(b.total, heads, 1, generator=g)) for _ in range(2))
    return b, cache, k.to(dtype), v.to(dtype)


CASES = [
    ([1], [0], 1, 64, 16),
    ([1] * 70, list(range(70)), 8, 128, 32),
    ([5, 0, 33, 1], [0, 10, 15, 64], 3, 64, 64),
    ([300, 17], [0, 1000], 2, 128, 256),
    ([129, 1, 2], [5, 127, 126], 17, 128, 128),
]


@pytest.mark.parametrize("rows,ctx,heads,D,page", CASES)
@pytest.mark.parametrize("cache_dtype,dtype", [(E4, BF), (E4, HF), (BF, BF), (HF, HF)])
def test_append_and_read(rows, ctx, heads, D, page, cache_dtype, dtype):
    b, cache, k, v = setup(rows, ctx, heads, D, page, cache_dtype, dtype, seed=len(rows), tail=3)
    kp, vp, ke, ve = cache
    table, cu, lens = b.table.cuda(), b.cu.cuda(), b.len_t.cuda()
    kvcache.kv_cache_append(k.cuda(), v.cuda(), kp, vp, table, cu, lens, k_exp=ke, v_exp=ve)
    starts = lens - (cu[1:] - cu[:-1])
    out = tuple(torch.full((b.total, heads, D), 9.0, dtype=dtype, device="cuda") for _ in range(2))
    got = kvcache.kv_cache_read(kp, vp, table, cu, b.total, starts=starts, k_exp=ke, v_exp=ve,
                                dtype=dtype, out=out)
    torch.cuda.synchronize()
    assert fattn.fa_device_error() == fattn.FA_OK
    n = sum(rows)
    where = torch.zeros(kp.shape[:2], dtype=torch.bool)
    for w, (x, y, exp) in enumerate(zip((k, v), got, (ke, ve))):
        if cache_dtype == E4:
            ref, e = R.quantise(x[:n])
            # dequantised values fit bf16 exactly and fp16 to its rounding
            assert torch.equal(y[:n].cpu(), ref.to(dtype))
            at = 0
            for s, r in enumerate(rows):
                for i in range(r):
                    pos = b.lens[s] - r + i
                    pg = int(b.table[s, pos // page])
                    assert torch.equal(exp[pg, :, pos % page].cpu(), e[at])
                    where[pg, pos % page] = True
                    at += 1
        else:
            assert torch.equal(y[:n].cpu(), x[:n])
            at = 0
            for s, r in enumerate(rows):
                for i in range(r):
                    pos = b.lens[s] - r + i
                    where[int(b.table[s, pos // page]), pos % page] = True
        assert (y[n:] == 9).all()  # rows behind the last sequence
    # slots that no row went to are as they were
    for t in (kp, vp):
        assert not bytes_of(t).cpu().view(*kp.shape[:2], -1)[~where].any()


def special(dtype):
    x = torch.zeros(12, 1, 64)
    x[0] = 0.0
    x[1, 0, 3] = 448.0
    x[2, 0, 3] = 448.0 + 2  # rounds into the next binade's scale
    x[3, 0, :] = torch.linspace(-1, 1, 64)
    x[4, 0, 0], x[4, 0, 1] = math.inf, 1.0
    x[5, 0, 0], x[5, 0, 1] = math.nan, 3.0
    x[6, 0, :] = math.nan
    x[7, 0, 0] = -math.inf
    x[8, 0, 9] = torch.finfo(dtype).max
    x[9, 0, 9] = torch.finfo(dtype).tiny
    x[10, 0, 9] = torch.finfo(dtype).smallest_normal * 2 ** -6
    x[11, 0, :] = torch.tensor([1.0625, 1.1875, 17 / 16 * 256, 19 / 16 * 256] * 16)  # ties
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_special_rows(dtype):
    x = special(dtype)
    n = x.shape[0]
    kp, vp, ke, ve = kvcache.alloc_kv_cache(1, 16, 1, 64, E4)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    kvcache.kv_cache_append(x.cuda(), x.cuda(), kp, vp, table, cu, lens, k_exp=ke, v_exp=ve)
    y, _ = kvcache.kv_cache_read(kp, vp, table, cu, n, k_exp=ke, v_exp=ve, dtype=BF)
    ref, e = R.quantise(x)
    assert torch.equal(ke[0, 0, :n].cpu(), e[:, 0])
    ref, got = ref.to(BF), y.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    ok = ~torch.isnan(ref)
    assert torch.equal(got[ok], ref[ok])


def test_strided_rows_and_pages():
    b, _, k, v = setup([20, 3], [4, 40], 2, 64, 16, BF, BF)
    qkv = torch.zeros(b.total, 3, 4, 64, dtype=BF, device="cuda")
    qkv[:, 1, :2], qkv[:, 2, 2:] = k.cuda(), v.cuda()
    kv = torch.zeros(b.pool.shape[1], 2, 2, 16, 64, dtype=BF, device="cuda")  # heads before tokens
    kp, vp = kv[:, 0].transpose(1, 2), kv[:, 1].transpose(1, 2)
    args = b.table.cuda(), b.cu.cuda(), b.len_t.cuda()
    kvcache.kv_cache_append(qkv[:, 1, :2], qkv[:, 2, 2:], kp, vp, *args)
    gk, gv = kvcache.kv_cache_read(kp, vp, args[0], args[1], b.total,
                                   starts=torch.tensor([4, 40], dtype=torch.int32, device="cuda"))
    assert torch.equal(gk.cpu(), k) and torch.equal(gv.cpu(), v)


def test_bad_pages_are_contained():
    b, (kp, vp, ke, ve), k, v = setup([3, 20, 2], [0, 30, 5], 2, 64, 16, E4, BF)
    table = b.table.clone()
    table[1, 2], table[2, 0] = kp.shape[0], -1
    args = table.cuda(), b.cu.cuda(), b.len_t.cuda()
    kvcache.kv_cache_append(k.cuda(), v.cuda(), kp, vp, *args, k_exp=ke, v_exp=ve)
    assert fattn.fa_device_error() == fattn.FA_ERR_INVALID_ARG
    starts = torch.tensor([0, 30, 5], dtype=torch.int32, device="cuda")
    gk, _ = kvcache.kv_cache_read(kp, vp, args[0], args[1], b.total, starts=starts, k_exp=ke,
                                  v_exp=ve)
    assert fattn.fa_device_error() == fattn.FA_ERR_INVALID_ARG
    ref, _ = R.quantise(k)
    good = [0, 1, 2, 3, 4] + list(range(21, 23))  # rows of whole pages
    assert torch.equal(gk[good].cpu(), ref[good].to(BF))
    assert not gk[5:21].any() and not gk[23:].any()
    # lengths beyond the table, and shorter than the rows
    lens = torch.tensor([2, 1 << 30, -4], dtype=torch.int32, device="cuda")
    kvcache.kv_cache_append(k.cuda(), v.cuda(), kp, vp, b.table.cuda(), args[1], lens, k_exp=ke,
                            v_exp=ve)
    assert fattn.fa_device_error() == fattn.FA_ERR_INVALID_ARG


def test_a_decoder_layer_from_prompt_to_tokens():
    """Rotary, cache and attention as they are used: a ragged prompt, then
    single tokens, against the dense 64-bit attention of the whole sequence."""
    g = torch.Generator().manual_seed(0)
    H, Hk, D, page, steps = 8, 2, 64, 16, 3
    prompts = [37, 5, 64]
    freq, mag = rotary.rotary_frequencies(D)
    full = [p + steps for p in prompts]
    x = [[torch.randn(n, h, D, generator=g).to(BF) for h in (H, Hk, Hk)] for n in full]
    kp, vp, _, _ = kvcache.alloc_kv_cache(40, page, Hk, D)
    table = torch.randperm(40, generator=g)[:3 * 6].view(3, 6).to(torch.int32).cuda()
    done = [0, 0, 0]
    outs = [[] for _ in prompts]
    turned = [[] for _ in prompts]
    for step in range(steps + 1):
        new = prompts if step == 0 else [1, 1, 1]
        cut = [[t[d:d + n] for t in seq] for seq, d, n in zip(x, done, new)]
        q, k, v = (torch.cat([c[i] for c in cut]).cuda() for i in range(3))
        pos = torch.cat([torch.arange(d, d + n) for d, n in zip(done, new)]).cuda()
        done = [d + n for d, n in zip(done, new)]
        cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
        lens = torch.tensor(done, dtype=torch.int32).cuda()
        q, k = rotary.rotary_func(q, k, freq, positions=pos, inplace=True)
        kvcache.kv_cache_append(k, v, kp, vp, table, cu, lens)
        o = attention.flash_attn_paged_func(q, kp, vp, table, cu, lens)
        at = 0
        for s, n in enumerate(new):
            outs[s].append(o[at:at + n].cpu())
            turned[s].append((q[at:at + n].cpu(), k[at:at + n].cpu()))
            at += n
    torch.cuda.synchronize()
    assert fattn.fa_device_error() == fattn.FA_OK
    for s, n in enumerate(full):
        q, k = (torch.cat([t[i] for t in turned[s]]) for i in range(2))
        dense = R.Batch([n], [0], Hk, D, page, BF, False)
        dense.k, dense.v = [k.double()], [x[s][2].double()]
        ref, lse, A, S = R.attention(dense, q, D ** -0.5)
        tol, _ = R.attention_bounds(ref, lse, A, S, BF, R.EPS[BF], D)
        assert ((torch.cat(outs[s]).double() - ref).abs() <= tol).all()
        # and the rows went in turned by their positions
        want = R.rotary(x[s][0][None], torch.arange(n)[None], freq.cpu())[0]
        assert ((q.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18).all()


@pytest.mark.parametrize("cache_dtype,D", [(BF, 128), (E4, 128), (E4, 64)])
def test_chunks_and_tokens_attend_to_what_the_cache_reads_back(cache_dtype, D):
    """A prompt in chunks beside sequences that generate, an idle one among
    them: each step attends to exactly the keys and values read back."""
    g = torch.Generator().manual_seed(7)
    H, Hk, page = 6, 3, 32
    freq, _ = rotary.rotary_frequencies(D)
    kp, vp, ke, ve = kvcache.alloc_kv_cache(60, page, Hk, D, cache_dtype)
    table = torch.randperm(60, generator=g)[:4 * 12].view(4, 12).to(torch.int32).cuda()
    kw = dict(k_exp=ke, v_exp=ve)
    done = [0, 0, 0, 0]
    for new in ([70, 3, 0, 20], [150, 1, 1, 0], [9, 1, 1, 1], [1, 1, 0, 1]):
        q, k, v = (torch.randn(sum(new), h, D, generator=g).to(BF).cuda() for h in (H, Hk, Hk))
        pos = torch.cat([torch.arange(d, d + n) for d, n in zip(done, new)]).cuda()
        ctx, done = done, [d + n for d, n in zip(done, new)]
        cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
        lens = torch.tensor(done, dtype=torch.int32).cuda()
        q, k = rotary.rotary_func(q, k, freq, positions=pos)
        kvcache.kv_cache_append(k, v, kp, vp, table, cu, lens, **kw)
        o, lse = attention.flash_attn_paged_func(q, kp, vp, table, cu, lens, return_lse=True, **kw)
        every = torch.tensor([0] + done).cumsum(0).to(torch.int32).cuda()
        kr, vr = kvcache.kv_cache_read(kp, vp, table, every, sum(done), **kw)
        torch.cuda.synchronize()
        assert fattn.fa_device_error() == fattn.FA_OK
        b = R.Batch(new, ctx, Hk, D, page, BF, False)
        b.k, b.v = ([t.cpu().double() for t in x.split(done)] for x in (kr, vr))
        ref, rl, A, S = R.attention(b, q.cpu(), D ** -0.5)
        tol_o, tol_l = R.attention_bounds(ref, rl, A, S, BF, R.EPS[BF], D)
        assert ((o.cpu().double() - ref).abs() <= tol_o).all()
        assert ((lse.cpu().double() - rl).abs() <= tol_l).all()


@pytest.mark.parametrize("cache_dtype", [BF, E4])
def test_append_and_read_in_a_graph_on_another_stream(cache_dtype):
    b, (kp, vp, ke, ve), k, v = setup([3, 20, 1], [30, 0, 5], 2, 64, 16, cache_dtype, BF)
    table, cu, lens = b.table.cuda(), b.cu.cuda(), b.len_t.cuda()
    starts = torch.tensor([30, 0, 5], dtype=torch.int32, device="cuda")
    kd, vd = k.cuda(), v.cuda()
    out = torch.zeros_like(kd), torch.zeros_like(vd)

    def step():
        kvcache.kv_cache_append(kd, vd, kp, vp, table, cu, lens, k_exp=ke, v_exp=ve)
        kvcache.kv_cache_read(kp, vp, table, cu, b.total, starts=starts, k_exp=ke, v_exp=ve,
                              dtype=BF, out=out)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    first = [t.clone() for t in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    n = sum(b.rows)
    for swap in (True, False):
        kd.copy_(v if swap else k)
        vd.copy_(k if swap else v)
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = first[::-1] if swap else first
        assert torch.equal(out[0][:n], want[0][:n]) and torch.equal(out[1][:n], want[1][:n])
    assert fattn.fa_device_error() == fattn.FA_OK


def test_written_tensors_are_seen_by_autograd():
    b, (kp, vp, ke, ve), k, v = setup([3, 2], [0, 5], 2, 64, 16, BF, BF)
    table, cu, lens = b.table.cuda(), b.cu.cuda(), b.len_t.cuda()
    w = torch.ones(64, device="cuda", dtype=BF, requires_grad=True)
    y = (kp * w).sum()  # saves kp
    kvcache.kv_cache_append(k.cuda(), v.cuda(), kp, vp, table, cu, lens)
    with pytest.raises(RuntimeError):
        y.backward()


def test_overlapping_results_are_refused():
    b, (kp, vp, ke, ve), k, v = setup([3, 2], [0, 5], 2, 64, 16, BF, BF)
    table, cu, lens = b.table.cuda(), b.cu.cuda(), b.len_t.cuda()
    kd, vd = k.cuda(), v.cuda()
    with pytest.raises(fattn.FattnError):
        kvcache.kv_cache_append(kd, vd, kp, kp, table, cu, lens)
    one = kp[:, :, :1].expand(-1, -1, 2, -1)
    with pytest.raises(fattn.FattnError):
        kvcache.kv_cache_append(kd, vd, one, vp, table, cu, lens)
    with pytest.raises(fattn.FattnError):
        kvcache.kv_cache_read(kp, vp, table, cu, b.total, out=(kd, kd))
    with pytest.raises(fattn.FattnError):
        kvcache.kv_cache_read(kp, vp, table, cu, b.total, out=(kd, vd[:1].expand(b.total, -1, -1)))
    both = torch.zeros(kp.shape[0], 2, *kp.shape[1:], device="cuda", dtype=BF)  # interleaved pages
    kvcache.kv_cache_append(kd, vd, both[:, 0], both[:, 1], table, cu, lens)
    kvcache.kv_cache_append(kd, vd, kp, vp, table, cu, lens)
    assert torch.equal(both[:, 0], kp) and torch.equal(both[:, 1], vp)


def test_a_batch_without_rows():
    b, (kp, vp, ke, ve), k, v = setup([0, 0], [4, 0], 2, 64, 16, BF, BF)
    table, cu, lens = b.table.cuda(), b.cu.cuda(), b.len_t.cuda()
    none = torch.zeros(0, 2, 64, device="cuda", dtype=BF)
    kvcache.kv_cache_append(none, none, kp, vp, table, cu, lens)
    ko, vo = kvcache.kv_cache_read(kp, vp, table, cu, 0)
    o, lse = attention.flash_attn_paged_func(torch.zeros(0, 6, 64, device="cuda", dtype=BF), kp, vp,
                                             table, cu, lens, return_lse=True)
    torch.cuda.synchronize()
    assert ko.shape == vo.shape == (0, 2, 64) and o.shape == (0, 6, 64) and lse.shape == (6, 0)
    assert not kp.any() and not vp.any() and fattn.fa_device_error() == fattn.FA_OK


def test_inference_mode():
    with torch.inference_mode():
        b, (kp, vp, ke, ve), k, v = setup([3, 2], [0, 5], 2, 64, 16, E4, BF)
        table, cu, lens = b.table.cuda(), b.cu.cuda(), b.len_t.cuda()
        freq, _ = rotary.rotary_frequencies(64)
        q = torch.randn(5, 4, 64, device="cuda").to(BF)
        want = rotary.rotary_func(q, None, freq)
        assert rotary.rotary_func(q, None, freq, inplace=True) is q and torch.equal(q, want)
        kvcache.kv_cache_append(k.cuda(), v.cuda(), kp, vp, table, cu, lens, k_exp=ke, v_exp=ve)
        o = attention.flash_attn_paged_func(q, kp, vp, table, cu, lens, k_exp=ke, v_exp=ve)
        assert torch.isfinite(o).all() and fattn.fa_device_error() == fattn.FA_OK


def test_two_threads():
    """Calls from two threads on streams of their own give what one gives."""
    import threading
    b, (kp, vp, ke, ve), k, v = setup([1] * 6, [100, 900, 2500, 0, 40, 600], 2, 128, 16, E4, BF)
    kw = dict(k_exp=ke, v_exp=ve)
    table, cu, lens = b.table.cuda(), b.cu.cuda(), b.len_t.cuda()
    ends = torch.tensor([0] + b.lens).cumsum(0).to(torch.int32).cuda()
    g = torch.Generator().manual_seed(1)
    kk, vv = (torch.randn(sum(b.lens), 2, 128, generator=g).to(BF).cuda() for _ in range(2))
    kvcache.kv_cache_append(kk, vv, kp, vp, table, ends, lens, **kw)
    wide = torch.nn.functional.pad(table, (0, 200), value=-1)  # work may be cut and joined
    qs = [torch.randn(6, 8, 128, generator=g).to(BF).cuda() for _ in range(2)]
    want = [attention.flash_attn_paged_func(q, kp, vp, wide, cu, lens, **kw) for q in qs]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[i].append(attention.flash_attn_paged_func(qs[i], kp, vp, wide, cu, lens, **kw))
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert len(got[i]) == 20 and all(torch.equal(o, want[i]) for o in got[i])
