"""The calls of a decoder's step together, as they are used: tables from lengths, norm and
rotation, writing into the cache, attention over it with a prompt that sequences share;
eagerly and as one captured graph."""
import pytest
import torch

import paged_ref as R
from exact_attention_93_gb300 import attention, fattn, kvcache, rotary

pytestmark = pytest.mark.gpu
I32 = torch.int32


class Decoder:
    """One layer's worth of calls over 16-bit pages of 16."""

    def __init__(self, batch, pages, heads, heads_k, D, dtype, cache, by_slots):
        g = torch.Generator().manual_seed(1)
        self.page, self.by_slots, self.D = 16, by_slots, D
        self.pages = kvcache.alloc_kv_cache(pages, 16, heads_k, D, cache)
        self.table = torch.zeros(batch, 60, dtype=I32, device="cuda")
        self.free = torch.randperm(pages, generator=g).to(I32).cuda()
        self.count = torch.tensor([pages], dtype=I32, device="cuda")
        self.lens = torch.zeros(batch, dtype=I32, device="cuda")
        self.freq, self.magnitude = rotary.rotary_frequencies(D)
        self.wq, self.wk = (1 + 0.1 * torch.randn(D, generator=g).to(dtype).cuda() for _ in range(2))

    def step(self, q, k, v, new, **groups):
        s = kvcache.kv_cache_reserve(new, self.lens, self.table, self.free, self.count, self.page,
                                     q.shape[0], inplace=True)
        q, k = rotary.qk_norm_rotary_func(q, k, self.wq, self.wk, self.freq, positions=s.positions,
                                          magnitude=self.magnitude)
        self.turned = q, k
        kp, vp, ke, ve = self.pages
        if self.by_slots:
            kvcache.kv_cache_write(k, v, kp, vp, s.slots, ke, ve)
        else:
            kvcache.kv_cache_append(k, v, kp, vp, self.table, s.cu_seqlens, s.seqlens, ke, ve)
        o = attention.flash_attn_paged_func(q, kp, vp, self.table, s.cu_seqlens, s.seqlens, k_exp=ke,
                                            v_exp=ve, **groups)
        return o, s


@pytest.mark.parametrize("dtype,cache,by_slots", [
    (torch.bfloat16, torch.bfloat16, True), (torch.float16, R.E4M3, False)])
def test_prompt_then_tokens(dtype, cache, by_slots):
    heads, heads_k, D, batch, prompt, steps = 8, 2, 64, 4, 147, 6
    g = torch.Generator().manual_seed(2)
    draw = lambda n, h: torch.randn(n, h, D, generator=g).to(dtype)  # noqa: E731
    dec = Decoder(batch, 64, heads, heads_k, D, dtype, cache, by_slots)
    weights, freq = (dec.wq.cpu(), dec.wk.cpu()), dec.freq.cpu()
    held = lambda x: R.quantise(x)[0] if cache == R.E4M3 else x.double()  # noqa: E731
    keys, values = ([torch.empty(0, heads_k, D, dtype=torch.float64)] * batch for _ in "kv")

    def step(rows, pad, **groups):
        n = sum(rows)
        q, k, v = draw(n + pad, heads), draw(n + pad, heads_k), draw(n + pad, heads_k)
        before = dec.lens.tolist()
        o, s = dec.step(q.cuda(), k.cuda(), v.cuda(), torch.tensor(rows, dtype=I32, device="cuda"), **groups)
        assert s.slots[n:].tolist() == [-1] * pad and s.missing.tolist() == [0]
        # Rotated rows as the norm's own test holds them to the definition; from here on the
        # very values that the calls have rounded them to.
        pos = torch.tensor([p for b, r in enumerate(rows) for p in range(before[b], before[b] + r)])
        turned = []
        for x, w, y in zip((q, k), weights, dec.turned):
            f = x[:n].double()
            f = f * (f.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w.double()
            ref = R.rotary(f[None], pos[None], freq)[0]
            top = f.abs().amax(-1, keepdim=True) * 2 ** 0.5
            tol = R.EPS[dtype] * 1.01 * ref.abs() + (2.0 ** -21 + 40 * 2.0 ** -24) * top + 2.0 ** -25
            assert ((y[:n].cpu().double() - ref).abs() <= tol).all()
            turned.append(y[:n].cpu())
        at = 0
        for b, r in enumerate(rows):
            keys[b] = torch.cat((keys[b], held(turned[1][at:at + r])))
            values[b] = torch.cat((values[b], held(v[at:at + r])))
            at += r

        class Now:  # as paged_ref.attention wants it
            pass
        now = Now()
        now.rows, now.lens, now.heads_k = rows, [x.shape[0] for x in keys], heads_k
        now.k, now.v = keys, values
        ro, rl, A, S = R.attention(now, turned[0], D ** -0.5)
        p_eps = R.EPS[torch.float16 if cache == R.E4M3 else dtype]
        tol, _ = R.attention_bounds(ro, rl, A, S, dtype, p_eps, D)
        # fp16 weights below 2^-18 of the largest are off by 2^-29 of it at most
        tol = tol + 2.0 ** -28 * max(float(x.abs().sum(0).max()) for x in values if x.shape[0])
        assert ((o[:n].cpu().double() - ro).abs() <= tol).all()

    step([prompt, 0, 0, 0], 0)  # the prompt goes into sequence 0; its whole pages are then everybody's
    shared = prompt // 16
    dec.table[1:, :shared] = dec.table[0, :shared]
    dec.lens[1:] = shared * 16
    for x in (keys, values):
        x[1:] = [x[0][:shared * 16]] * (batch - 1)
    groups = dict(cu_groups=torch.tensor([0, batch], dtype=I32, device="cuda"),
                  shared_pages=torch.tensor([shared], dtype=I32, device="cuda"))
    for i in range(steps):
        step([1 + (b + i) % 2 for b in range(batch)], 2, **groups)
    assert fattn.fa_device_error() == fattn.FA_OK
    # what the cache holds is what has been written
    lens = dec.lens.tolist()
    assert lens == [x.shape[0] for x in keys]
    cu = torch.tensor([0] + lens).cumsum(0).to(I32).cuda()
    kp, vp, ke, ve = dec.pages
    k, v = kvcache.kv_cache_read(kp, vp, dec.table, cu, sum(lens), k_exp=ke, v_exp=ve, dtype=dtype)
    assert torch.equal(k.cpu().double(), torch.cat(keys)) and torch.equal(v.cpu().double(), torch.cat(values))


def test_generation_in_one_graph_equals_the_same_steps_one_by_one():
    heads, heads_k, D, batch, steps = 16, 4, 128, 5, 40
    dtype = torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(3)
    draw = lambda n, h: torch.randn(n, h, D, device="cuda", generator=gen).to(dtype)  # noqa: E731
    data = [(draw(batch, heads), draw(batch, heads_k), draw(batch, heads_k)) for _ in range(steps)]
    new = torch.ones(batch, dtype=I32, device="cuda")
    groups = dict(cu_groups=torch.tensor([0, 2, batch], dtype=I32, device="cuda"),
                  shared_pages=torch.tensor([0, 0], dtype=I32, device="cuda"))
    eager, want = Decoder(batch, 30, heads, heads_k, D, dtype, dtype, True), []
    for q, k, v in data:
        want.append(eager.step(q, k, v, new, **groups)[0])
    # 30 pages of 16 hold 40 tokens of 5 sequences in 15
    dec = Decoder(batch, 30, heads, heads_k, D, dtype, dtype, True)
    q, k, v = (torch.zeros_like(t) for t in data[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, s = dec.step(q, k, v, new, **groups)
    got = []
    for x in data:
        for a, b in zip((q, k, v), x):
            a.copy_(b)
        graph.replay()
        got.append(o.clone())
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert dec.lens.tolist() == [steps] * batch and dec.count.tolist() == [15]
    kvcache.kv_cache_release(torch.ones(batch, dtype=torch.bool, device="cuda"), dec.lens, dec.table,
                             dec.free, dec.count, 16)
    assert dec.count.tolist() == [30] and sorted(dec.free.tolist()) == list(range(30))
    assert fattn.fa_device_error() == fattn.FA_OK


def test_a_step_without_pages_does_nothing():
    heads, heads_k, D = 4, 2, 64
    dec = Decoder(2, 2, heads, heads_k, D, torch.float16, torch.float16, False)
    x = lambda n, h: torch.ones(n, h, D, device="cuda", dtype=torch.float16)  # noqa: E731
    new = torch.tensor([20, 20], dtype=I32, device="cuda")
    _, s = dec.step(x(40, heads), x(40, heads_k), x(40, heads_k), new)
    assert s.missing.tolist() == [2] and dec.lens.tolist() == [0, 0] and dec.count.tolist() == [2]
    for t in dec.pages[:2]:
        assert (t == 0).all()
    assert fattn.fa_device_error() == fattn.FA_OK


def test_a_step_in_inference_mode_and_from_two_threads():
    import threading
    heads, heads_k, D, batch = 8, 2, 128, 3
    dtype = torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(5)
    data = [[torch.randn(batch, h, D, device="cuda", generator=gen).to(dtype)
             for h in (heads, heads_k, heads_k)] for _ in range(20)]
    new = torch.ones(batch, dtype=I32, device="cuda")

    def generate(mode):
        with mode():
            dec = Decoder(batch, 12, heads, heads_k, D, dtype, dtype, True)
            return [dec.step(*x, new)[0].clone() for x in data], dec.lens.tolist()

    want, lens = generate(torch.no_grad)
    got, lens2 = generate(torch.inference_mode)
    assert lens == lens2 == [20] * batch
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # each thread on a stream and a cache of its own
    results = [None] * 2

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            results[i] = generate(torch.no_grad)
            torch.cuda.current_stream().synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for got, lens2 in results:
        assert lens2 == lens and all(torch.equal(a, b) for a, b in zip(want, got))
    assert fattn.fa_device_error() == fattn.FA_OK
