"""Rotary positions along several axes, and norms of queries and keys with the
rotation in the same pass, against 64 bits on the GPU: values, gradients, layouts."""
import math

import pytest
import torch

import paged_ref as R
from exact_attention_93_gb300 import fattn, rotary

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
SHAPES = [(1, 1, 1, 1), (2, 37, 5, 3), (3, 130, 17, 1), (1, 5, 40, 8)]


def axis_of_pair(sections, order):
    if order == "blocks":
        return sum(([a] * n for a, n in enumerate(sections)), [])
    left, out = list(sections), []
    while any(left):
        for a, n in enumerate(left):
            if n:
                out.append(a)
                left[a] -= 1
    return out


def turn(x, pos, freq, interleaved=False, magnitude=1.0, inverse=False, axis=None):
    """64-bit rotation; pos (B, N), or (axes, B, N) with `axis` naming each pair's."""
    if axis is None:
        return R.rotary(x, pos, freq, interleaved, magnitude, inverse)
    # pair by pair: each pair of all alone, at its own axis' positions
    y, n = x.double().clone(), freq.numel()
    for a in set(axis):
        f = torch.where(torch.tensor([i == a for i in axis]), freq.double(), 0.0)
        z = R.rotary(x, pos[a], f, interleaved, magnitude, inverse)
        for i in range(n):
            if axis[i] == a:
                for e in (2 * i, 2 * i + 1) if interleaved else (i, i + n):
                    y[..., e] = z[..., e]
    return y


def norm(x, w, eps):
    """x (..., D) in 64 bits: w x / sqrt(mean x^2 + eps), and 1 / sqrt(...)."""
    x = x.double()
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    return x * r * (1 if w is None else w.double()), r


def close(got, ref, tol):
    """Within tol; where the definition gives NaN (of infinities) the result has it too, and
    where a row has one the rest, zeros by the definition, are equal."""
    got, ref = got.detach().cpu().double(), ref.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    off = (got - ref).abs() - tol.nan_to_num(nan=0.0)
    off = off[~torch.isnan(ref)]
    assert not off.numel() or float(off.max()) <= 0, (float(off.max()), int((off > 0).sum()))


def fp16_floor(dtype):
    return 2.0 ** -25 if dtype == HF else 0.0


def bound_turn(ref, x, magnitude, dtype):
    """An angle is off by 2^-32 turns and its fp32 remainder by 2^-24 of pi/4, sine and
    cosine by 2^-23, so a pair by 2^-21 of its length, which is at most sqrt 2 times the
    row's largest element, times the magnitude; then one rounding to the type."""
    pair = x.double().abs().amax(-1, keepdim=True) * 2 ** 0.5 * max(1.0, abs(magnitude))
    return R.EPS[dtype] * 1.01 * ref.abs() + 2.0 ** -21 * pair + fp16_floor(dtype)


def bound_norm(ref, xn, magnitude, dtype, D):
    """The sum of D squares is off by D 2^-24 of itself, its root by half of that; the
    root's own rounding, eps, and the products add at most 8 more; then the rotation."""
    pair = xn.abs().amax(-1, keepdim=True) * 2 ** 0.5 * max(1.0, abs(magnitude))
    return (R.EPS[dtype] * 1.01 * ref.abs() + (2.0 ** -21 + (D / 2 + 8) * 2.0 ** -24) * pair +
            fp16_floor(dtype))


def norm_grads(x, dy, w, eps, turn_back):
    """The formulas' gradients (dx, dw) of w R x / |x| in 64 bits, with bounds on how far
    fp32 arithmetic may be off (before rounding to the type)."""
    D = x.shape[-1]
    x, (_, r) = x.double(), norm(x, None, eps)
    g = turn_back(dy)
    one = torch.ones(D, dtype=torch.float64) if w is None else w.double()
    mixed = (g * one * x).mean(-1, keepdim=True)
    dx = r * (g * one - x * r * r * mixed)
    dw = (g * x * r).flatten(0, -2).sum(0)
    # |g| is at most G, off by 2^-21 of that; sums of D products by (D + 2) 2^-24 of their
    # magnitudes, r by half of D 2^-24: the second term by (2 D + 16) 2^-24 in all
    G = g.abs().amax(-1, keepdim=True).maximum(
        dy.double().abs().amax(-1, keepdim=True) * 2 ** 0.5)
    W = one.abs().amax()
    size = r * (G * W + x.abs() * r * r * (G * W * x.abs()).mean(-1, keepdim=True))
    tol_x = (2.0 ** -21 + (2 * D + 16) * 2.0 ** -24) * size
    rows = x[..., 0].numel()
    tol_w = (2.0 ** -21 + (D / 2 + 8 + rows) * 2.0 ** -24) * (G * x.abs() * r).flatten(0, -2).sum(0)
    return dx, dw, tol_x, tol_w


SECTIONS = [((16, 24, 24), "blocks"), ((24, 20, 20), "turns"), ((0, 40, 8, 16), "turns"),
            ((1, 30, 1), "blocks"), ((32, 32), "blocks"), ((64,), "turns"),
            ((3, 1, 2, 1, 1, 4, 3, 1), "turns")]


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("sections,order", SECTIONS)
@pytest.mark.parametrize("interleaved", [False, True])
def test_axes(dtype, sections, order, interleaved):
    pairs = sum(sections)
    freq, mag = rotary.rotary_frequencies(2 * pairs, scaling="by_parts", factor=8.0,
                                          original_length=2048, device="cpu")
    axis = axis_of_pair(sections, order)
    g = torch.Generator().manual_seed(pairs + len(sections))
    for D in (64, 128):
        if 2 * pairs > D:
            continue
        for B, N, H, Hk in SHAPES:
            q = torch.randn(B, N, H, D, generator=g).to(dtype)
            k = torch.randn(B, N, Hk, D, generator=g).to(dtype)
            pos = torch.randint(-1000, 1 << 20, (len(sections), B, N), generator=g)
            yq, yk = rotary.rotary_func(q.cuda(), k.cuda(), freq.cuda(), positions=pos.cuda(),
                                        interleaved=interleaved, magnitude=mag, sections=sections,
                                        section_order=order)
            for x, y in ((q, yq), (k, yk)):
                ref = turn(x, pos, freq, interleaved, mag, axis=axis)
                assert y.shape == x.shape and y.dtype == dtype
                close(y, ref, bound_turn(ref, x, mag, dtype))
                assert torch.equal(y.cpu()[..., 2 * pairs:], x[..., 2 * pairs:])


def test_axes_positions_and_equal_places():
    # text has the same place on every axis: then sections change nothing, to the bit
    freq, _ = rotary.rotary_frequencies(128)
    q, k = (torch.randn(2, 61, h, 128, device="cuda").to(BF) for h in (8, 2))
    pos = torch.randint(0, 1 << 20, (2, 61), device="cuda")
    want = rotary.rotary_func(q, k, freq, positions=pos)
    for p in (pos.expand(3, 2, 61), pos.to(torch.int32).expand(3, 2, 61).contiguous(),
              pos.t().contiguous().t().expand(3, 2, 61)):
        for order in ("blocks", "turns"):
            got = rotary.rotary_func(q, k, freq, positions=p, sections=(20, 40, 4),
                                     section_order=order)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # (axes, seqlen) serves every batch, packed tensors have no other
    p = torch.randint(0, 5000, (2, 61), device="cuda", dtype=torch.int32)
    a = rotary.rotary_func(q, None, freq, positions=p, sections=(30, 34))
    b = rotary.rotary_func(q, None, freq, positions=p[:, None].expand(2, 2, 61), sections=(30, 34))
    c = rotary.rotary_func(q[1], None, freq, positions=p, sections=(30, 34))
    assert torch.equal(a, b) and torch.equal(a[1], c)
    assert rotary.rotary_func(q[:, :0], None, freq, positions=p[:, :0],
                              sections=(30, 34)).shape == (2, 0, 8, 128)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("order", ["blocks", "turns"])
def test_axes_gradients(interleaved, order):
    freq, _ = rotary.rotary_frequencies(64, device="cpu")
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(0, 100000, (3, 2, 33), generator=g)
    q, k = (torch.randn(2, 33, h, 128, generator=g).cuda().requires_grad_() for h in (6, 2))
    dq, dk = (torch.randn(t.shape, generator=g) for t in (q, k))
    call = lambda *x: rotary.rotary_func(*x, freq.cuda(), positions=pos.cuda(),  # noqa: E731
                                         interleaved=interleaved, magnitude=1.5,
                                         sections=(10, 18, 4), section_order=order)
    axis = axis_of_pair((10, 18, 4), order)
    got = torch.autograd.grad(call(q, k), (q, k), (dq.cuda(), dk.cuda()), create_graph=True)
    for d, x in zip((dq, dk), got):
        ref = turn(d, pos, freq, interleaved, 1.5, inverse=True, axis=axis)
        close(x, ref, bound_turn(ref, d, 1.5, F32))
    w = torch.randn_like(q, requires_grad=True)  # linear in what comes in: turned again
    gx, = torch.autograd.grad(call(q, None), (q,), (w,), create_graph=True)
    v = torch.randn(q.shape, generator=g)
    gw, = torch.autograd.grad(gx, (w,), (v.cuda(),))
    ref = turn(v, pos, freq, interleaved, 1.5, axis=axis)
    close(gw, ref, bound_turn(ref, v, 1.5, F32))


# ------------------------------------------------------------------- norm and rotation

def rows(g, shape, dtype):
    """Rows of very different magnitudes, zeros among them."""
    x = torch.randn(shape, generator=g) * torch.exp2(4 * torch.randn(shape[:-1] + (1,), generator=g))
    x[..., ::32] *= 4
    x.view(-1, shape[-1])[::7] *= 0.0 if x.view(-1, shape[-1]).shape[0] > 7 else 1.0
    return x.to(dtype)


CASES = [(D, rdim, sections) for D, rdim, sections in (
    (64, 64, None), (64, 16, (3, 5)), (128, 128, None), (128, 96, (16, 16, 16)), (128, 64, None))]


@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (HF, HF), (HF, F32), (F32, F32)])
@pytest.mark.parametrize("D,rdim,sections", CASES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_values(dtype, wdtype, D, rdim, sections, interleaved):
    g = torch.Generator().manual_seed(D + rdim)
    freq, mag = rotary.rotary_frequencies(rdim, scaling="by_parts", factor=8.0,
                                          original_length=2048, device="cpu")
    axis = None if sections is None else axis_of_pair(sections, "turns")
    for B, N, H, Hk in SHAPES:
        q, k = rows(g, (B, N, H, D), dtype), rows(g, (B, N, Hk, D), dtype)
        wq, wk = (1 + 0.3 * torch.randn(D, generator=g).to(wdtype) for _ in range(2))
        lead = () if sections is None else (len(sections),)
        pos = torch.randint(0, 1 << 20, lead + (B, N), generator=g)
        for eps in (1e-6, 1.0):
            got = rotary.qk_norm_rotary_func(
                q.cuda(), k.cuda(), wq.cuda(), wk.cuda(), freq.cuda(), positions=pos.cuda(),
                eps=eps, interleaved=interleaved, magnitude=mag, sections=sections,
                section_order="turns")
            for x, w, y in ((q, wq, got[0]), (k, wk, got[1])):
                xn, _ = norm(x, w, eps)
                ref = turn(xn, pos, freq, interleaved, mag, axis=axis)
                assert y.shape == x.shape and y.dtype == dtype
                close(y, ref, bound_norm(ref, xn, mag, dtype, D))


@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (HF, HF), (F32, F32)])
@pytest.mark.parametrize("D,rdim,sections", CASES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_gradients(dtype, wdtype, D, rdim, sections, interleaved):
    g = torch.Generator().manual_seed(D + rdim + 1)
    freq, mag = rotary.rotary_frequencies(rdim, device="cpu")[0], 1.25
    axis = None if sections is None else axis_of_pair(sections, "blocks")
    eps = 1e-3
    for B, N, H, Hk in SHAPES:
        x = [rows(g, (B, N, h, D), dtype) for h in (H, Hk)]
        w = [(1 + 0.3 * torch.randn(D, generator=g)).to(wdtype) for _ in range(2)]
        dy = [torch.randn(t.shape, generator=g).to(dtype) for t in x]
        lead = () if sections is None else (len(sections),)
        pos = torch.randint(0, 100000, lead + (B, N), generator=g)
        leaves = [t.cuda().requires_grad_() for t in x + w]
        y = rotary.qk_norm_rotary_func(*leaves, freq.cuda(), positions=pos.cuda(), eps=eps,
                                       interleaved=interleaved, magnitude=mag, sections=sections)
        got = torch.autograd.grad(y, leaves, [d.cuda() for d in dy])
        back = lambda d: turn(d, pos, freq, interleaved, mag, inverse=True, axis=axis)  # noqa: E731
        for i in range(2):
            dx, dw, tol_x, tol_w = norm_grads(x[i], dy[i], w[i], eps, back)
            tol_x = 1.3 * tol_x + R.EPS[dtype] * 1.01 * dx.abs() + fp16_floor(dtype)  # (magnitude 1.25)
            tol_w = 1.3 * tol_w + R.EPS[wdtype] * 1.01 * dw.abs() + fp16_floor(wdtype)
            assert got[i].dtype == dtype and got[2 + i].dtype == wdtype
            close(got[i], dx, tol_x)
            close(got[2 + i], dw, tol_w)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_without_eps(dtype):
    g = torch.Generator().manual_seed(4)
    freq, _ = rotary.rotary_frequencies(64, device="cpu")
    x = (torch.randn(1, 6, 3, 64, generator=g) * torch.tensor([1e-15, 1e-6, 1.0, 1e9, 1e15, 1.0])[:, None, None]).to(dtype)
    x[0, 5, 1] = 0.0  # 0 / 0 by the definition
    w = 1 + 0.3 * torch.randn(64, generator=g)
    dy = torch.randn(x.shape, generator=g).to(dtype)
    pos = torch.arange(6)[None]
    lx, lw = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    y = rotary.qk_norm_rotary_func(lx, None, lw, None, freq.cuda(), eps=0.0)
    gx, = torch.autograd.grad(y, (lx,), (dy.cuda(),))
    xn, _ = norm(x, w, 0.0)
    ref = turn(xn, pos, freq)
    close(y, ref, bound_norm(ref, xn, 1.0, dtype, 64))
    dx, _, tol, _ = norm_grads(x, dy, w, 0.0, lambda d: turn(d, pos, freq, inverse=True))
    close(gx, dx, tol + R.EPS[dtype] * 1.01 * dx.abs())


def test_norm_gradient_against_differences():
    # differences of the 64-bit definition: f(t) = sum of c * y(x + t dx, w + t dw)
    g = torch.Generator().manual_seed(5)
    freq, _ = rotary.rotary_frequencies(64, device="cpu")
    x, w = torch.randn(1, 9, 2, 64, generator=g), 1 + 0.2 * torch.randn(64, generator=g)
    c, dx, dw = (torch.randn(t.shape, generator=g) for t in (x, x, w))
    pos = torch.arange(9)[None]
    f = lambda t: (c.double() * R.rotary(norm(x.double() + t * dx, w.double() + t * dw, 1e-2)[0], pos,  # noqa: E731
                                         freq)).sum()
    h = 2.0 ** -16  # off by h^2 of third derivatives, and by 2^-52 of sums below 2^12 over h
    want = float((f(h) - f(-h)) / (2 * h))
    lx, lw = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    y = rotary.qk_norm_rotary_func(lx, None, lw, None, freq.cuda(), eps=1e-2)
    gx, gw = torch.autograd.grad(y, (lx, lw), (c.cuda(),))
    got = float((gx.cpu().double() * dx).sum() + (gw.cpu().double() * dw).sum())
    back = lambda d: R.rotary(d, pos, freq, inverse=True)  # noqa: E731
    _, _, tol_x, tol_w = norm_grads(x, c, w, 1e-2, back)
    tol = (tol_x * dx.abs()).sum() + (tol_w * dw.abs()).sum() + 1e-6
    assert abs(got - want) <= float(tol) + R.EPS[F32] * 1e4


def test_norm_parts_absent():
    g = torch.Generator().manual_seed(8)
    freq, _ = rotary.rotary_frequencies(64)
    q, k = (torch.randn(3, 20, h, 64, generator=g).cuda().requires_grad_() for h in (4, 2))
    w = torch.randn(64, generator=g).cuda().requires_grad_()
    one = torch.ones(64, device="cuda")
    d = torch.randn(3, 20, 4, 64, generator=g).cuda()
    dk = torch.randn(3, 20, 2, 64, generator=g).cuda()
    call = rotary.qk_norm_rotary_func
    # no weights are ones
    a, b = call(q, k, None, None, freq), call(q, k, one, one, freq)
    for x, y in zip(a + torch.autograd.grad(a, (q, k), (d, dk)),
                    b + torch.autograd.grad(b, (q, k), (d, dk))):
        assert torch.equal(x, y)
    # each operand and weight alone gives what it gives beside the others
    both = call(q, k, w, one, freq)
    gq, gk, gw = torch.autograd.grad(both, (q, k, w), (d, dk))
    y = call(q, None, w, None, freq)
    assert torch.equal(y, both[0])
    hq, hw = torch.autograd.grad(y, (q, w), (d,))
    assert torch.equal(hq, gq) and (hw - gw).abs().max() <= 2.0 ** -24 * 240 * 64 * 8
    mixed = call(q, k, w, None, freq)  # one result's gradient alone
    hk, = torch.autograd.grad(mixed[1], (k,), (dk,))
    assert torch.equal(hk, gk)
    qd, kd = q.detach(), k.detach()  # a weight that needs a gradient beside rows that do not
    hw2, = torch.autograd.grad(call(qd, kd, w, one, freq)[0], (w,), (d,))
    assert torch.equal(hw2, hw)
    assert torch.equal(call(qd, kd, w.detach(), one, freq)[0], both[0])
    # one weight for queries and keys
    yq, yk = call(q, k, w, w, freq)
    s, = torch.autograd.grad((yq, yk), (w,), (d, dk))
    kw, = torch.autograd.grad(call(kd, None, w, None, freq), (w,), (dk,))
    assert (s - hw - kw).abs().max() <= 2.0 ** -24 * 400 * 64 * 8


@pytest.mark.parametrize("dtype,D,H,Hk", [(F32, 64, 33000, 7), (BF, 128, 5, 30001), (HF, 64, 24, 40)])
def test_norm_many_heads(dtype, D, H, Hk):
    # more groups of heads than the gradient's kernel has warps, and uneven ones
    g = torch.Generator().manual_seed(H)
    freq, _ = rotary.rotary_frequencies(D, device="cpu")
    x = [torch.randn(1, 2, h, D, generator=g).to(dtype) for h in (H, Hk)]
    dy = [torch.randn(t.shape, generator=g).to(dtype) for t in x]
    w = [(1 + 0.3 * torch.randn(D, generator=g)) for _ in range(2)]
    pos = torch.tensor([[7, 1000]])
    leaves = [t.cuda().requires_grad_() for t in x + w]
    y = rotary.qk_norm_rotary_func(*leaves, freq.cuda(), positions=pos.cuda())
    got = torch.autograd.grad(y, leaves, [d.cuda() for d in dy])
    for i in range(2):
        xn, _ = norm(x[i], w[i], 1e-6)
        ref = turn(xn, pos, freq)
        close(y[i], ref, bound_norm(ref, xn, 1.0, dtype, D))
        dx, dw, tol_x, tol_w = norm_grads(x[i], dy[i], w[i], 1e-6, lambda d: turn(d, pos, freq, inverse=True))
        close(got[i], dx, tol_x + R.EPS[dtype] * 1.01 * dx.abs() + fp16_floor(dtype))
        close(got[2 + i], dw, tol_w + R.EPS[F32] * 1.01 * dw.abs())


def test_norm_broadcast_and_strided_gradients():
    g = torch.Generator().manual_seed(9)
    freq, _ = rotary.rotary_frequencies(64)
    x = torch.randn(2, 10, 1, 64, generator=g).cuda().requires_grad_()
    w = torch.ones(64, device="cuda", requires_grad=True)
    d = torch.randn(2, 10, 4, 64, generator=g).cuda()
    y = rotary.qk_norm_rotary_func(x.expand(2, 10, 4, 64), None, w, None, freq)
    up = d.transpose(1, 2).contiguous().transpose(1, 2)
    gx, gw = torch.autograd.grad(y, (x, w), (up,))
    z = rotary.qk_norm_rotary_func(x.repeat(1, 1, 4, 1), None, w, None, freq)
    hx, hw = torch.autograd.grad(z, (x, w), (d,))
    assert torch.equal(gw, hw) and (gx - hx).abs().max() <= 2.0 ** -20 * gx.abs().max()
    # a single broadcast number, and an odd address
    y = rotary.qk_norm_rotary_func(x, None, w, None, freq)
    a = torch.autograd.grad(y.sum(), (x, w), retain_graph=True)
    odd = torch.ones(2 * 10 * 64 + 1, device="cuda")[1:].view(2, 10, 1, 64)
    for u, v in zip(a, torch.autograd.grad(y, (x, w), (odd,))):
        assert torch.equal(u, v)


def test_norm_in_place_strided_streams_and_graphs():
    freq, _ = rotary.rotary_frequencies(128)
    w = torch.randn(128, device="cuda").to(BF)
    qkv = torch.randn(2, 21, 3, 4, 128, device="cuda").to(BF)
    keep = qkv.clone()
    call = lambda t, **kw: rotary.qk_norm_rotary_func(t[:, :, 0], t[:, :, 1], w, None, freq, **kw)  # noqa: E731
    want = call(keep)
    out = call(qkv, inplace=True)
    assert out[0].data_ptr() == qkv.data_ptr()
    assert torch.equal(qkv[:, :, 0], want[0]) and torch.equal(qkv[:, :, 1], want[1])
    assert torch.equal(qkv[:, :, 2], keep[:, :, 2])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = call(keep)
    s.synchronize()
    assert torch.equal(again[0], want[0])
    x = torch.zeros_like(keep)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = call(x)
        graphs.append((graph, y))
    x.copy_(keep)
    for graph, _ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for _, y in graphs:
        assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])


def test_norm_backward_in_a_graph_and_twice_the_same_bits():
    freq, _ = rotary.rotary_frequencies(64)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros(4, 700, 6, 64, device="cuda").requires_grad_()
    w = torch.ones(64, device="cuda").requires_grad_()
    d = torch.randn(x.shape, device="cuda", generator=gen)
    data = torch.randn(x.shape, device="cuda", generator=gen)

    def step():
        y = rotary.qk_norm_rotary_func(x, None, w, None, freq)
        return torch.autograd.grad(y, (x, w), (d,))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = step()
    torch.cuda.current_stream().wait_stream(s)
    with torch.no_grad():
        x.copy_(data)
    graph.replay()
    torch.cuda.synchronize()
    a, b = step(), step()
    for u, v, z in zip(got, a, b):
        assert torch.equal(u, v) and torch.equal(v, z)


def test_norm_empty_and_non_finite():
    freq, _ = rotary.rotary_frequencies(64)
    w = torch.ones(64, device="cuda", requires_grad=True)
    x = torch.zeros(2, 0, 4, 64, device="cuda", requires_grad=True)
    y = rotary.qk_norm_rotary_func(x, None, w, None, freq)
    gx, gw = torch.autograd.grad(y, (x, w), (torch.zeros_like(y),))
    assert y.shape == x.shape and gx.shape == x.shape and (gw == 0).all()
    # a row's values stay in the row, forward and back; the weights' gradient sees all
    x = torch.randn(1, 5, 3, 64, device="cuda")
    x[0, 2, 1, 7] = math.nan
    x[0, 4, 0, 9] = math.inf
    x.requires_grad_()
    y = rotary.qk_norm_rotary_func(x, None, w, None, freq)
    gx, = torch.autograd.grad(y, (x,), (torch.ones_like(y),))
    fine = torch.ones(5, 3, dtype=torch.bool, device="cuda")
    fine[2, 1] = fine[4, 0] = False
    for t in (y, gx):
        assert torch.isfinite(t[0][fine]).all() and not torch.isfinite(t[0, 2, 1]).any()


def test_norm_refusals():
    freq, _ = rotary.rotary_frequencies(64)
    x = torch.randn(2, 9, 3, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    call = rotary.qk_norm_rotary_func
    bad = [dict(q_weight=w[:32]), dict(q_weight=w.to(BF)), dict(k_weight=w), dict(q_weight=w.double()),
           dict(q_weight=torch.ones(64, 2, device="cuda")[:, 0]), dict(q_weight=torch.ones(64)),
           dict(sections=(10, 10)), dict(sections=(32,)), dict(sections=()),
           dict(sections=(16, 16), section_order="rows"), dict(sections=(-1, 33)),
           dict(sections=(16, 16), positions=torch.zeros(9, dtype=torch.int32, device="cuda")),
           dict(sections=(16, 16), positions=torch.zeros(3, 9, dtype=torch.int32, device="cuda"))]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            call(**{**dict(q=x, k=None, q_weight=w, k_weight=None, inv_freq=freq), **kw})
    for eps in (-1.0, math.nan, math.inf):
        with pytest.raises(fattn.FattnError):
            call(x, None, w, None, freq, eps=eps)
    with pytest.raises(ValueError):
        call(x, x, w, w, freq, inplace=True)
    with pytest.raises(ValueError):
        call(x, None, w.clone().requires_grad_(), None, freq, inplace=True)
    # once differentiable: a second time raises, and does not come out wrong
    x.requires_grad_()
    y = call(x, None, w, None, freq)
    gx, = torch.autograd.grad(y, (x,), (torch.ones_like(y),), create_graph=True)
    with pytest.raises(NotImplementedError):
        gx.sum().backward()
    # what the gradients need must not have changed
    y = call(x * 1, None, w, None, freq)
    z = x * 1
    y = call(z, None, w, None, freq)
    with torch.no_grad():
        z += 1
    with pytest.raises(RuntimeError):
        y.sum().backward()
    v = w.clone().requires_grad_()
    y = call(x * 1, None, v, None, freq)
    with torch.no_grad():
        v += 1
    with pytest.raises(RuntimeError):
        y.sum().backward()
