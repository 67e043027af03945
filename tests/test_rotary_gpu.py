"""Rotary positions against 64 bits on the GPU: values, gradients, layouts."""
import pytest
import torch

import paged_ref as R
from exact_attention_93_gb300 import fattn, rotary

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def bound(ref, x, magnitude, dtype):
    """The angle is off by 2^-32 turns and its fp32 remainder by 2^-24 of pi/4,
    sine and cosine by 2^-23, so a rotated pair by 2^-21 of its length times
    the magnitude; then one rounding to the type."""
    pair = x.double().abs().amax(-1, keepdim=True) * 2 ** 0.5 * max(1.0, abs(magnitude))
    return R.EPS[dtype] * 1.01 * ref.abs() + 2.0 ** -21 * pair + (2.0 ** -25 if dtype == HF else 0)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("D,rdim", [(64, 64), (64, 16), (128, 128), (128, 64), (128, 96)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_values(dtype, D, rdim, interleaved):
    g = torch.Generator().manual_seed(D + rdim)
    freq, mag = rotary.rotary_frequencies(rdim, scaling="by_parts", factor=8.0,
                                          original_length=2048, device="cpu")
    for B, N, H, Hk in ((1, 1, 1, 1), (2, 37, 5, 3), (3, 130, 17, 1), (1, 5, 40, 8)):
        q = torch.randn(B, N, H, D, generator=g).to(dtype)
        k = torch.randn(B, N, Hk, D, generator=g).to(dtype)
        pos = torch.randint(0, 1 << 20, (B, N), generator=g)
        yq, yk = rotary.rotary_func(q.cuda(), k.cuda(), freq.cuda(), positions=pos.cuda(),
                                    interleaved=interleaved, magnitude=mag)
        for x, y in ((q, yq), (k, yk)):
            ref = R.rotary(x, pos, freq, interleaved, mag)
            assert y.shape == x.shape and y.dtype == dtype
            assert ((y.cpu().double() - ref).abs() <= bound(ref, x, mag, dtype)).all()
            assert torch.equal(y.cpu()[..., rdim:], x[..., rdim:])


@pytest.mark.parametrize("kind", ["none", "int32", "shared", "packed", "negative"])
def test_positions(kind):
    g = torch.Generator().manual_seed(1)
    B, N, H, D = 2, 50, 4, 64
    freq, _ = rotary.rotary_frequencies(D, device="cpu")
    q = torch.randn(B, N, H, D, generator=g)
    pos, given = torch.arange(N).expand(B, N), None
    if kind == "int32":
        pos = torch.randint(0, 1 << 30, (B, N), generator=g)
        given = pos.to(torch.int32)
    elif kind == "shared":
        pos = torch.randint(0, 1 << 40, (N,), generator=g)
        given, pos = pos, pos.expand(B, N)
        # fp64 has no 2^-32 turns at such positions: integer angles keep it exact
        freq = torch.zeros_like(freq)
    elif kind == "negative":
        pos = -torch.randint(0, 1 << 16, (B, N), generator=g)
        given = pos
    if kind == "packed":
        y = rotary.rotary_func(q[0].cuda(), None, freq.cuda())[None]
        q, pos = q[:1], pos[:1]
    else:
        y = rotary.rotary_func(q.cuda(), None, freq.cuda(),
                               positions=None if given is None else given.cuda())
    ref = R.rotary(q, pos, freq)
    # the reference's own angle: position times 2^-53 of it
    own = pos.abs().double().amax() * 2.0 ** -52 * q.double().abs().amax() * 2
    assert ((y.cpu().double() - ref).abs() <= bound(ref, q, 1.0, F32) + own).all()


@pytest.mark.parametrize("scaling,factor", [(None, 1.0), ("linear", 4.0), ("ntk", 8.0),
                                            ("by_parts", 16.0)])
def test_round_trip_keeps_lengths_and_relative_products(scaling, factor):
    freq, mag = rotary.rotary_frequencies(128, scaling=scaling, factor=factor,
                                          original_length=4096)
    q = torch.randn(1, 64, 2, 128, device="cuda")
    k = torch.randn(1, 64, 2, 128, device="cuda")
    prods = []
    for shift in (0, 100000):
        pos = torch.arange(64, device="cuda") + shift
        a, b = rotary.rotary_func(q, k, freq, positions=pos, magnitude=mag)
        prods.append(torch.einsum("bihd,bjhd->bhij", a.double(), b.double()))
    # the product of a query and a key goes by their distance alone
    assert (prods[0] - prods[1]).abs().max() <= 2.0 ** -20 * 128 * 20 * mag ** 2


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients(dtype, interleaved):
    g = torch.Generator().manual_seed(3)
    B, N, D = 2, 33, 128
    freq, mag = rotary.rotary_frequencies(64, scaling="by_parts", factor=4.0, original_length=64)
    q = torch.randn(B, N, 6, D, generator=g).to(dtype).cuda().requires_grad_()
    k = torch.randn(B, N, 2, D, generator=g).to(dtype).cuda().requires_grad_()
    pos = torch.randint(0, 100000, (B, N), generator=g).cuda()
    yq, yk = rotary.rotary_func(q, k, freq, positions=pos, interleaved=interleaved, magnitude=mag)
    dq, dk = (torch.randn(t.shape, generator=g).to(dtype) for t in (yq, yk))
    # gradients as other operators leave them: transposed, and expanded over heads
    up = dq.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    got = torch.autograd.grad((yq, yk), (q, k), (up, dk.cuda()))
    for d, x in zip((dq, dk), got):
        ref = R.rotary(d, pos.cpu(), freq.cpu(), interleaved, mag, inverse=True)
        assert ((x.cpu().double() - ref).abs() <= bound(ref, d, mag, dtype)).all()
    # one output alone, and a gradient that is a single broadcast number
    yq, yk = rotary.rotary_func(q, k, freq, positions=pos, interleaved=interleaved, magnitude=mag)
    gk, = torch.autograd.grad(yk.sum(), (k,))
    ref = R.rotary(torch.ones(B, N, 2, D), pos.cpu(), freq.cpu(), interleaved, mag, inverse=True)
    assert ((gk.cpu().double() - ref).abs() <= bound(ref, torch.ones(1), mag, dtype)).all()


def test_gradient_against_differences():
    freq, mag = rotary.rotary_frequencies(64, scaling="linear", factor=2.0)
    x = torch.randn(1, 9, 2, 64, device="cuda", requires_grad=True)
    w = torch.randn(1, 9, 2, 64, device="cuda")
    f = lambda t: (rotary.rotary_func(t, None, freq, magnitude=1.5).double() * w).sum()  # noqa: E731
    gx, = torch.autograd.grad(f(x), (x,))
    d = torch.randn_like(x)
    with torch.no_grad():
        # linear in x, so the difference is exact up to fp32 rounding of the two values
        diff = (f(x + d) - f(x - d)) / 2
    assert abs(float(diff - (gx.double() * d).sum())) <= 2.0 ** -20 * 9 * 2 * 64 * 10


def test_heads_shared_by_expansion():
    freq, _ = rotary.rotary_frequencies(64)
    x = torch.randn(2, 10, 1, 64, device="cuda", requires_grad=True)
    y = rotary.rotary_func(x.expand(2, 10, 4, 64), None, freq)
    w = torch.randn_like(y)
    gx, = torch.autograd.grad(y, (x,), (w,))
    ref = R.rotary(w.cpu(), torch.arange(10).expand(2, 10), freq.cpu(), inverse=True).sum(2, True)
    assert ((gx.cpu().double() - ref).abs() <= 2.0 ** -20 * 4 * 8).all()


def test_in_place_strided_streams_and_graphs():
    freq, _ = rotary.rotary_frequencies(128)
    qkv = torch.randn(2, 21, 3, 4, 128, device="cuda").to(BF)
    keep = qkv.clone()
    want = rotary.rotary_func(keep[:, :, 0], keep[:, :, 1], freq)
    out = rotary.rotary_func(qkv[:, :, 0], qkv[:, :, 1], freq, inplace=True)
    assert out[0].data_ptr() == qkv.data_ptr()
    assert torch.equal(qkv[:, :, 0], want[0]) and torch.equal(qkv[:, :, 1], want[1])
    assert torch.equal(qkv[:, :, 2], keep[:, :, 2])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = rotary.rotary_func(keep[:, :, 0], keep[:, :, 1], freq)
    s.synchronize()
    assert torch.equal(again[0], want[0])
    x = torch.zeros_like(keep)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = rotary.rotary_func(x[:, :, 0], x[:, :, 1], freq)
    x.copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])


def test_non_finite_values_stay_in_their_pair():
    freq, _ = rotary.rotary_frequencies(64)
    x = torch.randn(1, 3, 1, 64, device="cuda")
    x[0, 1, 0, 5] = float("nan")
    y = rotary.rotary_func(x, None, freq)
    bad = torch.isnan(y).nonzero().tolist()
    assert bad == [[0, 1, 0, 5], [0, 1, 0, 37]]


def test_empty():
    freq, _ = rotary.rotary_frequencies(64)
    assert rotary.rotary_func(torch.zeros(2, 0, 4, 64, device="cuda"), None, freq).shape == (2, 0, 4, 64)


def test_second_derivative():
    # the gradient is linear in what comes in: its own gradient is the rotation
    freq, _ = rotary.rotary_frequencies(64)
    x = torch.randn(1, 5, 2, 64, device="cuda", requires_grad=True)
    w = torch.randn(1, 5, 2, 64, device="cuda", requires_grad=True)
    y = rotary.rotary_func(x, None, freq, magnitude=2.0)
    gx, = torch.autograd.grad(y, (x,), (w,), create_graph=True)
    v = torch.randn_like(x)
    gw, = torch.autograd.grad(gx, (w,), (v,))
    ref = R.rotary(v.cpu(), torch.arange(5)[None], freq.cpu(), magnitude=2.0)
    assert ((gw.cpu().double() - ref).abs() <= 2.0 ** -20 * 2 * 8).all()


def test_backward_on_another_stream_and_leaf_accumulation():
    freq, _ = rotary.rotary_frequencies(64)
    x = torch.randn(2, 9, 3, 64, device="cuda", requires_grad=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y, z = rotary.rotary_func(x, x[:, :, :1], freq)
        (y.sum() + 2 * z.sum()).backward()
    torch.cuda.current_stream().wait_stream(s)
    one = torch.ones(2, 9, 3, 64)
    pos = torch.arange(9).expand(2, 9)
    ref = R.rotary(one, pos, freq.cpu(), inverse=True)
    ref[:, :, :1] += 2 * R.rotary(one[:, :, :1], pos, freq.cpu(), inverse=True)
    assert ((x.grad.cpu().double() - ref).abs() <= 2.0 ** -20 * 8).all()


def test_in_place_refusals_and_versions():
    freq, _ = rotary.rotary_frequencies(64)
    x = torch.randn(2, 9, 3, 64, device="cuda")
    keep = x.clone()
    with pytest.raises(ValueError):  # both results in one place
        rotary.rotary_func(x, x, freq, inplace=True)
    with pytest.raises(ValueError):
        rotary.rotary_func(x.requires_grad_(), None, freq, inplace=True)
    x = x.detach()
    with pytest.raises(fattn.FattnError):  # heads that share their elements
        rotary.rotary_func(x[:, :, :1].expand(-1, -1, 3, -1), None, freq, inplace=True)
    assert torch.equal(x, keep)
    a, b = rotary.rotary_func(x, x, freq)  # two results: allowed
    assert torch.equal(a, b)
    with pytest.raises(ValueError):
        rotary.rotary_func(x, None, freq.clone().requires_grad_())
    w = torch.ones(64, device="cuda", requires_grad=True)
    y = (x * w).sum()  # saves x
    rotary.rotary_func(x, None, freq, inplace=True)
    with pytest.raises(RuntimeError):
        y.backward()
