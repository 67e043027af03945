"""Weights of the norm with rotation that lie at any address, as views into one buffer of a
model's parameters do."""
import pytest
import torch

from exact_attention_93_gb300 import rotary

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype,wtype", [(BF, BF), (HF, HF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_weights_at_any_address(D, dtype, wtype, interleaved):
    freq, _ = rotary.rotary_frequencies(D)
    g = torch.Generator(device="cuda").manual_seed(D)
    draw = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    q, k = draw(2, 19, 5, D).to(dtype), draw(2, 19, 2, D).to(dtype)
    dy, du = torch.randn_like(q), torch.randn_like(k)
    flat = draw(2 * D + 8).to(wtype)

    def run(first, second, copy):
        x, u, w = q.clone().requires_grad_(), k.clone().requires_grad_(), flat.clone().requires_grad_()
        wq, wk = w[first:first + D], w[second:second + D]
        if copy:
            wq, wk = wq.clone(), wk.clone()
        else:
            assert wq.data_ptr() % 8 or wk.data_ptr() % 8
        y, z = rotary.qk_norm_rotary_func(x, u, wq, wk, freq, interleaved=interleaved)
        with torch.no_grad():
            plain = rotary.qk_norm_rotary_func(x, u, wq, wk, freq, interleaved=interleaved)
        return (y, z, *plain, *torch.autograd.grad((y, z), (x, u, w), (dy, du)))

    for first, second in ((1, D + 5), (0, D + 1), (3, D + 4)):
        for a, b in zip(run(first, second, False), run(first, second, True)):
            assert torch.equal(a, b)
