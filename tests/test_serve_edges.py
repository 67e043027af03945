"""What the serving calls refuse on the host, beyond shapes and types, and how
their native module is built.  No kernel runs here."""
import pytest
import torch

from exact_attention_93_gb300 import attention, kvcache, rotary


def small():
    """A cache of one sequence of three keys, on the CPU: every call on it is refused."""
    kp, vp, _, _ = kvcache.alloc_kv_cache(2, 16, 2, 64, device="cpu")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    x, q = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    return x, q, kp, vp, (torch.zeros(1, 2, dtype=torch.int32), i32(0, 3), i32(3))


def test_tangents_are_refused():
    x, q, kp, vp, (table, cu, lens) = small()
    freq, _ = rotary.rotary_frequencies(64, device="cpu")
    with torch.autograd.forward_ad.dual_level():
        d = lambda t: torch.autograd.forward_ad.make_dual(t, torch.ones_like(t))  # noqa: E731
        for grad in (torch.enable_grad(), torch.no_grad()):
            with grad:
                for call in (lambda: rotary.rotary_func(d(x), None, freq),
                             lambda: rotary.rotary_func(x, d(x), freq, inplace=True),
                             lambda: rotary.rotary_func(x, None, d(freq)),
                             lambda: kvcache.kv_cache_append(x, d(x), kp, vp, table, cu, lens),
                             lambda: kvcache.kv_cache_read(kp, d(vp), table, cu, 3),
                             lambda: attention.flash_attn_paged_func(d(q), kp, vp, table, cu, lens)):
                    with pytest.raises(NotImplementedError):
                        call()
