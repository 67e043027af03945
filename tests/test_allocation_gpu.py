"""The calls' results are allocated as torch allocates its own: filled where deterministic
algorithms ask for that, and seen by dispatch modes and by the profiler."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import paged_ref as R
from exact_attention_93_gb300 import attention, kvcache, rotary

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture
def deterministic():
    before = torch.are_deterministic_algorithms_enabled()
    fills = torch.utils.deterministic.fill_uninitialized_memory
    torch.use_deterministic_algorithms(True)
    yield
    torch.use_deterministic_algorithms(before)
    torch.utils.deterministic.fill_uninitialized_memory = fills


def used_memory():
    """Leaves blocks that are no NaN to the allocator, whatever the calls then ask for."""
    for n in (1 << 10, 1 << 12, 1 << 14, 1 << 16, 1 << 20, 1 << 22):
        del_me = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
        del del_me


@pytest.mark.parametrize("dtype,fp8", [(BF, False), (HF, True)])
def test_rows_behind_the_last_sequence(deterministic, dtype, fp8):
    b = R.Batch([1, 2], [20, 30], 2, 64, 16, dtype, fp8, tail=5)
    k, v, table, cu, lens, kw = b.gpu()
    q = torch.randn(b.total, 4, 64, device="cuda").to(dtype)
    n = sum(b.rows)
    for fills in (True, False):
        torch.utils.deterministic.fill_uninitialized_memory = fills
        used_memory()
        o, lse = attention.flash_attn_paged_func(q, k, v, table, cu, lens, return_lse=True, **kw)
        assert not torch.isnan(o[:n]).any() and not torch.isnan(lse[:, :n]).any()
        kr, vr = kvcache.kv_cache_read(k, v, table, cu, b.total, dtype=dtype, **kw)
        assert not torch.isnan(kr[:n]).any() and not torch.isnan(vr[:n]).any()
        if fills:
            for t in (o[n:], lse[:, n:], kr[n:], vr[n:]):
                assert torch.isnan(t).all()


class Seen(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.names = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.names.append(str(func))
        return func(*args, **(kwargs or {}))


def calls():
    freq, _ = rotary.rotary_frequencies(64)
    x = torch.randn(9, 2, 64, device="cuda").to(BF)
    w = x.clone().requires_grad_()
    b = R.Batch([1, 2], [20, 30], 2, 64, 16, BF, False)
    k, v, table, cu, lens, _ = b.gpu()
    return [lambda: rotary.rotary_func(x, None, freq), lambda: rotary.rotary_func(w, None, freq),
            lambda: kvcache.kv_cache_read(k, v, table, cu, 3),
            lambda: attention.flash_attn_paged_func(x[:3], k, v, table, cu, lens)]


@pytest.mark.parametrize("which", range(4))
def test_dispatch_modes_see_the_allocations(which):
    call = calls()[which]
    with Seen() as seen:
        call()
    assert any(n.startswith("aten.empty.") for n in seen.names), seen.names


def test_the_profiler_sees_the_allocations():
    call = calls()[0]
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU]) as prof:
        call()
    assert any(e.key == "aten::empty" for e in prof.key_averages())
