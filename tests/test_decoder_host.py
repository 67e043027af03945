"""The entry points of include/fattn_decoder.h on the host: declared, exported, and
refusing bad arguments before anything reaches CUDA.  No kernel runs here."""
import ctypes
import math
import subprocess

import pytest
import torch

from exact_attention_93_gb300 import attention, build, fattn, kvcache, rotary
from paged_ref import KvPages, Ragged, RotaryOperand

FAKE = 1 << 20  # aligned and never dereferenced: every call below fails its checks first
OK, INV, UNS = fattn.FA_OK, fattn.FA_ERR_INVALID_ARG, fattn.FA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return fattn.load()


def test_declared_and_exported(lib):
    names = fattn.declared_symbols(fattn.DECODER_HEADER)
    assert names == ["fa_cache_release", "fa_cache_reserve", "fa_cache_write",
                     "fa_fwd_paged_shared", "fa_fwd_paged_shared_workspace_size",
                     "fa_qk_norm_rotary", "fa_qk_norm_rotary_bwd",
                     "fa_qk_norm_rotary_bwd_workspace_size", "fa_rotary_axes"]
    out = subprocess.run(["nm", "-D", "--defined-only", fattn.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    assert set(names) <= {line.split()[-1] for line in out.splitlines() if line.strip()}


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "x.c"
    src.write_text('#include "fattn_decoder.h"\nint main(void) { fa_reserve r; fa_positions p; '
                   '(void)r; (void)p; return 0; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", build.INCLUDE, "-c", str(src),
                    "-o", str(tmp_path / "x.o")], check=True)


class Positions(ctypes.Structure):
    _fields_ = [("positions", ctypes.c_void_p), ("bits", ctypes.c_int), ("axes", ctypes.c_int),
                ("axis_stride", ctypes.c_longlong), ("batch_stride", ctypes.c_longlong),
                ("axis_of_pair", ctypes.c_char_p)]


class Reserve(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("new_tokens", "seqlens", "block_table")] +
                [("table_stride", ctypes.c_longlong), ("max_pages", ctypes.c_int),
                 ("free_pages", ctypes.c_void_p), ("capacity", ctypes.c_int),
                 ("free_count", ctypes.c_void_p), ("batch", ctypes.c_int),
                 ("page_size", ctypes.c_int), ("total", ctypes.c_int)] +
                [(n, ctypes.c_void_p) for n in ("cu_seqlens", "seqlens_out", "positions", "slots",
                                                "free_count_out", "missing")])


def positions(**kw):
    d = dict(positions=FAKE, bits=32, axes=2, axis_stride=10, batch_stride=5,
             axis_of_pair=bytes([0, 1] * 16))
    return Positions(**{**d, **kw})


def operand(D=64, heads=2, x=FAKE, y=2 * FAKE, unit=64):
    s = fattn.FaStrides(10 * heads * unit, unit, heads * unit)
    return RotaryOperand(x, y, heads, s, s)


BAD_POSITIONS = [dict(axes=0), dict(axes=9), dict(positions=None), dict(positions=None, bits=0),
                 dict(bits=16), dict(axis_of_pair=None), dict(axis_of_pair=bytes([0, 2] * 16)),
                 dict(axis_stride=-1), dict(batch_stride=-1), dict(positions=FAKE + 2)]


@pytest.mark.parametrize("kw", BAD_POSITIONS)
def test_positions(lib, kw):
    q, p = operand(), positions(**kw)
    a, b = ctypes.addressof(q), ctypes.addressof(p)
    assert lib.fa_rotary_axes(a, None, 1, 5, 64, 64, FAKE, b, 1.0, 0, 0, 0, None) == INV
    assert lib.fa_qk_norm_rotary(a, None, FAKE, None, 0, 1e-6, 1, 5, 64, 64, FAKE, b, 1.0, 0, 0,
                                 None) == INV
    # no tokens: positions need no address
    assert lib.fa_rotary_axes(a, None, 1, 0, 64, 64, FAKE, None, 1.0, 0, 0, 0, None) == INV


def test_nothing_to_turn(lib):
    q, p = operand(), positions(positions=None, bits=0)
    a, b = ctypes.addressof(q), ctypes.addressof(p)
    assert lib.fa_rotary_axes(a, None, 1, 0, 64, 64, FAKE, b, 1.0, 0, 0, 0, None) == OK
    assert lib.fa_qk_norm_rotary(a, None, FAKE, None, 0, 1e-6, 0, 5, 64, 64, FAKE, b, 1.0, 0, 0,
                                 None) == OK


NORM_BAD = [(dict(eps=-1e-6), INV), (dict(eps=math.nan), INV), (dict(eps=math.inf), INV),
            (dict(qw=FAKE + 4), INV), (dict(kw=FAKE), INV), (dict(wtype=1), UNS),
            (dict(wtype=3), UNS), (dict(D=96), UNS), (dict(dtype=3), UNS), (dict(rdim=24), INV),
            (dict(freq=None), INV), (dict(magnitude=math.inf), INV), (dict(x=FAKE + 8), INV),
            (dict(heads=0), INV), (dict(unit=4), INV)]


@pytest.mark.parametrize("kw,status", NORM_BAD)
def test_norm_arguments(lib, kw, status):
    d = {**dict(eps=1e-6, qw=FAKE, kw=None, wtype=0, D=64, dtype=0, rdim=64, freq=FAKE,
                magnitude=1.0, x=FAKE, heads=2, unit=64), **kw}
    q, p = operand(heads=d["heads"], x=d["x"], unit=d["unit"]), positions(axes=1)
    a, b = ctypes.addressof(q), ctypes.addressof(p)
    assert lib.fa_qk_norm_rotary(a, None, d["qw"], d["kw"], d["wtype"], d["eps"], 1, 5, d["D"],
                                 d["rdim"], d["freq"], b, d["magnitude"], 0, d["dtype"],
                                 None) == status
    s = fattn.FaStrides(640, 64, 128)
    assert lib.fa_qk_norm_rotary_bwd(a, None, 3 * FAKE, s, None, s, d["qw"], d["kw"], FAKE, None,
                                     d["wtype"], d["eps"], 1, 5, d["D"], d["rdim"], d["freq"], b,
                                     d["magnitude"], 0, d["dtype"], FAKE, 1 << 30, None) == status


def test_norm_gradient_arguments(lib):
    n = ctypes.c_size_t(9)
    assert lib.fa_qk_norm_rotary_bwd_workspace_size(96, ctypes.byref(n)) == UNS and n.value == 0
    assert lib.fa_qk_norm_rotary_bwd_workspace_size(64, None) == INV
    assert lib.fa_qk_norm_rotary_bwd_workspace_size(64, ctypes.byref(n)) == OK and n.value > 0
    p = positions(axes=1)
    s = fattn.FaStrides(640, 64, 128)

    def call(op=None, g=3 * FAKE, gs=s, ws=FAKE, size=n.value, dw=FAKE, dkw=None):
        op = op or operand()
        return lib.fa_qk_norm_rotary_bwd(ctypes.addressof(op), None, g, gs, None, s, FAKE, None, dw,
                                         dkw, 0, 1e-6, 1, 5, 64, 64, FAKE, ctypes.addressof(p), 1.0,
                                         0, 0, ws, size, None)
    for kw in (dict(g=None), dict(g=FAKE + 8), dict(gs=fattn.FaStrides(640, 63, 128)),
               dict(gs=fattn.FaStrides(640, -64, 128)), dict(ws=None), dict(ws=FAKE + 128),
               dict(size=n.value - 1), dict(dw=FAKE + 4), dict(dkw=FAKE),
               dict(op=operand(y=FAKE)), dict(g=2 * FAKE)):
        assert call(**kw) == INV, kw


RESERVE_BAD = [dict(new_tokens=None), dict(seqlens=FAKE + 2), dict(block_table=None),
               dict(table_stride=7), dict(max_pages=0), dict(max_pages=1 << 27, table_stride=1 << 27),
               dict(free_pages=None), dict(capacity=-1), dict(free_count=None), dict(batch=0),
               dict(batch=(1 << 20) + 1), dict(page_size=8), dict(page_size=48),
               dict(page_size=512), dict(total=-1), dict(total=(1 << 29) + 1),
               dict(cu_seqlens=None), dict(seqlens_out=None), dict(positions=None),
               dict(slots=FAKE + 4), dict(free_count_out=None), dict(missing=None)]


@pytest.mark.parametrize("kw", RESERVE_BAD)
def test_reserve_arguments(lib, kw):
    d = {n: FAKE for n, t in Reserve._fields_ if t is ctypes.c_void_p}
    d.update(table_stride=8, max_pages=8, capacity=100, batch=3, page_size=16, total=50)
    r = Reserve(**{**d, **kw})
    assert lib.fa_cache_reserve(ctypes.addressof(r), None) == INV
    assert lib.fa_cache_reserve(None, None) == INV


@pytest.mark.parametrize("kw", [dict(done=None), dict(lens=None), dict(keep=FAKE + 1), dict(table=None),
                                dict(stride=7), dict(pages=0), dict(free=None), dict(cap=-1),
                                dict(count=None), dict(batch=0), dict(size=100)])
def test_release_arguments(lib, kw):
    d = {**dict(done=FAKE, lens=FAKE, keep=None, table=FAKE, stride=8, pages=8, free=FAKE, cap=10,
                count=FAKE, batch=3, size=16), **kw}
    assert lib.fa_cache_release(*(d[n] for n in ("done", "lens", "keep", "table", "stride", "pages",
                                                 "free", "cap", "count", "batch", "size")),
                                None) == INV


def pages(**kw):
    d = dict(k=FAKE, v=2 * FAKE, k_exp=None, v_exp=None, k_page=16 * 128, k_token=128, k_head=64,
             v_page=16 * 128, v_token=128, v_head=64, pages=4, page_size=16, heads=2, head_dim=64,
             type=fattn.FA_ELEM_BF16)
    return KvPages(**{**d, **kw})


@pytest.mark.parametrize("kw,call,status", [
    (dict(k=None), {}, INV), (dict(page_size=24), {}, UNS), (dict(head_dim=96), {}, UNS),
    (dict(type=1), {}, UNS), (dict(type=3), {}, INV), (dict(v=FAKE), {}, INV),
    (dict(k_token=32), {}, INV), ({}, dict(slots=None), INV), ({}, dict(slots=FAKE + 4), INV),
    ({}, dict(total=-1), INV), ({}, dict(total=(1 << 29) + 1), INV), ({}, dict(k=FAKE + 2), INV),
    ({}, dict(stride=-128), INV)])
def test_write_arguments(lib, kw, call, status):
    c = pages(**kw)
    d = {**dict(slots=FAKE, total=5, k=FAKE, stride=128), **call}
    assert lib.fa_cache_write(ctypes.addressof(c), d["slots"], d["total"], d["k"], d["stride"], 64,
                              FAKE, 128, 64, 0, None) == status
    assert lib.fa_cache_write(None, FAKE, 5, FAKE, 128, 64, FAKE, 128, 64, 0, None) == INV
    if not kw:
        assert lib.fa_cache_write(ctypes.addressof(c), None, 0, None, 128, 64, None, 128, 64, 0,
                                  None) == OK


def test_shared_arguments(lib):
    c = pages()
    r = Ragged(FAKE, 200, 200, FAKE, FAKE, 4, 4)
    n = ctypes.c_size_t(7)
    r.max_pages = r.table_stride = 1 << 20  # so wide that sharing pays
    size = lambda groups, total=4: lib.fa_fwd_paged_shared_workspace_size(  # noqa: E731
        4, total, 4, 2, 64, 1 << 24, groups, ctypes.byref(n))
    assert size(-1) == INV and size(5) == INV
    assert size(0) == OK
    plain = ctypes.c_size_t()
    assert lib.fa_fwd_paged_workspace_size(4, 4, 4, 2, 64, 1 << 24, ctypes.byref(plain)) == OK
    assert n.value == plain.value
    assert size(2) == OK and n.value > plain.value + 2 * 4 * 4 * 64 * 4

    def call(groups=2, cu=FAKE, shared=FAKE, ws=FAKE, bytes_=n.value, q=FAKE, o=2 * FAKE, scale=0.1):
        return lib.fa_fwd_paged_shared(q, 256, 64, o, 256, 64, FAKE, ctypes.addressof(c),
                                       ctypes.addressof(r), cu, shared, groups, 4, scale, 0, ws,
                                       bytes_, None)
    for kw in (dict(groups=-1), dict(groups=5), dict(cu=None), dict(cu=FAKE + 2), dict(shared=None),
               dict(ws=None), dict(ws=FAKE + 64), dict(bytes_=n.value // 2), dict(q=None),
               dict(o=FAKE), dict(scale=math.nan)):
        assert call(**kw) == INV, kw


# ---- the Python calls, on the CPU: refused for what they are before the device

def i32(*v):
    return torch.tensor(v, dtype=torch.int32)


def test_python_refusals():
    x, w = torch.zeros(2, 9, 3, 64), torch.ones(64)
    freq, _ = rotary.rotary_frequencies(64, device="cpu")
    p2 = torch.zeros(2, 9, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        rotary.rotary_func(x, None, freq, positions=p2, sections=(16, 16))
    with pytest.raises(ValueError, match="CUDA"):
        rotary.qk_norm_rotary_func(x, None, w, None, freq)
    for kw, what in ((dict(sections=(16, 15)), "add up"), (dict(sections=(16, 16)), "need positions"),
                     (dict(sections=(40, -8), positions=p2), "add up"),
                     (dict(sections=(4,) * 9, positions=p2), "1 to 8"),
                     (dict(sections=(16, 16), positions=p2[0]), "axes"),
                     (dict(sections=(16, 16), positions=p2[:, :8]), "axes"),
                     (dict(sections=(16, 16), positions=p2, section_order="x"), "section_order"),
                     (dict(sections=(16, 16), positions=p2, section_order=None), "section_order")):
        for call in (lambda **k: rotary.rotary_func(x, None, freq, **k),
                     lambda **k: rotary.qk_norm_rotary_func(x, None, w, None, freq, **k)):
            with pytest.raises(ValueError, match=what):
                call(**kw)
    for bad in (5, (16.0, 16), ("16", "16")):
        with pytest.raises(TypeError):
            rotary.rotary_func(x, None, freq, positions=p2, sections=bad)
    with torch.autograd.forward_ad.dual_level():
        d = lambda t: torch.autograd.forward_ad.make_dual(t, torch.ones_like(t))  # noqa: E731
        for a in ((d(x), None, w, None, freq), (x, None, d(w), None, freq), (x, d(x), w, None, freq),
                  (x, x, w, d(w), freq)):
            with pytest.raises(NotImplementedError):
                rotary.qk_norm_rotary_func(*a)


def test_python_table_refusals():
    table, free = torch.zeros(3, 4, dtype=torch.int32), i32(*range(9))
    n, c = i32(1, 1, 1), i32(9)
    good = dict(new_tokens=n, seqlens=n, block_table=table, free_pages=free, free_count=c,
                page_size=16, total=3)
    with pytest.raises(ValueError, match="CUDA"):
        kvcache.kv_cache_reserve(**good)
    for kw in (dict(new_tokens=n.long()), dict(seqlens=n[:2]), dict(block_table=table.t()),
               dict(block_table=table.long()), dict(block_table=table[0]), dict(free_pages=free[::2]),
               dict(block_table=table[:, :3].as_strided((3, 4), (2, 1))),
               dict(free_count=i32(1, 2)), dict(page_size=20), dict(total=-1), dict(total=1 << 40)):
        with pytest.raises(ValueError) as e:
            kvcache.kv_cache_reserve(**{**good, **kw})
        assert "CUDA" not in str(e.value), kw
    done = torch.zeros(3, dtype=torch.bool)
    rel = dict(done=done, seqlens=n, block_table=table, free_pages=free, free_count=c, page_size=16)
    with pytest.raises(ValueError, match="CUDA"):
        kvcache.kv_cache_release(**rel)
    for kw in (dict(done=n), dict(done=done[:2]), dict(keep_pages=n[:2]), dict(keep_pages=n.long())):
        with pytest.raises(ValueError) as e:
            kvcache.kv_cache_release(**{**rel, **kw})
        assert "CUDA" not in str(e.value), kw
    kp, vp, _, _ = kvcache.alloc_kv_cache(2, 16, 2, 64, device="cpu")
    x, slots = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        kvcache.kv_cache_write(x, x, kp, vp, slots)
    for s in (slots.int(), slots[:2], torch.zeros(6, dtype=torch.int64)[::2]):
        with pytest.raises(ValueError, match="slots"):
            kvcache.kv_cache_write(x, x, kp, vp, s)
    with pytest.raises(ValueError, match="no gradients"):
        kvcache.kv_cache_write(x.clone().requires_grad_(), x, kp, vp, slots)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    args = (q, kp, vp, torch.zeros(1, 2, dtype=torch.int32), i32(0, 3), i32(3))
    for kw in (dict(cu_groups=i32(0, 1)), dict(shared_pages=i32(1)),
               dict(cu_groups=i32(0, 1), shared_pages=i32(1), causal=False),
               dict(cu_groups=i32(0, 1, 1), shared_pages=i32(1, 0))):
        with pytest.raises(ValueError) as e:
            attention.flash_attn_paged_func(*args, **kw)
        assert "CUDA" not in str(e.value), kw
