"""The entry points of include/fattn_cache.h on the host: declared, exported,
and refusing bad arguments before anything reaches CUDA.  No kernel runs
here."""
import ctypes
import math
import subprocess

import pytest
import torch

from exact_attention_93_gb300 import attention, build, fattn, kvcache, rotary
from paged_ref import KvPages, Ragged, RotaryOperand

FAKE = 1 << 20  # aligned and never dereferenced: every call below fails its checks first
INV, UNS = fattn.FA_ERR_INVALID_ARG, fattn.FA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return fattn.load()


def test_declared_and_exported(lib):
    names = fattn.declared_symbols(fattn.CACHE_HEADER)
    assert names == ["fa_cache_append", "fa_cache_read", "fa_fwd_paged",
                     "fa_fwd_paged_workspace_size", "fa_rotary"]
    out = subprocess.run(["nm", "-D", "--defined-only", fattn.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert set(names) <= exported


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "x.c"
    src.write_text('#include "fattn_cache.h"\nint main(void) { fa_kv_pages c; (void)c; return 0; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", build.INCLUDE, "-c", str(src),
                    "-o", str(tmp_path / "x.o")], check=True)


def pages(**kw):
    D = kw.get("head_dim", 64)
    d = dict(k=FAKE, v=FAKE, k_exp=None, v_exp=None, k_page=16 * 2 * D, k_token=2 * D, k_head=D,
             v_page=16 * 2 * D, v_token=2 * D, v_head=D, pages=4, page_size=16, heads=2,
             head_dim=64, type=fattn.FA_ELEM_BF16)
    d.update(kw)
    return KvPages(**d)


def ragged(**kw):
    d = dict(block_table=FAKE, table_stride=8, max_pages=8, cu_seqlens=FAKE, seqlens=FAKE, batch=2,
             total=5)
    d.update(kw)
    return Ragged(**d)


BAD_CACHE = [
    (dict(k=None), {}, INV), (dict(v=FAKE + 8), {}, INV), (dict(pages=0), {}, INV),
    (dict(heads=0), {}, INV), (dict(page_size=24), {}, UNS), (dict(page_size=8), {}, UNS),
    (dict(page_size=512), {}, UNS), (dict(head_dim=96), {}, UNS), (dict(type=2), {}, UNS),
    (dict(type=fattn.FA_ELEM_FP16), {}, UNS),                   # not the rows' type
    (dict(type=fattn.FA_ELEM_E4M3), {}, INV),                   # no exponents
    (dict(k_token=-128), {}, INV), (dict(k_head=4), {}, INV), (dict(v_page=1 << 50), {}, INV),
    ({}, dict(batch=0), INV), ({}, dict(total=-1), INV), ({}, dict(max_pages=0), INV),
    ({}, dict(table_stride=7), INV), ({}, dict(block_table=None), INV),
    ({}, dict(cu_seqlens=FAKE + 2), INV), ({}, dict(max_pages=1 << 27, table_stride=1 << 27), INV),
    ({}, dict(total=1 << 30), INV),
]


@pytest.mark.parametrize("c,b,status", BAD_CACHE)
def test_cache_arguments(lib, c, b, status):
    c, b = pages(**c), ragged(**b)
    pc, pb = ctypes.addressof(c), ctypes.addressof(b)
    assert lib.fa_cache_append(pc, pb, FAKE, 128, 64, FAKE, 128, 64, 0, None) == status
    assert lib.fa_cache_read(pc, pb, None, FAKE, 128, 64, FAKE, 128, 64, 0, None) == status
    assert lib.fa_fwd_paged(FAKE, 256, 64, FAKE, 256, 64, FAKE, pc, pb, 4, None, 0.125, 1, 0, FAKE,
                            1 << 30, None) == status


def test_rows_and_null_structs(lib):
    c, b = pages(), ragged()
    pc, pb = ctypes.addressof(c), ctypes.addressof(b)
    assert lib.fa_cache_append(None, pb, FAKE, 128, 64, FAKE, 128, 64, 0, None) == INV
    assert lib.fa_cache_append(pc, None, FAKE, 128, 64, FAKE, 128, 64, 0, None) == INV
    assert lib.fa_cache_append(pc, pb, None, 128, 64, FAKE, 128, 64, 0, None) == INV
    assert lib.fa_cache_append(pc, pb, FAKE, 128, 64, FAKE, 128, 60, 0, None) == INV
    assert lib.fa_cache_append(pc, pb, FAKE, 128, 64, FAKE, 128, 64, 2, None) == UNS
    assert lib.fa_cache_read(pc, pb, FAKE + 1, FAKE, 128, 64, FAKE, 128, 64, 0, None) == INV
    n = ragged(seqlens=None)
    assert lib.fa_cache_append(pc, ctypes.addressof(n), FAKE, 128, 64, FAKE, 128, 64, 0,
                               None) == INV
    e = pages(v=2 * FAKE, v_head=0)  # heads, or keys and values, that share elements
    assert lib.fa_cache_append(ctypes.addressof(e), pb, FAKE, 128, 64, FAKE, 128, 64, 0,
                               None) == INV
    assert lib.fa_cache_append(pc, pb, FAKE, 128, 64, FAKE, 128, 64, 0, None) == INV
    assert lib.fa_cache_read(pc, pb, None, FAKE, 128, 64, FAKE, 128, 64, 0, None) == INV
    assert lib.fa_cache_read(pc, pb, None, FAKE, 0, 64, 2 * FAKE, 128, 64, 0, None) == INV
    z = ragged(total=0)  # nothing to do, nothing to check the rows of
    assert lib.fa_cache_append(pc, ctypes.addressof(z), None, 0, 0, None, 0, 0, 0, None) == 0


def paged(lib, heads=4, scale=0.125, opts=None, ws=FAKE, ws_bytes=1 << 30, q=FAKE, q_token=256,
          o=FAKE, lse=FAKE):
    c, b = pages(), ragged(max_pages=1000, table_stride=1000)
    return lib.fa_fwd_paged(q, q_token, 64, o, 256, 64, lse, ctypes.addressof(c),
                            ctypes.addressof(b), heads,
                            None if opts is None else ctypes.addressof(opts), scale, 1, 0, ws,
                            ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(heads=3), INV), (dict(heads=0), INV), (dict(heads=2 * 129), INV),
    (dict(scale=math.nan), INV), (dict(scale=math.inf), INV), (dict(ws=None), INV),
    (dict(ws=FAKE + 128), INV), (dict(ws_bytes=64), INV), (dict(q=FAKE + 2), INV),
    (dict(q_token=252), INV), (dict(o=None), INV), (dict(o=FAKE), INV), (dict(lse=FAKE + 1), INV),
    (dict(opts=fattn.FaOptions(-2, 0, None, 0, None, 0)), INV),
    (dict(opts=fattn.FaOptions(0, -2, None, 0, None, 0)), INV),
    (dict(opts=fattn.FaOptions(-1, -1, FAKE + 2, 0, None, 0)), INV),
    (dict(opts=fattn.FaOptions(-1, -1, None, 0, FAKE, 0)), UNS),  # block masks
])
def test_paged_arguments(lib, kw, status):
    assert paged(lib, **kw) == status


def test_workspace_size(lib):
    n = ctypes.c_size_t()
    size = lambda *a: (lib.fa_fwd_paged_workspace_size(*a, ctypes.byref(n)), n.value)  # noqa: E731
    st, long = size(1, 1, 8, 2, 64, 1 << 20)
    assert st == fattn.FA_OK and long > 0 and long % 256 == 0
    assert size(1, 1, 8, 2, 64, 16) == (fattn.FA_OK, 0)  # short tables need none
    assert size(1, 1000, 8, 2, 64, 1 << 20)[1] > long    # more rows, larger blocks
    # single tokens, and with a chunk among them: either kernel's blocks fit
    assert size(200, 200, 8, 2, 64, 1 << 20)[1] < size(200, 701, 8, 2, 64, 1 << 20)[1]
    for bad, want in (((0, 1, 8, 2, 64, 16), INV), ((1, 1, 8, 3, 64, 16), INV),
                      ((1, 1, 8, 2, 96, 16), UNS), ((1, -1, 8, 2, 64, 16), INV),
                      ((1, 1, 8, 2, 64, -1), INV)):
        assert size(*bad) == (want, 0)
    assert lib.fa_fwd_paged_workspace_size(1, 1, 8, 2, 64, 16, None) == INV


def rot(lib, B=1, N=4, D=64, r=64, freq=FAKE, pos=None, bits=0, stride=0, mag=1.0, dtype=0, x=FAKE,
        y=2 * FAKE, heads=2, xs=(512, 64, 128), ys=(512, 64, 128)):
    op = RotaryOperand(x, y, heads, fattn.FaStrides(*xs), fattn.FaStrides(*ys))
    return lib.fa_rotary(ctypes.addressof(op), None, B, N, D, r, freq, pos, bits, stride, mag, 0, 0,
                         dtype, None)


@pytest.mark.parametrize("kw,status", [
    (dict(D=96), UNS), (dict(dtype=3), UNS), (dict(r=0), INV), (dict(r=80), INV), (dict(r=24), INV),
    (dict(B=-1), INV), (dict(freq=None), INV), (dict(freq=FAKE + 4), INV), (dict(bits=32), INV),
    (dict(pos=FAKE, bits=16), INV), (dict(pos=FAKE + 4, bits=64), INV),
    (dict(pos=FAKE, bits=32, stride=-1), INV), (dict(mag=math.nan), INV), (dict(x=None), INV),
    (dict(y=FAKE + 8), INV), (dict(heads=0), INV), (dict(xs=(512, 60, 128)), INV),
    (dict(xs=(512, -64, 128)), INV),
    (dict(y=FAKE, ys=(512, 64, 192)), INV),   # in place with other strides
    (dict(ys=(512, 0, 128)), INV),            # heads written over each other
    (dict(y=FAKE, xs=(512, 0, 128), ys=(512, 0, 128)), INV),
])
def test_rotary_arguments(lib, kw, status):
    assert rot(lib, **kw) == status


def test_rotary_of_nothing(lib):
    assert rot(lib, N=0, x=None, y=None) == fattn.FA_OK


# ---- the Python entry points refuse on the host as well

def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def i32(*v):
    return torch.tensor(v, dtype=torch.int32)


def test_python_refusals():
    kp, vp, _, _ = kvcache.alloc_kv_cache(2, 16, 2, 64, device="cpu")
    table, cu, lens = torch.zeros(1, 2, dtype=torch.int32), i32(0, 3), i32(3)
    x = t(3, 2, 64)
    args = (kp, vp, table, cu, lens)
    with pytest.raises(ValueError):  # CPU tensors
        kvcache.kv_cache_append(x, x, *args)
    with pytest.raises(ValueError):
        kvcache.kv_cache_read(kp, vp, table, cu, 3)
    with pytest.raises(ValueError):
        attention.flash_attn_paged_func(t(3, 4, 64), *args)
    for bad in ((x, t(3, 1, 64)), (t(3, 2, 128), t(3, 2, 128)), (x, x.half())):
        with pytest.raises(ValueError):
            kvcache.kv_cache_append(*bad, *args)
    for bad in (torch.zeros(1, 2), torch.zeros(2, dtype=torch.int32)):
        with pytest.raises(ValueError):
            kvcache.kv_cache_append(x, x, kp, vp, bad, cu, lens)
    with pytest.raises(ValueError):
        kvcache.kv_cache_append(x, x, kp, vp, table, cu.long(), lens)
    with pytest.raises(ValueError):
        kvcache.kv_cache_append(x, x, kp, vp, table, cu, i32(3, 3))
    with pytest.raises(TypeError):
        kvcache.kv_cache_append(x, x, kp, vp, table, cu, None)
    with pytest.raises(TypeError):
        kvcache.kv_cache_append(x, "x", kp, vp, table, cu, lens)
    with pytest.raises(TypeError):  # neither bf16 nor fp16
        kvcache.kv_cache_read(kp, vp, table, cu, 3, dtype=torch.float32)
    with pytest.raises(ValueError):  # a result of another size
        kvcache.kv_cache_read(kp, vp, table, cu, 3, out=(t(2, 2, 64), t(2, 2, 64)))
    with pytest.raises(ValueError):  # half a result
        kvcache.kv_cache_read(kp, vp, table, cu, 3, out=(t(3, 2, 64), None))
    with pytest.raises(ValueError):  # exponents with a 16-bit cache, and an e4m3 one without
        kvcache.kv_cache_append(x, x, *args, k_exp=torch.zeros(2, 2, 16, dtype=torch.uint8))
    k8, v8, ke, ve = kvcache.alloc_kv_cache(2, 16, 2, 64, torch.float8_e4m3fn, device="cpu")
    with pytest.raises(ValueError):
        kvcache.kv_cache_append(x, x, k8, v8, table, cu, lens)
    with pytest.raises(ValueError):
        kvcache.kv_cache_append(x, x, k8, v8, table, cu, lens, k_exp=ke, v_exp=ve[:1])
    with pytest.raises(ValueError):  # gradients would be lost
        kvcache.kv_cache_append(x.clone().requires_grad_(), x, *args)
    with pytest.raises(ValueError):
        attention.flash_attn_paged_func(t(3, 4, 64).requires_grad_(), *args)
    with pytest.raises(ValueError):
        attention.flash_attn_paged_func(t(3, 3, 64), *args)
    with pytest.raises(ValueError):
        attention.flash_attn_paged_func(t(3, 4, 64), *args, window_size=(-3, 0))
    with pytest.raises(ValueError):
        attention.flash_attn_paged_func(t(3, 4, 64), *args, alibi_slopes=torch.ones(3))
    for kw in (dict(page_size=24), dict(headdim=80)):
        with pytest.raises(ValueError):
            kvcache.alloc_kv_cache(**{**dict(pages=1, page_size=16, nheads=1, headdim=64,
                                             device="cpu"), **kw})
    with pytest.raises(TypeError):
        kvcache.alloc_kv_cache(1, 16, 1, 64, torch.float32, device="cpu")


def test_python_rotary_refusals():
    freq, _ = rotary.rotary_frequencies(64, device="cpu")
    q = t(1, 4, 2, 64)
    for bad in (dict(q=t(4, 64)), dict(k=t(1, 5, 2, 64)), dict(k=t(1, 4, 2, 64).half()),
                dict(inv_freq=freq.float()), dict(positions=torch.zeros(5, dtype=torch.int32)),
                dict()):  # the last: CPU tensors
        with pytest.raises(ValueError):
            rotary.rotary_func(**{**dict(q=q, k=None, inv_freq=freq), **bad})
    with pytest.raises(TypeError):
        rotary.rotary_func(q, None, freq, positions=torch.zeros(4))


@pytest.mark.parametrize("kw", [dict(rotary_dim=20), dict(rotary_dim=0), dict(base=0.0),
                                dict(factor=0.5), dict(scaling="half"), dict(scaling="by_parts")])
def test_frequency_refusals(kw):
    with pytest.raises(ValueError):
        rotary.rotary_frequencies(**{**dict(rotary_dim=64, device="cpu"), **kw})


def test_frequencies():
    f, m = rotary.rotary_frequencies(64, device="cpu")
    assert m == 1.0 and f[0] == 1.0 and abs(float(f[-1]) - 10000 ** (-62 / 64)) < 1e-15
    lin, _ = rotary.rotary_frequencies(64, scaling="linear", factor=4, device="cpu")
    assert torch.equal(lin, f / 4)
    ntk, _ = rotary.rotary_frequencies(64, scaling="ntk", factor=4, device="cpu")
    assert ntk[0] == 1.0 and abs(float(ntk[-1] * 4 / f[-1]) - 1) < 1e-12
    by, m = rotary.rotary_frequencies(64, scaling="by_parts", factor=4, original_length=2048,
                                      device="cpu")
    turns = 2048 * f / (2 * math.pi)
    assert torch.equal(by[turns >= 32], f[turns >= 32])
    assert torch.allclose(by[turns <= 1], f[turns <= 1] / 4, rtol=1e-15)
    assert abs(m - (0.1 * math.log(4) + 1)) < 1e-15
