"""A paged key/value cache: allocation, writing and reading back.

Keys and values live in pages of page_size tokens, (pages, page_size, nheads,
headdim) tensors in bf16, fp16 or e4m3; a block table names the pages of each
sequence.  An e4m3 cache stores every (token, head) row at its own power-of-two
scale, whose exponent byte e is in k_exp / v_exp, (pages, nheads, page_size)
uint8: values are code * 2 ** (e - 127).

Sequences are packed along their tokens: rows cu_seqlens[b] .. cu_seqlens[b +
1] - 1 of a (total, nheads, headdim) tensor belong to sequence b.
attention.flash_attn_paged_func attends over what is cached here.
"""
from __future__ import annotations

import torch

from . import fattn

__all__ = ["alloc_kv_cache", "kv_cache_append", "kv_cache_read"]


def alloc_kv_cache(pages, page_size, nheads, headdim, dtype=torch.bfloat16, device="cuda"):
    """(k_pages, v_pages, k_exp, v_exp) of an empty cache, zeros; the exponent
    tensors are None unless dtype is torch.float8_e4m3fn."""
    if page_size not in (16, 32, 64, 128, 256):
        raise ValueError("page_size must be 16, 32, 64, 128 or 256")
    if headdim not in (64, 128):
        raise ValueError("headdim must be 64 or 128")
    fp8 = dtype == torch.float8_e4m3fn
    if not fp8 and dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"unsupported dtype {dtype}; use bfloat16, float16 or float8_e4m3fn")
    shape = (pages, page_size, nheads, headdim)
    make = lambda s, t: torch.zeros(s, dtype=t, device=device)  # noqa: E731
    if not fp8:
        return make(shape, dtype), make(shape, dtype), None, None
    exp = (pages, nheads, page_size)
    return (make(shape, torch.uint8).view(dtype), make(shape, torch.uint8).view(dtype),
            make(exp, torch.uint8), make(exp, torch.uint8))


def _check_rows(k, v, k_pages):
    shape, page = k.shape, k_pages.shape
    if (len(shape) != 3 or shape != v.shape or shape[1:] != page[2:] or k.dtype != v.dtype
            or k.stride(2) != 1 or v.stride(2) != 1):
        raise ValueError(f"k and v must be packed (total, {page[2]}, {page[3]}) tensors of one "
                         "type with the head dimension contiguous")
    return shape[0]


def kv_cache_append(k, v, k_pages, v_pages, block_table, cu_seqlens, seqlens, k_exp=None,
                    v_exp=None):
    """Writes the packed new keys and values ((total, nheads, headdim), bf16 or
    fp16) into the cache, in place: row i of sequence b becomes key seqlens[b]
    - (rows of b) + i, so seqlens (int32, (batch,)) are the lengths with the new
    tokens.  block_table: int32 (batch, max_pages); cu_seqlens: int32 (batch +
    1,).  A 16-bit cache has the rows' type; an e4m3 one gets each row at its
    own power-of-two scale, rounded to nearest even.  Rows of `total` behind the
    last sequence, and rows whose key would be negative, are not written.  The
    slots that one call writes must be distinct."""
    if torch.is_grad_enabled() and (k.requires_grad or v.requires_grad):
        raise ValueError("the cache keeps no gradients: call under torch.no_grad()")
    cache = fattn.kv_pages(k_pages, v_pages, k_exp, v_exp)
    total = _check_rows(k, v, k_pages)
    if seqlens is None:
        raise ValueError("seqlens is needed")
    batch = fattn.ragged(block_table, cu_seqlens, seqlens, total)
    device = fattn.one_device(k, v, k_pages, v_pages, block_table, cu_seqlens, seqlens)
    with fattn.on_device(device):
        fattn.fa_cache_append(cache, batch, k, v, fattn.raw_stream(device))


def kv_cache_read(k_pages, v_pages, block_table, cu_seqlens, total, starts=None, k_exp=None,
                  v_exp=None, dtype=None, out=None):
    """(k, v): cached keys and values as packed (total, nheads, headdim)
    tensors.  Row i of sequence b is key starts[b] + i (starts None: key i).
    dtype (bf16 or fp16) defaults to a 16-bit cache's own type, which it must
    be, and to bf16, which holds every e4m3 row exactly.  out: a (k, v) pair to
    write into; rows behind the last sequence are left as they were
    (uninitialised without out)."""
    cache = fattn.kv_pages(k_pages, v_pages, k_exp, v_exp)
    if dtype is None:
        dtype = torch.bfloat16 if k_pages.dtype == torch.float8_e4m3fn else k_pages.dtype
    total = int(total)
    if out is None:
        # one allocation: [0] keys, [1] values
        k, v = torch.empty((2, total, *k_pages.shape[2:]), dtype=dtype,
                           device=k_pages.device).unbind()
    else:
        k, v = out
        if _check_rows(k, v, k_pages) != total or k.dtype != dtype:
            raise ValueError("out must hold `total` rows of dtype")
    batch = fattn.ragged(block_table, cu_seqlens, starts, total)
    device = fattn.one_device(k_pages, v_pages, k, v, block_table, cu_seqlens, starts)
    with fattn.on_device(device):
        fattn.fa_cache_read(cache, batch, starts, k, v, fattn.raw_stream(device))
    return k, v
