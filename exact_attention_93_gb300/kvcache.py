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

_ELEMS = {torch.bfloat16: fattn.FA_ELEM_BF16, torch.float16: fattn.FA_ELEM_FP16}


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


def kv_cache_append(k, v, k_pages, v_pages, block_table, cu_seqlens, seqlens, k_exp=None,
                    v_exp=None):
    """Writes the packed new keys and values ((total, nheads, headdim), bf16 or
    fp16) into the cache, in place: row i of sequence b becomes key seqlens[b]
    - (rows of b) + i, so seqlens (int32, (batch,)) are the lengths with the new
    tokens.  block_table: int32 (batch, max_pages); cu_seqlens: int32 (batch +
    1,).  A 16-bit cache has the rows' type; an e4m3 one gets each row at its
    own power-of-two scale, rounded to nearest even.  Rows of `total` behind the
    last sequence, and rows whose key would be negative, are not written.  The
    slots that one call writes must be distinct, and k_pages and v_pages must not
    overlap (they may be interleaved views of one tensor)."""
    status = fattn.bind().append(k, v, k_pages, v_pages, block_table, cu_seqlens, seqlens, k_exp,
                                 v_exp)
    if status:
        fattn._check(status, "fa_cache_append")


def kv_cache_read(k_pages, v_pages, block_table, cu_seqlens, total, starts=None, k_exp=None,
                  v_exp=None, dtype=None, out=None):
    """(k, v): cached keys and values as packed (total, nheads, headdim)
    tensors.  Row i of sequence b is key starts[b] + i (starts None: key i).
    dtype (bf16 or fp16) defaults to a 16-bit cache's own type, which it must
    be, and to bf16, which holds every e4m3 row exactly.  out: a (k, v) pair to
    write into; rows behind the last sequence are left as they were
    (uninitialised without out).  The cache keeps no gradients: outside
    torch.no_grad(), tensors that need one are refused, here as in
    kv_cache_append."""
    k, v = (None, None) if out is None else out
    got = fattn.bind().read(k_pages, v_pages, block_table, cu_seqlens, total, starts, k_exp, v_exp,
                            -1 if dtype is None else _ELEMS.get(dtype, fattn.FA_ELEM_FP32), k, v)
    if type(got) is int:
        fattn._check(got, "fa_cache_read")
    return got
