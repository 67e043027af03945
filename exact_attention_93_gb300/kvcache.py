"""A paged key/value cache: allocation, writing and reading back.

Keys and values live in pages of page_size tokens, (pages, page_size, nheads,
headdim) tensors in bf16, fp16 or e4m3; a block table names the pages of each
sequence.  An e4m3 cache stores every (token, head) row at its own power-of-two
scale, whose exponent byte e is in k_exp / v_exp, (pages, nheads, page_size)
uint8: values are code * 2 ** (e - 127).

Sequences are packed along their tokens: rows cu_seqlens[b] .. cu_seqlens[b +
1] - 1 of a (total, nheads, headdim) tensor belong to sequence b.
attention.flash_attn_paged_func attends over what is cached here.

kv_cache_reserve builds a step's tables on the GPU from how many tokens each
sequence brings, taking pages from a stack of free ones; kv_cache_release gives
pages back.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import fattn

__all__ = ["CacheStep", "alloc_kv_cache", "kv_cache_append", "kv_cache_read", "kv_cache_release",
           "kv_cache_reserve", "kv_cache_write"]

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


class CacheStep(NamedTuple):
    """What kv_cache_reserve gives; all on the GPU."""
    cu_seqlens: torch.Tensor  # int32 (batch + 1,): the packed rows of each sequence
    seqlens: torch.Tensor     # int32 (batch,): lengths with the new tokens
    positions: torch.Tensor   # int32 (total,): of each packed row, in its sequence
    slots: torch.Tensor       # int64 (total,): page * page_size + place in the page
    free_count: torch.Tensor  # int32 (1,): free pages left
    missing: torch.Tensor     # int32 (1,): 0, or why nothing was taken


def kv_cache_reserve(new_tokens, seqlens, block_table, free_pages, free_count, page_size, total,
                     inplace=False):
    """The tables of a step in which sequence b, seqlens[b] keys long, brings
    new_tokens[b] more (int32 (batch,)): a CacheStep for rotary_func, kv_cache_append or
    kv_cache_write, and attention, without a look at the lengths on the host.

    Pages that a sequence lacks for its new tokens are taken from the end of
    free_pages[:free_count] (int32; free_count int32 (1,)), in the order of the
    sequences and of their keys, and written into block_table (int32 (batch,
    max_pages)); its entries for pages that the sequences hold already are read, the
    others left alone.  total is how many rows the packed tensors of the step have; rows
    behind the last sequence get position 0 and slot -1.  A page below zero where a new
    key goes, in the table or among the free ones, is recorded as an error, and its rows
    get slot -1 too.

    All or nothing: if the free pages do not suffice, missing says how many more it
    takes, and for bad lengths (negative, beyond the table, more new tokens than
    total) or a free_count outside free_pages it is -1, with an error recorded as for
    the other calls.  The table, seqlens and free_count then stay as they were, and
    cu_seqlens is all zeros, so that what follows in the same step does nothing.

    inplace=True writes the new lengths and the count over seqlens and free_count
    instead of into new tensors.  (Without it, the call can be made again on the same
    inputs, with the same result.)"""
    got = fattn.bind().reserve(new_tokens, seqlens, block_table, free_pages, free_count, page_size,
                               total, inplace)
    if type(got) is int:
        fattn._check(got, "fa_cache_reserve")
    return CacheStep(*got)


def kv_cache_release(done, seqlens, block_table, free_pages, free_count, page_size,
                     keep_pages=None):
    """Gives the pages of every sequence b with done[b] (bool or uint8 (batch,)) back to
    the end of free_pages[:free_count], all in place: free_count grows, seqlens[b]
    becomes 0, block_table stays.  keep_pages (int32 (batch,)): how many first pages of
    each sequence are left out, because others share them, say.  Bad lengths, or more
    pages than free_pages has room for, change nothing and are recorded as an error."""
    status = fattn.bind().release(done, seqlens, block_table, free_pages, free_count, page_size,
                                  keep_pages)
    if status:
        fattn._check(status, "fa_cache_release")


def kv_cache_write(k, v, k_pages, v_pages, slots, k_exp=None, v_exp=None):
    """kv_cache_append by slots: packed row i of k and v goes to slots[i] (int64 (total,),
    page * page_size + place in the page; kv_cache_reserve's).  Rows with a negative
    slot are not written, nor those beyond the cache, which are recorded as an error.
    The slots of one call must be distinct."""
    status = fattn.bind().write(k, v, k_pages, v_pages, slots, k_exp, v_exp)
    if status:
        fattn._check(status, "fa_cache_write")
