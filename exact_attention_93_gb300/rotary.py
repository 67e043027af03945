"""Rotary positions with autograd: rotary_func turns queries and keys before
attention.flash_attn_func, or before they go into a paged cache
(kvcache.kv_cache_append) and over it (attention.flash_attn_paged_func).

Pair i of the first rotary_dim elements of a head at position p is turned by
the angle p * inv_freq[i].  rotary_frequencies gives inv_freq for the usual
bases and for contexts stretched beyond the trained length.
"""
from __future__ import annotations

import math

import torch

from . import fattn

__all__ = ["rotary_frequencies", "rotary_func"]


def rotary_frequencies(rotary_dim, base=10000.0, scaling=None, factor=1.0, original_length=None,
                       beta_fast=32.0, beta_slow=1.0, device="cuda"):
    """(inv_freq, magnitude): the fp64 (rotary_dim / 2) angles per position
    base ** (-2 i / rotary_dim), and what rotated values are multiplied by.
    scaling stretches the context by `factor`:

    None        as trained; magnitude 1.
    "linear"    every angle divided by factor (positions interpolated).
    "ntk"       base * factor ** (rotary_dim / (rotary_dim - 2)): the slowest
                pair is interpolated by factor, the fastest not at all.
    "by_parts"  pairs that turn beta_fast times or more within original_length
                positions stay, those that turn beta_slow times or less are
                divided by factor, with a linear ramp between; magnitude
                0.1 ln(factor) + 1.
    """
    if rotary_dim < 16 or rotary_dim % 16:
        raise ValueError("rotary_dim must be a positive multiple of 16")
    if not base > 0 or not factor >= 1:
        raise ValueError("base must be positive and factor at least 1")
    if scaling not in (None, "linear", "ntk", "by_parts"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling == "ntk":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    i = torch.arange(0, rotary_dim, 2, dtype=torch.float64)
    freq, magnitude = base ** (-i / rotary_dim), 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "by_parts":
        if not original_length or not beta_fast > beta_slow:
            raise ValueError("by_parts needs original_length, and beta_fast above beta_slow")
        turns = original_length * freq / (2 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0, 1)
        freq = freq * keep + freq / factor * (1 - keep)
        magnitude = 0.1 * math.log(factor) + 1.0
    return freq.to(device), magnitude


def rotary_func(q, k, inv_freq, positions=None, interleaved=False, magnitude=1.0, inplace=False):
    """q and k (k may be None) with the first 2 * len(inv_freq) elements of
    every head turned by position, the others unchanged: (batch, seqlen,
    nheads, headdim) or packed (total, nheads, headdim) CUDA tensors of bf16,
    fp16 or fp32, headdim 64 or 128 and contiguous, the other strides multiples
    of 16 bytes; q and k may have different numbers of heads.

    inv_freq is a float64 tensor of angles per position (rotary_frequencies),
    positions an int32 or int64 (seqlen,) or (batch, seqlen) tensor (None: 0,
    1, 2, ...).  Pairs are elements (i, i + rotary_dim / 2), or (2 i, 2 i + 1)
    when interleaved.  Rotated elements are multiplied by magnitude.

    Returns new tensors (q, k), or q alone when k is None.  Differentiable in q
    and k (the gradient is the rotation back), any number of times; tensors with
    a forward-mode tangent are refused.
    inplace=True writes over q and k instead and returns them; it is for
    inference, refuses tensors that need a gradient, and q and k must not
    overlap.  (A backward pass can be captured into a CUDA graph while no eager
    graph of the same leaves is alive: torch ties their gradients to the stream
    of the graph that came first.)"""
    out = fattn.bind().rotary(q, k, inv_freq, positions, magnitude, interleaved, inplace)
    if type(out) is int:
        fattn._check(out, "fa_rotary")
    return out
