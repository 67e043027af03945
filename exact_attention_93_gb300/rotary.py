"""Rotary positions with autograd: rotary_func turns queries and keys before
attention.flash_attn_func, or before they go into a paged cache
(kvcache.kv_cache_append) and over it (attention.flash_attn_paged_func).

Pair i of the first rotary_dim elements of a head at position p is turned by
the angle p * inv_freq[i].  rotary_frequencies gives inv_freq for the usual
bases and for contexts stretched beyond the trained length.
"""
from __future__ import annotations

import contextlib
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


def _check(q, k, inv_freq, positions):
    if q.dim() not in (3, 4):
        raise ValueError("expected (batch, seqlen, nheads, headdim) or packed "
                         "(total, nheads, headdim) tensors")
    if k is not None and (k.dim() != q.dim() or k.shape[:-2] != q.shape[:-2]
                          or k.shape[-1] != q.shape[-1] or k.dtype != q.dtype):
        raise ValueError("q and k must agree in type and in every dimension but the heads")
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous float64 (rotary_dim / 2) tensor")
    B, N = (q.shape[0], q.shape[1]) if q.dim() == 4 else (1, q.shape[0])
    if positions is not None:
        if positions.dtype not in (torch.int32, torch.int64):
            raise TypeError("positions must be int32 or int64")
        if positions.shape != (N,) and (q.dim() != 4 or positions.shape != (B, N)):
            raise ValueError("positions must have shape (seqlen,) or (batch, seqlen)")
    for t in (q, k, inv_freq, positions):
        if t is not None and (not t.is_cuda or t.device != q.device):
            raise ValueError("libfattn takes CUDA tensors of one device only")
    return B, N


def _turn(xs, ys, inv_freq, positions, magnitude, interleaved, inverse):
    """Turns the tensors xs (one or two) into ys."""
    x = xs[0]
    B, N = (x.shape[0], x.shape[1]) if x.dim() == 4 else (1, x.shape[0])
    bits, stride, at = 0, 0, None
    if positions is not None:
        if positions.stride(-1) != 1:
            positions = positions.contiguous()
        bits, at = 32 if positions.dtype == torch.int32 else 64, positions.data_ptr()
        stride = positions.stride(0) if positions.dim() == 2 else 0
    ops = [fattn.rotary_operand(a, b) for a, b in zip(xs, ys)]
    here = (contextlib.nullcontext() if x.device.index == torch.cuda.current_device()
            else torch.cuda.device(x.device))
    with here:
        fattn.fa_rotary(ops[0], ops[1] if len(ops) > 1 else None, B, N, x.shape[-1],
                        2 * inv_freq.numel(), inv_freq.data_ptr(), at, bits, stride, magnitude,
                        interleaved, inverse, fattn.elem_code(x.dtype))


def _grad_operand(g):
    """The incoming gradient as the kernels need it: D contiguous, 16-byte
    aligned rows.  Anything else is copied once (argument marshalling)."""
    if g.stride(-1) != 1 or any(s % 8 for s in g.stride()[:-1]) or g.data_ptr() % 16:
        g = g.contiguous()
    return g


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, inv_freq, positions, magnitude, interleaved):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(inv_freq, positions)
        ctx.magnitude, ctx.interleaved = magnitude, interleaved
        xs = [q] if k is None else [q, k]
        ys = [torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in xs]
        _turn(xs, ys, inv_freq, positions, magnitude, interleaved, False)
        return (ys[0], None) if k is None else tuple(ys)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq, dk):
        inv_freq, positions = ctx.saved_tensors
        grads = [None if g is None else _grad_operand(g) for g in (dq, dk)]
        outs = [None if g is None else torch.empty(g.shape, dtype=g.dtype, device=g.device)
                for g in grads]
        have = [i for i in range(2) if grads[i] is not None]
        if have:
            _turn([grads[i] for i in have], [outs[i] for i in have], inv_freq, positions,
                  ctx.magnitude, ctx.interleaved, True)
        return outs[0], outs[1], None, None, None, None


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
    and k.  inplace=True writes over q and k instead and returns them; it is
    for inference and refuses tensors that need a gradient."""
    _check(q, k, inv_freq, positions)
    magnitude, interleaved = float(magnitude), bool(interleaved)
    grad = torch.is_grad_enabled() and (q.requires_grad or (k is not None and k.requires_grad))
    if grad and not inplace:
        q, k = _Rotary.apply(q, k, inv_freq, positions, magnitude, interleaved)
        return q if k is None else (q, k)
    xs = [q] if k is None else [q, k]
    if inplace:
        if grad:
            raise ValueError("inplace=True would overwrite tensors that need a gradient")
        ys = xs
    else:
        ys = [torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in xs]
    _turn(xs, ys, inv_freq, positions, magnitude, interleaved, False)
    return ys[0] if k is None else tuple(ys)
