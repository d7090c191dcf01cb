"""Rotary positions of queries and keys, before they are attended and cached.

As in the rest of the binding, only arguments are marshalled here
(include/libgdn.h has the contract) and there is no other implementation.

  rope(q, k, inv_freq, lens=... | positions=..., ...) -> (q, k)
  rope_frequencies(rot, ...) -> (inv_freq, factor)
"""
from __future__ import annotations

import math
from ctypes import byref

import torch

from . import _lib
from .paged import _IO, _checked, _i32, _library, _on, _ptr, _raw_stream, _short


def rope_frequencies(rot, *, base=10000.0, scaling=None, scale=1.0, trained=None, slow=1.0, fast=32.0, device=None):
    """The angle a position of each of rot / 2 pairs, base^(-2i / rot), for
    contexts longer than those a model was trained for: (inv_freq [rot / 2]
    float64, factor), as rope takes them.

    scaling None: as they are; "linear": positions divided by scale; "base": the
    base raised so that the slowest pair turns 1 / scale as far and the fastest
    as before; "parts": pairs that turn at least `fast` times within the `trained`
    positions stay, those that turn at most `slow` times are slowed by scale,
    those between in proportion to their turns.  factor is 1 but for "parts" with
    scale over 1: 0.1 ln(scale) + 1, the lengthening that keeps the softmax of
    a longer context as sharp (give rope 1.0 for a model without it).
    """
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2, got %s" % (rot,))
    if not base > 0 or not scale > 0:
        raise ValueError("base and scale must be positive")
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    factor = 1.0
    if scaling == "base" and rot > 2:
        base = base * scale ** (rot / (rot - 2))
    f = float(base) ** (-i / rot)
    if scaling == "linear":
        f = f / scale
    elif scaling == "parts":
        if trained is None or not trained > 0 or not fast > slow:
            raise ValueError("parts needs trained positions, and fast above slow")
        keep = ((trained * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        f = f * (keep + (1 - keep) / scale)
        factor = 0.1 * math.log(scale) + 1.0 if scale > 1 else 1.0
    elif scaling not in (None, "base"):
        raise ValueError("scaling must be None, linear, base or parts, got %r" % (scaling,))
    return f.to(device) if device is not None else f, factor


def _strides(x):
    """Token and head strides of [.., tokens, heads, d] rows of tokens one
    stride apart; x itself where they are, else a copy: (x, token, head)."""
    if x.is_contiguous():
        return x, x.shape[-2] * x.shape[-1], x.shape[-1]
    st = x.stride()
    if st[-1] != 1 and x.shape[-1] > 1 or (x.dim() == 4 and x.shape[0] > 1 and x.shape[1] > 1
                                           and st[0] != x.shape[1] * st[1]):
        x = x.contiguous()
        return x, x.shape[-2] * x.shape[-1], x.shape[-1]
    d = x.shape[-1]
    token = d if x.shape[:-2].numel() == 1 else st[0] if x.dim() == 4 and x.shape[1] == 1 else st[-3]
    return x, token, (st[-2] if x.shape[-2] > 1 else d)


def rope_args(q, k, inv_freq, *, lens=None, cu_seqlens=None, positions=None, interleaved=False, factor=1.0, out=None):
    """Validate shapes and build the gdn_rope_args struct (device-agnostic):
    returns (args, tensors to keep alive, (q, k) outputs)."""
    dtype, shape = q.dtype, q.shape
    if dtype not in _IO:
        raise ValueError("unsupported dtype %s (float32 or bfloat16)" % dtype)
    if len(shape) not in (3, 4):
        raise ValueError("q must be [tokens, hq, d] or [B, T, hq, d]")
    if k is not None and (k.dtype is not dtype or k.dim() != len(shape) or k.shape[:-2] != shape[:-2]
                          or k.shape[-1] != shape[-1]):
        raise ValueError("k must have q's dtype, tokens and head size, got %s %s" % (k.dtype, tuple(k.shape)))
    lead = shape[:-2]
    total, d = lead.numel(), shape[-1]
    if inv_freq.dim() != 1 or inv_freq.dtype not in (torch.float64, torch.float32):
        raise ValueError("inv_freq must be [rot / 2] float64 or float32")
    rot = 2 * inv_freq.shape[0]
    if not 2 <= rot <= d:
        raise ValueError("inv_freq must hold between 1 and d / 2 angles, got %d for d = %d" % (inv_freq.shape[0], d))
    if inv_freq.dtype is not torch.float64 or not inv_freq.is_contiguous():
        inv_freq = inv_freq.to(torch.float64).contiguous()
    batch, i64 = 0, 0
    if (positions is None) == (lens is None):
        raise ValueError("give either positions or lens")
    if positions is not None:
        if cu_seqlens is not None:
            raise ValueError("cu_seqlens goes with lens")
        if positions.shape != lead or positions.dtype not in (torch.int32, torch.int64):
            raise ValueError("positions must be int32 or int64 %s" % (tuple(lead),))
        positions = positions if positions.is_contiguous() else positions.contiguous()
        i64 = int(positions.dtype is torch.int64)
    else:
        if lens.dim() != 1:
            raise ValueError("lens must be [B]")
        batch = lens.shape[0]
        if cu_seqlens is not None:
            if len(shape) != 3:
                raise ValueError("with cu_seqlens q and k must be [tokens, heads, d]")
            cu_seqlens = _i32(cu_seqlens, "cu_seqlens", (batch + 1,))
        elif len(shape) != 4 or shape[0] != batch:
            raise ValueError("without cu_seqlens q and k must be [B, T, heads, d]")
        lens = _i32(lens, "lens", (batch,))
    if out is not None and len(out) != 2:
        raise ValueError("out must be (q, k)")
    # tokens of no row: zeros where all of it is new
    make = torch.zeros if (cu_seqlens is not None and out is not None) or (lens is not None and batch == 0) else torch.empty
    ins, outs = [], []
    for n, x in enumerate((q, k)):
        if x is None:
            ins.append((None, 0, 0))
            outs.append((None, 0, 0))
            continue
        ins.append(_strides(x))
        y = None if out is None else out[n]
        if y is None:
            y = make(x.shape, dtype=dtype, device=x.device)
        elif y.shape != x.shape or y.dtype is not dtype:
            raise ValueError("out must have the inputs' shapes and dtype")
        to = _strides(y)
        if to[0] is not y or min(to[1:]) < d:
            raise ValueError("out must have a dense last dimension, its rows apart and tokens one stride apart")
        if y.data_ptr() == x.data_ptr() and ins[n][0] is not x:
            raise ValueError("in place needs a dense last dimension and tokens one stride apart")
        outs.append(to)
    p = lambda x: (_ptr(x[0]), x[1], x[2])
    a = _lib.RopeArgs(
        total, batch, shape[-2], 0 if k is None else k.shape[-2], d, rot, _IO[dtype], int(bool(interleaved)),
        float(factor), *p(ins[0]), *p(ins[1]), *p(outs[0]), *p(outs[1]), inv_freq.data_ptr(), _ptr(positions), i64,
        _ptr(lens), _ptr(cu_seqlens), int(out is None))
    return a, (ins, inv_freq, positions, lens, cu_seqlens), (outs[0][0], outs[1][0])


def rope(q, k, inv_freq, *, lens=None, cu_seqlens=None, positions=None, interleaved=False, factor=1.0, out=None,
         stream=None):
    """Rotary positions of queries and keys.

    q [B, T, hq, d] or packed [tokens, hq, d], k likewise with hkv heads (None:
    queries only), float32 or bfloat16.  inv_freq [rot / 2] (float64; float32 is
    converted each call): the angle a position of each pair; the first rot
    dimensions of a head are turned, the others copied.  Pair i is dimensions
    (i, i + rot / 2), or with interleaved (2i, 2i + 1).  factor multiplies the
    turned values.  rope_frequencies gives both for long contexts.

    A token's position follows from lens [B] as in kv_append: lens[b] - n + i for
    token i of row b's n, T for every row or with cu_seqlens [B + 1] packed; or
    positions, of q's leading shape, gives it.  Angles are formed in 64 bits.
    out: (q, k) to write to: each its own input, or apart from both, also as
    slices of one buffer that do not overlap; new tensors when None.
    Packed tokens of no row are left as they were there, and zeros in new ones.
    Returns (q, k).
    """
    if out is None and stream is None and q.is_cuda:
        got = _short("rope", q, k, inv_freq, lens, cu_seqlens, positions, interleaved, factor)
        if got is not None:
            return got
    dev = q.device
    ctx = _on(stream, dev, (k, inv_freq, lens, cu_seqlens, positions) + tuple(out or ()))
    if ctx is not None:
        with ctx:
            return rope(q, k, inv_freq, lens=lens, cu_seqlens=cu_seqlens, positions=positions, interleaved=interleaved,
                        factor=factor, out=out)
    a, keep, out = rope_args(q, k, inv_freq, lens=lens, cu_seqlens=cu_seqlens, positions=positions,
                             interleaved=interleaved, factor=factor, out=out)
    _checked(_library().gdn_rope(byref(a), _raw_stream(dev.index)))
    del keep
    return out
