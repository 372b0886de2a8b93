"""Norms before and after a block, fused with its gate and residual.

    norm_rows:  n = x / sqrt(mean x^2 + eps) * weight
    join_rows:  h = beta * residual + alpha * gate * norm(y), then norm(h) for the next block

A norm is written in a type of 16 or 32 bits, or quantized for the product that
follows, straight from fp32: 8-bit integers (int8.py) or blocks of 4 or 8 bits
(mxfp4.py).  Argument marshalling only: the kernels are in csrc/norms.hip.

    norm_rows(h, norm_weight, q=xq, scale=x_scale)
    plan.run(xq, x_scale, y)                                    # the block: PreparedInt8 or PreparedMxfp4
    join_rows(h, y, h, weight=post_weight, alpha=0.5, next_weight=next_norm_weight, q=xq, scale=x_scale)
"""
from __future__ import annotations

import struct

import torch

from . import load_library
from .calls import call_on
from .int8 import TYPES, _rows, _scales
from .mxfp4 import BITS, BLOCK, _codes, _powers, _values

NONE, INT8, MX4, MX8 = range(4)         # skinny_rows_kind
# skinny_norm_args and skinny_join_args
_NORM = struct.Struct("@5P4qd6i")
_JOIN = struct.Struct("@9P7qd2f10i")


def _weight(name, t, k, index):
    kind = TYPES.get(t.dtype)
    if kind is None or t.shape != (k,) or not t.is_contiguous() or t.get_device() != index:
        raise ValueError(f"{name} must be a contiguous BF16, FP16 or fp32 [{k}] on cuda:{index}, got {tuple(t.shape)} "
                         f"{t.dtype} on {t.device}")
    return t.data_ptr(), kind


def _out(name, t, m, k, index):
    kind = TYPES.get(t.dtype)
    if kind is None:
        raise ValueError(f"{name} must be BF16, FP16 or fp32, is {t.dtype}")
    return t.data_ptr(), kind, _rows(name, t, t.dtype, m, k, index)


def _quantized(q, scale, m, k, index):
    """kind, addresses and pitches of quantized rows, by q's type."""
    if q is None:
        if scale is not None:
            raise ValueError("scale without q")
        return NONE, 0, 0, 0, 0
    if scale is None:
        raise ValueError("q without scale")
    if q.dtype == torch.int8:
        ldq = _rows("q", q, torch.int8, m, k, index)
        _scales("scale", scale, m, index)
        return INT8, q.data_ptr(), scale.data_ptr(), ldq, 0
    if q.dtype not in BITS:
        raise ValueError(f"q must be torch.int8, float8_e4m3fn, or uint8 or float4_e2m1fn_x2 for 4 bits, is {q.dtype}")
    if k % BLOCK:
        raise ValueError(f"rows to quantize must be whole blocks of {BLOCK}, have {k} values")
    bits, ldq = _codes("q", q, m, k, index)
    return MX8 if bits == 8 else MX4, q.data_ptr(), scale.data_ptr(), ldq, _powers("scale", scale, m, k, index)


def norm_rows(x, weight, out=None, q=None, scale=None, eps=1e-6, stream=None):
    """The root-mean-square norm of x's rows [M, K] times weight [K], on the
    current (or given) stream: to out [>= M, K], to q and scale, or to both
    (quantized from fp32, not from out); returns (out, q, scale) as given.

    x, weight and out: BF16, FP16 or fp32, free of each other; out may be x.  q
    and scale: int8.quantize_rows' (torch.int8, fp32 [>= M]) or
    mxfp4.quantize_blocks' (K a multiple of 32).  The squares are summed in 64
    bits.  Any K and pitch; K a multiple of 8 on 16-byte aligned rows is fastest.
    Capturable in a graph."""
    kind, index, ldx = _values("x", x)
    m, k = x.shape
    wp, wt = _weight("weight", weight, k, index)
    op, ot, ldo = (0, 0, 0) if out is None else _out("out", out, m, k, index)
    qk, qp, sp, ldq, lds = _quantized(q, scale, m, k, index)
    if out is None and q is None:
        raise ValueError("norm_rows needs out, or q and scale")
    call_on(index, stream, load_library().skinny_norm_rows,
            _NORM.pack(x.data_ptr(), wp, op, qp, sp, ldx, ldo, ldq, lds, eps, kind, wt, ot, qk, m, k))
    return out, q, scale


def join_rows(residual, y, out, weight=None, gate=None, sigmoid=False, alpha=1.0, beta=1.0, next_weight=None,
              next_out=None, q=None, scale=None, eps=1e-6, stream=None):
    """out[:M] = beta residual + alpha (gate z) on the current (or given)
    stream, with z = the norm of y [M, K] by weight [K], or y without one;
    returns out.  residual and out [>= M, K] have one type, out may be residual.
    gate: [M, K] or [K] (one for all rows), as it is or, with sigmoid, 1 / (1 +
    exp(-gate)); None: 1.

    With next_weight [K], also the norm of out (as it is held) for the block
    that follows: to next_out [>= M, K], to q and scale as norm_rows, or both.
    All but residual and out may differ in type: BF16, FP16 or fp32.  eps serves
    both norms.  Capturable in a graph."""
    yt, index, ldy = _values("y", y)
    m, k = y.shape
    rp, rt, ldr = _out("residual", residual, m, k, index)
    if out.dtype != residual.dtype:
        raise ValueError(f"out and residual must have one type, got {out.dtype} and {residual.dtype}")
    ldo = _rows("out", out, out.dtype, m, k, index)
    wp, wt = (0, 0) if weight is None else _weight("weight", weight, k, index)
    gp = gt = ldg = 0
    if gate is not None:
        if gate.dim() == 1:
            gp, gt = _weight("gate", gate, k, index)
        elif gate.shape == y.shape:
            gp, gt, ldg = _out("gate", gate, m, k, index)
        else:
            raise ValueError(f"gate must be [{m}, {k}] or [{k}], got {tuple(gate.shape)}")
    np_ = nt = op = ot = ldn = 0
    if next_weight is not None:
        np_, nt = _weight("next_weight", next_weight, k, index)
        if next_out is None and q is None:
            raise ValueError("next_weight needs next_out, or q and scale")
    elif next_out is not None or q is not None:
        raise ValueError("next_out and q need next_weight")
    if next_out is not None:
        op, ot, ldn = _out("next_out", next_out, m, k, index)
    qk, qp, sp, ldq, lds = _quantized(q, scale, m, k, index)
    call_on(index, stream, load_library().skinny_join_rows,
            _JOIN.pack(rp, y.data_ptr(), wp, gp, out.data_ptr(), np_, op, qp, sp, ldr, ldy, ldg, ldo, ldn, ldq, lds,
                       eps, alpha, beta, rt, yt, wt, gt, nt, ot, qk, sigmoid, m, k))
    return out
