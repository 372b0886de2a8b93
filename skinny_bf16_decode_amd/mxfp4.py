"""Products with weights in 4 bits: blocks of 32 values with a power of two.

    v[m, k]   = q[m, k] * 2^(scale[m, k // 32] - 127)
    out[m, n] = sum_k x[m, k] w[n, k] (+ residual[m, n])

The formats of OCP Microscaling Formats v1.0: values in 4 bits (e2m1, two a
byte) or 8 (e4m3), powers of two in a byte (e8m0).  Weights have 4 bits, half
the bytes of the 8-bit integers' (int8.py), tokens 4 or 8; one plan serves
decode steps and prompts.  Argument marshalling only: the kernels are in
csrc/mxfp4.hip.

    wq, w_scale = quantize_blocks(W, torch.empty(N, K // 2, uint8), torch.empty(N, K // 32, uint8))
    plan = PreparedMxfp4(wq, w_scale)          # keeps a copy: wq may be freed
    xq, x_scale = quantize_blocks(x, xq, x_scale)   # xq: float8_e4m3fn [M, K], or uint8 [M, K // 2]
    plan.run(xq, x_scale, out)                 # out: [M, N]
"""
from __future__ import annotations

import ctypes

import torch

from . import _raise, load_library
from .calls import call_on, stream_handle
from .int8 import TYPES, _rows

BLOCK = 32
# bits of a code by the type of its tensor; a byte holds two of 4
BITS = {torch.float8_e4m3fn: 8, torch.uint8: 4, torch.float4_e2m1fn_x2: 4}
POWERS = (torch.uint8, torch.float8_e8m0fnu)


def _codes(name, t, rows, k, index):
    """Checks [>= rows, k] codes with contiguous rows; returns their bits and pitch in bytes."""
    bits = BITS.get(t.dtype)
    if bits is None:
        raise ValueError(f"{name} must be torch.float8_e4m3fn, or torch.uint8 or float4_e2m1fn_x2 for 4 bits, is {t.dtype}")
    return bits, _rows(name, t, t.dtype, rows, k * bits // 8, index)


def _powers(name, t, rows, k, index):
    dtype = t.dtype
    if dtype not in POWERS:
        raise ValueError(f"{name} must be torch.uint8 or float8_e8m0fnu, is {dtype}")
    return _rows(name, t, dtype, rows, k // BLOCK, index)


def _values(name, t):
    """The type, GPU and pitch of a matrix of values."""
    kind = TYPES.get(t.dtype)
    index = t.get_device()                      # -1: not on a GPU
    if kind is None or t.dim() != 2 or index < 0:
        raise ValueError(f"{name} must be a 2-D BF16, FP16 or fp32 tensor on a GPU")
    m, k = t.shape
    ld, unit = t.stride()
    if unit != 1 and k > 1:
        raise ValueError(f"{name} rows must have unit stride")
    return kind, index, ld if m > 1 else k


def quantize_blocks(x, q, scale, gate=None, stream=None):
    """Rows of x [M, K] (BF16, FP16 or fp32) to blocks in q and scale, on the
    current (or given) stream; returns (q, scale).  q: torch.float8_e4m3fn
    [>= M, K], or 4 bits in torch.uint8 (or float4_e2m1fn_x2) [>= M, K / 2], the
    first of two in the low half; scale: torch.uint8 or float8_e8m0fnu [>= M,
    K / 32].  K is a multiple of 32.  With a gate [M, K] of x's type, of x
    silu(gate).

    A block's power is floor(log2 max |x|) - 2 (4 bits) or - 8; values go to the
    nearest, ties to even, and are clipped at 6 or 448.  A block with an
    infinity or NaN has the power NaN (255) and codes 0.  Rows may be pitched
    and unaligned; whole 16-byte vectors are fastest.  Capturable in a graph."""
    kind, index, ldx = _values("x", x)
    m, k = x.shape
    if k % BLOCK:
        raise ValueError(f"x must have whole blocks of {BLOCK} in a row, has {k} values")
    bits, ldq = _codes("q", q, m, k, index)
    lds = _powers("scale", scale, m, k, index)
    gp, ldg = None, 0
    if gate is not None:
        if gate.shape != x.shape:
            raise ValueError(f"gate must have x's shape {tuple(x.shape)}, has {tuple(gate.shape)}")
        ldg = _rows("gate", gate, x.dtype, m, k, index)
        gp = gate.data_ptr()
    call_on(index, stream, load_library().skinny_quantize_blocks, x.data_ptr(), kind, m, k, ldx, gp, ldg, bits,
            q.data_ptr(), ldq, scale.data_ptr(), lds)
    return q, scale


def expand_blocks(q, scale, out, stream=None):
    """out[:M] = the values that M = q.shape[0] rows of codes q (of
    quantize_blocks' types) with powers scale [>= M, K / 32] stand for, rounded
    once to out's type: BF16, FP16 or fp32 [>= M, K]; returns out."""
    kind, index, ldo = _values("out", out)
    m, k = q.shape[0], out.shape[1]
    if k % BLOCK:
        raise ValueError(f"out must have whole blocks of {BLOCK} in a row, has {k} values")
    bits, ldq = _codes("q", q, m, k, index)
    lds = _powers("scale", scale, m, k, index)
    if out.shape[0] < m:
        raise ValueError(f"out must have at least {m} rows, has {out.shape[0]}")
    call_on(index, stream, load_library().skinny_expand_blocks, q.data_ptr(), bits, m, k, ldq, scale.data_ptr(), lds,
            out.data_ptr(), kind, ldo)
    return out


class PreparedMxfp4:
    """A prepared 4-bit weight: a copy in the matrix units' order, with its
    powers.  ``weight`` is 4-bit codes [N, K / 2] (torch.uint8 or
    float4_e2m1fn_x2) with contiguous rows (a pitch is allowed), K a multiple of
    32 up to 2^22; ``w_scale`` torch.uint8 or float8_e8m0fnu [N, K / 32];
    ``out_dtype`` BF16, FP16 or fp32.  Runs change nothing in a plan: it may run
    on several streams at once."""

    def __init__(self, weight, w_scale, out_dtype=None, stream=None):
        self._plan = ctypes.c_void_p()
        out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
        if weight.dim() != 2 or BITS.get(weight.dtype) != 4 or not weight.is_cuda:
            raise ValueError("weight must be a 2-D torch.uint8 or float4_e2m1fn_x2 tensor on a GPU")
        if out_dtype not in TYPES:
            raise ValueError(f"unsupported output dtype {out_dtype}")
        self.n, self.k = weight.shape[0], 2 * weight.shape[1]
        if self.k % BLOCK:
            raise ValueError(f"weight must have whole blocks of {BLOCK} in a row, has {self.k} values")
        index = weight.get_device()
        _, ldw = _codes("weight", weight, self.n, self.k, index)
        ldws = _powers("w_scale", w_scale, self.n, self.k, index)
        self.out_dtype = out_dtype
        self.device = weight.device
        self._index = index
        with torch.cuda.device(self.device):
            _raise(load_library().skinny_mxfp4_prepare(weight.data_ptr(), self.n, self.k, ldw, w_scale.data_ptr(), ldws,
                                                       TYPES[out_dtype], stream_handle(stream, index),
                                                       ctypes.byref(self._plan)))

    def run(self, xq, x_scale, out, stream=None, residual=None):
        """out[:M] = x @ weight^T (+ residual[:M]) with M = xq.shape[0] >= 0,
        on the current (or given) stream; returns out.  xq: codes of 8 or 4 bits
        (quantize_blocks' types), 16-byte aligned with a pitch that is a
        multiple of 16 bytes; x_scale [>= M, K / 32]; out and residual:
        out_dtype [>= M, N], may be row-pitched; residual may be out itself.

        8-bit tokens go through BF16: with powers below 2^-124 (byte 3; blocks
        with nothing above 2^-116) their values are rounded to multiples of
        2^-133; powers above 2^119 (byte 246), of the weight above 2^125 (252),
        which quantize_blocks never gives, make infinities.  4-bit tokens are
        exact at every power."""
        if not self._plan:
            raise ValueError("the plan is closed")
        m = xq.shape[0]
        index = self._index
        bits, ldx = _codes("xq", xq, m, self.k, index)
        ldxs = _powers("x_scale", x_scale, m, self.k, index)
        ldo = _rows("out", out, self.out_dtype, m, self.n, index)
        res, ldr = None, 0
        if residual is not None:
            ldr = _rows("residual", residual, self.out_dtype, m, self.n, index)
            res = residual.data_ptr()
        call_on(index, stream, load_library().skinny_mxfp4_run, self._plan, xq.data_ptr(), bits, ldx,
                x_scale.data_ptr(), ldxs, res, ldr, out.data_ptr(), ldo, m)
        return out

    def close(self):
        if self._plan:
            load_library().skinny_mxfp4_destroy(self._plan)
            self._plan = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
