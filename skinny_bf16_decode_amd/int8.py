"""Products in 8-bit integers with a scale for each token and output channel.

    q[m, k]   = round(x[m, k] * 127 / max_k |x[m, k]|),  scale[m] = max_k |x[m, k]| / 127
    out[m, n] = (sum_k q[m, k] wq[n, k]) * scale[m] * w_scale[n] (+ residual[m, n])

Half the weight bytes of the BF16 projection for the same layer, and no limit
on the token count: one plan serves decode steps and prompts.  The integers'
sums are exact; an output is rounded to fp32, scaled, and rounded once to its
type.  Argument marshalling only: the kernels are in csrc/int8.hip.

    wq, w_scale = quantize_rows(W, torch.empty(N, K, int8), torch.empty(N, float32))
    plan = PreparedInt8(wq, w_scale)          # keeps a copy: wq may be freed
    q, scale = quantize_rows(x, q, scale)     # x: bf16, fp16 or fp32 [M, K]
    plan.run(q, scale, out)                   # out: [M, N]
"""
from __future__ import annotations

import ctypes

import torch

from . import _raise, load_library
from .calls import call_on, stream_handle

TYPES = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}


def _rows(name, t, dtype, rows, cols, index):
    """Checks a [>= rows, cols] matrix with contiguous rows; returns its pitch."""
    shape = t.shape
    if t.dtype != dtype or len(shape) != 2 or shape[1] != cols or shape[0] < rows:
        raise ValueError(f"{name} must be {dtype} [>= {rows}, {cols}], got {tuple(shape)} {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, is on {t.device}")
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name} rows must have unit stride")
    return ld if shape[0] > 1 else cols


def _scales(name, t, count, index):
    shape = t.shape
    if t.dtype != torch.float32 or len(shape) != 1 or shape[0] < count or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous torch.float32 [>= {count}], got {tuple(shape)} {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, is on {t.device}")


def quantize_rows(x, q, scale, stream=None):
    """Rows of x [M, K] (BF16, FP16 or fp32) to 8-bit integers in q [>= M, K]
    and scale [>= M] (fp32), on the current (or given) stream; returns
    (q, scale).  A row of zeros has scale 0, a row with an infinity or NaN
    scale NaN, both q = 0.  Rows may be pitched; whole 16-byte vectors (8-byte
    in q) are fastest.  Capturable in a graph."""
    kind = TYPES.get(x.dtype)
    index = x.get_device()                      # -1: not on a GPU
    if kind is None or x.dim() != 2 or index < 0:
        raise ValueError("x must be a 2-D BF16, FP16 or fp32 tensor on a GPU")
    m, k = x.shape
    ldx, unit = x.stride()
    if unit != 1 and k > 1:
        raise ValueError("x rows must have unit stride")
    ldq = _rows("q", q, torch.int8, m, k, index)
    _scales("scale", scale, m, index)
    call_on(index, stream, load_library().skinny_quantize_rows, x.data_ptr(), kind, m, k, ldx if m > 1 else k,
            q.data_ptr(), ldq, scale.data_ptr())
    return q, scale


class PreparedInt8:
    """A prepared 8-bit weight: a copy in the matrix units' order, with its
    channel scales.  ``weight`` is torch.int8 [N, K] with contiguous rows (a
    pitch is allowed), K a multiple of 16 below 131072; ``w_scale`` fp32 [N];
    ``out_dtype`` BF16, FP16 or fp32.  Runs change nothing in a plan: it may
    run on several streams at once."""

    def __init__(self, weight, w_scale, out_dtype=None, stream=None):
        self._plan = ctypes.c_void_p()
        out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
        if weight.dim() != 2 or weight.dtype != torch.int8 or not weight.is_cuda:
            raise ValueError("weight must be a 2-D torch.int8 tensor on a GPU")
        if out_dtype not in TYPES:
            raise ValueError(f"unsupported output dtype {out_dtype}")
        self.n, self.k = weight.shape
        index = weight.get_device()
        ldw = _rows("weight", weight, torch.int8, self.n, self.k, index)
        _scales("w_scale", w_scale, self.n, index)
        self.out_dtype = out_dtype
        self.device = weight.device
        self._index = index
        with torch.cuda.device(self.device):
            _raise(load_library().skinny_int8_prepare(weight.data_ptr(), self.n, self.k, ldw, w_scale.data_ptr(),
                                                      TYPES[out_dtype], stream_handle(stream, index),
                                                      ctypes.byref(self._plan)))

    def run(self, xq, x_scale, out, stream=None, residual=None):
        """out[:M] = (xq @ weight^T) * x_scale * w_scale (+ residual[:M]) with
        M = xq.shape[0] >= 0, on the current (or given) stream; returns out.
        xq: torch.int8 [M, K], 16-byte aligned with a pitch that is a multiple
        of 16; x_scale: fp32 [>= M]; out and residual: out_dtype [>= M, N],
        may be row-pitched; residual may be out itself."""
        if not self._plan:
            raise ValueError("the plan is closed")
        m = xq.shape[0]
        index = self._index
        ldx = _rows("xq", xq, torch.int8, m, self.k, index)
        _scales("x_scale", x_scale, m, index)
        ldo = _rows("out", out, self.out_dtype, m, self.n, index)
        res, ldr = None, 0
        if residual is not None:
            ldr = _rows("residual", residual, self.out_dtype, m, self.n, index)
            res = residual.data_ptr()
        call_on(index, stream, load_library().skinny_int8_run, self._plan, xq.data_ptr(), ldx, x_scale.data_ptr(),
                res, ldr, out.data_ptr(), ldo, m)
        return out

    def close(self):
        if self._plan:
            load_library().skinny_int8_destroy(self._plan)
            self._plan = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
