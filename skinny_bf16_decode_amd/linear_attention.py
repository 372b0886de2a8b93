"""Linear attention with a decay for each head and token.

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,    o_t = scale q_t^T S_t

for every head, over packed sequences of prompts (``prompt``: chunks on the
matrix units, long sequences split over the chip) or for one new token of each
sequence (``step``).  The states stay in a pool of fp32 [dk, dv] matrices, one
[heads, dk, dv] slot a sequence.  q, k, v and out are views with a contiguous
last dimension, so the column ranges of a packed projection's output can be
passed in place.  States and sums are fp32; a prompt's matrix products take
fp32 operands with all 24 bits for BF16 inputs and with 22 for FP16 ones.
Argument marshalling only: the kernels are in csrc/linear_attention.hip.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import IN_BF16, IN_F16, load_library
from .calls import call_on

_TYPES = {torch.bfloat16: IN_BF16, torch.float16: IN_F16}
_P, _LL, _I = ctypes.c_void_p, ctypes.c_longlong, ctypes.c_int


class _Args(ctypes.Structure):
    _fields_ = ([(n, _P) for n in ("q", "k", "v", "out", "log_decay", "state_in", "state_out", "starts", "slots",
                                   "workspace")] + [("workspace_bytes", ctypes.c_size_t)] +
                [(n, _LL) for n in ("q_token", "q_head", "k_token", "k_head", "v_token", "v_head", "out_token",
                                    "out_head", "decay_token", "decay_head", "in_state_slot", "in_state_head",
                                    "out_state_slot", "out_state_head")] +
                [(n, _I) for n in ("type", "tokens", "sequences", "heads", "key_heads", "dk", "dv", "pool")] +
                [("scale", ctypes.c_float)])


# the same as bytes, which take a fifth of the time to make: decode steps of few sequences wait for this
_ARGS = struct.Struct("@10PQ14q8if0P")
assert _ARGS.size == ctypes.sizeof(_Args)


def workspace_bytes(tokens: int, sequences: int, heads: int, dk: int, dv: int) -> int:
    """Bytes of workspace a prompt call of these sizes needs (may be 0): no less for more tokens or sequences."""
    return load_library().skinny_linear_workspace(tokens, sequences, heads, dk, dv)


def _state(name, t, heads, dk, dv, index):
    shape = t.shape
    if t.dtype != torch.float32 or len(shape) != 4 or tuple(shape[1:]) != (heads, dk, dv):
        raise ValueError(f"{name} must be torch.float32 [pool, {heads}, {dk}, {dv}], got {tuple(shape)} {t.dtype}")
    slot, head, row, unit = t.stride()
    if unit != 1 or row != dv:
        raise ValueError(f"{name}'s [dk, dv] matrices must be contiguous")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, is on {t.device}")
    return t.data_ptr(), shape[0], slot, head


def _ints(name, t, count, index):
    if t.dtype != torch.int32 or t.shape != (count,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous torch.int32 [{count}], got {tuple(t.shape)} {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, is on {t.device}")
    return t.data_ptr()


def _workspace(nbytes, device, stream):
    """Memory for one call on `stream` (an object, a handle or None, the
    current one).  It comes from that stream's own memory and goes back to it:
    the allocator orders what is freed and taken again on one stream only, and
    on another one a block may still be in use, before the call or after it."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if not hasattr(stream, "cuda_stream"):
        # the default stream's handle is 0, of which ExternalStream makes a new stream
        stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _call(entry, q, k, v, log_decay, out, sequences, starts, state_in, state_out, slots, scale, workspace, stream):
    dtype, shape = v.dtype, v.shape
    kind = _TYPES.get(dtype)
    index = v.get_device()                      # -1: not on a GPU
    if kind is None or len(shape) != 3 or index < 0:
        raise ValueError("v must be a BF16 or FP16 [tokens, heads, dv] tensor on a GPU")
    tokens, heads, dv = shape
    q_shape = q.shape
    if len(q_shape) != 3 or q_shape[0] != tokens or k.shape != q_shape:
        raise ValueError(f"q and k must be [{tokens}, key_heads, dk] alike, got {tuple(q.shape)} and {tuple(k.shape)}")
    key_heads, dk = q_shape[1:]
    if out.shape != shape:
        raise ValueError(f"out must have v's shape {tuple(shape)}, got {tuple(out.shape)}")
    if log_decay.dtype != torch.float32 or log_decay.shape != (tokens, heads):
        raise ValueError(f"log_decay must be torch.float32 [{tokens}, {heads}], got {tuple(log_decay.shape)} "
                         f"{log_decay.dtype}")
    qt, qh, qu = q.stride()
    kt, kh, ku = k.stride()
    vt, vh, vu = v.stride()
    ot, oh, ou = out.stride()
    if qu != 1 or ku != 1 or vu != 1 or ou != 1:
        raise ValueError("q, k, v and out must have a contiguous last dimension")
    if q.dtype != dtype or k.dtype != dtype or out.dtype != dtype:
        raise ValueError(f"q, k, v and out must have one type, got {q.dtype}, {k.dtype}, {v.dtype} and {out.dtype}")
    if (q.get_device() != index or k.get_device() != index or out.get_device() != index or
            log_decay.get_device() != index):
        raise ValueError("q, k, v, out and log_decay must be on the same device")
    pool = ip = op = slot_ptr = start_ptr = wp = wb = 0
    i_slot = i_head = o_slot = o_head = 0
    if state_in is not None:
        ip, pool, i_slot, i_head = _state("state_in", state_in, heads, dk, dv, index)
    if state_out is not None:
        op, count, o_slot, o_head = _state("state_out", state_out, heads, dk, dv, index)
        if state_in is not None and count != pool:
            raise ValueError(f"state_in and state_out hold {pool} and {count} states")
        pool = count
    if slots is not None:
        slot_ptr = _ints("slots", slots, sequences, index)
    if starts is not None:
        start_ptr = _ints("starts", starts, sequences + 1, index)
    if workspace is not None:
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous and on the same device")
        wp, wb = workspace.data_ptr(), workspace.nbytes
    if scale is None:
        scale = dk ** -0.5
    if tokens <= 1:                     # the strides of a single token say nothing
        qt = kt = vt = ot = 0
    gt, gh = log_decay.stride()
    call_on(index, stream, entry,
            _ARGS.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), log_decay.data_ptr(), ip, op, start_ptr,
                       slot_ptr, wp, wb, qt, qh, kt, kh, vt, vh, ot, oh, gt, gh, i_slot, i_head, o_slot, o_head, kind,
                       tokens, sequences, heads, key_heads, dk, dv, pool, scale))


def prompt(q, k, v, log_decay, out, starts, state_in=None, state_out=None, slots=None, scale=None, workspace=None,
           stream=None):
    """out[t] = scale q_t^T S_t over packed sequences, on the current (or given) stream; returns out.

    q, k [tokens, key_heads, dk]; v, out [tokens, heads, dv]; BF16 or FP16,
    dk <= 256 and dv <= 1024 multiples of 8, any strides that are multiples of 8
    elements on 16-byte aligned tensors.  log_decay fp32 [tokens, heads], at
    most 0.  starts int32 [sequences + 1] on the GPU: sequence i has the
    tokens starts[i] .. starts[i + 1] (none is allowed).  state_in (None: zero)
    and state_out (None: not kept; may be state_in) are fp32 [pool, heads, dk,
    dv]; slots int32 [sequences] names each sequence's state, all different
    (None: 0, 1, ...); a slot outside the pool is no state.  scale: dk ** -0.5
    if None.  workspace: a tensor of at least workspace_bytes(...) bytes, which
    must not serve two calls at once; None allocates one for the call, in the
    memory of the stream that it runs on."""
    if starts.dim() != 1 or starts.shape[0] < 1:
        raise ValueError("starts must be int32 [sequences + 1]")
    sequences = starts.shape[0] - 1
    if workspace is None and v.dim() == 3 and q.dim() == 3:
        need = workspace_bytes(v.shape[0], sequences, v.shape[1], q.shape[2], v.shape[2])
        if need:
            workspace = _workspace(need, v.device, stream)
    _call(load_library().skinny_linear_prompt, q, k, v, log_decay, out, sequences, starts, state_in, state_out,
          slots, scale, workspace, stream)
    return out


def step(q, k, v, log_decay, out, state_in=None, state_out=None, slots=None, scale=None, stream=None):
    """One new token of each sequence: prompt's arguments with tokens == sequences and no starts; returns out."""
    _call(load_library().skinny_linear_step, q, k, v, log_decay, out, v.shape[0], None, state_in, state_out, slots,
          scale, None, stream)
    return out
