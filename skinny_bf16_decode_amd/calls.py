"""Calls of the C entry points on a GPU and stream: what the operators' modules share.

A decode step of few sequences waits for the host, so this adds as little as it can."""
from __future__ import annotations

import torch

from . import _raise


def stream_handle(stream, index):
    """hipStream_t of the given stream (an object or a handle), or of the current one of GPU `index`."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    if not hasattr(stream, "cuda_stream"):
        return int(stream)
    if stream.device_index != index:
        raise ValueError(f"the tensors are on cuda:{index}, the stream is of cuda:{stream.device_index}")
    return int(stream.cuda_stream)


def call_on(index, stream, entry, *args):
    """entry(*args, handle of the stream), its error raised, with GPU `index`
    current: a default stream's handle names the current GPU's, whichever that is.
    The tensors of a call on a given stream are the caller's to order with that
    stream and to keep until it has run."""
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream_handle(stream, index)
    if torch._C._cuda_getDevice() == index:
        status = entry(*args, handle)
    else:
        with torch.cuda.device(index):
            status = entry(*args, handle)
    if status:
        _raise(status)
