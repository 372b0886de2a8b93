"""What the 8-bit product's and linear attention's Python entries pass to the
library, with stand-ins for the GPU's tensors, streams and library."""
from __future__ import annotations

import contextlib
import types

import pytest
import torch

from skinny_bf16_decode_amd import linear_attention as la


EMPTY = torch.empty


class OnGpu:
    """A tensor on GPU `index` as far as the entries look at one."""

    def __init__(self, dtype, shape, index=0, address=0x10000):
        self._meta = EMPTY(shape, dtype=dtype, device="meta")
        self.dtype, self.shape, self.index, self.address = dtype, self._meta.shape, index, address
        self.device, self.nbytes, self.is_cuda = torch.device("cuda", index), self._meta.nbytes, True

    def dim(self):
        return len(self.shape)

    def stride(self):
        return self._meta.stride()

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.index

    def data_ptr(self):
        return self.address


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle
        self.device_index = 0 if device is None else torch.device(device).index
        self.device = torch.device("cuda", self.device_index)


CURRENT = 0x77          # the current stream of every stand-in GPU


@pytest.fixture
def gpu(monkeypatch):
    """Records (call, device, stream) of what runs on the stand-in GPUs, device 0 the current one."""
    g = types.SimpleNamespace(log=[], device=0, stream=CURRENT, need=1000)

    @contextlib.contextmanager
    def on_stream(stream):
        before = g.stream, g.device
        g.stream, g.device = stream.cuda_stream, stream.device_index
        yield
        g.stream, g.device = before

    @contextlib.contextmanager
    def on_device(device):
        before = g.device
        g.device = device if isinstance(device, int) else torch.device(device).index
        yield
        g.device = before

    def empty(*shape, dtype=None, device=None):
        index = torch.device(device).index
        # a stream's context changes the current stream of its own device only
        g.log.append(("alloc", index, g.stream if index == g.device else CURRENT))
        return OnGpu(dtype, shape, index, 0x20000)

    def entry(name):
        def call(*args):
            g.log.append((name, g.device, args[-1]))
            return 0
        return call

    lib = types.SimpleNamespace(skinny_linear_workspace=lambda *a: g.need,
                                **{n: entry(n) for n in ("skinny_linear_prompt", "skinny_linear_step",
                                                         "skinny_quantize_rows", "skinny_int8_run")})
    import skinny_bf16_decode_amd as sk
    from skinny_bf16_decode_amd import int8
    for module in (la, int8, sk):
        monkeypatch.setattr(module, "load_library", lambda: lib)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", on_stream)
    monkeypatch.setattr(torch.cuda, "device", on_device)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle, device))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: CURRENT, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: g.device, raising=False)
    return g


def attention_args(index=0, tokens=8, step=False):
    h = [OnGpu(torch.bfloat16, (tokens, 2, 32), index) for _ in range(4)]
    args = h[:3] + [OnGpu(torch.float32, (tokens, 2), index), h[3]]
    return args if step else args + [OnGpu(torch.int32, (3,), index)]


@pytest.mark.parametrize("stream,handle", [(None, CURRENT), (Stream(0x55), 0x55), (0x55, 0x55)])
def test_workspace_is_of_the_stream_that_the_prompt_runs_on(gpu, stream, handle):
    la.prompt(*attention_args(), stream=stream)
    assert gpu.log == [("alloc", 0, handle), ("skinny_linear_prompt", 0, handle)]
