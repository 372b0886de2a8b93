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
    # as torch's: of handle 0 a new stream
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle or 0x99, device))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0, device))
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


def calls(index):
    """name, call(stream) of every entry, with tensors on GPU `index`."""
    from skinny_bf16_decode_amd import int8
    x, q, scale = (OnGpu(t, s, index) for t, s in ((torch.bfloat16, (4, 64)), (torch.int8, (4, 64)),
                                                   (torch.float32, (4,))))
    plan = int8.PreparedInt8.__new__(int8.PreparedInt8)
    plan.n, plan.k, plan.out_dtype, plan._index, plan._plan = 32, 64, torch.bfloat16, index, None
    out = OnGpu(torch.bfloat16, (4, 32), index)

    def run(stream):
        plan._plan = 1
        try:
            plan.run(q, scale, out, stream=stream)
        finally:
            plan._plan = None               # nothing to destroy

    return [("skinny_quantize_rows", lambda stream: int8.quantize_rows(x, q, scale, stream=stream)),
            ("skinny_int8_run", run),
            ("skinny_linear_prompt", lambda stream: la.prompt(*attention_args(index), stream=stream)),
            ("skinny_linear_step", lambda stream: la.step(*attention_args(index, step=True), stream=stream))]


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("which", range(4))
def test_calls_run_on_their_tensors_gpu(gpu, which, index):
    """The library launches on the current GPU: it has to be the tensors', whichever is current outside."""
    gpu.need = 0
    name, call = calls(index)[which]
    for stream, handle in ((None, CURRENT), (Stream(0x55, f"cuda:{index}"), 0x55), (0x55, 0x55)):
        gpu.log.clear()
        call(stream)
        assert gpu.log == [(name, index, handle)] and gpu.device == 0


@pytest.mark.parametrize("which", range(4))
def test_a_stream_of_another_gpu_is_refused(gpu, which):
    gpu.need = 0
    with pytest.raises(ValueError, match="cuda:1, the stream is of cuda:0"):
        calls(1)[which][1](Stream(0x55, "cuda:0"))
    assert gpu.log == []


def test_workspace_on_another_gpu(gpu):
    for stream, handle in ((None, CURRENT), (Stream(0x55, "cuda:1"), 0x55), (0x55, 0x55)):
        gpu.log.clear()
        la.prompt(*attention_args(1), stream=stream)
        assert gpu.log == [("alloc", 1, handle), ("skinny_linear_prompt", 1, handle)]


@pytest.mark.parametrize("index", [0, 1])
def test_workspace_on_the_default_stream_by_its_handle(gpu, index):
    """Which is 0, what torch.cuda.current_stream().cuda_stream mostly is."""
    la.prompt(*attention_args(index), stream=0)
    assert gpu.log == [("alloc", index, 0), ("skinny_linear_prompt", index, 0)]
