"""Calls on a stream of the caller's, with the current stream at work beside them: the current stream's bits."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("given", ["stream", "handle"])
def test_prompt_on_a_stream_without_a_workspace(given):
    """Memory of the workspace's size is taken, written and freed on the current stream before and after the call."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from skinny_bf16_decode_amd import linear_attention as la
    from .test_gpu_linear_attention import make, run
    c = make([1500, 3, 700], 4, 4, 64, 128, "bf16", 51)
    want, new = run(la, c)
    need = la.workspace_bytes(2203, 3, 4, 64, 128)
    assert need > 0
    side = torch.cuda.Stream()
    keep = c["slots"].long()
    for _ in range(5):
        o, n = torch.zeros_like(want), torch.zeros_like(new)
        torch.cuda.synchronize()
        before = [torch.full((need // 4,), math.nan, device="cuda") for _ in range(2)]
        del before
        la.prompt(c["q"], c["k"], c["v"], c["log_decay"], o, c["starts"], state_in=c["states"], state_out=n,
                  slots=c["slots"], scale=c["scale"], stream=side if given == "stream" else side.cuda_stream)
        after = [torch.full((need // 4,), math.nan, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(n[keep], new[keep])
        assert all(bool(x.isnan().all()) for x in after)
