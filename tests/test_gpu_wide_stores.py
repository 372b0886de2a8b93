"""The widest form of linear attention, whose lanes store 16 bytes of output at once: right, and the same in every run."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("lengths", [[320] * 22 + [64, 1], [8000]])
def test_outputs_stored_16_bytes_at_a_time(lengths, kind):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from skinny_bf16_decode_amd import linear_attention as la
    from .test_gpu_linear_attention import check, make, run, say
    say("wide stores", kind, lengths[:2], len(lengths))
    c = make(lengths, 12, 12, 128, 128, kind, 95)
    out, new = run(la, c)
    check(c, out, new, (kind, lengths[:2]))
    for _ in range(10):
        again, _ = run(la, c)
        assert torch.equal(again.view(torch.int16), out.view(torch.int16))
