"""One workspace, of the largest prompt, for prompts of all sizes, full of NaN before each; states in place."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# few sequences and many parts, then more sequences than parts, some of them cut
PROMPTS = [[5000], [1, 2047, 0, 640, 0, 3000], [90] * 40 + [900, 0, 700, 1300] + [64] * 6, [60] * 60 + [1500], [400], [30]]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(2, 2, 128, 128), (12, 4, 64, 128), (1, 1, 32, 40), (600, 600, 8, 8)])
def test_one_workspace_for_all_prompts(shape, kind):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from skinny_bf16_decode_amd import linear_attention as la
    from .test_gpu_linear_attention import check, make, run, say
    heads, _, dk, dv = shape
    size = la.workspace_bytes(max(map(sum, PROMPTS)), max(map(len, PROMPTS)), heads, dk, dv)
    ws = torch.empty(-(-size // 4), device="cuda")
    for lengths in PROMPTS:
        say("workspace", kind, shape, lengths[:4], len(lengths))
        c = make(lengths, *shape, kind, 63)
        out, new = run(la, c, workspace=ws.fill_(math.nan))
        check(c, out, new, (kind, shape, lengths[:4]))
        again, same = run(la, c, workspace=ws.fill_(math.nan), state_out=c["states"])
        keep = c["slots"].long()
        assert torch.equal(again, out) and torch.equal(same[keep], new[keep])
