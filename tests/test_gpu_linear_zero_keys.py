"""Linear attention over keys that are zero, as padded tokens have them: finite
data stays on the matrix units.

A chunk that is not finite is done again token by token, which costs a rounded
decay a token where the chunk's own way costs one for 64 tokens.  Without
values to add, a state is its start times the decays, and the two ways can be
told apart by its error: chunk by chunk at most, for each chunk, an exp2 good to
2^-23 of an argument below 2 that is rounded to 2^-24, and a product rounded to
2^-24: 2^-22 in all.  Token by token the same rounded decay enters 300 times, up
to 300 times 2^-24 and more.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("size", [1.0, 70000.0])
@pytest.mark.parametrize("zero", ["all", "tiles", "none"])
@pytest.mark.parametrize("dk,dv,heads", [(64, 64, 8), (128, 128, 8), (32, 40, 4), (200, 128, 4)])
def test_zero_keys_stay_in_chunks(dk, dv, heads, zero, size, kind):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from skinny_bf16_decode_amd import linear_attention as la
    from .test_gpu_linear_attention import check, definition, make, run, say
    say("zero keys", kind, dk, dv, zero, size)
    tokens = 300                                    # five chunks, the last one part full
    c = make([tokens], heads, heads, dk, dv, kind, 81)
    c["v"].zero_()
    at = torch.arange(tokens, device="cuda") % 64
    if zero == "all":
        c["k"].zero_()
    elif zero == "tiles":
        c["k"][(at < 16) | (at >= 32)] = 0          # the scores of whole 16 x 32 tiles
    # 64 of them stay below 2 in the exponent of 2
    c["log_decay"].copy_((-0.003 - 0.0021 * torch.arange(heads, device="cuda")).expand(tokens, heads))
    c["states"] *= size
    out, new = run(la, c)
    check(c, out, new, (dk, dv, zero, size))
    _, S = definition(c)
    got = new[c["slots"].long()].double()
    assert bool(((got - S).abs() <= 5 * 2.0 ** -22 * S.abs()).all()), float(((got - S).abs() / S.abs()).max())
