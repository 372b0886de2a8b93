"""Outputs of prompts whose large state is orthogonal to the queries: what is
left after the terms cancel has fp32's error, as a step's has.

Tolerance.  Let r = (sum_k (scale q_k S_k)^2)^(1/2), the size of a sum of the
terms with random signs.  fp32 rounds each state once or twice (2^-24 of it) and
the sum over dk some dozen times (2^-24 of a partial sum, about r), all of either
sign: less than 2^-22 r in the norm over all outputs, held to twice that, beside
the output's own rounding.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("entry", ["prompt", "step"])
@pytest.mark.parametrize("shape,b,length", [((2, 2, 128, 128), 3, 70), ((2, 1, 64, 64), 2, 130), ((3, 3, 200, 72), 1, 64),
                                            ((12, 12, 128, 128), 24, 64), ((4, 2, 32, 40), 2, 33)])
def test_what_cancellation_leaves(shape, b, length, entry, kind):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from skinny_bf16_decode_amd import linear_attention as la
    from .test_gpu_linear_attention import make, run, say
    heads, key_heads, dk, dv = shape
    if entry == "step":
        length = 1
    say("cancel", kind, entry, shape, b, length)
    c = make([length] * b, *shape, kind, 97)
    c["scale"] = 1.0
    c["log_decay"].zero_()
    c["q"].copy_(c["q"][:1].expand_as(c["q"]).clone())              # one query for all tokens
    c["v"] *= 0.125
    q = c["q"][0].double().repeat_interleave(heads // key_heads, 0)[None]        # [1, heads, dk]
    S = 4096.0 * c["states"].double()
    S -= q[..., None] * (q[..., None] * S).sum(2, keepdim=True) / (q * q).sum(-1)[..., None, None]
    c["states"].copy_(S)
    if entry == "prompt":
        out, _ = run(la, c)
    else:
        out = torch.empty_like(c["v"])
        la.step(c["q"], c["k"], c["v"], c["log_decay"], out, state_in=c["states"], slots=c["slots"], scale=1.0)
        torch.cuda.synchronize()
    S = c["states"][c["slots"].long()].double()
    k = c["k"].double().repeat_interleave(heads // key_heads, 1).view(b, length, heads, dk)
    v = c["v"].double().view(b, length, heads, dv)
    want, r = torch.empty_like(v), torch.empty_like(v)
    for t in range(length):
        S = S + k[:, t, :, :, None] * v[:, t, :, None]
        terms = q[..., None] * S
        want[:, t], r[:, t] = terms.sum(2), terms.square().sum(2).sqrt()
    assert float(want.norm()) < 2.0 ** -10 * float(r.norm())        # there is something to lose
    err = float((out.double().view_as(want) - want).norm())
    say(kind, entry, shape, "error", err / float(r.norm()), "of 2^-21:", err / float(r.norm()) * 2 ** 21)
    assert err <= 2.0 ** -21 * float(r.norm()) + torch.finfo(c["dtype"]).eps / 2 * float(want.norm())
