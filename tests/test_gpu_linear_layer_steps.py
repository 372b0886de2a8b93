"""The linear-attention layer's own steps against their formulas in 64 bits,
from the layer's inputs and weights.

Tolerances.  The 8-bit rows are exact (test_gpu_int8.py), so the projection's
sums are, and its columns are rounded to fp32, scaled twice (2^-24 each) and
rounded to BF16 (eps / 2): those bits are known.  A unit vector's elements are
off by the sum of squares' (128 fp32 roundings at most), the root's and the
quotient's roundings, below 2^-16, and the one to BF16.  A log decay: the
softplus and its product, a few ulps: 2^-20.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

EPS = torch.finfo(torch.bfloat16).eps


@pytest.fixture(scope="module")
def made():
    """(module, layer, its packed weight, decay rates): rows of all sizes, so that no column range passes for another."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from skinny_bf16_decode_amd import linear_layer as ll
    hidden = 384
    g = torch.Generator().manual_seed(101)
    packed = torch.randn(ll.PACKED_ROWS, hidden, generator=g) * hidden ** -0.5
    packed *= torch.exp(0.3 * torch.randn(ll.PACKED_ROWS, 1, generator=g))
    out = torch.randn(hidden, ll.WIDTH, generator=g) * ll.WIDTH ** -0.5
    rate = torch.exp(torch.linspace(-1.0, -7.0, ll.HEADS))
    return ll, ll.LinearLayer(packed.cuda(), out.cuda(), rate.cuda(), 4), packed, rate


def projected(layer, packed, x):
    """The BF16 rows of the packed projection, from the definition of the 8-bit rows and their product."""
    from .test_gpu_int8 import plain_rows
    (xq, xs), (wq, ws) = (tuple(map(torch.from_numpy, plain_rows(t.float().numpy()))) for t in (x, packed))
    sums = xq.double() @ wq.double().t().contiguous()
    return (sums.float() * xs[:, None] * ws[None, :]).bfloat16()


@pytest.mark.parametrize("tokens", [1, 5, 90])
def test_projection_lengths_and_decays(made, tokens):
    ll, layer, packed, rate = made
    x = torch.randn(tokens, layer.hidden, generator=torch.Generator().manual_seed(tokens)).bfloat16()
    q, k, v, gate, log_decay = (t.cpu() for t in layer.project(x.cuda()))
    rows = projected(layer, packed, x)
    parts = [rows[:, i * 1536:(i + 1) * 1536].reshape(tokens, 12, 128) for i in range(4)]
    assert torch.equal(v, parts[2]) and torch.equal(gate, parts[3])
    for got, part in ((q, parts[0]), (k, parts[1])):
        want = part.double() / part.double().norm(dim=-1, keepdim=True)
        assert bool(((got.double() - want).abs() <= (EPS / 2 + 2.0 ** -16) * want.abs()).all())
        assert float((got.double().norm(dim=-1) - 1).abs().max()) < EPS / 2 + 2.0 ** -16
    want = -rate.double() * torch.nn.functional.softplus(rows[:, 6272:6284].double())
    assert bool(((log_decay.double() - want).abs() <= 2.0 ** -20 * want.abs()).all())


def test_a_prompt_and_steps_from_the_inputs(made):
    """The whole layer: a prompt of two sequences and a step of both, from the hidden states to the residual."""
    ll, layer, packed, rate = made
    lengths, slots = [33, 70], [3, 1]
    x = torch.randn(sum(lengths) + 2, layer.hidden, generator=torch.Generator().manual_seed(9)).bfloat16()
    layer.states.zero_()
    seen, finish = [], layer.finish
    layer.finish = lambda mixed, gate, residual: (seen.append(mixed.clone()), finish(mixed, gate, residual))[1]
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")             # noqa: E731
    try:
        layer.prompt(x[:-2].cuda(), torch.zeros(sum(lengths), layer.hidden, device="cuda"), ints(0, 33, 103), ints(*slots))
        layer.step(x[-2:].cuda(), torch.zeros(2, layer.hidden, device="cuda"), ints(*slots))
    finally:
        layer.finish = finish
    rows = projected(layer, packed, x)
    q, k, v = (rows[:, i * 1536:(i + 1) * 1536].reshape(-1, 12, 128).double() for i in range(3))
    # q and k as the layer rounds them, to BF16 from the true quotient: off by half a step at most
    q, k = (t / t.norm(dim=-1, keepdim=True) for t in (q, k))
    decay = torch.exp(-rate.double() * torch.nn.functional.softplus(rows[:, 6272:6284].double()))
    got = torch.cat([s.cpu() for s in seen]).double()
    for seq, tokens in ((0, [*range(33), 103]), (1, [*range(33, 103), 104])):
        S = torch.zeros(12, 128, 128, dtype=torch.float64)
        big = torch.zeros_like(S)
        for t in tokens:
            S = decay[t][:, None, None] * S + k[t][:, :, None] * v[t][:, None]
            big = decay[t][:, None, None] * big + (k[t].abs()[:, :, None] * v[t].abs()[:, None])
            want = (q[t][:, :, None] * S).sum(1) * 128 ** -0.5
            most = (q[t].abs()[:, :, None] * big).sum(1) * 128 ** -0.5
            # q and k are off by eps / 2 each, the output is rounded by eps / 2
            assert bool(((got[t] - want).abs() <= 1.01 * EPS * most + EPS / 2 * want.abs()).all()), t
        state = layer.states[slots[seq]].cpu().double()
        assert bool(((state - S).abs() <= 1.01 * EPS / 2 * big).all())
