"""The layer that runs the 8-bit products and linear attention together.

Tolerances: a row's 8-bit projection does not depend on the rows beside it, so
a token has the same q, k, v and decay bits in a prompt and in a step.  Both
round attention's output once from sums good to a few 2^-24 of the terms'
magnitudes, so they differ by a BF16 step at most, 2 eps / 2 of the value, plus
1e-5 of the largest.  The states are fp32: 1e-5 of the largest.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ll():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from skinny_bf16_decode_amd import linear_layer
    return linear_layer


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def inputs(tokens, hidden, seed):
    return torch.randn(tokens, hidden, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def attended(ll, layer, call):
    """What finish is given: attention's output and the gate."""
    seen = []
    finish = layer.finish
    layer.finish = lambda mixed, gate, residual: (seen.append(mixed.clone()), finish(mixed, gate, residual))[1]
    out = call()
    layer.finish = finish
    return out, seen[0]


@pytest.mark.parametrize("hidden,lengths", [(512, [70, 0, 5]), (1024, [1, 400]), (512, [130])])
def test_prompt_is_prompt_and_steps(ll, hidden, lengths):
    """A prompt in one call, and all but its last tokens followed by steps."""
    live = [i for i, n in enumerate(lengths) if n > 0]
    tokens = sum(lengths)
    x = inputs(tokens, hidden, 3)
    starts = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
    slots = list(range(len(lengths)))[::-1]
    whole = ll.random_layer(hidden, len(lengths) + 1)
    res = torch.zeros(tokens, hidden, device="cuda")
    out, mixed = attended(ll, whole, lambda: whole.prompt(x, res, ints(*starts), ints(*slots)))
    assert out is res
    cut = ll.random_layer(hidden, len(lengths) + 1)
    shorter = [n - 1 if n else 0 for n in lengths]
    rest = [t for i, n in enumerate(lengths) for t in range(starts[i], starts[i] + shorter[i])]
    last = [starts[i] + lengths[i] - 1 for i in live]
    s2 = [sum(shorter[:i]) for i in range(len(lengths) + 1)]
    cut.prompt(x[rest], torch.zeros(len(rest), hidden, device="cuda"), ints(*s2), ints(*slots))
    res2 = torch.zeros(len(last), hidden, device="cuda")
    _, mixed2 = attended(ll, cut, lambda: cut.step(x[last], res2, ints(*[slots[i] for i in live])))
    torch.cuda.synchronize()
    a, b = mixed[last].double(), mixed2.double()
    eps = torch.finfo(torch.bfloat16).eps
    assert bool(((a - b).abs() <= eps * a.abs().maximum(b.abs()) + 1e-5 * a.abs().max()).all())
    assert float((whole.states - cut.states).abs().max()) <= 1e-5 * float(whole.states.abs().max())
    assert bool((whole.states[len(lengths)] == 0).all())


def test_layer_against_the_formula(ll):
    """Attention from the projected bits, token by token in 64 bits; the output from the gated heads' 8 bits."""
    hidden, tokens = 512, 90
    layer = ll.random_layer(hidden, 1)
    x = inputs(tokens, hidden, 5)
    res = torch.randn(tokens, hidden, generator=torch.Generator().manual_seed(6)).cuda()
    before = res.double()
    q, k, v, gate, log_decay = layer.project(x)
    out, mixed = attended(ll, layer, lambda: layer.prompt(x, res, ints(0, tokens), ints(0)))
    state = torch.zeros(ll.HEADS, ll.DIM, ll.DIM, dtype=torch.float64, device="cuda")
    want = torch.empty(tokens, ll.HEADS, ll.DIM, dtype=torch.float64, device="cuda")
    for t in range(tokens):
        state = log_decay[t].double().exp()[:, None, None] * state + k[t].double()[:, :, None] * v[t].double()[:, None]
        want[t] = (q[t].double()[:, :, None] * state).sum(dim=1) * ll.DIM ** -0.5
    eps = torch.finfo(torch.bfloat16).eps
    # two split terms of the state and the scores: 2^-17 of the terms' magnitudes, below 1e-4 of the largest output
    assert bool(((mixed.double() - want).abs() <= eps / 2 * want.abs() + 1e-4 * want.abs().max()).all())
    xq, xs = layer._quantized((mixed * torch.sigmoid(gate)).view(tokens, ll.WIDTH))
    gen = torch.Generator(device="cuda").manual_seed(0)
    torch.randn(ll.PACKED_ROWS, hidden, generator=gen, device="cuda")
    wq, ws = layer._quantized(torch.randn(hidden, ll.WIDTH, generator=gen, device="cuda") * ll.WIDTH ** -0.5)
    p = (xq.double() @ wq.double().t().contiguous()) * torch.outer(xs.double(), ws.double())
    bound = 1.01 * (3 * 2.0 ** -24 * p.abs() + 2 * 2.0 ** -24 * (p + before).abs())
    assert bool(((out.double() - (p + before)).abs() <= bound).all())


def test_steps_in_a_graph(ll):
    """Replays of a captured step, eager work between them, give the eager step's bits."""
    hidden, slots = 512, ints(2, 0)
    eager, layer = ll.random_layer(hidden, 3), ll.random_layer(hidden, 3)
    x = inputs(2, hidden, 8)
    static, res = x.clone(), torch.zeros(2, hidden, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(static, res, slots)
    torch.cuda.current_stream().wait_stream(side)
    layer.states.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(static, res, slots)
    for replay in range(4):
        new = inputs(2, hidden, 20 + replay)
        static.copy_(new)
        res.zero_()
        graph.replay()
        want = eager.step(new, torch.zeros(2, hidden, device="cuda"), slots)
        torch.cuda.synchronize()
        assert torch.equal(res, want), replay
        assert torch.equal(layer.states, eager.states), replay


def test_layer_refusals(ll):
    w, o = torch.zeros(ll.PACKED_ROWS, 64, device="cuda"), torch.zeros(64, ll.WIDTH, device="cuda")
    rate = torch.ones(ll.HEADS, device="cuda")
    for bad in ((w[:-1], o, rate), (w, o[:-1], rate), (w, o, rate[:-1]), (w, o, rate.double())):
        with pytest.raises(ValueError):
            ll.LinearLayer(*bad, 2)
