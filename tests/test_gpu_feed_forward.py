"""4-bit products, blocks and norms as they are used together: feed-forward
blocks over prompts and decode steps, on other streams, and in captured graphs."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def ff():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from skinny_bf16_decode_amd import feed_forward
    return feed_forward


HIDDEN, INNER = 512, 1056


def stream_of(tokens, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(tokens, HIDDEN, generator=g).to(dtype).cuda()


def by_hand(blocks, h):
    """The same by the definitions, in 64 bits from one rounding to the next: each
    stage's result is rounded where the blocks round it, so that what is left
    between the two is a product's fp32 sum and a value that it carries over a border."""
    from skinny_bf16_decode_amd.mxfp4 import expand_blocks, quantize_blocks

    def tokens_of(v, bits):
        q = torch.empty(v.shape[0], v.shape[1] * bits // 8, dtype=torch.float8_e4m3fn if bits == 8 else torch.uint8,
                        device="cuda")
        s = torch.empty(v.shape[0], v.shape[1] // 32, dtype=torch.uint8, device="cuda")
        quantize_blocks(v.float().contiguous(), q, s)
        return expand_blocks(q, s, torch.empty(v.shape, device="cuda")).double()

    def norm(x, w):
        x = x.double()
        return x / torch.sqrt(x.square().mean(dim=1, keepdim=True) + 1e-6) * w.double()

    h = h.clone()
    for b, (gate_up, down) in blocks:
        rows = (tokens_of(norm(h, b.norm_weight), b.bits) @ gate_up.t()).bfloat16()
        gate, up = rows[:, :INNER].double(), rows[:, INNER:].double()
        y = (tokens_of(up * gate * torch.sigmoid(gate), b.bits) @ down.t()).bfloat16()
        z = y if b.post_weight is None else norm(y, b.post_weight)
        h = (h.double() + b.alpha * z.double()).to(h.dtype)
    return h


def make(ff, bits, post=True):
    """Two blocks and their weights as they are held."""
    from skinny_bf16_decode_amd.mxfp4 import expand_blocks, quantize_blocks
    g = torch.Generator().manual_seed(bits)
    made = []
    for _ in range(2):
        gate_up = (torch.randn(2 * INNER, HIDDEN, generator=g) * HIDDEN ** -0.5).cuda()
        down = (torch.randn(HIDDEN, INNER, generator=g) * INNER ** -0.5).cuda()
        norms = [(1 + 0.1 * torch.randn(HIDDEN, generator=g)).cuda() for _ in range(2)]
        held = []
        for w in (gate_up, down):
            n, k = w.shape
            q = torch.empty(n, k // 2, dtype=torch.uint8, device="cuda")
            s = torch.empty(n, k // 32, dtype=torch.uint8, device="cuda")
            quantize_blocks(w, q, s)
            held.append(expand_blocks(q, s, torch.empty(n, k, device="cuda")).double())
        made.append((ff.FeedForward(gate_up, down, norms[0], norms[1] if post else None, alpha=0.5, bits=bits), held))
    return made


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("tokens", [1, 5, 64, 300, 1100])
def test_blocks_against_their_definitions(ff, tokens, post, bits, dtype):
    """Two blocks: the result's distance over the whole is below a hundredth of a
    block's addition.  A value carried over a border of its type moves by a step
    of that type, 2^-3 of it in e4m3 and up to a half in e2m1; a bf16 rounding of
    the products differs for about 1 in 2^8 sums (fp32 errors of 2^-16 of a
    step's size), so that 2^-8 of the values move by a step of 2^-8, and of those
    that do 2^-5 cross a border: together below 2^-8 of the addition in norm."""
    blocks = make(ff, bits, post)
    h = stream_of(tokens, tokens, dtype)
    want = by_hand(blocks, h)
    got = ff.run_blocks([b for b, _ in blocks], h.clone())
    added = (want.double() - h.double()).norm()
    assert float((got.double() - want.double()).norm() / added) < 1e-2
    assert bool(torch.isfinite(got).all())


@pytest.mark.parametrize("bits", [8, 4])
def test_blocks_in_a_graph_and_on_a_stream(ff, bits):
    blocks = [b for b, _ in make(ff, bits)]
    tokens = 7
    h = torch.empty(tokens, HIDDEN, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        h.copy_(stream_of(tokens, 0))
        ff.run_blocks(blocks, h)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ff.run_blocks(blocks, h)
    for seed in range(1, 6):
        new = stream_of(tokens, seed)
        eager = ff.run_blocks(blocks, new.clone())          # between the replays, from the same plans
        h.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, eager), seed
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.current_stream())
            other = ff.run_blocks(blocks, new.clone())
        side.synchronize()
        assert torch.equal(other, eager), seed


def test_one_plan_on_two_streams(ff):
    """Runs that overlap: prompts on one stream, decode steps on another."""
    blocks = [b for b, _ in make(ff, 8)]
    prompt, step = stream_of(700, 1), stream_of(3, 2)
    want = ff.run_blocks(blocks, prompt.clone()), ff.run_blocks(blocks, step.clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    kept = []
    for _ in range(5):
        for s, x in zip(streams, (prompt, step)):
            with torch.cuda.stream(s):
                kept.append(ff.run_blocks(blocks, x.clone()))
    torch.cuda.synchronize()
    for i, got in enumerate(kept):
        assert torch.equal(got, want[i % 2]), i


def test_explicit_streams(ff):
    """Every entry point on a stream given by object and by handle."""
    from skinny_bf16_decode_amd import mxfp4, norms
    x = stream_of(9, 3)
    w = torch.ones(HIDDEN, device="cuda")
    want = None
    plan = make(ff, 8)[0][0].gate_up
    s = torch.cuda.Stream()
    for stream in (None, s, s.cuda_stream):
        s.wait_stream(torch.cuda.current_stream())
        q, p = ff.token_places(9, HIDDEN, 8, "cuda")
        out, n = torch.empty_like(x), torch.empty(9, HIDDEN, device="cuda")
        y = torch.empty(9, 2 * INNER, dtype=torch.bfloat16, device="cuda")
        v = torch.empty(9, HIDDEN, device="cuda")
        torch.cuda.synchronize()
        norms.norm_rows(x, w, out=n, stream=stream)
        norms.join_rows(x, n, out, alpha=0.5, stream=stream)
        mxfp4.quantize_blocks(out, q, p, stream=stream)
        mxfp4.expand_blocks(q, p, v, stream=stream)
        plan.run(q, p, y, stream=stream)
        torch.cuda.synchronize()
        got = (n, out, v, y)
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals(ff):
    w = torch.zeros(HIDDEN, device="cuda")
    with pytest.raises(ValueError, match="gate_up_weight"):
        ff.FeedForward(torch.zeros(INNER, HIDDEN, device="cuda"), torch.zeros(HIDDEN, INNER, device="cuda"), w)
    with pytest.raises(ValueError, match="8 or 4 bits"):
        ff.FeedForward(torch.zeros(2 * INNER, HIDDEN, device="cuda"), torch.zeros(HIDDEN, INNER, device="cuda"), w, bits=6)


def test_command(ff, capsys):
    ff.main()
    assert capsys.readouterr().out.count(" us") == 2


@pytest.mark.parametrize("post", [True, False])
def test_blocks_of_unlike_eps(ff, post):
    """Each block's norms have that block's eps: run together the same bits as
    entered one by one, from rows so small that eps is most of what they are
    divided by (squares of 2^-20 next to eps 2^-14 and 2^-24: a factor above 4)."""
    blocks = [b for b, _ in make(ff, 8, post)]
    blocks[0].eps, blocks[1].eps = 2.0 ** -14, 2.0 ** -24
    h = (stream_of(5, 3) * 2.0 ** -10).bfloat16()
    want = h.clone()
    for b in blocks:
        b.run(want, b.enter(want))
    got = ff.run_blocks(blocks, h.clone())
    assert torch.equal(got, want)
    blocks[1].eps = blocks[0].eps               # the border between the blocks sees the difference
    assert not torch.equal(ff.run_blocks(blocks, h.clone()), want)
