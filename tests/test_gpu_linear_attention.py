"""Linear attention with decay against the recurrence itself in 64 bits, token
by token.

Tolerances.  With |S|_t the same recurrence on absolute values, a state's error
is at most c |S|_t.  A term passes at most n = 64 + 64 + T / 64 + 16 fp32
roundings (products and sums inside a chunk, one decay a chunk, the joins), its
FP16 split keeps 22 bits, and a decay exp(-x) that still counts has x < 88 and
an argument good to x 2^-23, so c = (n + 4 + 88) 2^-23.  An output adds up to
dk + 64 terms of a state and of scores that are split to 16 bits:
    |err| <= ((n + 92 + dk) 2^-23 + 2^-15) scale |q| . |S|_t + eps / 2 |out| + tiny / 2.
Those are worst cases; roundings of either sign also bring the error's norm to
a few 2^-24 of the result's, held to 2^-20 (states) and 2^-15 + 0.6 eps (outputs:
the final rounding alone is eps / sqrt(12) to eps / 2 in the norm).
"""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def la():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from skinny_bf16_decode_amd import linear_attention
    return linear_attention


def say(*a):
    print(*a, flush=True)


def make(lengths, heads, key_heads, dk, dv, kind, seed, initial=True, rates=(0.3, 0.0005), order=None):
    g = torch.Generator().manual_seed(seed)
    n, b = sum(lengths), len(lengths)
    t = TYPES[kind]
    rnd = lambda *s: torch.randn(*s, generator=g)                    # noqa: E731
    c = {"q": torch.nn.functional.normalize(rnd(n, key_heads, dk), dim=-1).to(t),
         "k": torch.nn.functional.normalize(rnd(n, key_heads, dk), dim=-1).to(t), "v": rnd(n, heads, dv).to(t)}
    rate = torch.exp(torch.linspace(math.log(rates[0]), math.log(rates[1]), heads))
    c["log_decay"] = -rate * torch.nn.functional.softplus(rnd(n, heads) + 0.5)
    pool = b + 3
    c["states"] = rnd(pool, heads, dk, dv) if initial else None
    c["slots"] = torch.randperm(pool, generator=g)[:b].to(torch.int32)
    ends = [0]
    for x in lengths:
        ends.append(ends[-1] + x)
    c["starts"] = torch.tensor(ends, dtype=torch.int32)
    c.update(lengths=lengths, pool=pool, scale=dk ** -0.5, heads=heads, dk=dk, dv=dv, dtype=t)
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in c.items()}


def definition(c, absolute=False):
    """(out [tokens, heads, dv], new states [b, heads, dk, dv]) in 64 bits, the
    sequences in parallel, the tokens one by one."""
    heads, dk, dv, lengths = c["heads"], c["dk"], c["dv"], c["lengths"]
    b = len(lengths)
    share = heads // c["q"].shape[1]
    f = (lambda x: x.double().abs()) if absolute else (lambda x: x.double())
    q, k, v = f(c["q"]).repeat_interleave(share, 1), f(c["k"]).repeat_interleave(share, 1), f(c["v"])
    decay = c["log_decay"].double().exp()
    S = torch.zeros(b, heads, dk, dv, dtype=torch.float64, device="cuda")
    if c["states"] is not None:
        S = f(c["states"][c["slots"].long()])
    out = torch.zeros(v.shape, dtype=torch.float64, device="cuda")
    starts = [int(x) for x in c["starts"]]
    for t in range(max(lengths, default=0)):
        live = [i for i in range(b) if lengths[i] > t]
        at = torch.tensor([starts[i] + t for i in live], device="cuda")
        idx = torch.tensor(live, device="cuda")
        s = S[idx] * decay[at][:, :, None, None] + k[at][:, :, :, None] * v[at][:, :, None, :]
        S[idx] = s
        out[at] = (q[at][:, :, :, None] * s).sum(2) * c["scale"]
    return out, S


def run(la, c, **kw):
    new = torch.full((c["pool"], c["heads"], c["dk"], c["dv"]), 5.0, device="cuda")
    out = torch.full_like(c["v"], -3.0)
    args = dict(state_in=c["states"], state_out=new, slots=c["slots"], scale=c["scale"])
    args.update(kw)
    got = la.prompt(c["q"], c["k"], c["v"], c["log_decay"], out, c["starts"], **args)
    torch.cuda.synchronize()
    assert got is out
    return out, args["state_out"]


def check(c, out, new, what):
    want, S = definition(c)
    big, bigS = definition(c, absolute=True)
    T = max(c["lengths"], default=0)
    n = 64 + 64 + T / 64 + 16
    got = new[c["slots"].long()].double()
    far = (got - S).abs()
    bound = (n + 4 + 88) * 2.0 ** -23 * bigS + 1e-38
    assert bool((far <= bound).all()), (what, "state", float((far / bound).max()))
    norm = float(S.norm())
    assert float(far.norm()) <= 2.0 ** -20 * norm + 1e-37, (what, "state norm", float(far.norm()) / max(norm, 1e-300))
    fi = torch.finfo(c["dtype"])
    tiny = fi.smallest_normal * fi.eps / 2
    far = (out.double() - want).abs()
    bound = ((n + 92 + c["dk"]) * 2.0 ** -23 + 2.0 ** -15) * big + fi.eps / 2 * want.abs() + tiny
    assert bool((far <= bound).all()), (what, "out", float((far / bound).max()))
    norm = float(want.norm())
    lost = tiny * math.sqrt(max(1, want.numel()))                # outputs of subnormal size
    assert float(far.norm()) <= (2.0 ** -15 + 0.6 * fi.eps) * norm + lost, (what, "out norm", float(far.norm()))
    # slots of no sequence are not touched
    rest = [i for i in range(c["pool"]) if i not in set(c["slots"].tolist())]
    if c["states"] is None or new.data_ptr() != c["states"].data_ptr():
        assert bool((new[rest] == 5).all()), (what, "a free slot was written")


SHAPES = [  # heads, key_heads, dk, dv
    (1, 1, 8, 8), (3, 3, 32, 40), (4, 2, 64, 64), (6, 2, 64, 128), (2, 2, 96, 192), (12, 12, 128, 128),
    (3, 1, 128, 64), (2, 1, 200, 40), (2, 2, 256, 256), (1, 1, 136, 264), (5, 5, 40, 72), (2, 2, 16, 320)]
LENGTHS = [[1], [2], [63], [64], [65], [130], [0, 1, 77, 0, 64, 3], [300, 0, 1, 129]]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_prompt_shapes_and_lengths(la, kind, shape):
    for i, lengths in enumerate(LENGTHS):
        say("prompt", kind, shape, lengths)
        c = make(lengths, *shape, kind, 100 + i, initial=i % 2 == 0)
        out, new = run(la, c)
        check(c, out, new, (kind, shape, lengths))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape,lengths", [
    ((2, 2, 128, 128), [5000]), ((4, 2, 64, 128), [1, 2047, 0, 640, 0, 3000, 64, 0]), ((8, 4, 64, 64), [257] * 20),
    ((2, 1, 256, 192), [1500, 511, 1]), ((12, 12, 128, 128), [1024, 1025]), ((1, 1, 32, 40), [0, 4097, 0])])
def test_prompt_in_parts(la, kind, shape, lengths):
    """Sequences long enough to be cut into parts, with states that reach far."""
    c = make(lengths, *shape, kind, 7, initial=True)
    assert la.workspace_bytes(sum(lengths), len(lengths), shape[0], shape[2], shape[3]) > 0
    say("parts", kind, shape, lengths)
    out, new = run(la, c)
    check(c, out, new, (kind, shape, lengths))
    # with a workspace of the caller's, full of NaN: the same bits
    need = la.workspace_bytes(sum(lengths), len(lengths), shape[0], shape[2], shape[3])
    ws = torch.full((need // 4 + 1,), math.nan, device="cuda")
    out2, new2 = run(la, c, workspace=ws)
    assert torch.equal(out, out2) and torch.equal(new, new2)


@pytest.mark.parametrize("kind", TYPES)
def test_prompt_state_in_place_and_kept_out(la, kind):
    for lengths in ([70, 0, 5, 200], [3000, 10, 0]):
        c = make(lengths, 4, 2, 64, 128, kind, 21)
        want_out, want_new = run(la, c)
        before = c["states"].clone()
        out, _ = run(la, c, state_out=None)
        assert torch.equal(out, want_out) and torch.equal(c["states"], before)
        rest = [i for i in range(c["pool"]) if i not in set(c["slots"].tolist())]
        out, same = run(la, c, state_out=c["states"])
        assert torch.equal(out, want_out)
        assert torch.equal(same[c["slots"].long()], want_new[c["slots"].long()])
        assert torch.equal(same[rest], before[rest])


def test_prompt_is_steps(la):
    """A prompt continued token by token: the prompt's own outputs and state."""
    c = make([90, 40], 4, 2, 64, 128, "bf16", 3)
    out, new = run(la, c)
    S = c["states"].clone()
    starts = c["starts"].tolist()
    for t in range(40):
        rows = torch.tensor([starts[0] + t, starts[1] + t], device="cuda")
        o = torch.empty(2, 4, 128, dtype=torch.bfloat16, device="cuda")
        la.step(c["q"][rows], c["k"][rows], c["v"][rows], c["log_decay"][rows], o, state_in=S, state_out=S,
                slots=c["slots"], scale=c["scale"])
        assert float((o.double() - out[rows].double()).norm()) <= 2 * 0.6 * 2.0 ** -7 * float(out[rows].double().norm())
    seq1 = int(c["slots"][1])
    assert float((S[seq1] - new[seq1]).norm()) <= 2.0 ** -19 * float(new[seq1].norm())


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("b", [1, 5])
def test_step(la, kind, shape, b):
    c = make([1] * b, *shape, kind, 40 + b)
    new = torch.full((c["pool"], *c["states"].shape[1:]), 5.0, device="cuda")
    out = torch.empty_like(c["v"])
    assert la.step(c["q"], c["k"], c["v"], c["log_decay"], out, state_in=c["states"], state_out=new,
                   slots=c["slots"], scale=c["scale"]) is out
    torch.cuda.synchronize()
    check(c, out, new, (kind, shape, b))
    # from nothing, without slots
    c["states"], c["slots"] = None, torch.arange(b, dtype=torch.int32, device="cuda")
    new.fill_(5.0)
    la.step(c["q"], c["k"], c["v"], c["log_decay"], out, state_out=new, scale=c["scale"])
    torch.cuda.synchronize()
    check(c, out, new, (kind, shape, b, "from zero"))


@pytest.mark.parametrize("entry", ["prompt", "step"])
def test_views_of_a_packed_projection(la, entry):
    """q, k and v as column ranges of one [tokens, 6288] output, out into a
    wider buffer, transposed decays, states with a pitch: the packed call's bits."""
    heads, d = 12, 128
    lengths = [33, 0, 100, 1] if entry == "prompt" else [1] * 6
    c = make(lengths, heads, heads, d, d, "bf16", 17)
    n, b = sum(lengths), len(lengths)
    call = {"prompt": lambda *a, **k: la.prompt(*a, c["starts"], **k), "step": la.step}[entry]
    out = torch.empty_like(c["v"])
    new = torch.zeros_like(c["states"])
    kw = dict(slots=c["slots"], scale=c["scale"])
    call(c["q"], c["k"], c["v"], c["log_decay"], out, state_in=c["states"], state_out=new, **kw)
    rows = torch.full((n, 6288), math.nan, dtype=torch.bfloat16, device="cuda")
    views = []
    for i, x in enumerate((c["q"], c["k"], c["v"])):
        view = rows[:, i * heads * d:(i + 1) * heads * d].view(n, heads, d)
        view.copy_(x)
        views.append(view)
    wide = torch.full((n, heads, 2 * d), 9.0, dtype=torch.bfloat16, device="cuda")
    g = c["log_decay"].t().contiguous().t()
    pool = torch.full((c["pool"], heads + 1, d, d), 5.0, device="cuda")
    pool[:, :heads].copy_(c["states"])
    call(*views, g, wide[:, :, :d], state_in=pool[:, :heads], state_out=pool[:, :heads], **kw)
    torch.cuda.synchronize()
    assert torch.equal(wide[:, :, :d], out) and bool((wide[:, :, d:] == 9).all())
    assert torch.equal(pool[c["slots"].long(), :heads], new[c["slots"].long()])
    assert bool((pool[:, heads] == 5).all())


@pytest.mark.parametrize("kind", TYPES)
def test_decays_at_their_ends(la, kind):
    """No decay at all, decays that forget at once (-inf, the lowest value), and far sums."""
    c = make([200, 64, 65], 6, 3, 64, 64, kind, 8)
    g = c["log_decay"]
    g[:, 0] = 0.0
    g[:, 1] = -30.0
    g[::7, 2] = -math.inf
    g[::5, 3] = torch.finfo(torch.float32).min
    g[:, 4] = -1e-9
    g[:, 5] = -4.0
    out, new = run(la, c)
    check(c, out, new, kind)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("size", [2.0 ** -40, 2.0 ** -12, 2.0 ** 12, 2.0 ** 40])
def test_states_of_any_size(la, kind, size):
    """The state's magnitude is fp32's, whatever the 16-bit type's."""
    c = make([150], 2, 2, 64, 64, kind, 12)
    c["states"] *= size
    out, new = run(la, c)
    _, S = definition(c)
    assert float((new[c["slots"].long()].double() - S).norm()) <= 2.0 ** -20 * float(S.norm())
    if not (kind == "f16" and size > 1e5):          # those outputs are FP16 infinities
        check(c, out, new, (kind, size))


@pytest.mark.parametrize("kind", TYPES)
def test_values_of_any_size(la, kind):
    """Keys, queries and values near the ends of FP16."""
    for qs, ks, vs in ((2.0 ** -10, 2.0 ** -10, 2.0 ** -6), (2.0 ** 6, 2.0 ** 9, 2.0 ** -4), (2.0 ** -12, 2.0 ** 8, 2.0 ** 9)):
        c = make([150, 70], 2, 2, 64, 64, kind, 14, initial=False)
        c["q"], c["k"], c["v"] = (x * s for x, s in ((c["q"], qs), (c["k"], ks), (c["v"], vs)))
        out, new = run(la, c)
        check(c, out, new, (kind, qs, ks, vs))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("where", ["q", "k", "v", "log_decay", "states"])
@pytest.mark.parametrize("lengths", [[50, 100, 33], [1500, 700, 40]])
def test_values_that_are_not_finite(la, kind, bad, where, lengths):
    """An infinity or NaN reaches what depends on it and nothing else: no
    earlier token, other sequence, other head or other column."""
    if where == "log_decay" and bad < 0:
        pytest.skip("-inf is a decay")
    heads, dk, dv = 4, 72, 136
    c = make(lengths, heads, 2, dk, dv, kind, 31, rates=(0.05, 0.0005))
    mid = lengths[0] + lengths[1] // 2
    if where == "log_decay":
        c[where][mid, 1] = bad
    elif where == "states":
        c[where][int(c["slots"][1]), 2, 5, 17] = bad
    else:
        c[where][mid, 1, 9] = bad
    out, new = run(la, c)
    want, S = definition(c)
    got = new[c["slots"].long()]
    assert torch.equal(out.isnan(), want.isnan()) and torch.equal(out.isinf(), want.isinf())
    assert torch.equal(got.isnan(), S.isnan()) and torch.equal(got.isinf(), S.isinf())
    assert bool((torch.sign(got)[got.isinf()] == torch.sign(S)[got.isinf()]).all())
    assert bool(S.isfinite().any()) and bool(want.isfinite().any())
    o, w = out.double()[want.isfinite()], want[want.isfinite()]
    eps = torch.finfo(c["dtype"]).eps
    assert float((o - w).norm()) <= (2.0 ** -15 + 0.6 * eps) * float(w.norm())
    s, w = got.double()[S.isfinite()], S[S.isfinite()]
    assert float((s - w).norm()) <= 2.0 ** -20 * float(w.norm())


def test_neighbours_do_not_leak(la):
    """Rows beside a sequence -- other sequences, rows past the last -- may hold anything."""
    c = make([70, 30, 64], 2, 2, 64, 64, "bf16", 33)
    out, new = run(la, c)
    for x in ("q", "k", "v"):
        c[x][70:100] = math.nan
    c["log_decay"][70:100] = math.nan
    out2, new2 = run(la, c)
    keep = [0, 2]
    assert torch.equal(out2[:70], out[:70]) and torch.equal(out2[100:], out[100:])
    assert torch.equal(new2[c["slots"].long()[keep]], new[c["slots"].long()[keep]])


def test_slots_outside_the_pool_and_gaps_between_sequences(la):
    for lengths in ([40, 70, 5], [900, 1200, 5]):
        c = make(lengths, 2, 2, 64, 64, "bf16", 35)
        zero = dict(c, states=c["states"].clone())
        zero["states"][c["slots"][1].long()] = 0
        want, want_new = run(la, zero)
        bad = c["slots"].clone()
        for s in (-1, c["pool"], 2 ** 31 - 1, -2 ** 31):
            bad[1] = s
            out, new = run(la, c, slots=bad)
            assert torch.equal(out, want)
            assert bool((new[c["slots"][1].long()] == 5).all())
            for i in (0, 2):
                assert torch.equal(new[c["slots"][i].long()], want_new[c["slots"][i].long()])
        o1 = torch.empty(3, 2, 64, dtype=torch.bfloat16, device="cuda")
        new = torch.full_like(c["states"], 5.0)
        la.step(c["q"][:3], c["k"][:3], c["v"][:3], c["log_decay"][:3], o1, state_in=c["states"], state_out=new,
                slots=bad)
        assert bool((new[c["slots"][1].long()] == 5).all()) and bool(o1.isfinite().all())
    # tokens that belong to no sequence stay as they are
    c = make([40, 70, 5], 2, 2, 64, 64, "bf16", 36)
    starts = c["starts"].clone()
    starts[0] = 10
    out = torch.full_like(c["v"], -3.0)
    la.prompt(c["q"], c["k"], c["v"], c["log_decay"], out, starts[:3], scale=c["scale"])
    torch.cuda.synchronize()
    assert bool((out[:10] == -3).all()) and bool((out[110:] == -3).all())
    assert bool((out[10:110] != -3).any(dim=-1).all())


def test_no_sequences_and_no_tokens(la):
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    g = torch.empty(0, 2, device="cuda")
    la.step(e, e, e, g, torch.empty_like(e))
    la.prompt(e, e, e, g, torch.empty_like(e), torch.zeros(1, dtype=torch.int32, device="cuda"))
    states = torch.randn(4, 2, 64, 64, device="cuda")
    new = torch.zeros_like(states)
    la.prompt(e, e, e, g, torch.empty_like(e), torch.zeros(4, dtype=torch.int32, device="cuda"), state_in=states,
              state_out=new)
    torch.cuda.synchronize()
    assert torch.equal(new[:3], states[:3]) and bool((new[3] == 0).all())


def test_offsets_past_32_bits(la):
    """A pool whose last slots lie more than 2^31 elements in, and token strides as large."""
    heads, d = 8, 128
    slots = 2 ** 31 // (heads * d * d) + 3
    pool = torch.zeros(slots, heads, d, d, device="cuda")
    c = make([70, 1], heads, heads, d, d, "bf16", 41)
    ids = torch.tensor([slots - 1, slots - 2], dtype=torch.int32, device="cuda")
    pool[ids.long()] = c["states"][c["slots"].long()]
    out, new = run(la, c)
    out2, _ = run(la, c, state_in=pool, state_out=pool, slots=ids)
    assert torch.equal(out, out2) and torch.equal(pool[ids.long()], new[c["slots"].long()])
    assert bool((pool[:4] == 0).all())
    del pool
    step_ids = ids
    big = torch.empty(300, 2 ** 24 - 8, dtype=torch.bfloat16, device="cuda")
    c = make([200, 100], heads, heads, d, d, "bf16", 42)
    views = []
    for i, x in enumerate((c["q"], c["k"], c["v"])):
        view = big[:, i * heads * d:(i + 1) * heads * d].view(300, heads, d)
        view.copy_(x)
        views.append(view)
    out, new = run(la, c)
    c["q"], c["k"], c["v"] = views
    out2 = torch.empty(300, heads, d, dtype=torch.bfloat16, device="cuda")
    new2 = torch.full_like(new, 5.0)
    la.prompt(*views, c["log_decay"], out2, c["starts"], state_in=c["states"], state_out=new2, slots=c["slots"],
              scale=c["scale"])
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(new, new2)


def test_streams_and_graphs(la):
    """Another stream, and graph replays with eager work between them: the eager bits."""
    c = make([1500, 3, 700], 4, 4, 64, 128, "bf16", 51)
    out, new = run(la, c)
    st_out = torch.empty(3, 4, 128, dtype=torch.bfloat16, device="cuda")
    args = (c["q"][:3], c["k"][:3], c["v"][:3], c["log_decay"][:3])
    kw = dict(slots=c["slots"], scale=c["scale"])
    st_new = torch.zeros_like(c["states"])
    la.step(*args, st_out, state_in=c["states"], state_out=st_new, **kw)
    torch.cuda.synchronize()
    ws = torch.empty(la.workspace_bytes(2203, 3, 4, 64, 128), dtype=torch.uint8, device="cuda")
    o, n, so, sn = torch.zeros_like(out), torch.zeros_like(new), torch.zeros_like(st_out), torch.zeros_like(st_new)

    def both(stream=None):
        la.prompt(c["q"], c["k"], c["v"], c["log_decay"], o, c["starts"], state_in=c["states"], state_out=n,
                  workspace=ws, stream=stream, **kw)
        la.step(*args, so, state_in=c["states"], state_out=sn, stream=stream, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both(side)
    side.synchronize()
    keep = c["slots"].long()
    assert torch.equal(o, out) and torch.equal(n[keep], new[keep]) and torch.equal(so, st_out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for replay in range(4):
        for t in (o, n, so, sn):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(n[keep], new[keep]), replay
        assert torch.equal(so, st_out) and torch.equal(sn, st_new), replay
        run(la, make([900, 900], 4, 4, 64, 128, "bf16", 52))


def test_same_bits_every_time(la):
    c = make([2000, 100, 900], 6, 2, 64, 128, "f16", 61)
    out, new = run(la, c)
    for _ in range(3):
        out2, new2 = run(la, c)
        assert torch.equal(out, out2) and torch.equal(new, new2)


def test_refusals(la):
    c = make([10, 20], 4, 2, 64, 64, "bf16", 71)
    out = torch.empty_like(c["v"])

    def bad(**kw):
        a = dict(q=c["q"], k=c["k"], v=c["v"], log_decay=c["log_decay"], out=out, starts=c["starts"],
                 state_in=c["states"], state_out=None, slots=c["slots"])
        a.update(kw)
        with pytest.raises(ValueError):
            la.prompt(**a)

    bad(q=c["q"][:29])
    bad(q=c["q"].float())
    bad(k=c["k"].half())
    bad(q=c["q"][:, :, :60], k=c["k"][:, :, :60])               # dk % 8
    bad(v=c["v"][:, :3], out=out[:, :3], log_decay=c["log_decay"][:, :3], state_in=c["states"][:, :3])
    bad(out=out[:, :, ::2])
    bad(out=out.transpose(0, 1).contiguous())
    bad(log_decay=c["log_decay"].half())
    bad(log_decay=c["log_decay"][:29])
    bad(starts=c["starts"].long())
    bad(starts=c["starts"].cpu())
    bad(slots=c["slots"][:1])
    bad(slots=c["slots"].long())
    bad(state_in=c["states"].half())
    bad(state_in=c["states"][:, :, :, :32])
    bad(state_in=c["states"].transpose(2, 3))
    bad(state_out=torch.empty(3, 4, 64, 64, device="cuda"))      # another pool's size
    bad(slots=None, state_in=c["states"][:1])                    # fewer states than sequences
    bad(v=torch.empty(30 * 4 * 64 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(30, 4, 64))
    with pytest.raises(ValueError):
        la.step(c["q"], c["k"], c["v"], c["log_decay"], out, state_in=c["states"][:20], slots=None)
    long = make([4000], 4, 2, 64, 64, "bf16", 72)
    with pytest.raises(ValueError, match="workspace"):
        la.prompt(long["q"], long["k"], long["v"], long["log_decay"], torch.empty_like(long["v"]), long["starts"],
                  workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
