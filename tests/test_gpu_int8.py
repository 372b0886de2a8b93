"""Rows to 8-bit integers and the 8-bit product, against their formulas in 64
bits.

Tolerances: the integers' sum is exact.  It is rounded to fp32 (2^-24), scaled
twice (2^-24 each), a residual added (2^-24 of the sum) and the result rounded
to its type (eps / 2, or half the smallest subnormal), so
    |err| <= 3 * 2^-24 |product| + (2^-24 + eps / 2) |out| + tiny / 2,
with one part in 100 for the products of those factors.
"""
from __future__ import annotations

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def i8():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from skinny_bf16_decode_amd import int8
    return int8


def say(*a):
    print(*a, flush=True)


def subnormal_step(dtype):
    fi = torch.finfo(dtype)
    return fi.smallest_normal * fi.eps


# ---------------------------------------------------------------------------
# quantize_rows
# ---------------------------------------------------------------------------

def plain_rows(x):
    """The formula in fp32, whose operations numpy rounds as IEEE says; exact
    where the kernel's integers have to be."""
    x = x.astype(np.float32)
    top = np.max(np.abs(x), axis=1, initial=0)
    bad = ~np.isfinite(x).all(axis=1)
    lift = np.where(top < np.float32(2.0 ** -60), np.float32(2.0 ** 64), np.float32(1))
    safe = np.where(bad | (top == 0), np.float32(1), top)
    inverse = np.float32(127) / (safe * np.where(bad | (top == 0), np.float32(1), lift))
    with np.errstate(all="ignore"):
        q = np.rint((x * lift[:, None]) * inverse[:, None])
    q[bad | (top == 0)] = 0
    with np.errstate(all="ignore"):
        scale = np.where(bad, np.float32(np.nan), top / np.float32(127))
    return q.astype(np.int8), scale.astype(np.float32)


def check_rows(i8, x, q=None, scale=None):
    m, k = x.shape
    q = torch.full((m, k), 77, dtype=torch.int8, device="cuda") if q is None else q
    scale = torch.full((m,), 7.0, device="cuda") if scale is None else scale
    got_q, got_s = i8.quantize_rows(x, q, scale)
    torch.cuda.synchronize()
    assert got_q is q and got_s is scale
    want_q, want_s = plain_rows(x.float().cpu().numpy())
    assert np.array_equal(q[:m].cpu().numpy(), want_q)
    assert np.array_equal(scale[:m].cpu().numpy(), want_s, equal_nan=True)
    # and the definition: the integers are the nearest to x * 127 / max in 64 bits, but for the fp32 factors
    x64 = x.double().cpu().numpy()
    ok = np.isfinite(want_s) & (want_s > 0)
    exact = x64[ok] * (127.0 / np.abs(x64[ok]).max(axis=1, keepdims=True))
    assert np.abs(want_q[ok] - exact).max(initial=0) <= 0.5 + 127 * 4 * 2.0 ** -24


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,k", [(1, 1), (1, 7), (3, 16), (2, 33), (5, 512), (4, 7168), (33, 1000), (2, 18432),
                                 (2, 40960), (1, 100000), (300, 128)])
def test_quantize_sizes(i8, kind, m, k):
    g = torch.Generator().manual_seed(m * 1000 + k)
    x = torch.randn(m, k, generator=g) * torch.exp(2 * torch.randn(k, generator=g))
    check_rows(i8, x.to(TYPES[kind]).cuda())


@pytest.mark.parametrize("kind", TYPES)
def test_quantize_rows_that_go_wrong(i8, kind):
    t = TYPES[kind]
    fi = torch.finfo(t)
    g = torch.Generator().manual_seed(5)
    x = torch.randn(12, 264, generator=g).to(t)
    x[0] = 0
    x[1] = -0.0
    x[2, 100] = math.inf
    x[3, 0] = -math.inf
    x[4, 263] = math.nan
    x[5, 7] = fi.max
    x[6] = x[6].sign() * (fi.smallest_normal * fi.eps)       # the smallest subnormal
    x[7] = (x[7].double() * 2.0 ** (-75 if kind != "f16" else -14)).to(t)
    x[8] = 0
    x[8, 5] = -fi.smallest_normal
    x[9] = torch.arange(264).to(t)                          # halves: ties go to even
    x[9] = x[9] % 127 + 0.5
    x[9, 3] = 127
    x[10] = 1.0
    x[11, 17] = -1000.0
    check_rows(i8, x.cuda())


@pytest.mark.parametrize("kind", TYPES)
def test_quantize_pitched_and_unaligned(i8, kind):
    t = TYPES[kind]
    base = torch.randn(9, 700, generator=torch.Generator().manual_seed(3)).to(t).cuda()
    for lo, hi in ((0, 640), (3, 643), (8, 648), (16, 533)):
        for q_off in (0, 8, 5):
            q = torch.full((9, 720), 77, dtype=torch.int8, device="cuda")
            view = q[:, q_off:q_off + hi - lo]
            check_rows(i8, base[:, lo:hi], q=view)
            rest = q.clone()
            rest[:, q_off:q_off + hi - lo] = 77
            assert bool((rest == 77).all()), "columns outside the view were written"
    # more rows of space than rows
    q = torch.full((12, 640), 77, dtype=torch.int8, device="cuda")
    scale = torch.full((12,), 7.0, device="cuda")
    check_rows(i8, base[:, :640], q=q, scale=scale)
    assert bool((q[9:] == 77).all()) and bool((scale[9:] == 7).all())


def test_quantize_no_rows(i8):
    q, s = torch.empty(0, 64, dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda")
    i8.quantize_rows(torch.empty(0, 64, device="cuda"), q, s)
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------

def make(m, n, k, seed, out, residual):
    g = torch.Generator().manual_seed(seed)
    xq = torch.randint(-128, 128, (m, k), generator=g, dtype=torch.int8)
    wq = torch.randint(-128, 128, (n, k), generator=g, dtype=torch.int8)
    xs = torch.exp(torch.randn(m, generator=g)) / 128
    ws = torch.exp(torch.randn(n, generator=g)) / 128 / math.sqrt(k)
    res = torch.randn(m, n, generator=g).to(TYPES[out]) if residual else None
    return xq, wq, xs, ws, res


def definition(xq, wq, xs, ws, res):
    """(sum in 64 bits, product, out)"""
    xq, wq = xq.cuda().double(), wq.cuda().double()
    p = (xq @ wq.t().contiguous()) * torch.outer(xs.cuda().double(), ws.cuda().double())
    return p, p if res is None else p + res.cuda().double()


def check_product(got, p, want, dtype, what):
    fi = torch.finfo(dtype)
    bound = 1.01 * (3 * 2.0 ** -24 * p.abs() + (2.0 ** -24 + fi.eps / 2) * want.abs()) + subnormal_step(dtype) / 2
    far = (got.double() - want).abs()
    assert bool((far <= bound).all()), (what, float((far / bound).max()))


SIZES = [(1, 1, 16), (1, 17, 64), (2, 16, 48), (3, 40, 80), (16, 33, 1024), (17, 100, 7168), (31, 250, 400),
         (48, 129, 208), (49, 64, 64), (64, 96, 18432), (65, 130, 320), (100, 300, 1008), (128, 256, 512),
         (129, 257, 1040), (200, 16, 5120), (255, 700, 96), (257, 513, 272), (513, 1030, 144), (1000, 272, 2064),
         (1, 6288, 7168), (37, 3584, 7168), (2000, 1000, 528), (300, 6288, 128), (700, 40, 16)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("out,residual", [("bf16", False), ("f32", True), ("f16", False), ("bf16", True)])
def test_product_sizes(i8, m, n, k, out, residual):
    say("product", m, n, k, out, residual)
    xq, wq, xs, ws, res = make(m, n, k, m + n + k, out, residual)
    p, want = definition(xq, wq, xs, ws, res)
    plan = i8.PreparedInt8(wq.cuda(), ws.cuda(), out_dtype=TYPES[out])
    y = torch.full((m + 1, n), -7.0, dtype=TYPES[out], device="cuda")
    for again in range(2):                       # the second run finds what the first left behind
        got = plan.run(xq.cuda(), xs.cuda(), y, residual=None if res is None else res.cuda())
        torch.cuda.synchronize()
        assert got is y
        check_product(y[:m], p, want, TYPES[out], (m, n, k, out, again))
        assert bool((y[m:] == -7).all())
    plan.close()


def test_product_extremes_are_exact(i8):
    """Sums at the ends of the range: -128 * -128 over the longest K, and rows
    of 127 against -128; with scales of one, the fp32 output is the rounded sum."""
    k = 131056
    xq = torch.full((5, k), -128, dtype=torch.int8)
    wq = torch.full((20, k), -128, dtype=torch.int8)
    xq[1] = 127
    wq[3] = 127
    wq[4, ::2] = 0
    want = (xq.long() @ wq.long().t()).double()
    assert float(want.max()) < 2 ** 31
    plan = i8.PreparedInt8(wq.cuda(), torch.ones(20, device="cuda"), out_dtype=torch.float32)
    y = torch.empty(5, 20, device="cuda")
    plan.run(xq.cuda(), torch.ones(5, device="cuda"), y)
    assert torch.equal(y.cpu(), want.float())
    plan.close()


@pytest.mark.parametrize("m", [1, 40, 300])
def test_product_scales_that_are_not_finite(i8, m):
    """A NaN or infinite scale reaches its token or channel and no other."""
    n, k = 90, 160
    xq, wq, xs, ws, _ = make(m, n, k, 9, "f32", False)
    xs[0], ws[7], ws[50] = math.nan, math.inf, 0.0
    p, want = definition(xq, wq, xs, ws, None)
    plan = i8.PreparedInt8(wq.cuda(), ws.cuda(), out_dtype=torch.float32)
    y = plan.run(xq.cuda(), xs.cuda(), torch.empty(m, n, device="cuda"))
    assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y.isinf(), want.isinf())
    fine = want.isfinite()
    assert bool(((y.double() - want).abs()[fine] <= 4 * 2.0 ** -24 * p.abs()[fine]).all())
    plan.close()


@pytest.mark.parametrize("m", [3, 70, 260])
def test_product_views_and_in_place_residual(i8, m):
    n, k = 200, 320
    xq, wq, xs, ws, res = make(m, n, k, 11, "bf16", True)
    p, want = definition(xq, wq, xs, ws, res)
    big_x = torch.zeros(m, k + 48, dtype=torch.int8, device="cuda")
    big_x[:, 16:16 + k] = xq.cuda()
    big_w = torch.zeros(n, k + 5, dtype=torch.int8, device="cuda")
    big_w[:, 3:3 + k] = wq.cuda()
    plan = i8.PreparedInt8(big_w[:, 3:3 + k], ws.cuda())
    big_y = torch.full((m, n + 9), 3.0, dtype=torch.bfloat16, device="cuda")
    y = big_y[:, 5:5 + n]
    y.copy_(res)
    plan.run(big_x[:, 16:16 + k], xs.cuda(), y, residual=y)
    torch.cuda.synchronize()
    check_product(y, p, want, torch.bfloat16, m)
    assert bool((big_y[:, :5] == 3).all()) and bool((big_y[:, 5 + n:] == 3).all())
    plan.close()


def test_product_on_a_stream_and_in_a_graph(i8):
    """Graph replays, with eager runs of other sizes between, give the eager bits."""
    n, k = 512, 2048
    xq, wq, xs, ws, _ = make(300, n, k, 13, "bf16", False)
    plan = i8.PreparedInt8(wq.cuda(), ws.cuda())
    xq, xs = xq.cuda(), xs.cuda()
    sizes = (1, 40, 100, 300)
    eager = {m: plan.run(xq[:m], xs, torch.empty(m, n, dtype=torch.bfloat16, device="cuda")).clone() for m in sizes}
    x = torch.randn(300, k, device="cuda")
    want_q, want_s = (t.clone() for t in i8.quantize_rows(x, torch.empty_like(xq), torch.empty_like(xs)))
    torch.cuda.synchronize()
    outs = {m: torch.zeros(m, n, dtype=torch.bfloat16, device="cuda") for m in sizes}
    gq, gs = torch.zeros_like(xq), torch.zeros_like(xs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for m in sizes:
            plan.run(xq[:m], xs, outs[m])
    side.synchronize()
    for m in sizes:
        assert torch.equal(outs[m], eager[m])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for m in sizes:
            plan.run(xq[:m], xs, outs[m])
        i8.quantize_rows(x, gq, gs)
    for replay in range(4):
        for m in sizes:
            outs[m].zero_()
        gq.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for m in sizes:
            assert torch.equal(outs[m], eager[m]), (replay, m)
        assert torch.equal(gq, want_q) and torch.equal(gs, want_s)
        plan.run(xq[:77], xs, torch.empty(77, n, dtype=torch.bfloat16, device="cuda"))
        torch.cuda.synchronize()
    plan.close()


def test_product_refusals(i8):
    w, ws = torch.zeros(32, 64, dtype=torch.int8, device="cuda"), torch.zeros(32, device="cuda")
    with pytest.raises(ValueError):
        i8.PreparedInt8(w[:, :40], ws)                       # K % 16
    with pytest.raises(ValueError):
        i8.PreparedInt8(w, ws[:31])
    with pytest.raises(ValueError):
        i8.PreparedInt8(w, ws, out_dtype=torch.float64)
    plan = i8.PreparedInt8(w, ws)
    x, xs = torch.zeros(4, 64, dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda")
    y = torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda")
    bad = [(x[:, :48], xs, y, None), (x.float(), xs, y, None), (x, xs[:3], y, None), (x, xs, y[:3], None),
           (x, xs, y.float(), None), (x, xs, y[:, :31], None), (x, xs, y, y.float()), (x.cpu(), xs, y, None),
           (torch.zeros(4, 72, dtype=torch.int8, device="cuda")[:, :64], xs, y, None),      # pitch % 16
           (torch.zeros(4 * 64 + 1, dtype=torch.int8, device="cuda")[1:].view(4, 64), xs, y, None),
           (x.t().contiguous().t(), xs, y, None)]
    for x_, xs_, y_, r_ in bad:
        with pytest.raises(ValueError):
            plan.run(x_, xs_, y_, residual=r_)
    assert plan.run(x[:0], xs[:0], y[:0]).shape == (0, 32)
    plan.close()
    with pytest.raises(ValueError):
        plan.run(x, xs, y)
