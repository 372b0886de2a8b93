"""Norms before and after a block, against their formulas in 64 bits.

Tolerances: r is off by half a step of fp32 (2^-24; the 64-bit sum's own error
is below 2^-40 for rows of these lengths) and two products by as much each, so a
norm by 3 steps of 2^-24 and its type's rounding, eps / 2.  An int8 scale by the
same 3 and its division's, 4 steps.  Quantized rows have to be, bit by bit, what
int8.quantize_rows and mxfp4.quantize_blocks make of the fp32 norm.  A joined
row adds up to 3 products (gate, alpha, beta) and a sum, and a sigmoid of 4 steps
(an exponential of 2, a sum and a division): 2^-24 times 10 |alpha gate z| +
2 |beta residual| + |h|, then its type's rounding.  One part in 1000 is for the
products of those factors, half the smallest subnormal for what lies below.
"""
from __future__ import annotations

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
H = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def op():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from skinny_bf16_decode_amd import norms
    return norms


def tiny(dtype):
    fi = torch.finfo(dtype)
    return fi.smallest_normal * fi.eps


def exact_norm(x, w, eps=EPS):
    x = x.double()
    return x / torch.sqrt(x.square().mean(dim=1, keepdim=True) + eps) * w.double()


def close(got, want, tol, dtype):
    fi = torch.finfo(dtype)
    tol = 1.001 * (tol + fi.eps / 2 * want.abs()) + tiny(dtype) / 2
    # past the type's largest value the nearest are that value and, half a step on, infinity
    over = (want.abs() + tol > fi.max) & (got.double().abs() >= fi.max) & (got.double().sign() == want.sign())
    bad = ~(((got.double() - want).abs() <= tol) | over)
    assert not bool(bad.any()), (bad.nonzero()[:5].tolist(), got[bad][:5].tolist(), want[bad][:5].tolist())


def quantized_places(kind, m, k):
    if kind == "int8":
        return torch.full((m, k), 77, dtype=torch.int8, device="cuda"), torch.full((m,), 7.0, device="cuda")
    if kind == "mx8":
        return (torch.full((m, k), 0x77, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                torch.full((m, k // 32), 0x77, dtype=torch.uint8, device="cuda"))
    return (torch.full((m, k // 2), 0x77, dtype=torch.uint8, device="cuda"),
            torch.full((m, k // 32), 0x77, dtype=torch.uint8, device="cuda"))


def quantized(kind, n):
    """What the separate call makes of fp32 rows."""
    from skinny_bf16_decode_amd.int8 import quantize_rows
    from skinny_bf16_decode_amd.mxfp4 import quantize_blocks
    q, s = quantized_places(kind, *n.shape)
    return quantize_rows(n, q, s) if kind == "int8" else quantize_blocks(n, q, s)


def same_rows(got, want):
    assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8))
    assert torch.equal(torch.nan_to_num(got[1].float(), nan=-5.0), torch.nan_to_num(want[1].float(), nan=-5.0))


def rows(m, k, kind, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(m, k, generator=g) * torch.exp(spread * torch.randn(m, 1, generator=g))).to(TYPES[kind]).cuda()


def weights(k, kind, seed):
    return (1 + 0.3 * torch.randn(k, generator=torch.Generator().manual_seed(seed))).to(TYPES[kind]).cuda()


SIZES = [(1, 1), (3, 2), (5, 7), (2, 31), (7, 64), (1, 128), (9, 130), (4, 1000), (1, 7168), (6, 8200), (3, 18432),
         (2, 40960), (1, 100003), (600, 96), (1030, 1536), (520, 2051), (515, 7168), (514, 33024)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,k", SIZES)
def test_norm_sizes(op, kind, m, k):
    i = (m + k) % 3
    wk, ok = list(TYPES)[i], list(TYPES)[(i + m) % 3]
    x, w = rows(m, k, kind, m + k), weights(k, wk, k)
    out = torch.full((m + 1, k), 3.0, dtype=TYPES[ok], device="cuda")
    assert op.norm_rows(x, w, out=out) == (out, None, None)
    torch.cuda.synchronize()
    want = exact_norm(x, w)
    close(out[:m], want, 3 * H * want.abs(), TYPES[ok])
    assert bool((out[m] == 3).all())


@pytest.mark.parametrize("q", ["int8", "mx4", "mx8"])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,k", [(1, 32), (5, 96), (3, 544), (1, 7168), (4, 18432), (2, 40960), (700, 128), (520, 7168)])
def test_norm_quantized(op, kind, q, m, k):
    x, w = rows(m, k, kind, m * k), weights(k, "f32", 3)
    n = torch.empty(m, k, device="cuda")
    got = quantized_places(q, m, k)
    assert op.norm_rows(x, w, out=n, q=got[0], scale=got[1])[1:] == got
    alone = quantized_places(q, m, k)
    op.norm_rows(x, w, q=alone[0], scale=alone[1])
    want = exact_norm(x, w)
    close(n, want, 3 * H * want.abs(), torch.float32)
    same_rows(got, quantized(q, n))
    same_rows(alone, got)


@pytest.mark.parametrize("m,k", [(3, 77), (1, 1), (600, 1001)])
def test_norm_int8_any_length(op, m, k):
    x, w = rows(m, k, "f16", 4), weights(k, "bf16", 5)
    n = torch.empty(m, k, device="cuda")
    got = quantized_places("int8", m, k)
    op.norm_rows(x, w, out=n, q=got[0], scale=got[1])
    same_rows(got, quantized("int8", n))


@pytest.mark.parametrize("kind", TYPES)
def test_norm_rows_that_go_wrong(op, kind):
    t = TYPES[kind]
    fi = torch.finfo(t)
    x = torch.randn(10, 160, generator=torch.Generator().manual_seed(1)).to(t)
    x[0] = 0
    x[1] = fi.max
    x[2] = fi.smallest_normal * fi.eps
    x[3, 17] = math.nan
    x[4, 3] = math.inf
    x[5] = 0
    x[5, 159] = fi.max
    x[6] = x[6] * (1e-30 if kind != "f16" else 1e-6)
    x[7, 0] = -math.inf
    x = x.cuda()
    w = torch.ones(160, device="cuda")
    for q in ("int8", "mx4", "mx8"):
        n = torch.empty(10, 160, device="cuda")
        got = quantized_places(q, 10, 160)
        op.norm_rows(x, w, out=n, q=got[0], scale=got[1])
        same_rows(got, quantized(q, n))
    want = exact_norm(x, w)
    fine = torch.isfinite(want)
    assert torch.equal(n.isnan(), want.isnan())
    close(n[fine], want[fine], 3 * H * want[fine].abs(), torch.float32)
    assert bool(n[3].isnan().all()) and bool(n[0].eq(0).all())
    others = [0, 1, 2, 5, 6, 8, 9]
    assert bool(torch.isfinite(n[others]).all())


def test_norm_int8_ignores_what_lies_past_the_row(op):
    """r is infinite for no row, and the last octet of an odd row ends inside it."""
    x = torch.full((4, 13), 1e-30, device="cuda")
    w = torch.full((13,), 3.0, device="cuda")
    n = torch.empty(4, 13, device="cuda")
    got = quantized_places("int8", 4, 13)
    op.norm_rows(x, w, out=n, q=got[0], scale=got[1], eps=2.0 ** -110)
    same_rows(got, quantized("int8", n))
    assert bool((got[0] == 127).all())


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("lo,k", [(0, 640), (3, 640), (8, 608), (5, 333)])
def test_norm_pitched_unaligned_in_place(op, kind, lo, k):
    base = rows(530, 700, kind, 9)
    w = weights(k + 1, "bf16", 2)[1:]
    want = exact_norm(base[:, lo:lo + k], w)
    before = base.clone()
    x = base[:, lo:lo + k]
    op.norm_rows(x, w, out=x)
    torch.cuda.synchronize()
    close(x, want, 3 * H * want.abs(), TYPES[kind])
    assert torch.equal(base[:, :lo], before[:, :lo]) and torch.equal(base[:, lo + k:], before[:, lo + k:])


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("q", ["int8", "mx4", "mx8"])
def test_norm_quantized_into_pitched_places(op, q, off):
    m, k = 6, 160
    x, w = rows(m, k, "bf16", 1), weights(k, "bf16", 1)
    n = torch.empty(m, k, device="cuda")
    op.norm_rows(x, w, out=n)
    want = quantized(q, n)
    width = want[0].shape[1]
    wide = torch.full((m, width + 16), 0x55, dtype=torch.uint8, device="cuda")
    got = wide[:, off:off + width].view(want[0].dtype)
    scale = torch.empty_like(want[1])
    if q != "int8":
        scale = torch.empty(m, k // 32 + 3, dtype=torch.uint8, device="cuda")[:, 1:1 + k // 32]
    op.norm_rows(x, w, q=got, scale=scale)
    torch.cuda.synchronize()
    same_rows((got.contiguous(), scale.contiguous()), want)
    assert bool((wide[:, :off] == 0x55).all()) and bool((wide[:, off + width:] == 0x55).all())


STREAMS = [(255, 520), (256, 520), (257, 1536), (300, 8192), (1023, 7168), (1025, 512), (4096, 7168), (3073, 7168),
           (4003, 4096), (5000, 264), (300, 8200), (260, 16384), (259, 24576), (256, 24584), (2100, 1544)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,k", STREAMS)
def test_norm_many_rows(op, kind, m, k):
    """Around the sizes at which rows go otherwise: from workgroup to workgroup, four at a time, one octet to three a
    thread."""
    x, w = rows(m, k, kind, m + k), weights(k, list(TYPES)[m % 3], k)
    out = torch.full((m + 1, k), 3.0, dtype=TYPES[kind], device="cuda")
    n = torch.empty(m, k, device="cuda")
    got = quantized_places("int8", m, k)
    op.norm_rows(x, w, out=out)
    op.norm_rows(x, w, out=n, q=got[0], scale=got[1])
    want = exact_norm(x, w)
    close(out[:m], want, 3 * H * want.abs(), TYPES[kind])
    close(n, want, 3 * H * want.abs(), torch.float32)
    assert bool((out[m] == 3).all())
    same_rows(got, quantized("int8", n))
    if k % 32 == 0:
        for q in ("mx4", "mx8"):
            got = quantized_places(q, m, k)
            op.norm_rows(x, w, q=got[0], scale=got[1])
            same_rows(got, quantized(q, n))


def test_norm_many_rows_that_go_wrong(op):
    """A row of NaN, infinity, zeros, the largest and the smallest values among others that are not touched by it."""
    m, k = 4100, 1024
    x = rows(m, k, "bf16", 1)
    x[7], x[1030, 5], x[2050, 9], x[4099, 3] = 0, math.nan, math.inf, -math.inf
    x[8], x[9] = torch.finfo(torch.bfloat16).max, 2.0 ** -133
    w = weights(k, "f32", 1)
    want = exact_norm(x, w)
    for q in ("int8", "mx4", "mx8"):
        n = torch.empty(m, k, device="cuda")
        got = quantized_places(q, m, k)
        op.norm_rows(x, w, out=n, q=got[0], scale=got[1])
        assert torch.equal(n.isnan(), want.isnan())
        fine = torch.isfinite(want)
        close(n[fine], want[fine], 3 * H * want[fine].abs(), torch.float32)
        same_rows(got, quantized(q, n))


def test_no_rows(op):
    x, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    op.norm_rows(x, w, out=torch.empty(0, 64, device="cuda"))
    op.join_rows(x, x, torch.empty(0, 64, device="cuda"))
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# join_rows
# ---------------------------------------------------------------------------

def exact_join(res, y, w, gate, sigmoid, alpha, beta, eps=EPS):
    z = y.double() if w is None else exact_norm(y, w, eps)
    if gate is not None:
        z = z * (torch.sigmoid(gate.double()) if sigmoid else gate.double())
    return res.double() * beta + z * alpha, 10 * H * (z * alpha).abs() + 2 * H * (res.double() * beta).abs()


@pytest.mark.parametrize("gate,sigmoid", [(None, False), ("channel", False), ("channel", True), ("token", False),
                                          ("token", True)])
@pytest.mark.parametrize("weight", [None, "f32"])
@pytest.mark.parametrize("m,k", [(1, 1), (3, 77), (2, 1000), (1, 7168), (5, 18432), (1, 40961), (600, 130), (515, 7168),
                                 (513, 33024)])
def test_join_sizes(op, m, k, weight, gate, sigmoid):
    kinds = list(TYPES)
    i = m + k + sigmoid
    yk, rk, gk, nk, ok = (kinds[(i + j * (1 + (k & 1))) % 3] for j in range(5))
    res, y = rows(m, k, rk, 1, 0.5), rows(m, k, yk, 2, 0.5)
    w = None if weight is None else weights(k, weight, 1)
    g = {None: None, "channel": weights(k, gk, 4), "token": rows(m, k, gk, 3, 0.1)}[gate]
    nw = weights(k, nk, 6)
    out = torch.full((m + 1, k), 3.0, dtype=TYPES[rk], device="cuda")
    nxt = torch.full((m + 1, k), 4.0, dtype=TYPES[ok], device="cuda")
    assert op.join_rows(res, y, out, weight=w, gate=g, sigmoid=sigmoid, alpha=0.37, beta=1.25, next_weight=nw,
                        next_out=nxt) is out
    torch.cuda.synchronize()
    a, b = (float(torch.tensor(v, dtype=torch.float32)) for v in (0.37, 1.25))
    h, tol = exact_join(res, y, w, g, sigmoid, a, b)
    close(out[:m], h, tol + H * h.abs(), TYPES[rk])
    n = exact_norm(out[:m], nw)
    close(nxt[:m], n, 3 * H * n.abs(), TYPES[ok])
    assert bool((out[m] == 3).all()) and bool((nxt[m] == 4).all())


@pytest.mark.parametrize("gate,sigmoid", [(None, False), ("channel", True), ("token", True)])
@pytest.mark.parametrize("weight", [None, "bf16"])
@pytest.mark.parametrize("rk", TYPES)
@pytest.mark.parametrize("m,k", [(1023, 520), (1024, 520), (1025, 7168), (2600, 264), (1500, 8192), (1030, 8200)])
def test_join_many_rows(op, m, k, rk, weight, gate, sigmoid):
    yk = ["bf16", "f32", "f16"][(m + k) % 3]
    res, y = rows(m, k, rk, 1, 0.5), rows(m, k, yk, 2, 0.5)
    w = None if weight is None else weights(k, weight, 1)
    g = {None: None, "channel": weights(k, "f16", 4), "token": rows(m, k, "bf16", 3, 0.1)}[gate]
    nw = weights(k, "f32", 6)
    out = torch.full((m + 1, k), 3.0, dtype=TYPES[rk], device="cuda")
    nxt, n = torch.full((m + 1, k), 4.0, dtype=torch.float16, device="cuda"), torch.empty(m, k, device="cuda")
    op.join_rows(res, y, out, weight=w, gate=g, sigmoid=sigmoid, alpha=0.375, beta=1.25, next_weight=nw, next_out=nxt)
    h, tol = exact_join(res, y, w, g, sigmoid, 0.375, 1.25)
    close(out[:m], h, tol + H * h.abs(), TYPES[rk])
    want = exact_norm(out[:m], nw)
    close(nxt[:m], want, 3 * H * want.abs(), torch.float16)
    assert bool((out[m] == 3).all()) and bool((nxt[m] == 4).all())
    got = quantized_places("int8", m, k)
    again = res.clone()
    op.join_rows(again, y, again, weight=w, gate=g, sigmoid=sigmoid, alpha=0.375, beta=1.25, next_weight=nw, next_out=n,
                 q=got[0], scale=got[1])
    assert torch.equal(again, out[:m])
    same_rows(got, quantized("int8", n))


@pytest.mark.parametrize("q", ["int8", "mx4", "mx8"])
@pytest.mark.parametrize("m,k", [(1, 32), (4, 7168), (2, 40960), (700, 544), (1100, 2048)])
@pytest.mark.parametrize("rk", TYPES)
def test_join_next_is_norm_rows_of_what_is_held(op, rk, m, k, q):
    res, y = rows(m, k, rk, 1, 0.5), rows(m, k, "bf16", 2, 0.5)
    w, nw = weights(k, "bf16", 1), weights(k, "f32", 2)
    got = quantized_places(q, m, k)
    out = torch.empty_like(res)
    op.join_rows(res, y, out, weight=w, alpha=0.5, next_weight=nw, q=got[0], scale=got[1])
    want = quantized_places(q, m, k)
    op.norm_rows(out, nw, q=want[0], scale=want[1])
    same_rows(got, want)


@pytest.mark.parametrize("k", [1536, 1535, 40960])
def test_join_in_place(op, k):
    """The residual stream in place, over y's place, and repeated."""
    m = 9
    res, y, w, nw = rows(m, k, "bf16", 1), rows(m, k, "bf16", 2), weights(k, "bf16", 3), weights(k, "bf16", 4)
    apart, n1 = torch.empty_like(res), torch.empty_like(res)
    op.join_rows(res, y, apart, weight=w, next_weight=nw, next_out=n1)
    a, n2 = res.clone(), torch.empty_like(res)
    op.join_rows(a, y, a, weight=w, next_weight=nw, next_out=n2)
    b, n3 = y.clone(), torch.empty_like(res)
    op.join_rows(res, b, b, weight=w, next_weight=nw, next_out=n3)
    torch.cuda.synchronize()
    assert torch.equal(a, apart) and torch.equal(b, apart) and torch.equal(n1, n2) and torch.equal(n1, n3)


def test_join_values_that_are_not_finite_stay_in_their_rows(op):
    m, k = 8, 96
    res, y = rows(m, k, "f32", 1), rows(m, k, "f32", 2)
    g = rows(m, k, "f32", 3)
    res[0, 5], y[1, 6], g[2, 7], y[3, 8] = math.inf, math.nan, math.nan, math.inf
    out, n = torch.empty_like(res), torch.empty_like(res)
    w = torch.ones(k, device="cuda")
    op.join_rows(res, y, out, weight=w, gate=g, sigmoid=True, next_weight=w, next_out=n)
    h, _ = exact_join(res, y, w, g, True, 1.0, 1.0)
    assert torch.equal(out.isnan(), h.isnan()) and torch.equal(out.isinf(), h.isinf())
    assert bool(torch.isfinite(out[4:]).all()) and bool(torch.isfinite(n[4:]).all())
    want = exact_norm(out, w)
    assert torch.equal(n.isnan(), want.isnan())


@pytest.mark.parametrize("gk", TYPES)
def test_join_gates_at_their_ends(op, gk):
    g = torch.tensor([-200.0, -100.0, -80.0, -20.0, 0.0, 20.0, 80.0, 200.0, math.inf, -math.inf] * 4).to(TYPES[gk])
    k = g.numel()
    y, res = torch.full((2, k), 3.0, device="cuda"), torch.zeros(2, k, device="cuda")
    out = torch.empty(2, k, device="cuda")
    op.join_rows(res, y, out, gate=g.cuda(), sigmoid=True)
    want = (3.0 * torch.sigmoid(g.double())).cuda().expand(2, k)
    # exp(-g) past fp32 is infinite there and the gate 0, what is below 2^-126 of it is subnormal
    assert bool(((out.double() - want).abs() <= 6 * H * want + 3 * 2.0 ** -126).all())


def test_join_gate_rows_shared_by_expansion(op):
    m, k = 5, 64
    res, y, g = rows(m, k, "f32", 1), rows(m, k, "bf16", 2), weights(k, "f32", 3)
    a, b = torch.empty_like(res), torch.empty_like(res)
    op.join_rows(res, y, a, gate=g)
    op.join_rows(res, y, b, gate=g.expand(m, k))
    assert torch.equal(a, b)


@pytest.mark.parametrize("off", [1, 4])
def test_join_pitched_and_unaligned(op, off):
    m, k = 7, 320
    def wide(seed, kind):
        return rows(m, k + 12, kind, seed)
    res, y, g, out, n = (wide(i, kind) for i, kind in enumerate(["bf16", "f16", "f32", "bf16", "f16"]))
    before, nb = out.clone(), n.clone()
    cut = lambda t: t[:, off:off + k]                           # noqa: E731
    w, nw = weights(k, "f16", 8), weights(k, "bf16", 9)
    op.join_rows(cut(res), cut(y), cut(out), weight=w, gate=cut(g), next_weight=nw, next_out=cut(n))
    torch.cuda.synchronize()
    h, tol = exact_join(cut(res), cut(y), w, cut(g), False, 1.0, 1.0)
    close(cut(out), h, tol + H * h.abs(), torch.bfloat16)
    want = exact_norm(cut(out), nw)
    close(cut(n), want, 3 * H * want.abs(), torch.float16)
    for t, b in ((out, before), (n, nb)):
        assert torch.equal(t[:, :off], b[:, :off]) and torch.equal(t[:, off + k:], b[:, off + k:])
