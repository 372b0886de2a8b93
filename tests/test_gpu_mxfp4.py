"""Blocks of 32 values with a power of two, and the products with 4-bit weights,
against their formulas in 64 bits.

Codes and powers are exact.  An expanded value is one product of a code and a
power, exact in fp32, rounded once.  The product's tolerance: one MFMA sums 128
products of 4-bit tokens and what was there before; it is off by fp32's half step
for the sum and by terms cut at 2^-23 of the largest, for which 2^-22 of the
magnitudes' sum is allowed.  8-bit tokens take four MFMAs of 32 products, each a
quarter of that.  A chain over K has K / 128 of them, and 4 more sums join the
waves, so
    |err| <= (ceil(K / 128) + 5) 2^-22 S + (2^-24 + eps / 2) |out| + tiny / 2
with S the sum of |x w|, 2^-24 for the residual's sum, eps / 2 for the output's
type, and one part in 100 for the products of those factors.
"""
from __future__ import annotations

import math

import numpy as np
import pytest

from . import mx_reference as mx

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def op():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from skinny_bf16_decode_amd import mxfp4
    return mxfp4


def raw(t):
    """A tensor of codes or powers as bytes."""
    return t.contiguous().view(torch.uint8).cpu().numpy()


def places(m, k, bits, fill=0x77):
    q = torch.full((m, k * bits // 8), fill, dtype=torch.uint8, device="cuda")
    return (q.view(torch.float8_e4m3fn) if bits == 8 else q), torch.full((m, k // 32), fill, dtype=torch.uint8,
                                                                        device="cuda")


# ---------------------------------------------------------------------------
# quantize_blocks and expand_blocks
# ---------------------------------------------------------------------------

def check_blocks(op, x, bits, q=None, scale=None):
    m, k = x.shape
    if q is None:
        q, scale = places(m, k, bits)
    got = op.quantize_blocks(x, q, scale)
    torch.cuda.synchronize()
    assert got[0] is q and got[1] is scale
    want, byte = mx.blocks(x.double().cpu().numpy(), bits)
    assert np.array_equal(raw(scale[:m]), byte)
    have = mx.unpack(raw(q[:m]), bits)
    assert np.array_equal(have, want)
    assert np.array_equal(np.signbit(have), np.signbit(want)), "signs of zeros"


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,k", [(1, 32), (3, 64), (2, 96), (5, 544), (4, 7168), (33, 1056), (2, 18432), (1, 100000),
                                 (700, 1536)])
def test_quantize_sizes(op, kind, bits, m, k):
    g = torch.Generator().manual_seed(m * 1000 + k)
    x = torch.randn(m, k, generator=g) * torch.exp(2 * torch.randn(k, generator=g))
    check_blocks(op, x.to(TYPES[kind]).cuda(), bits)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("kind", TYPES)
def test_quantize_borders(op, kind, bits):
    """Every border between neighbouring values, a step to each side, at many powers; the clipped range."""
    t = TYPES[kind]
    values = np.unique(np.abs(mx.code_values(bits)[~np.isnan(mx.code_values(bits))]))
    mids = (values[1:] + values[:-1]) / 2
    points = np.concatenate([values, mids, [mx.LARGEST[bits] * 1.05, mx.LARGEST[bits] * 1.1, 2.0 ** (mx.TOP[bits] + 1) * 0.99]])
    rows = []
    for power in (-10, -2, 0, 1, 3):
        for d in (-1, 0, 1):
            p = torch.tensor(points * 2.0 ** power, dtype=torch.float64).to(t)
            near = torch.nextafter(p, torch.full_like(p, math.inf * d)) if d else p
            for i in range(0, len(near), 31):
                part = near[i:i + 31]
                row = torch.zeros(32, dtype=t)
                row[:len(part)] = part * (1 - 2 * (torch.arange(len(part)) % 2)).to(t)
                row[31] = 2.0 ** (mx.TOP[bits] + power)          # fixes the block's power
                if float(part.abs().max()) < 2.0 ** (mx.TOP[bits] + power + 1):
                    rows.append(row)
    check_blocks(op, torch.stack(rows).cuda(), bits)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("kind", TYPES)
def test_quantize_blocks_that_go_wrong(op, kind, bits):
    t = TYPES[kind]
    fi = torch.finfo(t)
    x = torch.randn(14, 96, generator=torch.Generator().manual_seed(5)).to(t)
    x[0] = 0
    x[1] = -0.0
    x[2, 40] = math.inf
    x[3, 0] = -math.inf
    x[4, 95] = math.nan
    x[5, 7] = fi.max
    x[6] = x[6].sign() * (fi.smallest_normal * fi.eps)           # the smallest subnormal
    x[7] = (x[7].double() * 2.0 ** (-120 if kind != "f16" else -14)).to(t)
    x[8] = 0
    x[8, 33] = -fi.smallest_normal
    x[9] = torch.tensor([2.0 ** (i % 60 - 30) for i in range(96)], dtype=torch.float64).clamp(max=60000).to(t)
    x[10] = -fi.max
    x[11, 32:64] = 0
    x[12, :32] = math.nan
    x[13] = x[13] * 1e-38 if kind != "f16" else x[13] * 1e-5
    check_blocks(op, x.cuda(), bits)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("kind", TYPES)
def test_quantize_pitched_and_unaligned(op, kind, bits):
    t = TYPES[kind]
    base = torch.randn(9, 700, generator=torch.Generator().manual_seed(3)).to(t).cuda()
    for lo, k in ((0, 640), (3, 640), (8, 608), (16, 32)):
        for off in (0, 8, 5):
            n = k * bits // 8
            q = torch.full((9, 720), 0x77, dtype=torch.uint8, device="cuda")
            s = torch.full((9, 41), 0x77, dtype=torch.uint8, device="cuda")
            view, sv = q[:, off:off + n], s[:, off:off + k // 32]
            check_blocks(op, base[:, lo:lo + k], bits, view.view(torch.float8_e4m3fn) if bits == 8 else view, sv)
            for full, part in ((q, view), (s, sv)):
                rest = full.clone()
                rest[:, off:off + part.shape[1]] = 0x77
                assert bool((rest == 0x77).all()), "bytes outside the view were written"
    q, s = places(12, 640, bits)
    check_blocks(op, base[:, :640], bits, q, s)
    assert (raw(q[9:]) == 0x77).all() and (raw(s[9:]) == 0x77).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,k,off", [(1, 32, 0), (5, 1056, 0), (300, 4096, 0), (7, 96, 1)])
def test_quantize_gated(op, kind, bits, m, k, off):
    """x silu(g) is rounded three times in fp32 and exp(-g) is within 2 steps: its error is 8 steps of 2^-24 at most,
    a block's largest may cross a power of two by that much, and a value a border."""
    t = TYPES[kind]
    gen = torch.Generator().manual_seed(m + k)
    x, g = (torch.randn(m, k + 8, generator=gen).to(t).cuda()[:, off:off + k] for _ in range(2))
    g = g * 3
    g[0, :4] = torch.tensor([-80.0, 80.0, 0.0, -200.0], dtype=t)
    q, s = places(m, k, bits)
    op.quantize_blocks(x, q, s, gate=g)
    torch.cuda.synchronize()
    v = x.double() * g.double() * torch.sigmoid(g.double())
    v = v.cpu().numpy()
    tol = 8 * 2.0 ** -24
    got = raw(s)
    assert ((got == mx.block_bytes(v * (1 - tol), bits)) | (got == mx.block_bytes(v * (1 + tol), bits))).all()
    u = v / np.repeat(mx.powers(got), 32, axis=1)
    limited = np.clip(u, -mx.LARGEST[bits], mx.LARGEST[bits])
    err = np.abs(mx.unpack(raw(q), bits) - limited)
    assert (err <= mx.step_at(limited, bits) / 2 * (1 + 1e-9) + tol * np.abs(u)).all()


def test_quantize_gated_infinities(op):
    x = torch.ones(4, 32, device="cuda")
    g = torch.ones(4, 32, device="cuda")
    g[0, 3], g[1, 3], g[2, 3] = math.inf, -math.inf, math.nan
    q, s = places(4, 32, 8)
    op.quantize_blocks(x, q, s, gate=g)
    assert raw(s)[:, 0].tolist()[:3] == [255] * 3 and raw(s)[3, 0] != 255 and (raw(q)[:3] == 0).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("off", [0, 1])
def test_expand_every_code_and_power(op, kind, bits, off):
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    k = 256 * 8 // bits
    byte = np.repeat(np.arange(256, dtype=np.uint8)[:, None], k // 32, axis=1)
    q = torch.zeros(256, 256 + off, dtype=torch.uint8, device="cuda")[:, off:]
    q.copy_(torch.from_numpy(codes))
    s = torch.from_numpy(byte).cuda().view(torch.float8_e8m0fnu)
    out = torch.full((257, k + off), 7.0, dtype=TYPES[kind], device="cuda")[:, off:]
    got = op.expand_blocks(q.view(torch.float8_e4m3fn) if bits == 8 else q, s, out)
    torch.cuda.synchronize()
    assert got is out and bool((out[256] == 7).all())
    exact = mx.expanded(codes, byte, bits)
    # fp32's range first: 448 2^127 is past it
    with np.errstate(over="ignore"):
        want = torch.from_numpy(exact.astype(np.float32)).to(TYPES[kind])
    assert torch.equal(torch.nan_to_num(out[:256].cpu().float(), nan=-3.5), torch.nan_to_num(want.float(), nan=-3.5))


def test_no_rows(op):
    q, s = torch.empty(0, 64, dtype=torch.uint8, device="cuda"), torch.empty(0, 4, dtype=torch.uint8, device="cuda")
    op.quantize_blocks(torch.empty(0, 128, device="cuda"), q, s)
    op.expand_blocks(q, s, torch.empty(0, 128, device="cuda"))
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------

def random_codes(gen, rows, k, bits, lo=120, hi=135):
    codes = torch.randint(0, 256, (rows, k * bits // 8), generator=gen, dtype=torch.uint8)
    if bits == 8:
        codes[(codes & 127) == 127] = 0x38
    return codes, torch.randint(lo, hi, (rows, k // 32), generator=gen, dtype=torch.uint8)


def on_gpu(codes, byte, bits):
    q = codes.cuda()
    return (q.view(torch.float8_e4m3fn) if bits == 8 else q), byte.cuda()


def subnormal_step(dtype):
    fi = torch.finfo(dtype)
    return fi.smallest_normal * fi.eps


def reference(xc, xs, wc, ws, bits, residual=None):
    x, w = mx.expanded(xc.numpy(), xs.numpy(), bits), mx.expanded(wc.numpy(), ws.numpy(), 4)
    y, S = x @ w.T, np.abs(x) @ np.abs(w).T
    if residual is not None:
        y = y + residual.double().cpu().numpy()
    return y, S


def check_product(got, y, S, k, dtype):
    got = got.double().cpu().numpy()
    fi = torch.finfo(dtype)
    tol = (math.ceil(k / 128) + 5) * 2.0 ** -22 * S + (2.0 ** -24 + fi.eps / 2) * np.abs(y)
    tol = 1.01 * tol + subnormal_step(dtype) / 2
    # past the type's largest value the nearest are that value and, half a step on, infinity
    over = (np.abs(y) + tol > fi.max) & (np.abs(got) >= fi.max) & (np.sign(got) == np.sign(y))
    bad = ~((np.abs(got - y) <= tol) | over)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], y[bad][:5], tol[bad][:5])


def run_case(op, m, n, k, bits, out, residual, seed, xs_off=0):
    g = torch.Generator().manual_seed(seed)
    dtype = TYPES[out]
    xc, xs = random_codes(g, m, k, bits)
    wc, ws = random_codes(g, n, k, 4, 115, 125)
    plan = op.PreparedMxfp4(*on_gpu(wc, ws, 4), out_dtype=dtype)
    q, s = on_gpu(xc, xs, bits)
    if xs_off:
        wide = torch.full((m, k // 32 + 2 * xs_off), 255, dtype=torch.uint8, device="cuda")
        s = wide[:, xs_off:xs_off + k // 32]
        s.copy_(xs)
    res = torch.randn(m, n, generator=g).to(dtype).cuda() if residual else None
    got = torch.full((m + 1, n), 3.0, dtype=dtype, device="cuda")
    assert plan.run(q, s, got, residual=res) is got
    torch.cuda.synchronize()
    assert bool((got[m] == 3).all())
    check_product(got[:m], *reference(xc, xs, wc, ws, bits, res), k, dtype)
    plan.close()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("m,n,k", [
    (1, 1, 32), (1, 16, 32), (2, 17, 96), (16, 33, 256), (17, 100, 288), (31, 64, 544), (33, 130, 1024), (48, 257, 512),
    (64, 96, 2080), (65, 40, 768), (1, 6288, 7168), (7, 3584, 7168), (5, 512, 18432), (100, 300, 1536), (200, 1000, 1056),
    (257, 513, 2304), (300, 77, 96), (600, 520, 1312), (513, 2049, 256)])
def test_product_sizes(op, m, n, k, bits):
    run_case(op, m, n, k, bits, ["bf16", "f16", "f32"][(m + n) % 3], (m + k) % 2 == 0, m * 7 + n)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("m", [1, 6, 13, 20, 50, 90, 400, 1100])
@pytest.mark.parametrize("n,k", [(1536, 128), (50, 384), (4000, 640), (300, 1152), (260, 2176)])
def test_product_half_units(op, m, n, k, bits):
    """Whole dwords of powers that end in the middle of a unit of 256."""
    run_case(op, m, n, k, bits, "f32", False, m + k)


@pytest.mark.parametrize("m", [2, 40, 200])
@pytest.mark.parametrize("xb,wb", [(7, 127), (1, 140), (0, 160), (10, 120), (127, 3), (140, 0), (236, 60), (60, 240),
                                   (240, 20)])
def test_product_powers_at_their_ends(op, m, xb, wb):
    """Values at the ends of what a power can hold: 8-bit ones above 2^-126, the smallest normal, are exact, and 4-bit
    ones at any power (their products are left to fp32's range)."""
    n, k = 70, 256
    g = torch.Generator().manual_seed(m)
    for bits in (4, 8):
        xc, _ = exact_codes(g, m, k, bits)
        wc, _ = exact_codes(g, n, k, 4)
        xs, ws = torch.full((m, k // 32), xb, dtype=torch.uint8), torch.full((n, k // 32), wb, dtype=torch.uint8)
        plan = op.PreparedMxfp4(*on_gpu(wc, ws, 4), out_dtype=torch.float32)
        got = torch.empty(m, n, device="cuda")
        plan.run(*on_gpu(xc, xs, bits), got)
        y, _ = reference(xc, xs, wc, ws, bits)
        if bits == 8 and min(xb, wb) < 2:
            continue                                    # values below BF16's normal range
        got = got.cpu().numpy().astype(np.float64)
        assert (np.abs(got - y) <= 2.0 ** -149).all(), (bits, np.abs(got - y).max(), np.abs(y).max())


def test_four_bit_type(op):
    """torch's own type of two 4-bit values a byte."""
    g = torch.Generator().manual_seed(4)
    x, w = torch.randn(5, 256, generator=g).cuda(), torch.randn(48, 256, generator=g).cuda()
    made = []
    for t in (torch.uint8, torch.float4_e2m1fn_x2):
        xq, xs = places(5, 256, 4)
        wq, ws = places(48, 256, 4)
        xs, ws = (xs, ws) if t == torch.uint8 else (xs.view(torch.float8_e8m0fnu), ws.view(torch.float8_e8m0fnu))
        op.quantize_blocks(x, xq.view(t), xs)
        op.quantize_blocks(w, wq.view(t), ws)
        out = torch.empty(5, 48, device="cuda")
        op.PreparedMxfp4(wq.view(t), ws, out_dtype=torch.float32).run(xq.view(t), xs, out)
        made.append((xq, raw(xs), out, op.expand_blocks(xq.view(t), xs, torch.empty(5, 256, device="cuda"))))
    assert torch.equal(made[0][0], made[1][0]) and np.array_equal(made[0][1], made[1][1])
    assert torch.equal(made[0][2], made[1][2]) and torch.equal(made[0][3], made[1][3])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("m", [3, 40, 300])
@pytest.mark.parametrize("k", [160, 288, 1024])
@pytest.mark.parametrize("off", [1, 2, 3, 4])
def test_product_scales_at_any_address(op, m, k, off, bits):
    """Powers between others that stand for NaN."""
    run_case(op, m, 300, k, bits, "f32", False, m + k + off, xs_off=off)


def exact_codes(gen, rows, k, bits):
    """Multiples of 0.5 up to 6 with powers of 0 to 2: sums of 2048 products are exact in fp32."""
    if bits == 4:
        codes = torch.randint(0, 256, (rows, k // 2), generator=gen, dtype=torch.uint8)
    else:
        table = torch.tensor([0x00, 0x30, 0x38, 0x3C, 0x40, 0x44, 0x48, 0x4C, 0xB0, 0xB8, 0xC8], dtype=torch.uint8)
        codes = table[torch.randint(0, len(table), (rows, k), generator=gen)]
    return codes, torch.randint(127, 130, (rows, k // 32), generator=gen, dtype=torch.uint8)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("m,n,k", [(1, 50, 2048), (16, 64, 1984), (30, 600, 1024), (64, 200, 2048), (130, 300, 512),
                                   (500, 1100, 2016), (260, 4000, 320), (1030, 270, 1056)])
def test_product_exact(op, m, n, k, bits):
    """Where no sum is rounded, each code and power has to be in its place."""
    g = torch.Generator().manual_seed(n + k)
    xc, xs = exact_codes(g, m, k, bits)
    wc, ws = exact_codes(g, n, k, 4)
    plan = op.PreparedMxfp4(*on_gpu(wc, ws, 4), out_dtype=torch.float32)
    got = torch.empty(m, n, device="cuda")
    plan.run(*on_gpu(xc, xs, bits), got)
    y, S = reference(xc, xs, wc, ws, bits)
    assert S.max() * 4 < 2 ** 24
    assert np.array_equal(got.cpu().numpy().astype(np.float64), y)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("m", [4, 70, 300])
def test_product_nan_stays_in_its_row(op, m, bits):
    """A power of NaN, and in 8 bits a NaN code, in the first block and in the last: one row or column, no other."""
    n, k = 90, 416
    g = torch.Generator().manual_seed(m)
    xc, xs = random_codes(g, m, k, bits)
    wc, ws = random_codes(g, n, k, 4, 115, 125)
    xs[1, 0], xs[2, k // 32 - 1], ws[5, 3] = 255, 255, 255
    if bits == 8:
        xc[0, k - 1] = 0x7F
        xc[3, 0] = 0xFF
    plan = op.PreparedMxfp4(*on_gpu(wc, ws, 4), out_dtype=torch.float32)
    got = torch.empty(m, n, device="cuda")
    plan.run(*on_gpu(xc, xs, bits), got)
    want = torch.zeros(m, n, dtype=torch.bool)
    want[1] = want[2] = want[:, 5] = True
    if bits == 8:
        want[0] = want[3] = True
    assert torch.equal(got.isnan().cpu(), want)
    y, S = reference(xc, xs, wc, ws, bits)
    ok = ~want.numpy()
    check_product(got[torch.from_numpy(ok).cuda()], y[ok], S[ok], k, torch.float32)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("m", [9, 150])
def test_product_pitched_in_place(op, m, bits):
    n, k = 203, 608
    g = torch.Generator().manual_seed(m)
    xc, xs = random_codes(g, m, k, bits)
    wc, ws = random_codes(g, n, k, 4, 115, 125)
    width = k * bits // 8
    wide = torch.full((m, width + 32), 0x7F, dtype=torch.uint8, device="cuda")
    wide[:, 16:16 + width] = xc.cuda()
    q = wide[:, 16:16 + width]
    weight = torch.zeros(n, k // 2 + 3, dtype=torch.uint8, device="cuda")[:, 1:1 + k // 2]
    weight.copy_(wc)
    plan = op.PreparedMxfp4(weight, ws.cuda(), out_dtype=torch.bfloat16)
    out = torch.full((m, n + 7), 5.0, dtype=torch.bfloat16, device="cuda")
    view = out[:, 3:3 + n]
    res = torch.randn(m, n, generator=g).bfloat16()
    view.copy_(res)
    plan.run(q.view(torch.float8_e4m3fn) if bits == 8 else q, xs.cuda(), view, residual=view)
    torch.cuda.synchronize()
    check_product(view, *reference(xc, xs, wc, ws, bits, res), k, torch.bfloat16)
    assert bool((out[:, :3] == 5).all()) and bool((out[:, 3 + n:] == 5).all())


def test_product_no_tokens_and_same_bits_twice(op):
    g = torch.Generator().manual_seed(1)
    wc, ws = random_codes(g, 700, 7168, 4)
    plan = op.PreparedMxfp4(*on_gpu(wc, ws, 4))
    empty = torch.empty(0, 7168, dtype=torch.float8_e4m3fn, device="cuda")
    plan.run(empty, torch.empty(0, 224, dtype=torch.uint8, device="cuda"), torch.empty(0, 700, dtype=torch.bfloat16,
                                                                                     device="cuda"))
    for m in (1, 64, 400):
        xc, xs = random_codes(g, m, 7168, 8)
        outs = [torch.empty(m, 700, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
        for o in outs:
            plan.run(*on_gpu(xc, xs, 8), o)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
