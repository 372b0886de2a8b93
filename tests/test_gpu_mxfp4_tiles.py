"""The 4-bit product in every kernel and tile that it can take, against its
formula in 64 bits.  test_mxfp4_tiles_cpu.py asks the library's own choice
whether these sizes reach them all.

Tolerances: those of test_gpu_mxfp4.py, which hold for any number of K's steps added
one after the other.  Where the sums are exact, so has the product to be.
"""
from __future__ import annotations

import math

import numpy as np
import pytest

from . import mx_reference as mx

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# tokens and rows: no multiples of 16, so that the last tiles are part full
ROWS = [(3, 333), (7, 100), (13, 50), (37, 100), (3, 6290), (7, 4099), (13, 6290), (39, 2053), (19, 4103), (37, 3585),
        (3, 8199), (7, 8203), (13, 9001), (35, 4103), (29, 12301), (60, 7001), (6150, 35)]
# 256 rows by 32 t tokens, few wide and many narrow tiles: t = 2 to 4 at any address of x's powers,
# the others where these are whole dwords
ANY = [(135, 16403), (201, 16403), (299, 16403), (14728, 131), (21833, 98), (24607, 98)]
WORDS = {4: [(393, 16403), (489, 16403), (585, 16403), (681, 16403), (32821, 65), (40961, 65), (49175, 65), (57352, 65),
             (4003, 6289)],
         8: [(393, 16403), (489, 16403), (32821, 98), (46437, 65), (1501, 6289)]}
BOTH = [(bits, *size) for bits in (4, 8) for size in ANY]
ALL = BOTH + [(bits, *size) for bits in (4, 8) for size in WORDS[bits]]


@pytest.fixture(scope="module", autouse=True)
def op():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from skinny_bf16_decode_amd import mxfp4
    return mxfp4


def random_codes(gen, rows, k, bits, lo, hi):
    codes = torch.randint(0, 256, (rows, k * bits // 8), generator=gen, dtype=torch.uint8, device="cuda")
    if bits == 8:
        codes[(codes & 127) == 127] = 0x38
    return codes, torch.randint(lo, hi, (rows, k // 32), generator=gen, dtype=torch.uint8, device="cuda")


def exact_codes(gen, rows, k, bits):
    """Multiples of 0.5 up to 6 with powers of 0 to 2: sums of up to 2048 products are exact in fp32."""
    if bits == 4:
        codes = torch.randint(0, 256, (rows, k // 2), generator=gen, dtype=torch.uint8, device="cuda")
    else:
        table = torch.tensor([0x00, 0x30, 0x38, 0x3C, 0x40, 0x44, 0x48, 0x4C, 0xB0, 0xB8, 0xC8], dtype=torch.uint8,
                             device="cuda")
        codes = table[torch.randint(0, len(table), (rows, k), generator=gen, device="cuda")]
    return codes, torch.randint(127, 130, (rows, k // 32), generator=gen, dtype=torch.uint8, device="cuda")


def expanded(codes, byte, bits):
    """What codes stand for, in float64; NaN where they do."""
    table = torch.from_numpy(mx.code_values(bits)).cuda()
    if bits == 4:
        codes = torch.stack((codes & 15, codes >> 4), dim=-1).view(codes.shape[0], -1)
    powers = torch.from_numpy(mx.powers(np.arange(256))).cuda()
    return table[codes.long()] * powers[byte.long()].repeat_interleave(32, dim=1)


def reference(x, w, bits, residual=None):
    a, b = expanded(*x, bits), expanded(*w, 4)
    y, S = a @ b.t(), a.abs() @ b.abs().t()
    return (y if residual is None else y + residual.double()), S


def typed(codes, bits):
    return codes.view(torch.float8_e4m3fn) if bits == 8 else codes


def check_product(got, y, S, k, dtype):
    fi = torch.finfo(dtype)
    tol = (math.ceil(k / 128) + 5) * 2.0 ** -22 * S + (2.0 ** -24 + fi.eps / 2) * y.abs()
    tol = 1.01 * tol + fi.smallest_normal * fi.eps / 2
    got = got.double()
    over = (y.abs() + tol > fi.max) & (got.abs() >= fi.max) & (got.sign() == y.sign())
    bad = ~(((got - y).abs() <= tol) | over)
    assert not bool(bad.any()), (bad.nonzero()[:5].tolist(), got[bad][:5].tolist(), y[bad][:5].tolist())


def between(rows, off, fill=255):
    """These rows with `fill` before and behind each."""
    m, n = rows.shape
    wide = torch.full((m, n + 2 * off), fill, dtype=torch.uint8, device="cuda")
    view = wide[:, off:off + n]
    view.copy_(rows)
    return view


def fill_lds_with_nan(plan_of, m, n, bits):
    """The same tiles over codes and powers of NaN: what a workgroup's LDS holds of them must not reach the next product."""
    k = 1024
    plan = plan_of(torch.zeros(n, k // 2, dtype=torch.uint8, device="cuda"),
                   torch.full((n, k // 32), 255, dtype=torch.uint8, device="cuda"), out_dtype=torch.float32)
    x = torch.full((m, k * bits // 8), 0x7F, dtype=torch.uint8, device="cuda")
    s = torch.full((m, k // 32), 255, dtype=torch.uint8, device="cuda")
    out = torch.empty(m, n, device="cuda")
    plan.run(typed(x, bits), s, out)
    assert bool(out.isnan().all())
    plan.close()


def run_random(op, bits, m, n, k, off):
    print("random", bits, m, n, k, off, flush=True)
    gen = torch.Generator("cuda").manual_seed(m + 7 * n + k + off)
    dtype = list(TYPES.values())[(m + n + k // 32) % 3]
    x, w = random_codes(gen, m, k, bits, 120, 135), random_codes(gen, n, k, 4, 115, 125)
    res = torch.randn(m, n, generator=gen, device="cuda").to(dtype) if k % 64 else None
    plan = op.PreparedMxfp4(*w, out_dtype=dtype)
    out = torch.full((m + 1, n), 3.0, dtype=dtype, device="cuda")
    plan.run(typed(x[0], bits), between(x[1], off) if off else x[1], out, residual=res)
    torch.cuda.synchronize()
    assert bool((out[m] == 3).all())
    check_product(out[:m], *reference(x, w, bits, res), k, dtype)
    plan.close()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("m,n", ROWS)
@pytest.mark.parametrize("k", [96, 640, 2336])
def test_row_kernels(op, bits, m, n, k):
    run_random(op, bits, m, n, k, 0)


@pytest.mark.parametrize("bits,m,n", ALL)
@pytest.mark.parametrize("k", [128, 640, 1152, 2048])
def test_tiles(op, bits, m, n, k):
    """Steps of 128: one, an odd count that is longer than the rings, and whole units of 256."""
    run_random(op, bits, m, n, k, 0)


@pytest.mark.parametrize("bits,m,n", BOTH)
@pytest.mark.parametrize("k,off", [(32, 0), (160, 0), (800, 0), (1312, 0), (256, 1), (384, 2), (1024, 3), (1152, 5)])
def test_tiles_with_powers_at_any_address(op, bits, m, n, k, off):
    """K that ends inside a dword of powers, and whole ones at odd addresses, between powers of NaN."""
    run_random(op, bits, m, n, k, off)


@pytest.mark.parametrize("bits,m,n,k,off", [(*c, k, 0) for c in ALL for k in (128, 640, 2048)] +
                         [(*c, *ko) for c in BOTH for ko in ((32, 1), (416, 1), (1056, 3))])
def test_tiles_are_exact_after_nan(op, bits, m, n, k, off):
    """Each code and power in its place, and nothing that lies past K or is left in LDS."""
    print("exact", bits, m, n, k, off, flush=True)
    gen = torch.Generator("cuda").manual_seed(n + k)
    x, w = exact_codes(gen, m, k, bits), exact_codes(gen, n, k, 4)
    fill_lds_with_nan(op.PreparedMxfp4, m, n, bits)
    plan = op.PreparedMxfp4(*w, out_dtype=torch.float32)
    got = torch.empty(m, n, device="cuda")
    # NaN codes beside a row's own
    q = between(x[0], 16, 0x7F) if off else x[0]
    plan.run(typed(q, bits), between(x[1], off) if off else x[1], got)
    y, S = reference(x, w, bits)
    assert float(S.max()) * 4 < 2 ** 24
    assert torch.equal(got.double(), y)
    plan.close()


@pytest.mark.parametrize("bits,m,n", ALL)
def test_nan_stays_in_its_row(op, bits, m, n):
    """A power of NaN, and in 8 bits a NaN code, in the first block and in the last: one row or column, no other."""
    print("nan", bits, m, n, flush=True)
    k = 416 if (m, n) in ANY else 640
    gen = torch.Generator("cuda").manual_seed(m)
    x, w = random_codes(gen, m, k, bits, 120, 135), random_codes(gen, n, k, 4, 115, 125)
    x[1][1, 0], x[1][m - 2, k // 32 - 1], w[1][5, 3], w[1][n - 1, k // 32 - 1] = 255, 255, 255, 255
    if bits == 8:
        x[0][0, k - 1], x[0][m - 1, 0] = 0x7F, 0xFF
    plan = op.PreparedMxfp4(*w, out_dtype=torch.float32)
    got = torch.empty(m, n, device="cuda")
    plan.run(typed(x[0], bits), x[1], got)
    y, S = reference(x, w, bits)
    want = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    want[[1, m - 2]] = True
    want[:, [5, n - 1]] = True
    if bits == 8:
        want[[0, m - 1]] = True
    assert torch.equal(got.isnan(), want) and torch.equal(y.isnan(), want)
    check_product(got[~want], y[~want], S[~want], k, torch.float32)
    plan.close()


@pytest.mark.parametrize("bits,m,n", ALL)
def test_tiles_pitched_in_place_on_two_streams(op, bits, m, n):
    """Rows of x and out with pitches, out unaligned and its own residual; one plan on two streams at once."""
    print("pitched", bits, m, n, flush=True)
    k = 384
    gen = torch.Generator("cuda").manual_seed(m + 1)
    x, w = random_codes(gen, m, k, bits, 120, 135), random_codes(gen, n, k, 4, 115, 125)
    plan = op.PreparedMxfp4(*w, out_dtype=torch.bfloat16)
    q = typed(between(x[0], 16, 0x7F), bits)
    res = torch.randn(m, n, generator=gen, device="cuda").bfloat16()
    outs = [torch.full((m, n + 7), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    for o in outs:
        o[:, 3:3 + n] = res
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, o in enumerate(outs):
        plan.run(q, x[1], o[:, 3:3 + n], residual=o[:, 3:3 + n], stream=streams[i % 2])
    torch.cuda.synchronize()
    check_product(outs[0][:, 3:3 + n], *reference(x, w, bits, res), k, torch.bfloat16)
    assert bool((outs[0][:, :3] == 5).all()) and bool((outs[0][:, 3 + n:] == 5).all())
    assert all(torch.equal(o, outs[0]) for o in outs[1:])
    plan.close()
