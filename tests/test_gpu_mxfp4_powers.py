"""8-bit tokens with powers at the ends of what BF16 holds, through which their products go.

BF16's subnormals are multiples of 2^-133.  e4m3's are multiples of 2^-9, so that a
power of 2^-124 (byte 3) and more is exact; below, a value is off by half a step,
2^-134.  4-bit values are multiples of 0.5 and exact at every power down to 2^-127.
The product's own tolerance is test_gpu_mxfp4.py's.
"""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# product_rows, and tiles with powers at any address and in whole dwords
SIZES = [(127, 70, 32), (5, 90, 256), (135, 16403, 160), (135, 16403, 256)]


@pytest.fixture(scope="module", autouse=True)
def op():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from skinny_bf16_decode_amd import mxfp4
    return mxfp4


def product(op, x, w):
    plan = op.PreparedMxfp4(*w, out_dtype=torch.float32)
    out = torch.empty(x[0].shape[0], w[0].shape[0], device="cuda")
    plan.run(x[0].view(torch.float8_e4m3fn), x[1], out)
    return out.double()


def powers(rows, k, byte):
    return torch.full((rows, k // 32), byte, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("xb", range(13))
@pytest.mark.parametrize("m,n,k", SIZES)
def test_low_powers_of_tokens(op, m, n, k, xb):
    from .test_gpu_mxfp4_tiles import check_product, expanded, random_codes, reference
    print("tokens", m, n, k, xb, flush=True)
    gen = torch.Generator("cuda").manual_seed(xb)
    # all magnitudes, the smallest codes most often; the sums are far from fp32's own ends
    below = torch.randint(1, 127, (m, 1), generator=gen, device="cuda").byte()
    x = random_codes(gen, m, k, 8, 0, 1)[0] % below, powers(m, k, xb)
    w = random_codes(gen, n, k, 4, 0, 1)[0], powers(n, k, 200)
    got = product(op, x, w)
    y, S = reference(x, w, 8)
    if xb >= 3:
        check_product(got, y, S, k, torch.float32)
    else:
        off = 2.0 ** -134 * expanded(*w, 4).abs().sum(dim=1)
        tol = 1.01 * ((math.ceil(k / 128) + 5) * 2.0 ** -22 * (S + off) + 2.0 ** -23 * y.abs() + off)
        assert bool(((got - y).abs() <= tol).all())


@pytest.mark.parametrize("xb,wb", [(3, 252), (4, 140), (9, 252), (10, 250), (246, 0), (246, 1), (246, 2), (230, 3), (2, 200)])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_single_values_are_exact(op, m, n, k, xb, wb):
    """One code a token (every magnitude) and one a row: no sum, and every product has 24 bits and lies in fp32's
    normal range; at byte 2 those of the odd smallest codes are rounded, to even."""
    from .test_gpu_mxfp4_tiles import reference
    print("single", m, n, k, xb, wb, flush=True)
    at = 37 % k
    x, w = torch.zeros(m, k, dtype=torch.uint8, device="cuda"), torch.zeros(n, k // 2, dtype=torch.uint8, device="cuda")
    x[:, at] = (torch.arange(m, device="cuda") % 127).byte()
    w[:, at // 2] = (torch.arange(n, device="cuda") % 16).byte() * (16 if at % 2 else 1)
    x, w = (x, powers(m, k, xb)), (w, powers(n, k, wb))
    got = product(op, x, w)
    y, _ = reference(x, w, 8)
    if xb < 3:
        step = 2.0 ** -133
        v = torch.round(reference(x, (torch.full_like(w[0], 0x22), powers(n, k, 127)), 8)[0][:, :1] / step) * step
        y = v * reference((torch.full_like(x[0][:1], 0x38), powers(1, k, 127)), w, 8)[0]
    assert torch.equal(got, y)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_blocks_of_the_smallest_normal_values(op, m, n, k, bits):
    """What quantize_blocks makes of values about 2^-110 (powers below 2^-117) is what the product takes."""
    from .test_gpu_mxfp4_tiles import check_product, random_codes, reference, typed
    print("small", m, n, k, bits, flush=True)
    gen = torch.Generator("cuda").manual_seed(m)
    v = torch.randn(m, k, generator=gen, device="cuda") * 2.0 ** -112
    q = torch.empty(m, k * bits // 8, dtype=torch.uint8, device="cuda")
    s = torch.empty(m, k // 32, dtype=torch.uint8, device="cuda")
    op.quantize_blocks(v, typed(q, bits), s)
    assert int(s.min()) >= 3 and (bits == 4 or int(s.max()) < 10)
    w = random_codes(gen, n, k, 4, 195, 200)
    plan = op.PreparedMxfp4(*w, out_dtype=torch.float32)
    out = torch.empty(m, n, device="cuda")
    plan.run(typed(q, bits), s, out)
    check_product(out, *reference((q, s), w, bits), k, torch.float32)
