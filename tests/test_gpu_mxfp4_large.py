"""4-bit products, blocks and norms past 2^32 bytes and elements: rows behind that
border have to be what the same rows are by themselves."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_rows_past_four_billion_elements():
    from skinny_bf16_decode_amd import mxfp4, norms
    m, k = 66000, 65536
    x = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
    line = torch.randn(4096, k, generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
    for at in range(0, m, 4096):
        x[at:at + 4096] = line[:m - at]
    x[:, 0] = torch.arange(m, device="cuda").bfloat16()
    rows = [0, 1, 32767, 32768, 65535, 65536, m - 1]
    w = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    q, s = torch.empty(m, k, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(m, k // 32, dtype=torch.uint8, device="cuda")
    small = torch.empty(1, k, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(1, k // 32, dtype=torch.uint8, device="cuda")

    def same(fill):
        for r in rows:
            fill(x[r:r + 1], *small)
            assert torch.equal(q[r].view(torch.uint8), small[0][0].view(torch.uint8)) and torch.equal(s[r], small[1][0]), r

    mxfp4.quantize_blocks(x, q, s)
    same(mxfp4.quantize_blocks)
    norms.norm_rows(x, w, q=q, scale=s)
    same(lambda v, a, b: norms.norm_rows(v, w, q=a, scale=b))
    out = torch.empty_like(x)
    mxfp4.expand_blocks(q, s, out)
    for r in rows:
        one = torch.empty(1, k, dtype=torch.bfloat16, device="cuda")
        mxfp4.expand_blocks(q[r:r + 1], s[r:r + 1], one)
        assert torch.equal(out[r], one[0]), r
    norms.join_rows(x, out, out, weight=w)
    for r in rows:
        a, b = torch.empty(1, k, dtype=torch.bfloat16, device="cuda"), torch.empty(1, k, dtype=torch.bfloat16, device="cuda")
        norms.norm_rows(x[r:r + 1], w, q=small[0], scale=small[1])
        mxfp4.expand_blocks(*small, a)
        norms.join_rows(x[r:r + 1], a, b, weight=w)
        assert torch.equal(out[r], b[0]), r


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("m", [3, 200])
def test_weight_past_four_gigabytes(m, bits):
    from skinny_bf16_decode_amd import mxfp4
    n, k = 140000, 65536
    g = torch.Generator("cuda").manual_seed(2)
    w = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8, device="cuda")
    ws = torch.randint(115, 122, (n, k // 32), generator=g, dtype=torch.uint8, device="cuda")
    x = torch.randint(0, 256, (m, k * bits // 8), generator=g, dtype=torch.uint8, device="cuda")
    if bits == 8:
        x[(x & 127) == 127] = 0x38
        x = x.view(torch.float8_e4m3fn)
    xs = torch.randint(120, 127, (m, k // 32), generator=g, dtype=torch.uint8, device="cuda")
    plan = mxfp4.PreparedMxfp4(w, ws, out_dtype=torch.float32)
    out = torch.empty(m, n, device="cuda")
    plan.run(x, xs, out)
    plan.close()
    for lo in (0, 65536, 131072, n - 512):
        part = mxfp4.PreparedMxfp4(w[lo:lo + 512], ws[lo:lo + 512], out_dtype=torch.float32)
        want = torch.empty(m, 512, device="cuda")
        part.run(x, xs, want)
        S = mxfp4.expand_blocks(x, xs, torch.empty(m, k, device="cuda")).abs() @ \
            mxfp4.expand_blocks(w[lo:lo + 512], ws[lo:lo + 512], torch.empty(512, k, device="cuda")).abs().t()
        # other tiles may sum in another order: each sum is within (K / 128 + 5) 2^-22 of the magnitudes' sum
        assert bool(((out[:, lo:lo + 512] - want).abs() <= 2 * (k // 128 + 5) * 2.0 ** -22 * S * 1.01).all()), lo
        part.close()


def test_many_tokens_past_four_gigabytes():
    from skinny_bf16_decode_amd import mxfp4
    m, n, k = 300000, 40, 16384
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.randint(0, 120, (m, k), generator=g, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    xs = torch.randint(120, 127, (m, k // 32), generator=g, dtype=torch.uint8, device="cuda")
    w = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8, device="cuda")
    ws = torch.randint(115, 122, (n, k // 32), generator=g, dtype=torch.uint8, device="cuda")
    plan = mxfp4.PreparedMxfp4(w, ws, out_dtype=torch.float32)
    out = torch.empty(m, n, device="cuda")
    plan.run(x, xs, out)
    wide = mxfp4.expand_blocks(w, ws, torch.empty(n, k, device="cuda")).double()
    for lo in (0, 131072, 262144, m - 64):
        v = mxfp4.expand_blocks(x[lo:lo + 64], xs[lo:lo + 64], torch.empty(64, k, device="cuda")).double()
        want, S = v @ wide.t(), v.abs() @ wide.abs().t()
        assert bool(((out[lo:lo + 64] - want).abs() <= 1.01 * (k // 128 + 5) * 2.0 ** -22 * S + 2.0 ** -23 * want.abs()).all()), lo
