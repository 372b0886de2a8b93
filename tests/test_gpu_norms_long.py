"""Norms and joins of the longest rows: lengths whose octets, counted up, pass 2^31.

The tolerances of test_gpu_norms.py, with what a 64-bit sum of this many squares
adds: each of 1024 threads adds 2^21 of them one by one, 2^21 2^-53 = 2^-32 of the
sum, half of it in r, which 2^-31 covers together with the reference's own sum.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

CHUNK = 1 << 27
LONG = 2.0 ** -31


@pytest.fixture(scope="module", autouse=True)
def op():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from skinny_bf16_decode_amd import norms
    yield norms
    torch.cuda.empty_cache()


def row(k, seed, dtype=torch.float16, about=0.0, spread=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.empty(1, k, dtype=dtype, device="cuda").normal_(about, spread, generator=g)


def chunks(k):
    return [slice(a, min(a + CHUNK, k)) for a in range(0, k, CHUNK)]


def factor(x):
    total = sum(float(x[0, c].double().square().sum()) for c in chunks(x.shape[1]))
    return 1 / (total / x.shape[1] + 1e-6) ** 0.5


@pytest.mark.parametrize("k", [2147483641, 2147483647])
def test_norm_of_the_longest_rows(op, k):
    from .test_gpu_norms import H, close
    print("norm", k, flush=True)
    x, w = row(k, 1), row(k, 2, about=1.0, spread=0.2)[0]
    n, q = torch.full((1, k), 7.0, device="cuda"), torch.full((1, k), 77, dtype=torch.int8, device="cuda")
    scale = torch.zeros(1, device="cuda")
    op.norm_rows(x, w, out=n, q=q, scale=scale)
    torch.cuda.synchronize()
    r = factor(x)
    for c in chunks(k):
        want = x[:, c].double() * r * w[c].double()
        close(n[:, c], want, (3 * H + LONG) * want.abs(), torch.float32)
    # the integers are those of the fp32 norm, by int8.quantize_rows' formula
    top = max(n[0, c].abs().max() for c in chunks(k))
    assert torch.equal(scale[0], top / torch.full_like(top, 127.0))
    inverse = torch.full_like(top, 127.0) / top
    for c in chunks(k):
        assert torch.equal(q[0, c], torch.round(n[0, c] * inverse).to(torch.int8)), c


def test_join_of_the_longest_rows(op):
    from .test_gpu_norms import H, close
    k = 2147483647
    print("join", k, flush=True)
    res, y, w, nw = row(k, 1), row(k, 2), row(k, 3, about=1.0, spread=0.2)[0], row(k, 4, about=1.0, spread=0.2)[0]
    out, n = torch.full((1, k), 7.0, dtype=torch.float16, device="cuda"), torch.full((1, k), 7.0, dtype=torch.float16,
                                                                                   device="cuda")
    op.join_rows(res, y, out, weight=w, alpha=0.375, next_weight=nw, next_out=n)
    torch.cuda.synchronize()
    r, rn = factor(y), factor(out)
    for c in chunks(k):
        z = 0.375 * y[:, c].double() * r * w[c].double()
        h = res[:, c].double() + z
        close(out[:, c], h, (10 * H + LONG) * z.abs() + 2 * H * res[:, c].double().abs() + H * h.abs(), torch.float16)
        want = out[:, c].double() * rn * nw[c].double()
        close(n[:, c], want, (3 * H + LONG) * want.abs(), torch.float16)
