"""4-bit products, blocks and norms of more rows than one launch has: rows on both
sides of the border are what the same rows are in a small call, since they repeat."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U8, F16 = torch.uint8, torch.float16
PERIOD = 1000
ROWS = 268_436_000          # 16 threads a row: 268435424 in a launch of norms; 2^30 octets in one of blocks


@pytest.fixture(autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def repeated(t, count):
    """t's rows `count` / PERIOD times, into one allocation."""
    assert t.shape[0] == PERIOD and count % PERIOD == 0
    out = torch.empty(count // PERIOD, *t.shape, dtype=t.dtype, device="cuda")
    out.copy_(t)
    return out.view(count, *t.shape[1:])


def repeats(got, want):
    """Whether got's rows are want's, again and again."""
    a = got.view(-1, *want.shape)
    return all(bool((a[i:i + 50_000] == want).all()) for i in range(0, a.shape[0], 50_000))


def some(*shape, seed=1, dtype=F16):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def test_norm_to_values_and_integers():
    from skinny_bf16_decode_amd import norms
    print("norm", ROWS, flush=True)
    x, w = some(PERIOD, 1), some(1, seed=2)

    def call(x):
        m = x.shape[0]
        out, q, s = torch.full_like(x, 7.0), torch.full((m, 1), 77, dtype=torch.int8, device="cuda"), torch.full((m,), 7.0, device="cuda")
        norms.norm_rows(x, w, out=out, q=q, scale=s)
        return out, q, s

    want = call(x)
    for got, one in zip(call(repeated(x, ROWS)), want):
        assert repeats(got, one)


@pytest.mark.parametrize("bits", [4, 8])
def test_norm_to_blocks(bits):
    from skinny_bf16_decode_amd import norms
    print("norm to blocks", ROWS, bits, flush=True)
    x, w = some(PERIOD, 32), some(32, seed=2)

    def call(x):
        m = x.shape[0]
        q, s = torch.full((m, 4 * bits), 0x77, dtype=U8, device="cuda"), torch.full((m, 1), 0x77, dtype=U8, device="cuda")
        norms.norm_rows(x, w, q=q.view(torch.float8_e4m3fn) if bits == 8 else q, scale=s)
        return q, s

    want = call(x)
    for got, one in zip(call(repeated(x, ROWS)), want):
        assert repeats(got, one)


def test_join():
    from skinny_bf16_decode_amd import norms
    print("join", ROWS, flush=True)
    res, y, g = some(PERIOD, 1, dtype=torch.float32), some(PERIOD, 1, seed=3), some(PERIOD, 1, seed=4, dtype=torch.bfloat16)
    w, nw = some(1, seed=5), some(1, seed=6)

    def call(res, y, g):
        m = y.shape[0]
        out, n = torch.full_like(res, 7.0), torch.full_like(y, 7.0)
        q, s = torch.full((m, 1), 77, dtype=torch.int8, device="cuda"), torch.full((m,), 7.0, device="cuda")
        norms.join_rows(res, y, out, weight=w, gate=g, alpha=0.5, next_weight=nw, next_out=n, q=q, scale=s)
        return out, n, q, s

    want = call(res, y, g)
    for got, one in zip(call(*(repeated(t, ROWS) for t in (res, y, g))), want):
        assert repeats(got, one)


@pytest.mark.parametrize("pitched", [False, True])
def test_blocks_and_back(pitched):
    from skinny_bf16_decode_amd import mxfp4
    print("blocks", ROWS, pitched, flush=True)
    x, g = some(PERIOD, 32), some(PERIOD, 32, seed=2)
    more = 8 if pitched else 0

    def call(x, g):
        m = x.shape[0]
        q, s = torch.full((m, 16 + more), 0x77, dtype=U8, device="cuda"), torch.full((m, 1 + more), 0x77, dtype=U8, device="cuda")
        out = torch.full((m, 32 + more), 7.0, dtype=F16, device="cuda")
        mxfp4.quantize_blocks(x[:, :32], q[:, :16], s[:, :1], gate=g[:, :32])
        mxfp4.expand_blocks(q[:, :16], s[:, :1], out[:, :32])
        return q, s, out

    x, g = (torch.nn.functional.pad(t, (0, more)) for t in (x, g))
    want = call(x, g)
    for got, one in zip(call(repeated(x, ROWS), repeated(g, ROWS)), want):
        assert repeats(got, one)


# 32 x 32 tiles in 4 bits, 16 x 16 in 8
@pytest.mark.parametrize("bits,m", [(4, 268_436_000), (8, 134_218_000)])
def test_product_of_more_tokens_than_a_launch_has(bits, m):
    from skinny_bf16_decode_amd import mxfp4
    from .test_gpu_mxfp4_tiles import exact_codes, typed
    n, k = 7, 32
    print("tokens", m, bits, flush=True)
    gen = torch.Generator("cuda").manual_seed(bits)
    x, w = exact_codes(gen, PERIOD, k, bits), exact_codes(gen, n, k, 4)
    plan = mxfp4.PreparedMxfp4(*w, out_dtype=torch.float32)
    res = some(PERIOD, n, dtype=torch.float32).round()

    def call(q, s, r):
        out = torch.full((q.shape[0], n), 7.0, device="cuda")
        return plan.run(typed(q, bits), s, out, residual=r)

    want = call(*x, res)
    assert repeats(call(repeated(x[0], m), repeated(x[1], m), repeated(res, m)), want)


@pytest.mark.parametrize("bits", [4, 8])
def test_product_of_more_rows_than_a_launch_has(bits):
    """64 x 16 tiles: 536870848 rows in a launch; 69 GB of weight, as it is laid out."""
    from skinny_bf16_decode_amd import mxfp4
    from .test_gpu_mxfp4_tiles import exact_codes, typed
    m, n, k = 2, 536_872_000, 32
    print("rows", n, bits, flush=True)
    gen = torch.Generator("cuda").manual_seed(bits)
    x, w = exact_codes(gen, m, k, bits), exact_codes(gen, PERIOD, k, 4)

    def call(q, s):
        plan = mxfp4.PreparedMxfp4(q, s, out_dtype=F16)
        out = torch.full((m, q.shape[0]), 7.0, dtype=F16, device="cuda")
        plan.run(typed(x[0], bits), x[1], out)
        torch.cuda.synchronize()
        plan.close()
        return out

    want, got = call(*w), call(repeated(w[0], n), repeated(w[1], n))
    for i in range(m):
        assert repeats(got[i], want[i]), i
