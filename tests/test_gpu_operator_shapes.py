"""The 8-bit product at sizes that reach each of its tiles, and linear
attention at shapes that reach each way of cutting sequences and columns, with
the definitions and tolerances of test_gpu_int8.py and test_gpu_linear_attention.py.
"""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# tokens and rows that take: rows kernel, 16 r rows by 16 t tokens (one token tile, then several)
ROWS = [(1, 300), (17, 2053), (33, 3000), (64, 3500), (9, 4200), (17, 4097), (33, 4119), (49, 4103), (1, 8195),
        (17, 8196), (33, 8204), (49, 8220), (2053, 17), (4138, 33), (33, 2054), (6165, 33), (65, 4102), (200, 6288)]
# tiles kernel, 256 rows by 32 t tokens, t = 1 .. 8
TILES = [(194, 8205), (6651, 257), (5481, 514), (8168, 536), (6551, 1041), (8166, 1041), (8150, 1287), (8140, 1552)]


@pytest.mark.parametrize("m,n", ROWS + TILES)
@pytest.mark.parametrize("k", [16, 144, 400, 1040])
def test_product_tiles_of_every_size(m, n, k):
    """K of one, two, four and nine stages of 128, the last one part full: shorter and longer than the rings."""
    from skinny_bf16_decode_amd.int8 import PreparedInt8
    from .test_gpu_int8 import TYPES, check_product, definition, make, say
    out = ("bf16", "f32", "f16")[(m + n + k) % 3]
    residual = (m + k // 16) % 2 == 0
    say("product", m, n, k, out, residual)
    xq, wq, xs, ws, res = make(m, n, k, m + n + k, out, residual)
    p, want = definition(xq, wq, xs, ws, res)
    plan = PreparedInt8(wq.cuda(), ws.cuda(), out_dtype=TYPES[out])
    y = torch.full((m + 1, n), -7.0, dtype=TYPES[out], device="cuda")
    plan.run(xq.cuda(), xs.cuda(), y, residual=None if res is None else res.cuda())
    torch.cuda.synchronize()
    check_product(y[:m], p, want, TYPES[out], (m, n, k, out))
    assert bool((y[m:] == -7).all())
    plan.close()


def test_product_tiles_on_views_and_two_streams():
    """Pitched rows at an odd column offset; one plan on two streams at once."""
    from skinny_bf16_decode_amd.int8 import PreparedInt8
    from .test_gpu_int8 import check_product, definition, make
    m, n, k = 5481, 514, 272
    xq, wq, xs, ws, _ = make(m, n, k, 5, "bf16", False)
    p, want = definition(xq, wq, xs, ws, None)
    plan = PreparedInt8(wq.cuda(), ws.cuda())
    x = torch.zeros(m, k + 48, dtype=torch.int8, device="cuda")
    x[:, 16:16 + k] = xq.cuda()
    xs = xs.cuda()
    outs = [torch.full((m, n + 9), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in outs]
    torch.cuda.synchronize()
    for _ in range(5):
        for y, s in zip(outs, streams):
            plan.run(x[:, 16:16 + k], xs, y[:, 5:5 + n], stream=s)
    torch.cuda.synchronize()
    for y in outs:
        check_product(y[:, 5:5 + n], p, want, torch.bfloat16, "stream")
        assert bool((y[:, :5] == 3).all()) and bool((y[:, 5 + n:] == 3).all())
    plan.close()


# heads, key_heads, dk, dv; lengths
ATTENTION = {
    "eight waves, one sequence cut": ((12, 12, 128, 128), [40, 0, 1, 700, 130, 64, 65, 90, 33, 128, 2, 77]),
    "eight waves, shared keys, narrow dk": ((12, 4, 96, 128), [100, 0, 129, 300, 1, 64, 65, 90, 33, 128, 2, 600]),
    "eight waves, two column tiles": ((4, 2, 128, 256), [50] * 10 + [0, 1, 500, 64, 65, 90, 33, 127]),
    "many sequences, wide columns": ((12, 12, 128, 128), [90] * 20 + [0, 1, 500, 64]),
    "parts of one chunk": ((1, 1, 128, 64), [500, 0, 130, 64, 65]),
    "one long sequence": ((2, 2, 128, 128), [4100]),
    "one long sequence, shared keys": ((4, 1, 64, 64), [4100, 3]),
    "parts of 192": ((12, 12, 64, 128), [700, 1, 0, 193, 192]),
}


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("name", ATTENTION)
def test_prompt_cut_every_way(name, kind):
    from skinny_bf16_decode_amd import linear_attention as la
    from .test_gpu_linear_attention import check, make, run, say
    shape, lengths = ATTENTION[name]
    for initial in (True, False):
        say("prompt", name, kind, initial)
        c = make(lengths, *shape, kind, 41, initial=initial)
        out, new = run(la, c)
        check(c, out, new, (name, kind, initial))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("where", ["q", "k", "v", "log_decay", "states"])
def test_eight_waves_with_values_that_are_not_finite(where, bad, kind):
    """They reach what the formula says, in a sequence that is cut and in a whole one."""
    from skinny_bf16_decode_amd import linear_attention as la
    from .test_gpu_linear_attention import definition, make, run, say
    lengths = [40, 0, 1, 700, 130, 64, 65, 90, 33, 128, 2, 77]
    c = make(lengths, 12, 12, 128, 128, kind, 43, rates=(0.05, 0.0005))
    starts = c["starts"].tolist()
    for seq in (3, 7):
        at = starts[seq] + lengths[seq] // 2
        if where == "log_decay":
            c[where][at, 1] = bad
        elif where == "states":
            c[where][int(c["slots"][seq]), 2, 5, 17] = bad
        else:
            c[where][at, 1, 9] = bad
    say("not finite", where, bad, kind)
    out, new = run(la, c)
    want, S = definition(c)
    got = new[c["slots"].long()]
    assert torch.equal(out.isnan(), want.isnan()) and torch.equal(out.isinf(), want.isinf())
    assert torch.equal(got.isnan(), S.isnan()) and torch.equal(got.isinf(), S.isinf())
    fine = S.isfinite()
    assert float((got.double() - S)[fine].norm()) <= 2.0 ** -20 * float(S[fine].norm())
    fine = want.isfinite()
    eps = torch.finfo(c["dtype"]).eps
    assert float((out.double() - want)[fine].norm()) <= (2.0 ** -15 + 0.6 * eps) * float(want[fine].norm())
