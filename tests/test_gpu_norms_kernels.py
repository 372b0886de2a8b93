"""Norms and joins in every kernel that they can take, also where rows end
between the turns of a workgroup.  test_norm_shape_cpu.py asks the library's own
choice whether these calls reach them all.

Definitions and tolerances of test_gpu_norms.py; quantized rows have to be, bit by
bit, what the separate calls make of the fp32 norm.
"""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# rows, length, at an unaligned place, quantized kind
NORMS = [(5, 320, 0, "mx8"), (3, 12288, 0, "mx4"), (2, 30816, 0, "int8"), (515, 96, 0, "mx8"), (514, 9216, 0, None),
         (513, 32768, 0, "mx4"), (3, 65536, 0, "mx8"),                     # whole vectors
         (7, 320, 1, "mx8"), (600, 96, 1, "mx4"), (3, 8224, 1, "mx8"), (2, 20000, 1, "mx4"),   # blocks, one element at a time
         (5, 333, 0, "int8"), (600, 77, 1, None), (3, 8201, 0, "int8"), (2, 12289, 1, None), (3, 16384, 1, "int8"),
         (520, 8193, 1, None), (2, 24577, 0, "int8"), (260, 20001, 1, None)]
# rows in turns: four at a time, with one to three in the last; one at a time, of one to three octets a thread
STREAMED = [(4003, 7168), (3075, 7168), (12285, 2048), (4097, 4096), (3999, 7168), (4090, 8192), (2500, 7168), (300, 1544),
            (261, 12288), (259, 24576), (1027, 16640)]
# more of each kind of join: rows, length, unaligned, kind, a gate for each token
JOINS = [(5, 320, 0, "mx8", True), (3, 12288, 0, "mx4", False), (2, 30816, 0, "int8", True), (514, 9216, 0, None, True),
         (3, 65536, 0, "mx8", False), (1300, 1056, 0, "mx4", True),
         (7, 320, 1, "mx8", False), (600, 96, 1, "mx4", True), (3, 8224, 1, "mx8", True), (2, 20000, 1, "mx4", False),
         (5, 333, 0, "int8", True), (3, 8201, 0, "int8", False), (2, 12289, 1, None, True), (520, 8193, 1, None, False),
         (2, 24577, 0, "int8", True), (1100, 1001, 0, "int8", False)]
JOINED = [(1025, 520), (1100, 7168), (2047, 8192), (3001, 2048)]


@pytest.fixture(scope="module", autouse=True)
def op():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from skinny_bf16_decode_amd import norms
    return norms


def at(t, off):
    """The same values at a place `off` elements on, with a pitch, between values that are NaN (77 in integers)."""
    if not off:
        return t
    bad = math.nan if t.dtype.is_floating_point and t.element_size() > 1 else 77
    byte = t.view(torch.uint8) if t.element_size() == 1 else t
    wide = torch.full((t.shape[0], t.shape[1] + off + 2), bad, dtype=byte.dtype, device="cuda")
    view = wide[:, off:off + t.shape[1]]
    view.copy_(byte)
    return view.view(t.dtype) if t.element_size() == 1 else view


def places(q, m, k, off):
    from .test_gpu_norms import quantized_places
    if q is None:
        return None, None
    a, b = quantized_places(q, m + 1, k)
    return at(a, off), b


def same(got, want, m):
    """The first m rows, and that the one behind them is as it was."""
    from .test_gpu_norms import same_rows
    same_rows((got[0][:m].contiguous(), got[1][:m]), (want[0][:m].contiguous(), want[1][:m]))
    q, s = got
    assert bool((q[m].view(torch.uint8) == (77 if q.dtype == torch.int8 else 0x77)).all())
    assert bool((s[m:].float() == (7 if s.dtype == torch.float32 else 0x77)).all())


def separately(q, n):
    from .test_gpu_norms import quantized
    return quantized(q, n)


def check_norm(op, m, k, off, q, kind):
    from .test_gpu_norms import H, close, exact_norm, rows, weights
    print("norm", m, k, off, q, kind, flush=True)
    x, w = rows(m, k, kind, m + k), weights(k, list(TYPES)[(m + k) % 3], k)
    want = exact_norm(x, w)
    n = torch.full((m + 1, k), 3.0, device="cuda")
    out = torch.full((m + 1, k), 3.0, dtype=TYPES[kind], device="cuda")
    x = at(x, off)
    qa, sa = places(q, m, k, off)
    op.norm_rows(x, w, out=n, q=qa, scale=sa)
    nb = at(out, off)
    op.norm_rows(x, w, out=nb)
    torch.cuda.synchronize()
    close(n[:m], want, 3 * H * want.abs(), torch.float32)
    close(nb[:m], want, 3 * H * want.abs(), TYPES[kind])
    assert bool((n[m] == 3).all()) and bool((nb[m] == 3).all())
    if q is not None:
        same((qa, sa), separately(q, n[:m]), m)
        qb, sb = places(q, m, k, off)
        op.norm_rows(x, w, q=qb, scale=sb)
        same((qb, sb), (qa, sa), m)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,k,off,q", NORMS)
def test_norm_kernels(op, m, k, off, q, kind):
    check_norm(op, m, k, off, q, kind)


@pytest.mark.parametrize("q", ["int8", "mx4", "mx8"])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,k", STREAMED)
def test_norm_rows_in_turns(op, m, k, kind, q):
    check_norm(op, m, k, 0, q if k % 32 == 0 else "int8", kind)


def check_join(op, m, k, off, q, token, yk, rk):
    from .test_gpu_norms import H, close, exact_join, exact_norm, rows, weights
    print("join", m, k, off, q, token, yk, rk, flush=True)
    kinds = list(TYPES)
    res, y = rows(m, k, rk, 1, 0.5), rows(m, k, yk, 2, 0.5)
    w, nw = weights(k, kinds[m % 3], 1), weights(k, kinds[k % 3], 6)
    g = rows(m, k, kinds[(m + k) % 3], 3, 0.1) if token else weights(k, "f16", 4)
    sigmoid = (m + k) % 2 == 1
    h, tol = exact_join(res, y, w, g, sigmoid, 0.375, 1.25)
    res, y = at(res, off), at(y, off)
    if token:
        g = at(g, off)
    args = dict(weight=w, gate=g, sigmoid=sigmoid, alpha=0.375, beta=1.25, next_weight=nw)
    out, n = at(torch.full((m + 1, k), 3.0, dtype=TYPES[rk], device="cuda"), off), torch.full((m + 1, k), 4.0, device="cuda")
    qa, sa = places(q, m, k, off)
    op.join_rows(res, y, out, next_out=n, q=qa, scale=sa, **args)
    torch.cuda.synchronize()
    close(out[:m], h, tol + H * h.abs(), TYPES[rk])
    want = exact_norm(out[:m], nw)
    close(n[:m], want, 3 * H * want.abs(), torch.float32)
    assert bool((out[m] == 3).all()) and bool((n[m] == 4).all())
    # the same by itself, in place, and without the norm's values
    qb, sb = places(q, m, k, off)
    nb = at(torch.full((m + 1, k), 4.0, dtype=TYPES[rk], device="cuda"), off) if q is None else None
    op.join_rows(res, y, res, next_out=nb, q=qb, scale=sb, **args)
    assert torch.equal(res, out[:m])
    if q is None:
        close(nb[:m], want, 3 * H * want.abs(), TYPES[rk])
    else:
        same((qa, sa), separately(q, n[:m]), m)
        same((qb, sb), (qa, sa), m)


@pytest.mark.parametrize("rk", TYPES)
@pytest.mark.parametrize("yk", TYPES)
@pytest.mark.parametrize("m,k,off,q,token", JOINS)
def test_join_kernels(op, m, k, off, q, token, yk, rk):
    check_join(op, m, k, off, q, token, yk, rk)


@pytest.mark.parametrize("q", ["int8", "mx4", "mx8"])
@pytest.mark.parametrize("rk", TYPES)
@pytest.mark.parametrize("yk", TYPES)
@pytest.mark.parametrize("m,k", JOINED)
def test_join_rows_in_turns(op, m, k, yk, rk, q):
    check_join(op, m, k, 0, q if k % 32 == 0 else "int8", False, yk, rk)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_norm_turns_with_rows_that_go_wrong(op, kind):
    """NaN, infinity and zeros among four rows that share their steps, and in the ones of the last turn."""
    from .test_gpu_norms import H, close, exact_norm, quantized_places, rows, same_rows, weights
    m, k = 4003, 7168
    t = TYPES[kind]
    x = rows(m, k, kind, 1, 0.5)
    x[1], x[1026, 5], x[4000, 9], x[4001], x[4002, 7167] = 0, math.nan, math.inf, torch.finfo(t).max, -math.inf
    w = weights(k, "f32", 1)
    want = exact_norm(x, w)
    for q in ("int8", "mx4", "mx8"):
        n = torch.empty(m, k, device="cuda")
        got = quantized_places(q, m, k)
        op.norm_rows(x, w, out=n, q=got[0], scale=got[1])
        assert torch.equal(n.isnan(), want.isnan())
        fine = torch.isfinite(want)
        close(n[fine], want[fine], 3 * H * want[fine].abs(), torch.float32)
        same_rows(got, separately(q, n))
