"""The 4-bit products' and the norms' entry points on the CPU: every refusal
comes before any device call, and the Python calls name their tensors' GPU and stream."""
from __future__ import annotations

import ctypes

import pytest
import torch

import skinny_bf16_decode_amd as sk
from skinny_bf16_decode_amd import mxfp4, norms

from .test_operator_calls_cpu import CURRENT, EMPTY, OnGpu, Stream, gpu   # noqa: F401

OK, INVALID, SHAPE, ALIGN = 0, 1, 2, 3
P = 0x10000          # a 16-byte aligned address that is never read
E4M3 = torch.float8_e4m3fn


def lib():
    return sk.load_library()


@pytest.mark.parametrize("change,want", [
    (dict(type=3), INVALID), (dict(bits=6), INVALID), (dict(m=-1), INVALID), (dict(k=0), INVALID), (dict(k=48), SHAPE),
    (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(scale=None), INVALID), (dict(ldx=63), SHAPE),
    (dict(ldg=63, gate=P), SHAPE), (dict(ldq=31), SHAPE), (dict(ldq=63, bits=8), SHAPE), (dict(lds=1), SHAPE),
    (dict(x=P + 1), ALIGN), (dict(x=P + 2, type=1), ALIGN), (dict(gate=P + 1), ALIGN),
    (dict(m=0, x=None, q=None, scale=None), OK),
])
def test_quantize_blocks_refusals(change, want):
    a = dict(x=P, type=0, m=4, k=64, ldx=64, gate=None, ldg=64, bits=4, q=P, ldq=64, scale=P, lds=2)
    a.update(change)
    assert lib().skinny_quantize_blocks(*a.values(), None) == want, sk.last_error()


@pytest.mark.parametrize("change,want", [
    (dict(type=3), INVALID), (dict(bits=0), INVALID), (dict(m=-1), INVALID), (dict(k=0), INVALID), (dict(k=33), SHAPE),
    (dict(q=None), INVALID), (dict(scale=None), INVALID), (dict(out=None), INVALID), (dict(ldq=31), SHAPE),
    (dict(lds=1), SHAPE), (dict(ldo=63), SHAPE), (dict(out=P + 1), ALIGN), (dict(out=P + 2, type=1), ALIGN),
    (dict(m=0, q=None, scale=None, out=None), OK),
])
def test_expand_blocks_refusals(change, want):
    a = dict(q=P, bits=4, m=4, k=64, ldq=32, scale=P, lds=2, out=P, type=0, ldo=64)
    a.update(change)
    assert lib().skinny_expand_blocks(*a.values(), None) == want, sk.last_error()


@pytest.mark.parametrize("change,want", [
    (dict(w=None), INVALID), (dict(ws=None), INVALID), (dict(n=0), INVALID), (dict(k=0), INVALID), (dict(out=5), INVALID),
    (dict(k=80), SHAPE), (dict(k=(1 << 22) + 32, ldw=1 << 22, ldws=1 << 18), SHAPE), (dict(ldw=31), SHAPE),
    (dict(ldws=1), SHAPE), (dict(n=0x7FFFF001), SHAPE), (dict(n=1 << 26, k=1 << 22, ldw=1 << 22, ldws=1 << 18), SHAPE),
])
def test_mxfp4_prepare_refusals(change, want):
    a = dict(w=P, n=16, k=64, ldw=32, ws=P, ldws=2, out=0)
    a.update(change)
    plan = ctypes.c_void_p(123)
    st = lib().skinny_mxfp4_prepare(*a.values(), None, ctypes.byref(plan))
    assert st == want and plan.value is None and sk.last_error(), sk.last_error()


def test_mxfp4_null_plans():
    assert lib().skinny_mxfp4_prepare(P, 16, 64, 32, P, 2, 0, None, None) == INVALID
    assert lib().skinny_mxfp4_run(None, P, 4, 32, P, 2, None, 0, P, 16, 4, None) == INVALID
    lib().skinny_mxfp4_destroy(None)


class Plan(ctypes.Structure):
    """A skinny_mxfp4_plan of 16 rows and K = 64, for refusals alone."""
    _fields_ = [("n", ctypes.c_int), ("k", ctypes.c_int), ("units", ctypes.c_int), ("out", ctypes.c_int),
                ("device", ctypes.c_int), ("w", ctypes.c_void_p), ("w_scale", ctypes.c_void_p)]


@pytest.mark.parametrize("change,want", [
    (dict(bits=5), INVALID), (dict(m=-1), INVALID), (dict(m=0x7FFFF001), SHAPE), (dict(x=None), INVALID),
    (dict(xs=None), INVALID), (dict(out=None), INVALID), (dict(ldx=16), SHAPE), (dict(ldx=40), SHAPE),
    (dict(ldx=(1 << 22) + 16), SHAPE), (dict(bits=8, ldx=48), SHAPE), (dict(ldxs=1), SHAPE),
    (dict(ldxs=(1 << 22) + 1), SHAPE), (dict(ldo=15), SHAPE), (dict(res=P, ldr=15), SHAPE), (dict(x=P + 8), ALIGN),
    (dict(out=P + 1), ALIGN), (dict(res=P + 1), ALIGN), (dict(m=0, x=None, xs=None, out=None), OK),
])
def test_mxfp4_run_refusals(change, want):
    a = dict(x=P, bits=4, ldx=32, xs=P, ldxs=2, res=None, ldr=16, out=P, ldo=16, m=4)
    a.update(change)
    plan = Plan(16, 64, 1, 0, 0, None, None)
    assert lib().skinny_mxfp4_run(ctypes.byref(plan), *a.values(), None) == want, sk.last_error()


NORM_FIELDS = "x weight out q scale ldx ldo ldq lds eps x_type weight_type out_type q_kind m k".split()
JOIN_FIELDS = ("residual y weight gate out next_weight next_out q scale ldr ldy ldg ldo ldn ldq lds eps alpha beta "
               "residual_type y_type weight_type gate_type next_weight_type next_type q_kind sigmoid m k").split()


def norm_args(**change):
    a = dict(x=P, weight=P, out=P, q=P, scale=P, ldx=64, ldo=64, ldq=64, lds=2, eps=1e-6, x_type=0, weight_type=0,
             out_type=0, q_kind=norms.MX8, m=4, k=64)
    a.update(change)
    return norms._NORM.pack(*(a[f] or 0 for f in NORM_FIELDS))


def join_args(**change):
    a = dict(residual=P, y=P, weight=P, gate=P, out=P, next_weight=P, next_out=P, q=P, scale=P, ldr=64, ldy=64, ldg=64,
             ldo=64, ldn=64, ldq=64, lds=2, eps=1e-6, alpha=1.0, beta=1.0, residual_type=0, y_type=0, weight_type=0,
             gate_type=0, next_weight_type=0, next_type=0, q_kind=norms.MX8, sigmoid=0, m=4, k=64)
    a.update(change)
    return norms._JOIN.pack(*(a[f] or 0 for f in JOIN_FIELDS))


# what a norm's places are refused for, in norm_rows' and join_rows' names
PLACES = [
    (dict(weight_type=3), INVALID), (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(eps=1e-40), INVALID),
    (dict(out_type=3), INVALID), (dict(ldo=63), SHAPE), (dict(q_kind=4), INVALID), (dict(q_kind=-1), INVALID),
    (dict(out=None, q_kind=0), INVALID), (dict(q=None), INVALID), (dict(scale=None), INVALID), (dict(ldq=63), SHAPE),
    (dict(ldq=31, q_kind=norms.MX4), SHAPE), (dict(ldq=63, q_kind=norms.INT8), SHAPE), (dict(lds=1), SHAPE),
    (dict(k=48), SHAPE), (dict(out=P + 1), ALIGN), (dict(weight=P + 1), ALIGN),
    (dict(scale=P + 2, q_kind=norms.INT8), ALIGN),
]


@pytest.mark.parametrize("change,want", PLACES + [
    (dict(x_type=3), INVALID), (dict(m=-1), INVALID), (dict(k=0), INVALID), (dict(x=None), INVALID),
    (dict(weight=None), INVALID), (dict(ldx=63), SHAPE), (dict(x=P + 1), ALIGN), (dict(x=P + 2, x_type=1), ALIGN),
    (dict(m=0, x=None), OK),
])
def test_norm_refusals(change, want):
    assert lib().skinny_norm_rows(norm_args(**change), None) == want, sk.last_error()


IN_JOIN = {"weight": "next_weight", "weight_type": "next_weight_type", "out": "next_out", "out_type": "next_type",
           "ldo": "ldn"}


@pytest.mark.parametrize("change,want", [({IN_JOIN.get(f, f): v for f, v in c.items()}, w) for c, w in PLACES] + [
    (dict(residual_type=3), INVALID), (dict(y_type=-1), INVALID), (dict(gate_type=3), INVALID),
    (dict(weight_type=3), INVALID), (dict(m=-1), INVALID), (dict(k=0), INVALID), (dict(residual=None), INVALID),
    (dict(y=None), INVALID), (dict(out=None), INVALID), (dict(ldr=63), SHAPE), (dict(ldy=63), SHAPE),
    (dict(ldo=63), SHAPE), (dict(ldg=63), SHAPE), (dict(residual=P + 1), ALIGN), (dict(y=P + 1), ALIGN),
    (dict(out=P + 1), ALIGN), (dict(gate=P + 1), ALIGN), (dict(weight=P + 1), ALIGN),
    (dict(next_weight=None), INVALID), (dict(next_weight=None, next_out=None), INVALID),
    (dict(m=0, residual=None), OK),
])
def test_join_refusals(change, want):
    assert lib().skinny_join_rows(join_args(**change), None) == want, sk.last_error()


def test_null_args():
    assert lib().skinny_norm_rows(None, None) == INVALID and lib().skinny_join_rows(None, None) == INVALID


# ---------------------------------------------------------------------------
# the Python entries, with stand-ins for the GPU's tensors
# ---------------------------------------------------------------------------

@pytest.fixture
def log(gpu, monkeypatch):                              # noqa: F811
    names = ("skinny_quantize_blocks", "skinny_expand_blocks", "skinny_mxfp4_run", "skinny_norm_rows",
             "skinny_join_rows")

    def entry(name):
        def call(*args):
            gpu.log.append((name, gpu.device, args[-1]))
            return 0
        return call

    fake = type("Library", (), {n: staticmethod(entry(n)) for n in names})
    for module in (mxfp4, norms):
        monkeypatch.setattr(module, "load_library", lambda: fake)
    return gpu


def t(dtype, *shape, index=0):
    return OnGpu(dtype, shape, index)


BF, F32, U8, I8 = torch.bfloat16, torch.float32, torch.uint8, torch.int8


def calls(index):
    def g(dtype, *shape):
        return t(dtype, *shape, index=index)

    plan = mxfp4.PreparedMxfp4.__new__(mxfp4.PreparedMxfp4)
    plan.n, plan.k, plan.out_dtype, plan._index, plan._plan = 32, 64, BF, index, None

    def run(stream):
        plan._plan = 1
        try:
            plan.run(g(E4M3, 4, 64), g(U8, 4, 2), g(BF, 4, 32), stream=stream)
        finally:
            plan._plan = None

    return [("skinny_quantize_blocks", lambda s: mxfp4.quantize_blocks(g(BF, 4, 64), g(U8, 4, 32), g(U8, 4, 2), stream=s)),
            ("skinny_expand_blocks", lambda s: mxfp4.expand_blocks(g(U8, 4, 32), g(U8, 4, 2), g(BF, 4, 64), stream=s)),
            ("skinny_mxfp4_run", run),
            ("skinny_norm_rows", lambda s: norms.norm_rows(g(BF, 4, 64), g(BF, 64), out=g(BF, 4, 64), stream=s)),
            ("skinny_join_rows", lambda s: norms.join_rows(g(F32, 4, 64), g(BF, 4, 64), g(F32, 4, 64), stream=s))]


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("which", range(5))
def test_calls_run_on_their_tensors_gpu(log, which, index):
    name, call = calls(index)[which]
    for stream, handle in ((None, CURRENT), (Stream(0x55, f"cuda:{index}"), 0x55), (0x55, 0x55)):
        log.log.clear()
        call(stream)
        assert log.log == [(name, index, handle)] and log.device == 0


@pytest.mark.parametrize("which", range(5))
def test_a_stream_of_another_gpu_is_refused(log, which):
    with pytest.raises(ValueError, match="cuda:1, the stream is of cuda:0"):
        calls(1)[which][1](Stream(0x55, "cuda:0"))
    assert log.log == []


def plan_run(xq, xs, out, residual=None):
    plan = mxfp4.PreparedMxfp4.__new__(mxfp4.PreparedMxfp4)
    plan.n, plan.k, plan.out_dtype, plan._index, plan._plan = 32, 64, BF, 0, 1
    try:
        plan.run(xq, xs, out, residual=residual)
    finally:
        plan._plan = None


Q, N, J = mxfp4.quantize_blocks, norms.norm_rows, norms.join_rows
REFUSED = [
    (lambda: Q(torch.zeros(4, 64), t(U8, 4, 32), t(U8, 4, 2)), "on a GPU"),
    (lambda: Q(t(torch.float64, 4, 64), t(U8, 4, 32), t(U8, 4, 2)), "BF16, FP16 or fp32"),
    (lambda: Q(t(BF, 64), t(U8, 4, 32), t(U8, 4, 2)), "2-D"),
    (lambda: Q(t(BF, 4, 48), t(U8, 4, 24), t(U8, 4, 2)), "whole blocks"),
    (lambda: Q(t(BF, 4, 64), t(I8, 4, 32), t(U8, 4, 2)), "float8_e4m3fn"),
    (lambda: Q(t(BF, 4, 64), t(U8, 4, 64), t(U8, 4, 2)), "q must be"),
    (lambda: Q(t(BF, 4, 64), t(E4M3, 3, 64), t(U8, 4, 2)), "q must be"),
    (lambda: Q(t(BF, 4, 64), t(U8, 4, 32), t(I8, 4, 2)), "scale must be"),
    (lambda: Q(t(BF, 4, 64), t(U8, 4, 32), t(U8, 4, 1)), "scale must be"),
    (lambda: Q(t(BF, 4, 64), t(U8, 4, 32, index=1), t(U8, 4, 2)), "cuda:0"),
    (lambda: Q(t(BF, 4, 64), t(U8, 4, 32), t(U8, 4, 2), gate=t(BF, 4, 32)), "gate must have"),
    (lambda: Q(t(BF, 4, 64), t(U8, 4, 32), t(U8, 4, 2), gate=t(F32, 4, 64)), "gate must be"),
    (lambda: mxfp4.expand_blocks(t(U8, 4, 32), t(U8, 4, 2), t(BF, 3, 64)), "at least 4 rows"),
    (lambda: mxfp4.expand_blocks(t(U8, 4, 32), t(U8, 4, 2), t(BF, 4, 128)), "q must be"),
    (lambda: mxfp4.expand_blocks(t(U8, 4, 20), t(U8, 4, 2), t(BF, 4, 40)), "whole blocks"),
    (lambda: mxfp4.PreparedMxfp4(torch.zeros(16, 32, dtype=U8), torch.zeros(16, 2, dtype=U8)), "on a GPU"),
    (lambda: mxfp4.PreparedMxfp4(t(E4M3, 16, 64), t(U8, 16, 2)), "uint8 or float4"),
    (lambda: mxfp4.PreparedMxfp4(t(U8, 16, 24), t(U8, 16, 2)), "whole blocks"),
    (lambda: mxfp4.PreparedMxfp4(t(U8, 16, 32), t(U8, 15, 2)), "w_scale must be"),
    (lambda: mxfp4.PreparedMxfp4(t(U8, 16, 32), t(U8, 16, 2), out_dtype=torch.float64), "output dtype"),
    (lambda: plan_run(t(U8, 4, 64), t(U8, 4, 2), t(BF, 4, 32)), "xq must be"),
    (lambda: plan_run(t(BF, 4, 64), t(U8, 4, 2), t(BF, 4, 32)), "float8_e4m3fn"),
    (lambda: plan_run(t(E4M3, 4, 64), t(F32, 4, 2), t(BF, 4, 32)), "x_scale must be"),
    (lambda: plan_run(t(E4M3, 4, 64), t(U8, 4, 2), t(F32, 4, 32)), "out must be"),
    (lambda: plan_run(t(E4M3, 4, 64), t(U8, 4, 2), t(BF, 4, 32), t(BF, 4, 31)), "residual must be"),
    (lambda: N(t(BF, 4, 64), t(BF, 64)), "needs out"),
    (lambda: N(t(BF, 4, 64), t(BF, 63), out=t(BF, 4, 64)), "weight must be"),
    (lambda: N(t(BF, 4, 64), t(I8, 64), out=t(BF, 4, 64)), "weight must be"),
    (lambda: N(t(BF, 4, 64), t(BF, 64, index=1), out=t(BF, 4, 64)), "weight must be"),
    (lambda: N(t(BF, 4, 64), t(BF, 64), out=t(I8, 4, 64)), "out must be"),
    (lambda: N(t(BF, 4, 64), t(BF, 64), out=t(BF, 3, 64)), "out must be"),
    (lambda: N(t(BF, 4, 64), t(BF, 64), q=t(I8, 4, 64)), "q without scale"),
    (lambda: N(t(BF, 4, 64), t(BF, 64), out=t(BF, 4, 64), scale=t(F32, 4)), "scale without q"),
    (lambda: N(t(BF, 4, 64), t(BF, 64), q=t(I8, 4, 64), scale=t(U8, 4)), "scale must be"),
    (lambda: N(t(BF, 4, 64), t(BF, 64), q=t(BF, 4, 64), scale=t(U8, 4, 2)), "q must be"),
    (lambda: N(t(BF, 4, 48), t(BF, 48), q=t(U8, 4, 24), scale=t(U8, 4, 2)), "whole blocks"),
    (lambda: J(t(F32, 4, 64), t(BF, 4, 64), t(BF, 4, 64)), "one type"),
    (lambda: J(t(F32, 3, 64), t(BF, 4, 64), t(F32, 4, 64)), "residual must be"),
    (lambda: J(t(F32, 4, 64), t(BF, 4, 64), t(F32, 4, 64), gate=t(BF, 4, 32)), "gate must be"),
    (lambda: J(t(F32, 4, 64), t(BF, 4, 64), t(F32, 4, 64), gate=t(BF, 32)), "gate must be"),
    (lambda: J(t(F32, 4, 64), t(BF, 4, 64), t(F32, 4, 64), next_out=t(BF, 4, 64)), "need next_weight"),
    (lambda: J(t(F32, 4, 64), t(BF, 4, 64), t(F32, 4, 64), next_weight=t(BF, 64)), "needs next_out"),
]


@pytest.mark.parametrize("which", range(len(REFUSED)))
def test_python_refusals(log, which):
    call, text = REFUSED[which]
    with pytest.raises(ValueError, match=text):
        call()
    assert log.log == []


def test_a_closed_plan_is_refused():
    plan = mxfp4.PreparedMxfp4.__new__(mxfp4.PreparedMxfp4)
    plan._plan = ctypes.c_void_p()
    with pytest.raises(ValueError, match="closed"):
        plan.run(None, None, None)
