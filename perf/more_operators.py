"""What is measured of a decode block's operators in 4-bit weights, next to the
8-bit products and linear attention of operators.py.

  quantize   rows of activations to blocks of 32 values with one power of two each: 4-bit
             floating point (e2m1) or 8-bit (e4m3); with a gate g, of x silu(g)
  product    out[M, N] = sum over blocks 2^(x_scale + w_scale) (x . w) (+ residual), a 4-bit weight
  norm       n = x / sqrt(mean x^2 + eps) * weight, to a 16-bit type and to blocks or 8-bit integers
  join       h = beta residual + alpha gate norm(y), and the next block's norm of h

Each case names one operator and its sizes.  `run` computes the plain form, in
elementary torch operations, or (`own`) calls the framework's operators.  8-bit
results are returned in their own types (e4m3 values and e8m0 powers of two),
4-bit ones expanded to the values that they stand for.
"""
from __future__ import annotations

import functools
import importlib
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 32
EPS = 1e-6
# largest exponent and largest value of e2m1 and e4m3
TOP_EXPONENT = {4: 2, 8: 8}
LARGEST = {4: 6.0, 8: 448.0}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the activations of four decode tokens before a projection: a call of a few microseconds
        {"name": "quantize decode", "op": "quantize", "m": 4, "k": 7168, "type": "bf16", "bits": 8, "gate": False},
        # a prompt's activations (an uneven count) to 4 bits, and back to values
        {"name": "quantize prompt", "op": "quantize", "m": 6001, "k": 7168, "type": "bf16", "bits": 4, "gate": False},
        # the gated half of a feed-forward block on its way into the long-K projection
        {"name": "quantize gated", "op": "quantize", "m": 1000, "k": 18432, "type": "f16", "bits": 8, "gate": True},
        # one sequence decoding through the packed projection: weight bytes alone count
        {"name": "product one token", "op": "product", "m": 1, "n": 6288, "k": 7168, "bits": 8, "out": "bf16",
         "residual": False},
        # a ragged decode batch into the fp32 residual stream
        {"name": "product ragged batch", "op": "product", "m": 37, "n": 3584, "k": 7168, "bits": 8, "out": "f32",
         "residual": True},
        # a full decode batch through the long-K down projection
        {"name": "product long K", "op": "product", "m": 64, "n": 7168, "k": 18432, "bits": 4, "out": "bf16",
         "residual": False},
        # a prompt through the packed projection, tokens in 4 bits: bound by the matrix units
        {"name": "product prompt", "op": "product", "m": 4000, "n": 6288, "k": 7168, "bits": 4, "out": "bf16",
         "residual": False},
        # a shorter prompt with its tokens in 8 bits
        {"name": "product prompt 8 bit", "op": "product", "m": 1501, "n": 6288, "k": 7168, "bits": 8, "out": "f16",
         "residual": False},
        # one token's norm before a projection: a call of a few microseconds
        {"name": "norm decode", "op": "norm", "m": 1, "k": 7168, "type": "bf16", "weight": "bf16", "out": None,
         "q": "mx8"},
        # a prompt's norm before a projection, kept in 16 bits too
        {"name": "norm prompt", "op": "norm", "m": 4003, "k": 7168, "type": "bf16", "weight": "f32", "out": "bf16",
         "q": "mx8"},
        # a decode batch between two blocks of an fp32 residual stream
        {"name": "join decode", "op": "join", "m": 8, "k": 7168, "type": "bf16", "residual": "f32", "weight": "bf16",
         "gate": "channel", "sigmoid": False, "next": "mx8"},
        # a prompt between two blocks, with a gate for each token and channel
        {"name": "join prompt", "op": "join", "m": 4000, "k": 7168, "type": "bf16", "residual": "bf16",
         "weight": "bf16", "gate": "token", "sigmoid": True, "next": "bf16"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "norm", "join"])
    if op == "product":
        n, k = _log(rng, 16, 7168), BLOCK * _log(rng, 1, 576)
        bits = rng.choice([4, 8])
        # 8-bit tokens take the matrix units twice the time
        most = max(1, min(8192, int(4000 * 6288 * 7168 * 4 / bits / (n * k))))
        return {"op": op, "m": _log(rng, 1, most), "n": n, "k": k, "bits": bits,
                "out": rng.choice(["bf16", "f16", "f32"]), "residual": rng.random() < 0.4}
    if op == "quantize":
        k = BLOCK * _log(rng, 2, 576)
        most = max(1, min(8192, 20_000_000 // k))
        return {"op": op, "m": _log(rng, 1, most), "k": k, "type": rng.choice(["bf16", "f16", "f32"]),
                "bits": rng.choice([4, 8]), "gate": rng.random() < 0.4}
    # rows of whole blocks, or of any length where nothing is quantized
    whole = rng.random() < 0.7
    k = BLOCK * _log(rng, 2, 576) if whole else _log(rng, 64, 18432)
    most = max(1, min(8192, 20_000_000 // k))
    case = {"op": op, "m": _log(rng, 1, most), "k": k, "type": rng.choice(["bf16", "f16"]),
            "weight": rng.choice(["bf16", "f16", "f32"])}
    if op == "norm":
        q = rng.choice(["mx4", "mx8", "int8", None]) if whole else rng.choice(["int8", None])
        out = rng.choice(["bf16", "f16", "f32"]) if q is None or rng.random() < 0.5 else None
        return {**case, "out": out, "q": q}
    after = rng.choice(["mx4", "mx8", "bf16", "f16", None]) if whole else rng.choice(["bf16", "f16", None])
    return {**case, "residual": rng.choice(["bf16", "f16", "f32"]),
            "weight": rng.choice([None, "bf16", "f32"]), "gate": rng.choice([None, "channel", "token"]),
            "sigmoid": rng.random() < 0.4, "next": after}


def _result_bytes(kind, m, k):
    """Bytes of rows in a result's type."""
    if kind is None:
        return 0
    if kind == "int8":
        return m * k + 4 * m
    if kind in ("mx4", "mx8"):
        return m * k * int(kind[2]) // 8 + m * k // BLOCK
    return BYTES[kind] * m * k


def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    if op == "quantize":
        read = BYTES[case["type"]] * m * k * (2 if case["gate"] else 1)
        written = _result_bytes("mx%d" % case["bits"], m, k) + (2 * m * k if case["bits"] == 4 else 0)
        return {"bytes": read + written, "flops": m * k * (8 if case["gate"] else 3)}
    if op == "product":
        n, bits = case["n"], case["bits"]
        o = BYTES[case["out"]] * m * n * (2 if case["residual"] else 1)
        return {"bytes": n * k // 2 + n * k // BLOCK + _result_bytes("mx%d" % bits, m, k) + o, "flops": 2 * m * n * k}
    if op == "norm":
        done = _result_bytes(case["out"], m, k) + _result_bytes(case["q"], m, k)
        back = 2 * m * k if case["q"] == "mx4" else 0
        return {"bytes": BYTES[case["type"]] * m * k + BYTES[case["weight"]] * k + done + back, "flops": 4 * m * k}
    read = (BYTES[case["type"]] + BYTES[case["residual"]]) * m * k
    gate = {None: 0, "channel": k, "token": m * k}[case["gate"]] * BYTES[case["type"]]
    done = BYTES[case["residual"]] * m * k + _result_bytes(case["next"], m, k)
    back = 2 * m * k if case["next"] == "mx4" else 0
    return {"bytes": read + gate + done + back, "flops": 12 * m * k}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(gen, m, k):
    """Hidden states: a few channels far above the rest."""
    return _normal(gen, m, k) * torch.exp(0.5 * _normal(gen, k))


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, m, k = case["op"], case["m"], case["k"]
    if op == "product":
        n = case["n"]
        xq, xs = _plain_blocks(_activations(gen, m, k), case["bits"])
        wq, ws = _plain_blocks(_normal(gen, n, k) * 0.02 * torch.exp(0.2 * _normal(gen, n, 1)), 4)
        return {"xq": _held(xq, case["bits"]), "x_scale": xs, "wq": _held(wq, 4), "w_scale": ws,
                "residual": _normal(gen, m, n).to(TYPES[case["out"]]) if case["residual"] else None}
    kind = TYPES[case["type"]]
    s = {"x": _activations(gen, m, k).to(kind)}
    if op == "quantize":
        s["gate"] = (2 * _normal(gen, m, k)).to(kind) if case["gate"] else None
        return s
    # weights of norms lie about one
    if op == "norm":
        s["weight"] = (1 + 0.2 * _normal(gen, k)).to(TYPES[case["weight"]])
        return s
    s["residual"] = (3 * _activations(gen, m, k)).to(TYPES[case["residual"]])
    s["weight"] = (1 + 0.2 * _normal(gen, k)).to(TYPES[case["weight"]]) if case["weight"] else None
    rows = {None: None, "channel": (k,), "token": (m, k)}[case["gate"]]
    s["gate"] = _normal(gen, *rows).to(kind) if rows else None
    s["next_weight"] = (1 + 0.2 * _normal(gen, k)).to(kind) if case["next"] else None
    # the branch is scaled down as deep stacks have it
    s["alpha"], s["beta"] = 0.25, 1.0
    return s


def _places(m, k, kind):
    """Empty rows for a result of this type: out, q and scale."""
    def empty(*shape, dtype):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if kind == "int8":
        return None, empty(m, k, dtype=torch.int8), empty(m, dtype=torch.float32)
    if kind == "mx8":
        return None, empty(m, k, dtype=torch.float8_e4m3fn), empty(m, k // BLOCK, dtype=torch.float8_e8m0fnu)
    if kind == "mx4":
        return None, empty(m, k // 2, dtype=torch.uint8), empty(m, k // BLOCK, dtype=torch.float8_e8m0fnu)
    return (None if kind is None else empty(m, k, dtype=TYPES[kind])), None, None


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    op, m, k = case["op"], case["m"], case["k"]
    kinds = {"quantize": "mx%d" % case.get("bits", 8), "norm": case.get("q"), "join": case.get("next"), "product": None}
    s["next_out"], s["q"], s["scale"] = _places(m, k, kinds[op])
    if kinds[op] == "mx4":
        s["values"] = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
    if op == "norm":
        s["y"] = _places(m, k, case["out"])[0]
    elif op == "join":
        s["y"] = torch.empty_like(s["residual"])
    elif op == "product":
        s["y"] = torch.empty(m, case["n"], dtype=TYPES[case["out"]], device="cuda")
        if own:
            s["plan"] = _framework("mxfp4").PreparedMxfp4(s.pop("wq"), s.pop("w_scale"), out_dtype=TYPES[case["out"]])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

@functools.cache
def _framework(module):
    return importlib.import_module("skinny_bf16_decode_amd." + module)


def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _own_held(s):
    """The quantized rows as the values they stand for."""
    if s["q"] is not None and s["q"].dtype == torch.uint8:
        return _framework("mxfp4").expand_blocks(s["q"], s["scale"], s["values"])
    return s["q"], s["scale"]


def _own_quantize(s):
    _framework("mxfp4").quantize_blocks(s["x"], s["q"], s["scale"], gate=s["gate"])
    return _own_held(s)


def _own_product(s):
    return s["plan"].run(s["xq"], s["x_scale"], s["y"], residual=s["residual"])


def _own_norm(s):
    _framework("norms").norm_rows(s["x"], s["weight"], out=s["y"], q=s["q"], scale=s["scale"], eps=EPS)
    return s["y"], _own_held(s)


def _own_join(s):
    _framework("norms").join_rows(s["residual"], s["x"], s["y"], weight=s["weight"], gate=s["gate"],
                                  sigmoid=s["case"]["sigmoid"], alpha=s["alpha"], beta=s["beta"],
                                  next_weight=s["next_weight"], next_out=s["next_out"], q=s["q"], scale=s["scale"],
                                  eps=EPS)
    return s["y"], s["next_out"], _own_held(s)


_run_own = {"quantize": _own_quantize, "product": _own_product, "norm": _own_norm, "join": _own_join}


def _plain_blocks(v, bits):
    """Values in fp32 to the values of the block's type (fp32) and its powers of two (e8m0).  The power is that of
    the block's largest magnitude less the type's own largest exponent, from the bits of both; what is past the type's
    largest value is clipped.  Blocks with an infinity or NaN have the power NaN and values 0."""
    m, k = v.shape
    v = v.view(m, k // BLOCK, BLOCK)
    top = v.abs().amax(dim=-1, keepdim=True)
    fine = torch.isfinite(top)
    # subnormal magnitudes have powers below the smallest byte's
    power = ((top.view(torch.int32) >> 23) - 127 - TOP_EXPONENT[bits]).clamp(min=-127)
    inverse = ((127 - power) << 23).view(torch.float32)
    scaled = torch.where(fine, v * inverse, torch.zeros_like(v)).clamp(-LARGEST[bits], LARGEST[bits])
    if bits == 8:
        q = scaled.to(torch.float8_e4m3fn).float()
    else:
        a = scaled.abs()
        # borders between neighbouring values; ties go to the even one
        q = 0.5 * ((a > 0.25).float() + (a >= 0.75).float() + (a > 1.25).float() + (a >= 1.75).float())
        q = q + (a > 2.5).float() + (a >= 3.5).float() + 2 * (a > 5.0).float()
        q = torch.copysign(q, scaled)
    byte = torch.where(fine, power + 127, torch.full_like(power, 255)).to(torch.uint8)
    return q.view(m, k), byte.view(m, k // BLOCK).view(torch.float8_e8m0fnu)


def _held(q, bits):
    """The values of a block's type in its own bits; two 4-bit values a byte, the first in the low half."""
    if bits == 8:
        return q.to(torch.float8_e4m3fn)
    a = q.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code + 8 * torch.signbit(q).to(torch.uint8)
    return code[:, 0::2] + 16 * code[:, 1::2]


def _value_table(dtype):
    positive = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(positive + [-a for a in positive], device="cuda", dtype=dtype)


def _codes(q):
    return torch.stack((q & 15, q >> 4), dim=-1).view(q.shape[0], -1).long()


def _plain_values(q, scale):
    """What quantized rows stand for, in fp32."""
    values = _value_table(torch.float32)[_codes(q)] if q.dtype == torch.uint8 else q.float()
    m, k = values.shape
    return (values.view(m, k // BLOCK, BLOCK) * scale.float()[:, :, None]).view(m, k)


def _plain_held(s, v, kind):
    """Rows v (fp32) in the result's type, as the values they stand for."""
    if kind in ("mx4", "mx8"):
        bits = int(kind[2])
        q, scale = _plain_blocks(v, bits)
        if bits == 4:
            m, k = v.shape
            s["values"].copy_((q.view(m, k // BLOCK, BLOCK) * scale.float()[:, :, None]).view(m, k))
            return s["values"]
        s["q"].copy_(q)
        s["scale"].copy_(scale)
    elif kind == "int8":
        # scale = max |v| / 127, q = round to even (v * (127 / max |v|)); rows of zeros have scale 0
        top = v.abs().amax(dim=1)
        safe = torch.where(top > 0, top, torch.ones_like(top))
        s["q"].copy_(torch.round(v * (torch.full_like(top, 127.0) / safe)[:, None]))
        s["scale"].copy_(top / torch.full_like(top, 127.0))
    return s["q"], s["scale"]


def _plain_quantize(s):
    v = s["x"].float()
    if s["gate"] is not None:
        g = s["gate"].float()
        v = v * (g / (1 + torch.exp(-g)))
    return _plain_held(s, v, "mx%d" % s["case"]["bits"])


def _plain_product(s):
    y = _plain_values(s["xq"], s["x_scale"]) @ _plain_values(s["wq"], s["w_scale"]).t()
    if s["residual"] is not None:
        y = y + s["residual"].float()
    s["y"].copy_(y)
    return s["y"]


def _plain_rms(x, weight):
    """The mean of squares in 64 bits: the statistics are then the same in whatever order they are summed, and so are
    the quantized values, which would go the other way at a border."""
    r = torch.rsqrt(x.double().square().mean(dim=1, keepdim=True) + EPS).float()
    return x.float() * r * weight.float()


def _plain_norm(s):
    n = _plain_rms(s["x"], s["weight"])
    if s["y"] is not None:
        s["y"].copy_(n)
    return s["y"], _plain_held(s, n, s["case"]["q"])


def _plain_join(s):
    case = s["case"]
    z = s["x"].float() if s["weight"] is None else _plain_rms(s["x"], s["weight"])
    if s["gate"] is not None:
        g = s["gate"].float()
        z = z * (1 / (1 + torch.exp(-g)) if case["sigmoid"] else g)
    s["y"].copy_(s["residual"].float() * s["beta"] + z * s["alpha"])
    if s["next_weight"] is None:
        return s["y"], None, (None, None)
    n = _plain_rms(s["y"], s["next_weight"])
    if s["next_out"] is not None:
        s["next_out"].copy_(n)
    return s["y"], s["next_out"], _plain_held(s, n, case["next"])


_run_plain = {"quantize": _plain_quantize, "product": _plain_product, "norm": _plain_norm, "join": _plain_join}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _two_to(exponent):
    return ((exponent.long() + 1023) << 52).view(torch.float64)


def _exact_blocks(v, bits):
    """Values and powers of two, from logarithms and steps of the grid."""
    m, k = v.shape
    v = v.reshape(m, k // BLOCK, BLOCK)
    top = v.abs().amax(dim=-1, keepdim=True)
    # frexp: top = mantissa * 2^exponent, mantissa in [0.5, 1)
    exponent = torch.frexp(top)[1] - 1 - TOP_EXPONENT[bits]
    exponent = torch.where(top > 0, exponent, torch.full_like(exponent, -127)).clamp(min=-127)
    scale = _two_to(exponent)
    u = v / scale
    # a value of exponent e has steps of 2^(e - mantissa bits), down to the subnormals' step
    smallest, mantissa = (0, 1) if bits == 4 else (-6, 3)
    place = (torch.frexp(u)[1] - 1).clamp(min=smallest) - mantissa
    step = _two_to(place)
    u = (torch.round(u / step) * step).clamp(-LARGEST[bits], LARGEST[bits])
    return u, scale


def _exact_held(v, kind):
    if kind in ("mx4", "mx8"):
        u, scale = _exact_blocks(v, int(kind[2]))
        m, k = v.shape
        return (u * scale).reshape(m, k) if kind == "mx4" else (u.reshape(m, k), scale.reshape(m, k // BLOCK))
    return (None, v.abs().amax(dim=1) / 127) if kind == "int8" else (None, None)


def _exact_norm(x, weight):
    x = x.double()
    return x / torch.sqrt((x * x).sum(dim=1, keepdim=True) / x.shape[1] + EPS) * weight.double()


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "quantize":
        v = s["x"].double()
        if s["gate"] is not None:
            v = v * s["gate"].double() * torch.sigmoid(s["gate"].double())
        return _exact_held(v, "mx%d" % case["bits"])
    if op == "product":
        def values(q, scale):
            v = q.double() if q.dtype != torch.uint8 else _value_table(torch.float64)[_codes(q)]
            return v * scale.double().repeat_interleave(BLOCK, dim=1)

        y = torch.matmul(values(s["xq"], s["x_scale"]), values(s["wq"], s["w_scale"]).t().contiguous())
        return y if s["residual"] is None else y + s["residual"].double()
    if op == "norm":
        n = _exact_norm(s["x"], s["weight"])
        return n if case["out"] else None, _exact_held(n, case["q"])
    z = s["x"].double() if s["weight"] is None else _exact_norm(s["x"], s["weight"])
    if s["gate"] is not None:
        g = s["gate"].double()
        z = z * (torch.sigmoid(g) if case["sigmoid"] else g)
    h = s["residual"].double() * s["beta"] + z * s["alpha"]
    if s["next_weight"] is None:
        return h, None, (None, None)
    # the next norm reads the stream as it is held
    n = _exact_norm(h.to(TYPES[case["residual"]]), s["next_weight"])
    return h, n if case["next"] in TYPES else None, _exact_held(n, case["next"])
