"""What is measured of the decode layer's other operators, next to the projection
that bench.py measures.

  quantize   rows of activations (BF16, FP16 or fp32) to 8-bit integers with one scale a row
  product    out[M, N] = (xq[M, K] . wq[N, K]^T) * x_scale[m] * w_scale[n] (+ residual), 8-bit integers in
  prompt     linear attention with a decay for each head and token, over packed sequences:
             S_t = exp(g_t) S_{t-1} + k_t v_t^T,  o_t = scale q_t^T S_t
  step       the same recurrence for one new token of each sequence, on a pool of states

Each case names one operator and its sizes.  `run` computes the plain form, in
elementary torch operations, or (`own`) calls the framework's operators.
"""
from __future__ import annotations

import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}

# q, k, v and the gate of 12 heads of 128, then 144 more columns: the packed
# projection output [tokens, 6288], whose column ranges the operators read in place
PACKED_HEADS, PACKED_DIM, PACKED_TAIL = 12, 128, 144


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the activations of four decode tokens before a projection: a call of a few microseconds
        {"name": "quantize decode", "op": "quantize", "m": 4, "k": 7168, "type": "bf16"},
        # a prompt's activations, an uneven count of them
        {"name": "quantize prompt", "op": "quantize", "m": 6001, "k": 7168, "type": "bf16"},
        # one sequence decoding through the packed QKVG projection: weight bytes alone count
        {"name": "product one token", "op": "product", "m": 1, "n": 6288, "k": 7168, "out": "bf16", "residual": False},
        # a ragged decode batch into the fp32 residual stream
        {"name": "product ragged batch", "op": "product", "m": 37, "n": 3584, "k": 7168, "out": "f32", "residual": True},
        # a full decode batch through the long-K down projection
        {"name": "product long K", "op": "product", "m": 64, "n": 7168, "k": 18432, "out": "bf16", "residual": False},
        # a prompt through the packed projection: bound by the matrix units
        {"name": "product prompt", "op": "product", "m": 4000, "n": 6288, "k": 7168, "out": "bf16", "residual": False},
        # a short question: little work, few workgroups
        {"name": "prompt short", "op": "prompt", "tokens": 77, "sequences": 1, "uneven": False, "heads": 12,
         "key_heads": 12, "dk": 128, "dv": 128, "type": "bf16", "packed": True, "initial": False},
        # one long document: the sequence has to be split over the chip
        {"name": "prompt long", "op": "prompt", "tokens": 32768, "sequences": 1, "uneven": False, "heads": 12,
         "key_heads": 12, "dk": 128, "dv": 128, "type": "bf16", "packed": True, "initial": False},
        # a server's prompts of all lengths (empty and one-token ones among them) going on from kept states,
        # with key heads shared by three value heads
        {"name": "prompt ragged", "op": "prompt", "tokens": 12001, "sequences": 24, "uneven": True, "heads": 12,
         "key_heads": 4, "dk": 64, "dv": 128, "type": "f16", "packed": False, "initial": True},
        # a batch of prompts of one length
        {"name": "prompt batch", "op": "prompt", "tokens": 32768, "sequences": 16, "uneven": False, "heads": 12,
         "key_heads": 12, "dk": 128, "dv": 128, "type": "bf16", "packed": True, "initial": True},
        # one sequence decoding
        {"name": "step one", "op": "step", "sequences": 1, "heads": 12, "key_heads": 12, "dk": 128, "dv": 128,
         "type": "bf16", "packed": True},
        # a full decode batch: the states' bytes count
        {"name": "step full batch", "op": "step", "sequences": 64, "heads": 12, "key_heads": 12, "dk": 128, "dv": 128,
         "type": "bf16", "packed": True},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "prompt", "prompt", "step"])
    if op == "quantize":
        k = 16 * _log(rng, 4, 1152)
        m = _log(rng, 1, max(1, min(8192, 6001 * 7168 // k)))
        return {"op": op, "m": m, "k": k, "type": rng.choice(["bf16", "f16", "f32"]) if m * k < 20e6 else "bf16"}
    if op == "product":
        n, k = _log(rng, 16, 7168), 16 * _log(rng, 4, 1152)
        most = max(1, min(8192, int(4000 * 6288 * 7168 / (n * k))))
        return {"op": op, "m": _log(rng, 1, most), "n": n, "k": k, "out": rng.choice(["bf16", "f16", "f32"]),
                "residual": rng.random() < 0.4}
    packed = rng.random() < 0.4
    key_heads = PACKED_HEADS if packed else rng.choice([1, 2, 3, 4, 8])
    heads = PACKED_HEADS if packed else key_heads * rng.choice([1, 1, 2, 3])
    dk = PACKED_DIM if packed else rng.choice([32, 64, 96, 128, 128, 200, 256])
    dv = PACKED_DIM if packed else rng.choice([40, 64, 128, 128, 192, 256])
    kind = rng.choice(["bf16", "f16"])
    if op == "step":
        most = max(1, min(256, 64 * 12 * 128 * 128 // (heads * dk * dv)))
        return {"op": op, "sequences": _log(rng, 1, most), "heads": heads, "key_heads": key_heads, "dk": dk, "dv": dv,
                "type": kind, "packed": packed}
    most = 32768 * 12 * 128 * 128 // (heads * dk * dv)
    tokens = _log(rng, 1, min(32768, most))
    sequences = _log(rng, 1, max(1, min(64, tokens // 40 + 1)))
    return {"op": op, "tokens": tokens, "sequences": sequences, "uneven": rng.random() < 0.7, "heads": heads,
            "key_heads": key_heads, "dk": dk, "dv": dv, "type": kind, "packed": packed, "initial": rng.random() < 0.5}


def work(case):
    op = case["op"]
    if op == "quantize":
        m, k = case["m"], case["k"]
        return {"bytes": m * k * (BYTES[case["type"]] + 1) + 4 * m, "flops": 3 * m * k}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        o = BYTES[case["out"]] * m * n * (2 if case["residual"] else 1)
        return {"bytes": n * k + m * k + 4 * (m + n) + o, "flops": 2 * m * n * k}
    heads, kheads, dk, dv, b = case["heads"], case["key_heads"], case["dk"], case["dv"], case["sequences"]
    tokens = b if op == "step" else case["tokens"]
    per_token = BYTES[case["type"]] * (2 * kheads * dk + 2 * heads * dv) + 4 * heads
    states = (2 if op == "step" or case["initial"] else 1) * b * heads * dk * dv * 4
    return {"bytes": tokens * per_token + states, "flops": 4 * tokens * heads * dk * dv}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _lengths(case, seed):
    """The sequences' lengths: equal ones (the first takes what is over), or cut at random places, where the
    second sequence is empty and the third has one token if there are that many."""
    total, b = case["tokens"], case["sequences"]
    if not case["uneven"]:
        return [total - (b - 1) * (total // b)] + [total // b] * (b - 1)
    rng = random.Random(seed)
    fixed = [0, 1] if b >= 4 and total > 1 else []
    rest = b - len(fixed)
    left = total - sum(fixed)
    cuts = sorted(rng.randint(0, left) for _ in range(rest - 1))
    lengths = [hi - lo for lo, hi in zip([0] + cuts, cuts + [left])]
    return lengths[:1] + fixed + lengths[1:]


def _attention_inputs(case, seed, gen, tokens):
    heads, kheads, dk, dv = case["heads"], case["key_heads"], case["dk"], case["dv"]
    kind = TYPES[case["type"]]
    b = case["sequences"]
    # activations after a projection; keys and queries of unit length
    if case["packed"]:
        width = heads * dk
        rows = _normal(gen, tokens, 4 * width + PACKED_TAIL)
        for part in (0, 1):
            cols = rows[:, part * width:(part + 1) * width].view(tokens, heads, dk)
            cols /= cols.norm(dim=-1, keepdim=True)
        rows = rows.to(kind)
        q, k, v = (rows[:, i * width:(i + 1) * width].view(tokens, heads, dk) for i in range(3))
    else:
        q, k = (torch.nn.functional.normalize(_normal(gen, tokens, kheads, dk), dim=-1).to(kind) for _ in range(2))
        v = _normal(gen, tokens, heads, dv).to(kind)
    # log decays: each head forgets at a rate of its own, from a few tokens to a few thousand, scaled by the token
    rate = torch.exp(torch.linspace(math.log(0.3), math.log(0.0005), heads, device="cuda"))
    log_decay = -rate * torch.nn.functional.softplus(_normal(gen, tokens, heads) + 0.5)
    # the pool has free states too, and the sequences hold theirs in no order
    pool = b + 1 + b // 4
    slots = torch.randperm(pool, generator=gen, device="cuda")[:b].to(torch.int32)
    states = None
    if case["op"] == "step" or case["initial"]:
        states = 0.3 * _normal(gen, pool, heads, dk, dv)
    return {"q": q, "k": k, "v": v, "log_decay": log_decay.contiguous(), "slots": slots, "states": states,
            "pool": pool, "scale": dk ** -0.5}


def _inputs(case, seed):
    gen = _generator(seed)
    op = case["op"]
    if op == "quantize":
        # activations with a few channels far above the rest, as hidden states have them
        x = _normal(gen, case["m"], case["k"])
        x *= torch.exp(0.5 * _normal(gen, case["k"]))
        return {"x": x.to(TYPES[case["type"]])}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        s = {"xq": torch.clamp(torch.round(32 * _normal(gen, m, k)), -127, 127).to(torch.int8),
             "wq": torch.clamp(torch.round(32 * _normal(gen, n, k)), -127, 127).to(torch.int8),
             "x_scale": torch.exp(0.3 * _normal(gen, m)) / 32, "w_scale": 0.02 * torch.exp(0.2 * _normal(gen, n)) / 32,
             "residual": _normal(gen, m, n).to(TYPES[case["out"]]) if case["residual"] else None}
        return s
    tokens = case["sequences"] if op == "step" else case["tokens"]
    s = _attention_inputs(case, seed, gen, tokens)
    if op == "prompt":
        s["lengths"] = _lengths(case, seed)
        ends = [0]
        for length in s["lengths"]:
            ends.append(ends[-1] + length)
        s["starts"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    op = case["op"]
    if op == "quantize":
        s["q"] = torch.empty(case["m"], case["k"], dtype=torch.int8, device="cuda")
        s["scale"] = torch.empty(case["m"], dtype=torch.float32, device="cuda")
    elif op == "product":
        s["y"] = torch.empty(case["m"], case["n"], dtype=TYPES[case["out"]], device="cuda")
        if own:
            from skinny_bf16_decode_amd.int8 import PreparedInt8
            s["plan"] = PreparedInt8(s.pop("wq"), s["w_scale"], out_dtype=TYPES[case["out"]])
    else:
        tokens = s["v"].shape[0]
        s["out"] = torch.empty(tokens, case["heads"], case["dv"], dtype=TYPES[case["type"]], device="cuda")
        # the new states go to a second pool, as where the old ones are kept until a drafted token is accepted
        s["new_states"] = torch.zeros(s["pool"], case["heads"], case["dk"], case["dv"], device="cuda")
        if own and op == "prompt":
            from skinny_bf16_decode_amd import linear_attention
            size = linear_attention.workspace_bytes(tokens, case["sequences"], case["heads"], case["dk"], case["dv"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _own_quantize(s):
    from skinny_bf16_decode_amd.int8 import quantize_rows
    return quantize_rows(s["x"], s["q"], s["scale"])


def _own_product(s):
    return s["plan"].run(s["xq"], s["x_scale"], s["y"], residual=s["residual"])


def _own_prompt(s):
    from skinny_bf16_decode_amd import linear_attention
    linear_attention.prompt(s["q"], s["k"], s["v"], s["log_decay"], s["out"], s["starts"], state_in=s["states"],
                            state_out=s["new_states"], slots=s["slots"], scale=s["scale"], workspace=s["workspace"])
    return s["out"], s["new_states"]


def _own_step(s):
    from skinny_bf16_decode_amd import linear_attention
    linear_attention.step(s["q"], s["k"], s["v"], s["log_decay"], s["out"], state_in=s["states"],
                          state_out=s["new_states"], slots=s["slots"], scale=s["scale"])
    return s["out"], s["new_states"]


_run_own = {"quantize": _own_quantize, "product": _own_product, "prompt": _own_prompt, "step": _own_step}


def _plain_quantize(s):
    """scale = max |x| / 127, q = round to even (x * (127 / max |x|)); a row of zeros has scale 0, a row with an
    infinity or NaN scale NaN, both q = 0.  Rows below 2^-60 are lifted by 2^64 first, so that 127 / max is finite."""
    x = s["x"].float()
    top = x.abs().amax(dim=1)
    fine = torch.isfinite(top) & (top > 0)
    safe = torch.where(fine, top, torch.ones_like(top))
    lift = torch.where(safe < 2.0 ** -60, torch.full_like(top, 2.0 ** 64), torch.ones_like(top))
    inverse = torch.full_like(top, 127.0) / (safe * lift)
    q = torch.round((x * lift[:, None]) * inverse[:, None])
    q = torch.where(fine[:, None], q, torch.zeros_like(q)).to(torch.int8)
    scale = torch.where(torch.isfinite(top), top / torch.full_like(top, 127.0), torch.full_like(top, math.nan))
    s["q"].copy_(q)
    s["scale"].copy_(scale)
    return s["q"], s["scale"]


def _plain_product(s):
    y = s["xq"].float() @ s["wq"].float().t()
    y = y * s["x_scale"][:, None] * s["w_scale"][None, :]
    if s["residual"] is not None:
        y = y + s["residual"].float()
    s["y"].copy_(y)
    return s["y"]


def _shared(x, heads):
    """Key heads, each repeated for the value heads that share it."""
    return x.repeat_interleave(heads // x.shape[1], dim=1)


CHUNK = 64


def _plain_prompt(s):
    """Chunks of 64 tokens: inside a chunk ((q k^T) . decays) v, across chunks the states, summed over the chunks
    before with the decays between them.  Decays are differences of sums of logarithms, in 64 bits."""
    case, starts = s["case"], s["starts"].long()
    heads, b, tokens = case["heads"], case["sequences"], s["v"].shape[0]
    count = tokens // CHUNK + b                      # places for chunks; some stay empty
    base = starts[:-1] // CHUNK + torch.arange(b, device="cuda")
    place = torch.arange(count, device="cuda")
    seq = (torch.searchsorted(base, place, right=True) - 1).clamp(min=0)
    first = starts[seq] + (place - base[seq]) * CHUNK
    t = first[:, None] + torch.arange(CHUNK, device="cuda")
    valid = (t >= starts[seq][:, None]) & (t < starts[seq + 1][:, None])
    at = torch.where(valid, t, torch.zeros_like(t))

    def chunks(x):                                   # [tokens, heads, d] -> [chunk, heads, CHUNK, d]
        x = torch.where(valid[:, :, None, None], x.float()[at], torch.zeros((), device="cuda"))
        return x.transpose(1, 2).contiguous()

    q, k, v = (chunks(x) for x in (_shared(s["q"], heads), _shared(s["k"], heads), s["v"]))
    g = torch.where(valid[:, :, None], s["log_decay"].double().clamp(min=-200.0)[at], torch.zeros((), device="cuda"))
    g = g.transpose(1, 2).cumsum(dim=2)              # [chunk, heads, CHUNK]
    total = g[:, :, -1]
    seen = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda").tril()
    between = (g[:, :, :, None] - g[:, :, None, :]).masked_fill(~seen, -math.inf).float().exp()
    out = torch.matmul(torch.matmul(q, k.transpose(2, 3).contiguous()) * between, v)
    del between
    weight = (total[:, :, None] - g).float().exp()
    local = torch.matmul((k * weight[..., None]).transpose(2, 3).contiguous(), v)   # [chunk, heads, dk, dv]
    dk, dv = local.shape[2:]
    local = local.transpose(0, 1).reshape(heads, count, dk * dv)
    upto = total.cumsum(dim=0).t()                   # [heads, count], through this place
    before = upto - total.t()
    same = (seq[:, None] == seq[None, :]) & (place[:, None] > place[None, :])
    decay = (before[:, :, None] - upto[:, None, :]).masked_fill(~same, -math.inf).float().exp()
    state = torch.matmul(decay, local)               # at each chunk's start
    members = seq[None, :] == torch.arange(b, device="cuda")[:, None]
    last = torch.where(members, place, -1).amax(dim=1).clamp(min=0)
    end = upto[:, last]                              # [heads, b]
    decay = (end[:, :, None] - upto[:, None, :]).masked_fill(~members, -math.inf).float().exp()
    final = torch.matmul(decay, local).view(heads, b, dk, dv).transpose(0, 1)
    if s["states"] is not None:
        old = s["states"][s["slots"].long()]
        begin = before[:, base]                      # [heads, b]
        final = final + (end - begin).float().exp().t()[:, :, None, None] * old
        grown = (before - begin[:, seq]).float().exp()
        state = state + grown[:, :, None] * old.transpose(0, 1).reshape(heads, b, dk * dv)[:, seq]
    state = state.view(heads, count, dk, dv).transpose(0, 1)
    out = (out + torch.matmul(q * g.float().exp()[..., None], state)) * s["scale"]
    out = out.transpose(1, 2)[valid]                 # in the order of the tokens
    s["out"].copy_(out)
    s["new_states"][s["slots"].long()] = final
    return s["out"], s["new_states"]


def _plain_step(s):
    heads = s["case"]["heads"]
    q, k = (_shared(s[name], heads).float() for name in ("q", "k"))
    state = s["states"][s["slots"].long()] * s["log_decay"].exp()[:, :, None, None]
    state = state + k[:, :, :, None] * s["v"].float()[:, :, None, :]
    s["out"].copy_((state * q[:, :, :, None]).sum(dim=2) * s["scale"])
    s["new_states"][s["slots"].long()] = state
    return s["out"], s["new_states"]


_run_plain = {"quantize": _plain_quantize, "product": _plain_product, "prompt": _plain_prompt, "step": _plain_step}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "quantize":
        return None, s["x"].double().abs().amax(dim=1) / 127
    if op == "product":
        # the integers' products and sums are exact in 64 bits
        y = torch.matmul(s["xq"].double(), s["wq"].double().t().contiguous())
        y *= torch.outer(s["x_scale"].double(), s["w_scale"].double())
        return y if s["residual"] is None else y + s["residual"].double()
    heads, dk, dv = case["heads"], case["dk"], case["dv"]
    lengths = [1] * case["sequences"] if op == "step" else s["lengths"]
    b, most = len(lengths), max(lengths)
    share = heads // case["key_heads"]
    slots = s["slots"].long()
    pool = torch.zeros(s["pool"], heads, dk, dv, dtype=torch.float64, device="cuda")
    state = pool[slots] if s["states"] is None else s["states"][slots].double()
    v = s["v"].double()
    out = torch.zeros_like(v)
    starts = [sum(lengths[:i]) for i in range(b)]
    # the longest sequences first, so that those that still run are the first `live` ones
    order = sorted(range(b), key=lambda i: -lengths[i])
    first = torch.tensor([starts[i] for i in order], device="cuda")
    state = state[torch.tensor(order, device="cuda")]
    decay = s["log_decay"].double().exp()
    keys, queries = s["k"].double(), s["q"].double() * s["scale"]
    live = b
    for t in range(most):
        while lengths[order[live - 1]] <= t:
            live -= 1
        at = first[:live] + t
        run_ = state[:live]
        run_ *= decay[at][:, :, None, None]
        run_ += keys[at].repeat_interleave(share, dim=1)[:, :, :, None] * v[at][:, :, None, :]
        out[at] = torch.matmul(queries[at].repeat_interleave(share, dim=1)[:, :, None, :], run_)[:, :, 0]
    pool[slots[torch.tensor(order, device="cuda")]] = state
    return out, pool
