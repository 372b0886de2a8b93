"""A linear-attention layer in 8-bit weights, over prompts and decode steps.

    x -> 8 bits -> packed projection (q, k, v, gate, decay columns) -> linear
    attention on the columns in place -> gate -> 8 bits -> projection back,
    added to the residual stream

The packed projection has as many rows as kda.py's, and q, k, v and the gate of
12 heads of 128 in the same places (rows 0..6143); then come 128 rows that this
layer does not read, one decay logit a head, and pads.  It is another layer than
KDA's and KDA weights do not run on it: those decay each channel (their F_A rows,
through F_B), their rows 6272..6283 are beta, and their recurrence has a delta
term, which this one has not.  The two projections are PreparedInt8 plans, the
sequences' states a pool of fp32 [heads, 128, 128] matrices; a prompt of any
lengths and a decode step share both.  The elementwise parts between them
(lengths of q and k, gate, decay) are torch's.

    python -m skinny_bf16_decode_amd.linear_layer        # a prompt and decode steps on this GPU
"""
from __future__ import annotations

import torch

from . import linear_attention
from .int8 import PreparedInt8, quantize_rows

HEADS, DIM = 12, 128
WIDTH = HEADS * DIM
DECAY_COLUMN = 4 * WIDTH + 128
PACKED_ROWS = DECAY_COLUMN + HEADS + 4


class LinearLayer:
    """packed_weight [6288, hidden] and out_weight [hidden, 1536] (BF16 or
    fp32, quantized here, a scale for each row); decay_rate fp32 [12], how fast
    each head forgets: log decay = -decay_rate softplus(decay logit).  `slots`
    states are kept, zero at the start."""

    def __init__(self, packed_weight, out_weight, decay_rate, slots):
        hidden = packed_weight.shape[1]
        if packed_weight.shape[0] != PACKED_ROWS or tuple(out_weight.shape) != (hidden, WIDTH):
            raise ValueError(f"packed_weight must be [{PACKED_ROWS}, hidden] and out_weight [hidden, {WIDTH}], got "
                             f"{tuple(packed_weight.shape)} and {tuple(out_weight.shape)}")
        if decay_rate.dtype != torch.float32 or tuple(decay_rate.shape) != (HEADS,):
            raise ValueError(f"decay_rate must be torch.float32 [{HEADS}]")
        self.hidden, self.decay_rate = hidden, decay_rate
        self.packed = PreparedInt8(*self._quantized(packed_weight), out_dtype=torch.bfloat16)
        self.out = PreparedInt8(*self._quantized(out_weight), out_dtype=torch.float32)
        self.states = torch.zeros(slots, HEADS, DIM, DIM, device=packed_weight.device)

    @staticmethod
    def _quantized(x):
        m, k = x.shape
        return quantize_rows(x, torch.empty(m, k, dtype=torch.int8, device=x.device),
                             torch.empty(m, dtype=torch.float32, device=x.device))

    def project(self, x):
        """q, k, v [tokens, 12, 128], the gate and the log decays of the tokens x [tokens, hidden]."""
        tokens = x.shape[0]
        rows = torch.empty(tokens, PACKED_ROWS, dtype=torch.bfloat16, device=x.device)
        self.packed.run(*self._quantized(x), rows)
        q, k, v, gate = (rows[:, i * WIDTH:(i + 1) * WIDTH].view(tokens, HEADS, DIM) for i in range(4))
        for part in (q, k):                     # unit length, in place
            part /= part.float().norm(dim=-1, keepdim=True).clamp(min=1e-6)     # fp32, rounded once
        logit = rows[:, DECAY_COLUMN:DECAY_COLUMN + HEADS].float()
        return q, k, v, gate, -self.decay_rate * torch.nn.functional.softplus(logit)

    def finish(self, mixed, gate, residual):
        """residual [tokens, hidden] fp32, plus the projection of the gated heads (in place); returns it."""
        # gate and product in BF16, the type of both: their roundings, 2^-8 of a value, are about the 8 bits' that
        # follow, half a step of 127 to the row's largest
        gated = (mixed * torch.sigmoid(gate)).view(mixed.shape[0], WIDTH)
        return self.out.run(*self._quantized(gated), residual, residual=residual)

    def prompt(self, x, residual, starts, slots):
        """The tokens x [tokens, hidden] of packed sequences, starts int32 [sequences + 1], going on from the
        states in slots int32 [sequences], which they leave at their ends."""
        q, k, v, gate, log_decay = self.project(x)
        mixed = torch.empty_like(v, memory_format=torch.contiguous_format)
        linear_attention.prompt(q, k, v, log_decay, mixed, starts, state_in=self.states, state_out=self.states,
                                slots=slots)
        return self.finish(mixed, gate, residual)

    def step(self, x, residual, slots):
        """One new token of each sequence: x [sequences, hidden], slots int32 [sequences].  Capturable in a graph."""
        q, k, v, gate, log_decay = self.project(x)
        mixed = torch.empty_like(v, memory_format=torch.contiguous_format)
        linear_attention.step(q, k, v, log_decay, mixed, state_in=self.states, state_out=self.states, slots=slots)
        return self.finish(mixed, gate, residual)


def random_layer(hidden, slots, seed=0, device="cuda"):
    """A layer of random weights: states forget over a few tokens to a few thousand."""
    gen = torch.Generator(device=device).manual_seed(seed)
    packed = torch.randn(PACKED_ROWS, hidden, generator=gen, device=device) * hidden ** -0.5
    out = torch.randn(hidden, WIDTH, generator=gen, device=device) * WIDTH ** -0.5
    return LinearLayer(packed, out, torch.exp(torch.linspace(-1.0, -7.0, HEADS, device=device)), slots)


def main():
    hidden, lengths, steps = 7168, [1500, 0, 77, 423], 32
    layer = random_layer(hidden, slots=len(lengths) + 2)
    gen = torch.Generator(device="cuda").manual_seed(1)
    starts = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")
    slots = torch.tensor([5, 0, 3, 2], dtype=torch.int32, device="cuda")
    x = torch.randn(sum(lengths), hidden, generator=gen, device="cuda", dtype=torch.bfloat16)
    new = torch.randn(len(lengths), hidden, generator=gen, device="cuda", dtype=torch.bfloat16)
    residual = torch.zeros(len(lengths), hidden, device="cuda")

    def timed(what, count, fn):
        fn()
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        for _ in range(count):
            fn()
        end.record()
        end.synchronize()
        print(f"{what}: {1e3 * begin.elapsed_time(end) / count:.1f} us")

    timed(f"prompt of {sum(lengths)} tokens", 5, lambda: layer.prompt(x, torch.zeros(x.shape, device="cuda"), starts,
                                                                     slots))
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(new, residual, slots)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        layer.step(new, residual, slots)
    timed(f"decode step of {len(lengths)} sequences", steps, graph.replay)


if __name__ == "__main__":
    main()
