"""A gated feed-forward block in 4-bit weights, over prompts and decode steps.

    norm -> 8 or 4 bits -> gate and up projections -> silu(gate) * up -> 8 or 4
    bits -> down projection -> post norm, residual -> the next block's norm

Every step is one launch: norm_rows before the first block, then for each block
two PreparedMxfp4 products, quantize_blocks with its gate between them, and
join_rows, which ends the block and begins the next one.  The residual stream is
changed in place; nothing is kept between calls, so a block may run on several
streams at once.

    python -m skinny_bf16_decode_amd.feed_forward        # a prompt and decode steps on this GPU
"""
from __future__ import annotations

import torch

from .mxfp4 import BLOCK, PreparedMxfp4, quantize_blocks
from .norms import join_rows, norm_rows


def token_places(tokens, k, bits, device):
    """Empty codes of 8 or 4 bits and powers for rows of k values."""
    dtype = torch.float8_e4m3fn if bits == 8 else torch.uint8
    return (torch.empty(tokens, k * bits // 8, dtype=dtype, device=device),
            torch.empty(tokens, k // BLOCK, dtype=torch.uint8, device=device))


class FeedForward:
    """h + alpha post_norm(down (silu(gate x) * (up x))), x = norm(h).

    gate_up_weight [2 inner, hidden] (the gate's rows first) and down_weight
    [hidden, inner]: BF16, FP16 or fp32, quantized here; hidden and inner whole
    blocks of 32.  norm_weight [hidden]; post_weight
    [hidden], or None for no norm at the block's end.  Tokens go through the
    products in `bits`, 8 or 4."""

    def __init__(self, gate_up_weight, down_weight, norm_weight, post_weight=None, alpha=1.0, bits=8, eps=1e-6):
        hidden, inner = down_weight.shape
        if tuple(gate_up_weight.shape) != (2 * inner, hidden):
            raise ValueError(f"gate_up_weight must be [{2 * inner}, {hidden}], got {tuple(gate_up_weight.shape)}")
        if bits not in (4, 8):
            raise ValueError(f"tokens have 8 or 4 bits, not {bits}")
        self.hidden, self.inner, self.bits = hidden, inner, bits
        self.norm_weight, self.post_weight, self.alpha, self.eps = norm_weight, post_weight, alpha, eps
        self.gate_up = PreparedMxfp4(*self._quantized(gate_up_weight, 4))
        self.down = PreparedMxfp4(*self._quantized(down_weight, 4))

    @staticmethod
    def _quantized(x, bits, gate=None):
        return quantize_blocks(x, *token_places(*x.shape, bits, x.device), gate=gate)

    def enter(self, h):
        """The block's input of the residual stream h [tokens, hidden]: quantized rows and their powers."""
        q, scale = token_places(h.shape[0], self.hidden, self.bits, h.device)
        norm_rows(h, self.norm_weight, q=q, scale=scale, eps=self.eps)
        return q, scale

    def run(self, h, entered, following=None):
        """Adds the block of `entered` (its enter(h), or what the block before
        has returned) to h in place; returns `following`'s input, or None.
        Capturable in a graph."""
        tokens = h.shape[0]
        rows = torch.empty(tokens, 2 * self.inner, dtype=torch.bfloat16, device=h.device)
        self.gate_up.run(*entered, rows)
        y = torch.empty(tokens, self.hidden, dtype=torch.bfloat16, device=h.device)
        self.down.run(*self._quantized(rows[:, self.inner:], self.bits, gate=rows[:, :self.inner]), y)
        if following is None or following.eps != self.eps:      # join_rows has one eps for both its norms
            join_rows(h, y, h, weight=self.post_weight, alpha=self.alpha, eps=self.eps)
            return None if following is None else following.enter(h)
        q, scale = token_places(tokens, self.hidden, following.bits, h.device)
        join_rows(h, y, h, weight=self.post_weight, alpha=self.alpha, next_weight=following.norm_weight, q=q,
                  scale=scale, eps=self.eps)
        return q, scale


def run_blocks(blocks, h):
    """h [tokens, hidden] through the blocks, in place; returns h."""
    entered = blocks[0].enter(h)
    for block, following in zip(blocks, [*blocks[1:], None]):
        entered = block.run(h, entered, following)
    return h


def random_blocks(count, hidden, inner, bits=8, seed=0, device="cuda"):
    """Blocks of random weights with post norms, scaled down as deep stacks have them."""
    gen = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=device)

    return [FeedForward(normal(2 * inner, hidden) * hidden ** -0.5, normal(hidden, inner) * inner ** -0.5,
                        1 + 0.1 * normal(hidden), 1 + 0.1 * normal(hidden), alpha=(2 * count) ** -0.5, bits=bits)
            for _ in range(count)]


def main():
    hidden, inner, prompt, batch, steps = 7168, 18432, 2000, 8, 32
    blocks = random_blocks(2, hidden, inner)
    gen = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(prompt, hidden, generator=gen, device="cuda", dtype=torch.bfloat16)
    new = torch.randn(batch, hidden, generator=gen, device="cuda", dtype=torch.bfloat16)

    def timed(what, count, fn):
        fn()
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        for _ in range(count):
            fn()
        end.record()
        end.synchronize()
        print(f"{what}: {1e3 * begin.elapsed_time(end) / count:.1f} us")

    timed(f"{len(blocks)} blocks over a prompt of {prompt} tokens", 5, lambda: run_blocks(blocks, h))
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_blocks(blocks, new)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        run_blocks(blocks, new)
    timed(f"{len(blocks)} blocks, a decode step of {batch} tokens", steps, graph.replay)


if __name__ == "__main__":
    main()
