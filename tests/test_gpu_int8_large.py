"""8-bit products with more threads than one launch may have (2^32), in the weight's layout and in the product."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def free_gib():
    torch.cuda.empty_cache()
    return torch.cuda.mem_get_info()[0] / 2 ** 30


def test_more_tokens_than_a_launch_has():
    """64 tokens a workgroup of 512 threads."""
    if not torch.cuda.is_available() or free_gib() < 60:
        pytest.skip("no GPU with 60 GiB free")
    from skinny_bf16_decode_amd.int8 import PreparedInt8
    m, n, k, block = 540_000_000, 16, 16, 1000
    print("tokens", m, n, k, flush=True)
    xq = torch.randint(-128, 128, (block, k), dtype=torch.int8, device="cuda")
    xs = torch.rand(block, device="cuda") + 0.5
    wq = torch.randint(-128, 128, (n, k), dtype=torch.int8, device="cuda")
    plan = PreparedInt8(wq, torch.rand(n, device="cuda"))
    want = plan.run(xq, xs, torch.empty(block, n, dtype=torch.bfloat16, device="cuda"))
    out = torch.full((m, n), -7.0, dtype=torch.bfloat16, device="cuda")
    plan.run(xq.repeat(m // block, 1), xs.repeat(m // block), out)
    torch.cuda.synchronize()
    for part in out.view(-1, block, n).split(20000):
        assert torch.equal(part, want.expand_as(part))
    plan.close()


def test_a_weight_of_more_vectors_than_a_launch_has():
    """Rows past the 2^32nd vector of 16 bytes, 64 GiB."""
    if not torch.cuda.is_available() or free_gib() < 150:
        pytest.skip("no GPU with 150 GiB free")
    from skinny_bf16_decode_amd.int8 import PreparedInt8
    block, k = 1024, 131056
    n = block * 516                                             # 528384 rows of 2048 steps of 64 bytes
    print("weight", n, k, flush=True)
    w = torch.randint(-128, 128, (block, k), dtype=torch.int8, device="cuda")
    ws = torch.rand(block, device="cuda")
    xq = torch.randint(-128, 128, (2, k), dtype=torch.int8, device="cuda")
    xs = torch.rand(2, device="cuda")
    small = PreparedInt8(w, ws, out_dtype=torch.float32)
    want = small.run(xq, xs, torch.empty(2, block, device="cuda"))
    large = w.repeat(n // block, 1)
    plan = PreparedInt8(large, ws.repeat(n // block), out_dtype=torch.float32)
    del large
    out = plan.run(xq, xs, torch.full((2, n), -7.0, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(out.view(2, -1, block), want[:, None].expand(2, n // block, block))
    plan.close()
    small.close()
    torch.cuda.empty_cache()
