"""Linear attention over values whose columns differ in size by more than 16
bits span: each column of a state has fp32's accuracy by itself.  Definition and
tolerances of test_gpu_linear_attention.py, whose bounds hold for every element."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("shape,lengths", [
    ((2, 2, 64, 64), [150]), ((2, 1, 128, 128), [700, 5]), ((3, 3, 32, 40), [64, 1, 65]), ((2, 2, 96, 192), [130]),
    ((1, 1, 200, 72), [500, 77]), ((12, 12, 128, 128), [40, 0, 1, 700, 130, 64, 65, 90, 33, 128, 2, 77])])
def test_columns_of_unlike_sizes(shape, lengths, kind):
    """A few columns 2^26 times as large as the rest, as outlier channels are."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from skinny_bf16_decode_amd import linear_attention as la
    from .test_gpu_linear_attention import check, make, run, say
    say("columns", kind, shape, lengths)
    c = make(lengths, *shape, kind, 91)
    size = torch.full((shape[3],), 2.0 ** -13, device="cuda")
    size[3::7] = 2.0 ** 13                          # randn's largest values stay below FP16's 65504
    c["v"].copy_((c["v"].float() * size))
    c["states"] *= size
    out, new = run(la, c)
    check(c, out, new, (kind, shape, lengths))
