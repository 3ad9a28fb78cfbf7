"""Attention over a shared prefix: that a result's type rounds it and changes
nothing before that."""
import pytest
import torch

from tests.test_gpu_shared import BF16, F32, FP8, lengths_of, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 80, 96, 128, 192, 256])
@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("B,Hq,L,window", [(3, 8, 500, 0), (40, 16, 900, 0), (40, 8, 333, 200)])
def test_bf16_results_are_the_fp32_ones_rounded(ctx, D, dtype, B, Hq, L, window):
    """Probabilities keep their 24 bits whatever the results' type: nothing but the last rounding differs."""
    print("rounded", D, dtype, B, Hq, L, window, flush=True)
    _, _, cache, q, prefix, tables, n, _ = make(B, Hq, 2, D, 16, dtype, "hnd", L, lengths_of(B, L, 60, B, True), D)
    wide, e = run(ctx, cache, q, prefix, L, tables, n, D ** -0.5, F32, window)
    o, f = run(ctx, cache, q, prefix, L, tables, n, D ** -0.5, BF16, window)
    assert torch.equal(o, wide.to(BF16)) and torch.equal(e, f)
