"""Attention over a paged cache at the ends of its types' ranges, against the
64-bit form: what rounding a probability does to the mean of many results,
values near the largest next to vanished probabilities, infinite values, and
logits near the largest."""
import math

import pytest
import torch

from tests import decode_reference as ref
from tests.test_gpu_kv import BF16, F32, FP8, make_attend, run_attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_probabilities_are_not_cut_one_way(ctx, dtype):
    """bf16 results take probabilities of 16 bits.  Rounded to nearest they are
    off by at most 2^-17 in either direction, which cancels over results that
    are means of about 300 tokens each; cut, each is low by about 2^-17, and so
    is every result.  Measured against the correctly rounded results, so that
    only those that fall on the other side of a rounding border differ."""
    k, v, cache, q, tables, n, scales = make_attend(32, 64, 8, 128, 16, dtype, "hnd", [280 + b for b in range(32)], 21,
                                                    poison=False)
    g = torch.Generator().manual_seed(22)
    v = (torch.rand(v.shape, generator=g) + 1).to(dtype)
    cache.v.copy_(v)
    want, _ = ref.attend(k, v, q, tables, n, 128 ** -0.5, 0, scales, BF16)
    o, _ = run_attend(ctx, cache, q, tables, n, 128 ** -0.5, BF16)
    w = want[0]
    low = float(((o.cpu().double() - w.to(BF16).double()) / w).mean())
    assert abs(low) < 2.0 ** -18, low
