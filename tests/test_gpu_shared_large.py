"""Attention over a shared prefix with values near the largest, against the
64-bit form: sums of values times probabilities that pass the largest float, in
the prefix, in the own tokens and in the joining of both, where the result, their
mean, does not."""
import pytest
import torch

from tests import layer_reference as ref
from tests.decode_reference import close
from tests.test_gpu_shared import BF16, F32, lengths_of, make, run

pytestmark = pytest.mark.gpu


def check(ctx, k, v, cache, q, prefix, L, tables, n, out, window=0):
    cache.k.copy_(k)
    cache.v.copy_(v)
    want, tol = ref.attend_shared(k, v, q, prefix, L, tables, n, 1.0, window, (1, 1), out)
    assert bool(torch.isfinite(want[0]).all())
    o, lse = run(ctx, cache, q, prefix, L, tables, n, 1.0, out, window)
    close(o, want[0], tol[0])
    close(lse, want[1], tol[1])


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("D,B,Hq", [(64, 3, 2), (128, 3, 8), (80, 40, 8), (256, 5, 4), (96, 130, 2)])
@pytest.mark.parametrize("size", [1e37, 3e38])
@pytest.mark.parametrize("at", [70, 100, 290, 310])
def test_a_large_value_behind_logits_that_rise(ctx, out, D, B, Hq, size, at):
    """A large value at a logit a little above all before it, in the prefix (at < 300) or behind it: its probability is at
    most 1 whatever maximum is kept. The elements beside it are as good as ever."""
    L = 300
    lengths = [320 + b % 7 for b in range(B)]
    lengths[0], lengths[1] = 64, 0                       # one that does not see it, one that sees nothing
    k, v, cache, q, prefix, tables, n, _ = make(B, Hq, 2, D, 16, BF16, "hnd", L, lengths, D + at)
    used = torch.isfinite(k.float())
    k[..., 0] = torch.where(used[..., 0], torch.zeros(()), k[..., 0].float()).to(BF16)
    q[..., 0], q[..., 1:] = 1, 0
    for page, place in [(prefix[at // 16], at % 16)] if at < L else [(tables[b, (at - L) // 16], (at - L) % 16) for b in range(2, B)]:
        k[page, :, place, 0] = 4.875
        v[page, :, place, ::3], v[page, :, place, 1::3] = size, -size
    check(ctx, k, v, cache, q, prefix, L, tables, n, out)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 192])
@pytest.mark.parametrize("B,L,own", [(1, 2, 1), (3, 500, 100), (40, 100, 30), (3, 4000, 1500), (33, 1000, 0)])
@pytest.mark.parametrize("window", [0, 150])
def test_many_large_values(ctx, out, D, B, L, own, window):
    """Their sum passes the largest float in a part of the prefix or of the own tokens, and in the joining of parts that
    do not; their mean does not."""
    k, v, cache, q, prefix, tables, n, _ = make(B, 8, 2, D, 16, BF16, "nhd", L, lengths_of(B, L, own, B), D)
    g = torch.Generator().manual_seed(D + B)
    v[..., : D // 2] = torch.where(torch.isfinite(v.float()), (torch.rand(v.shape, generator=g) + 2) * 1e38, v.float())[..., : D // 2].to(BF16)
    k[...] = torch.where(torch.isfinite(k.float()), k.float() / 8, k.float()).to(BF16)
    check(ctx, k, v, cache, q, prefix, L, tables, n, out, window)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("B", [2, 40])
def test_infinite_and_large_values_together(ctx, out, B):
    """What is infinite or no number reaches the sequences that see it, in its own element, and no other."""
    L = 200
    lengths = [230] * B
    lengths[0] = 60
    k, v, cache, q, prefix, tables, n, _ = make(B, 4, 2, 64, 16, BF16, "hnd", L, lengths, 5, poison=False)
    k[...] = k / 8
    v[..., 3], v[..., 4], v[..., 5] = 3e38, -3e38, 1e38
    cache.k.copy_(k)
    clean, tol = ref.attend_shared(k, v, q, prefix, L, tables, n, 1.0, 0, (1, 1), out)
    v[prefix[100 // 16], 1, 100 % 16, 7], v[prefix[150 // 16], 1, 150 % 16, 8] = float("inf"), float("nan")
    cache.v.copy_(v)
    o, lse = run(ctx, cache, q, prefix, L, tables, n, 1.0, out)
    assert bool((o[1:, 2:, 7] == float("inf")).all()) and bool(torch.isnan(o[1:, 2:, 8]).all())
    keep = torch.ones(B, 4, 64, dtype=torch.bool)
    keep[1:, 2:, 7:9] = False
    close(o.cpu()[keep], clean[0][keep], tol[0][keep])
    close(lse, clean[1], tol[1])
