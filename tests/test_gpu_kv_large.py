"""Attention over a paged cache with values near the largest, against the 64-bit
form: sums of values times probabilities that pass the largest float, where the
result, their mean, does not."""
import pytest
import torch

import dense_linear_projection_amd as dlp
from tests import decode_reference as ref
from tests.test_gpu_kv import BF16, F32, make_attend, run_attend

pytestmark = pytest.mark.gpu


def check(ctx, k, v, cache, q, tables, n, out, window=0):
    cache.k.copy_(k)
    cache.v.copy_(v)
    want, tol = ref.attend(k, v, q, tables, n, 1.0, window, (1, 1), out)
    assert bool(torch.isfinite(want[0]).all())
    o, lse = run_attend(ctx, cache, q, tables, n, 1.0, out, window)
    ref.close(o, want[0], tol[0])
    ref.close(lse, want[1], tol[1])


def logits_of(k, q, tables, page, heights):
    """Keys and queries whose logits are heights[b][t] (exact in bf16), for every head."""
    k[..., 0], q[..., 0], q[..., 1:] = 0, 1, 0
    for b, row in enumerate(heights):
        for t, w in enumerate(row):
            k[tables[b, t // page], :, t % page, 0] = w


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("D,per", [(64, 1), (128, 4), (80, 20), (128, 20), (256, 3)])
@pytest.mark.parametrize("size", [1e37, 3e38])
def test_a_large_value_behind_logits_that_rise(ctx, out, D, per, size):
    """A large value at a logit a little above all before it: its probability is at most 1 whatever maximum is kept. The
    elements beside it are as good as ever."""
    lengths = [70, 40, 300, 5, 0, 333]
    k, v, cache, q, tables, n, _ = make_attend(len(lengths), 2 * per, 2, D, 16, BF16, "hnd", lengths, D + per)
    at = [69, 39, 290, 4, 0, 200]
    logits_of(k, q, tables, 16, [[4.875 if t == at[b] else 0.0 for t in range(m)] for b, m in enumerate(lengths)])
    for b, m in enumerate(lengths):
        if m:
            v[tables[b, at[b] // 16], :, at[b] % 16, ::3] = size
            v[tables[b, at[b] // 16], :, at[b] % 16, 1::3] = -size
    check(ctx, k, v, cache, q, tables, n, out)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 192])
@pytest.mark.parametrize("lengths", [[2, 40, 1, 100], [1000, 600], [7000], [300] * 40])
@pytest.mark.parametrize("window", [0, 150])
def test_many_large_values(ctx, out, D, lengths, window):
    """Their sum passes the largest float in a part, in the joining of the parts, and in both kinds of joining; their mean
    does not."""
    k, v, cache, q, tables, n, _ = make_attend(len(lengths), 8, 2, D, 16, BF16, "nhd", lengths, D)
    g = torch.Generator().manual_seed(D + len(lengths))
    near = torch.isfinite(v.float())
    v[..., : D // 2] = torch.where(near, (torch.rand(v.shape, generator=g) + 2) * 1e38, v.float())[..., : D // 2].to(BF16)
    k[..., :] = torch.where(torch.isfinite(k.float()), k.float() / 8, k.float()).to(BF16)
    check(ctx, k, v, cache, q, tables, n, out, window)


def test_large_values_that_cancel(ctx):
    k, v, cache, q, tables, n, _ = make_attend(2, 4, 1, 64, 16, BF16, "hnd", [600, 33], 3, poison=False)
    logits_of(k, q, tables, 16, [[0.0] * 600, [0.0] * 33])
    v[:, :, ::2, :5], v[:, :, 1::2, :5] = 3e38, -3e38
    check(ctx, k, v, cache, q, tables, n, F32)


@pytest.mark.parametrize("out", [BF16, F32])
def test_infinite_and_large_values_together(ctx, out):
    """What is infinite or no number stays so, in its own element."""
    k, v, cache, q, tables, n, _ = make_attend(2, 4, 2, 64, 16, BF16, "hnd", [500, 20], 4, poison=False)
    k[...] = k / 8
    v[..., 3], v[..., 4], v[..., 5] = 3e38, -3e38, 1e38
    cache.k.copy_(k)
    clean, tol = ref.attend(k, v, q, tables, n, 1.0, 0, (1, 1), out)
    v[tables[0, 3], 1, 5, 7], v[tables[0, 4], 1, 5, 8] = float("inf"), float("nan")
    cache.v.copy_(v)
    o, lse = run_attend(ctx, cache, q, tables, n, 1.0, out)
    assert bool((o[0, 2:, 7] == float("inf")).all()) and bool(torch.isnan(o[0, 2:, 8]).all())
    keep = torch.ones(2, 4, 64, dtype=torch.bool)
    keep[0, 2:, 7:9] = False
    ref.close(o.cpu()[keep], clean[0][keep], tol[0][keep])
    ref.close(lse, clean[1], tol[1])


def test_replays_follow_their_inputs(ctx):
    """Rows are worked out again, or not, as the values of the replay say; the counters of the joining are left at zero."""
    lengths = [700, 3, 260, 0]
    k, v, cache, q, tables, n, _ = make_attend(4, 8, 2, 128, 16, BF16, "hnd", lengths, 6, poison=False)
    cache.k.copy_(k / 8)
    dev = [t.cuda() for t in (q, tables, n)]
    o, lse = torch.empty(4, 8, 128, device="cuda"), torch.empty(4, 8, device="cuda")

    def call(o, lse):
        dlp.proj_kv_attend(ctx, cache, *dev, 1.0, o, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(o, lse)
    for size in (1.0, 1e38, 1.0, 1e37, 1.0):
        cache.v.copy_((torch.rand(v.shape) + 1) * size)
        o.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        a, b = torch.empty_like(o), torch.empty_like(lse)
        call(a, b)
        torch.cuda.synchronize()
        assert torch.equal(o, a) and torch.equal(lse, b)
        want, tol = ref.attend(cache.k.cpu(), cache.v.cpu(), q, tables, n, 1.0, 0, (1, 1), F32)
        ref.close(o, want[0], tol[0])
