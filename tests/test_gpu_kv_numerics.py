"""Attention over a paged cache at the ends of its types' ranges, against the
64-bit form: what rounding a probability does to the mean of many results,
values near the largest next to vanished probabilities, infinite values, and
logits near the largest."""
import math

import pytest
import torch

import dense_linear_projection_amd as dlp
from tests import decode_reference as ref
from tests.test_gpu_kv import BF16, F32, FP8, make_attend, run_attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_probabilities_are_not_cut_one_way(ctx, dtype):
    """Probabilities that met the values with 16 bits would be off by at most
    2^-17: rounded to nearest in either direction, which cancels over results
    that are means of about 300 tokens each, cut each low by about 2^-17, and
    so every result.  Measured against the correctly rounded results, so that
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


@pytest.mark.parametrize("D", [64, 80, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("per,lengths", [(4, [1, 500, 37, 0, 64]), (20, [900, 33]), (8, [7000])])
def test_bf16_results_are_the_fp32_ones_rounded(ctx, D, dtype, per, lengths):
    """Probabilities keep their 24 bits whatever the results' type: nothing but the last rounding differs."""
    k, v, cache, q, tables, n, scales = make_attend(len(lengths), 2 * per, 2, D, 16, dtype, "hnd", lengths, 28)
    wide, _ = run_attend(ctx, cache, q, tables, n, D ** -0.5, F32)
    o, _ = run_attend(ctx, cache, q, tables, n, D ** -0.5, BF16)
    assert torch.equal(o, wide.to(BF16))


def one_head(ctx, K, V, q, n, scale, out):
    """Results of one sequence of n tokens in one page, one head; K and V [16, 64], q [64]."""
    cache = dlp.kv_cache(K.view(1, 1, 16, 64).cuda(), V.view(1, 1, 16, 64).cuda())
    o, e = torch.empty(1, 1, 64, dtype=out, device="cuda"), torch.empty(1, 1, device="cuda")
    dlp.proj_kv_attend(ctx, cache, q.view(1, 1, 64).cuda(), torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                       torch.tensor([n], dtype=torch.int32, device="cuda"), scale, o, lse=e)
    return o[0], e[0]


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("low", [-20.0, -60.0, -80.0, -200.0, -3000.0])
def test_small_probability_of_a_large_value(ctx, out, low):
    """A value near the type's largest counts by its token's probability, also
    where that is nothing."""
    g = torch.Generator().manual_seed(23)
    K, V, q = torch.zeros(16, 64).to(BF16), torch.randn(16, 64, generator=g).to(BF16), torch.zeros(64).to(BF16)
    q[0], K[1, 0], V[1] = 1, low, 3e38
    want, tol = ref.attend(K.view(1, 1, 16, 64), V.view(1, 1, 16, 64), q.view(1, 1, 64), torch.zeros(1, 1, dtype=torch.int32),
                           torch.tensor([3]), 1.0, 0, (1.0, 1.0), out)
    o, e = one_head(ctx, K, V, q, 3, 1.0, out)
    ref.close(o[None], want[0], tol[0])
    ref.close(e[None], want[1], tol[1])


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("low", [0.0, -1.0, -20.0, -60.0])
def test_infinite_value_inside(ctx, out, low):
    """An infinite value whose token has a probability gives infinity, of its own sign, and no NaN."""
    g = torch.Generator().manual_seed(24)
    K, V, q = torch.zeros(16, 64).to(BF16), torch.randn(16, 64, generator=g).to(BF16), torch.zeros(64).to(BF16)
    q[0], K[1, 0], V[1, 5], V[1, 6] = 1, low, math.inf, -math.inf
    o, _ = one_head(ctx, K, V, q, 4, 1.0, out)
    assert float(o[0, 5]) == math.inf and float(o[0, 6]) == -math.inf
    assert int(torch.isfinite(o).sum()) == 62


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("logit", [-2.4e38, -3.38e38, 2.0e38, 2.4e38, 3.38e38])
def test_logits_near_the_largest(ctx, out, logit):
    """Every finite logit counts: tokens that all have the same share alike,
    one above the others takes all, however far from zero they are."""
    g = torch.Generator().manual_seed(25)
    K, V, q = torch.zeros(16, 64).to(BF16), torch.randn(16, 64, generator=g).to(BF16), torch.zeros(64).to(BF16)
    q[0], K[:, 0] = 1, logit
    o, e = one_head(ctx, K, V, q, 7, 1.0, out)
    mean = V[:7].double().mean(0)
    # seven equal probabilities: each fp32 sum's roundings, and the result's own
    ref.close(o[0], mean, 16 * ref.EPS32 * V[:7].double().abs().mean(0) + ref.HALF[out] * mean.abs())
    assert abs(float(e) / float(K[0, 0]) - 1) < 2 * ref.EPS32
    if logit < 0:
        K[5, 0] = 0
        o, e = one_head(ctx, K, V, q, 7, 1.0, out)
        assert torch.equal(o[0].cpu(), V[5].to(out)) and float(e) == 0
    K[:, 0], K[2, 0] = -logit, logit
    o, e = one_head(ctx, K, V, q, 7, 1.0, out)
    rest = [i for i in range(7) if i != 2]
    want = V[2].double() if logit > 0 else V[rest].double().mean(0)
    ref.close(o[0], want, 16 * ref.EPS32 * V[:7].double().abs().amax(0) + ref.HALF[out] * want.abs())


def test_large_negative_scale(ctx):
    """A negative scale turns the order of the logits round."""
    k, v, cache, q, tables, n, scales = make_attend(3, 8, 2, 64, 16, BF16, "hnd", [300, 17, 64], 26)
    want, tol = ref.attend(k, v, q, tables, n, -1.5, 0, scales, F32)
    o, e = run_attend(ctx, cache, q, tables, n, -1.5, F32)
    ref.close(o, want[0], tol[0])
    ref.close(e, want[1], tol[1])


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("rot", [64, 34])
def test_tokens_of_one_slot(ctx, dtype, rot):
    """Every element of a slot that several tokens go to is one of theirs; other slots keep what they had."""
    T, H, D = 300, 2, 64
    g = torch.Generator().manual_seed(27)
    qkv = torch.randn(T, 2 * H * D, generator=g).to(BF16)
    cache = dlp.kv_cache(*(torch.zeros(2, H, 16, D, device="cuda").to(dtype) for _ in range(2)))
    rope = torch.cat((torch.ones(1, rot // 2), torch.zeros(1, rot // 2)), 1).cuda()
    dlp.proj_kv_append(ctx, cache, qkv.cuda(), rope, torch.zeros(T, dtype=torch.int32, device="cuda"),
                       torch.full((T,), 21, device="cuda"))
    x = qkv.to(dtype).float().view(T, 2, H, D)
    for i, c in enumerate((cache.k, cache.v)):
        c = c.float().cpu()
        assert bool((c[1, :, 5] == x[:, i]).any(0).all())
        c[1, :, 5] = 0
        assert not c.any()
