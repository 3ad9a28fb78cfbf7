"""Attention over a shared prefix with scales at the ends of the range, against
the 64-bit form: a scale that base 2 takes past the largest float, one whose
product with the cache's scale vanishes, a scale of zero."""
import pytest
import torch

import dense_linear_projection_amd as dlp
from tests import layer_reference as ref
from tests.decode_reference import close
from tests.test_gpu_shared import BF16, F32, FP8, lengths_of, make, run

pytestmark = pytest.mark.gpu
GROUPS = ((3, 8), (40, 8))        # sequences and query heads: rows of one group, and of several


def case(B, Hq, dtype, k_scale=1.0):
    lengths = lengths_of(B, 150, 60, B)
    lengths[0] = 33
    k, v, cache, q, prefix, tables, n, scales = make(B, Hq, 2, 64, 16, dtype, "hnd", 150, lengths, 18)
    if dtype == FP8:
        cache = dlp.kv_cache(cache.k, cache.v, k_scale, scales[1])
        scales = (float(torch.tensor(k_scale).float()), scales[1])
    return k, v, cache, q, prefix, tables, n, scales


def check(ctx, k, v, cache, q, prefix, tables, n, scales, scale, window=0):
    scale = float(torch.tensor(scale).float())
    want, tol = ref.attend_shared(k, v, q, prefix, 150, tables, n, scale, window, scales, F32)
    o, lse = run(ctx, cache, q, prefix, 150, tables, n, scale, F32, window)
    close(o, want[0], tol[0])
    close(lse, want[1], tol[1])


@pytest.mark.parametrize("scale", [1e20, -1e31, 2.3e38, 2.5e38, -3e38])
@pytest.mark.parametrize("size", [4.0, 100.0])
@pytest.mark.parametrize("window", [0, 100])
def test_large_scales(ctx, scale, size, window):
    """Queries as small as the scale is large (but normal numbers): logits are ordinary."""
    for B, Hq in GROUPS:
        k, v, cache, q, prefix, tables, n, scales = case(B, Hq, BF16)
        used = torch.isfinite(k.float())
        k[...] = torch.where(used, torch.randint(-8, 9, k.shape, generator=torch.Generator().manual_seed(1)).float(), k.float()).to(BF16)
        cache.k.copy_(k)
        # one element of a query each, so that a logit is one product
        q[:] = 0
        at = torch.arange(q.shape[0] * q.shape[1]).view(q.shape[:2]) % 64
        q.scatter_(2, at[..., None], torch.full(q.shape, max(size / 8 / abs(scale), 2.0 ** -126)).to(BF16)[..., :1])
        check(ctx, k, v, cache, q, prefix, tables, n, scales, scale, window)


@pytest.mark.parametrize("scale,k_scale", [(1e-44, 0.01), (-1e-30, 1e-20), (1e-42, 1.0), (1e-38, 1e-38), (1e-45, 1e-45), (1e-30, 1e20),
                                           (1e30, 1e-30), (3e38, 1e-38), (-2e20, 1e10)])
@pytest.mark.parametrize("window", [0, 100])
def test_both_scales(ctx, scale, k_scale, window):
    """The scale times the cache's, which vanishes in fp32 though neither does, is ordinary though neither is, or is large."""
    for B, Hq in GROUPS:
        k, v, cache, q, prefix, tables, n, scales = case(B, Hq, FP8, k_scale)
        if abs(scale) * k_scale > 1e20:   # logits that differ are far apart, and those of one key are equal
            q[:] = 0
            q[..., 0] = 1
        check(ctx, k, v, cache, q, prefix, tables, n, scales, scale, window)


def test_a_scale_of_zero_of_what_is_no_number(ctx):
    """0 times NaN or infinity is NaN, in its own row; every other row is the mean."""
    k, v, cache, q, prefix, tables, n, scales = case(40, 8, BF16)
    n.clamp_(max=150)                                # tokens of the prefix alone
    want, tol = ref.attend_shared(k, v, q, prefix, 150, tables, n, 0.0, 0, scales, F32)
    q[7, 3, 5], q[9, 0, 63], q[11, 7, 0] = float("nan"), float("inf"), -float("inf")
    o, lse = run(ctx, cache, q, prefix, 150, tables, n, 0.0, F32)
    keep = torch.ones(40, 8, dtype=torch.bool)
    for b, h in ((7, 3), (9, 0), (11, 7)):
        keep[b, h] = False
        assert torch.isnan(o[b, h]).all() and torch.isnan(lse[b, h])
    close(o[keep], want[0][keep], tol[0][keep])
    close(lse[keep], want[1][keep], tol[1][keep])


@pytest.mark.parametrize("op", ["shared", "plain"])
def test_a_product_of_scales_past_the_largest_is_refused(ctx, op):
    k, v, cache, q, prefix, tables, n, _ = case(3, 8, FP8, 1e20)
    for scale in (1e20, -3e38):
        with pytest.raises(dlp.ProjError) as e:
            if op == "shared":
                run(ctx, cache, q, prefix, 150, tables, n, scale, F32)
            else:
                o = torch.empty(3, 8, 64, device="cuda")
                dlp.proj_kv_attend(ctx, cache, q.cuda(), tables.cuda(), n.cuda() * 0, scale, o)
        assert e.value.status == dlp.PROJ_ERR_INVALID_ARG


@pytest.mark.parametrize("scale", [1.0, 2e38])
def test_logits_near_the_largest(ctx, scale):
    """Logits as large as floats are: the largest takes all, equal ones share alike."""
    for B, Hq in GROUPS:
        k, v, cache, q, prefix, tables, n, scales = case(B, Hq, BF16)
        used = torch.isfinite(k.float())
        small = torch.randint(-5, 6, k.shape[:-1], generator=torch.Generator().manual_seed(2)).float() / 4
        k[..., 0] = torch.where(used[..., 0], small * (1 if scale > 1 else 2e38), k[..., 0].float()).to(BF16)
        cache.k.copy_(k)
        q[..., 0], q[..., 1:] = 1, 0
        want, _ = ref.attend_shared(k, v, q, prefix, 150, tables, n, float(torch.tensor(scale).float()), 0, scales, F32)
        o, lse = run(ctx, cache, q, prefix, 150, tables, n, scale, F32)
        # probabilities are 0, or one over how many there are: only sums of up to 210 of them round
        close(o, want[0], 300 * 2.0 ** -24 * torch.ones(o.shape).double() * 8)
        close(lse, want[1], 4 * 2.0 ** -24 * want[1].abs())
