"""Attention over a paged cache on its other kernels: more query heads to a
key head than one tile holds at every head size, long sequences joined by the
second kernel at every head size, and sequences of many page lists to a
workgroup, where nothing is split."""
import pytest
import torch

import dense_linear_projection_amd as dlp
from tests import decode_reference as ref
from tests.test_gpu_kv import BF16, F32, FP8, check_attend, make_attend, run_attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 80, 96, 128, 192, 256])
@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("per", [17, 20, 40])
def test_more_query_heads_than_a_tile(ctx, D, dtype, layout, per):
    check_attend(ctx, 3, 2 * per, 2, D, 16, dtype, layout, [150, 0, 33], D + per, F32)
    check_attend(ctx, 2, per, 1, D, 32, dtype, layout, [1100, 64], D + per + 1, BF16, 700)


@pytest.mark.parametrize("D", [64, 80, 96, 128, 192, 256])
@pytest.mark.parametrize("dtype,layout", [(BF16, "hnd"), (FP8, "nhd")])
@pytest.mark.parametrize("per", [1, 20])
def test_long_sequences_joined(ctx, D, dtype, layout, per):
    check_attend(ctx, 1, per, 1, D, 64, dtype, layout, [7000], D + per, F32)
    check_attend(ctx, 2, 2 * per, 2, D, 16, dtype, layout, [300, 6001], D + per + 1, BF16)


@pytest.mark.parametrize("page", [1, 16, 1024])
@pytest.mark.parametrize("dtype,layout", [(BF16, "nhd"), (FP8, "hnd")])
@pytest.mark.parametrize("window", [0, 4099])
def test_unsplit_sequences_of_many_pages(page, dtype, layout, window):
    small = dlp.proj_create(0, 0)                       # no workspace
    try:
        k, v, cache, q, tables, n, scales = make_attend(3, 4, 2, 64, page, dtype, layout, [5001, 2049, 0], page + window)
        want, tol = ref.attend(k, v, q, tables, n, 0.125, window, scales, F32)
        o, e = run_attend(small, cache, q, tables, n, 0.125, F32, window)
        ref.close(o, want[0], tol[0])
        ref.close(e, want[1], tol[1])
    finally:
        dlp.proj_destroy(small)


@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_cache_without_pages(ctx, dtype):
    """Nothing can be stored, and what is empty is attended: 0 and minus infinity, NaN where a token is asked for."""
    cache = dlp.kv_cache(*(torch.empty(0, 2, 16, 64, device="cuda").to(dtype) for _ in range(2)))
    qkv = torch.randn(3, 8 * 64, device="cuda").to(BF16)
    q, rope = torch.empty(3, 4, 64, device="cuda", dtype=BF16), torch.zeros(1, 0, device="cuda")
    dlp.proj_kv_append(ctx, cache, qkv, rope, torch.zeros(3, dtype=torch.int32, device="cuda"),
                       torch.tensor([0, -1, 5], device="cuda"), q)
    assert torch.equal(q, qkv[:, :256].view(3, 4, 64))
    o, e = run_attend(ctx, cache, q.cpu(), torch.zeros(3, 1, dtype=torch.int32), torch.tensor([0, 1, 0], dtype=torch.int32), 1.0, F32)
    assert not o[[0, 2]].any() and bool(torch.isneginf(e[[0, 2]]).all())
    assert bool(torch.isnan(o[1]).all()) and bool(torch.isnan(e[1]).all())
