"""4-bit projection at the sizes that take its other kernels: many columns for
few rows (32 and 64 columns to a workgroup, on 256 compute units), rows so
long that their scales do not fit LDS at once, large tiles over enough steps
that their rings go round, and the shapes of a serving model; and X of one
sign.  Wide results are compared on a part of their columns."""
import math

import pytest
import torch

from tests import decode_reference as ref
from tests.test_gpu_quant import BF16, F32, make, run

pytestmark = pytest.mark.gpu
ALL = [(True, BF16), (True, F32), (False, BF16), (False, F32)]      # zero points, scale type


def check(ctx, M, N, K, group, zeros, sdt, epi, out, columns=None, positive=False):
    print("quant", M, N, K, group, zeros, sdt, epi, out, flush=True)
    X, codes, scales, z, b = make(M, N, K, group, zeros, sdt, epi & 1, M + N + K + group)
    if positive:
        X = X.abs()
    got = run(ctx, X, codes, scales, z, group, b, epi, out).cpu()
    if columns is not None and N > columns:
        # the ends, and places spread over every tile's width
        at = torch.cat((torch.arange(40), torch.arange(N - 40, N), torch.arange(columns) * 1009 % N)).unique()
        got, codes, scales = got[:, at], codes[at], scales[at]
        z, b = None if z is None else z[at], None if b is None else b[at]
    want, tol = ref.quant(X, codes, scales, z, group, b, epi, out)
    if positive:
        # Within a group up to 132 roundings of sums of at most 47 |x| s a term, either way, so 11.5 of them in all;
        # groups independent of each other; then one rounding a group of a sum that grows to 15 |x| s a term.  Five
        # times that covers the largest of many.
        G = -(-K // group)
        size = X.double().abs() @ scales.double().abs()[:, torch.arange(K) // group].t()
        t = 5 * ref.EPS32 * (11.5 * 47 / math.sqrt(G) + 15 * math.sqrt(G / 3)) * size
        tol = t + ref.HALF[out] * (want.abs() + t)
    ref.close(got, want, tol)


@pytest.mark.parametrize("M", [1, 9, 16])
@pytest.mark.parametrize("N", [4097, 4100, 8192, 16384, 16385, 16400, 28672])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_many_columns_for_few_rows(ctx, M, N, group):
    for i, (zeros, sdt) in enumerate(ALL):
        check(ctx, M, N, 1024 if i % 2 else 1000, group, zeros, sdt, (3, 0, 1, 2)[i], F32 if i % 2 else BF16, 600)


@pytest.mark.parametrize("M,N,K,group", [(1, 100, 16512, 32), (16, 33, 17000, 32), (3, 40, 33024, 64), (16, 4100, 8320, 32),
                                         (2, 4100, 8456, 32), (20, 100, 8320, 32), (32, 70, 16640, 64), (17, 100, 8328, 32),
                                         (4, 16400, 4224, 32), (16, 16400, 4232, 32), (2, 16400, 8320, 64), (5, 16400, 16640, 128)])
def test_rows_whose_scales_come_in_parts(ctx, M, N, K, group):
    for zeros, sdt in ALL:
        check(ctx, M, N, K, group, zeros, sdt, 1, F32, 200)


@pytest.mark.parametrize("M,N,K", [(600, 7000, 640), (513, 7936, 1152), (600, 7000, 904), (1000, 4200, 1024)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_large_tiles_over_many_steps(ctx, M, N, K, group):
    for i, (zeros, sdt) in enumerate(ALL):
        check(ctx, M, N, K, group, zeros, sdt, (1, 2, 0, 3)[i], BF16 if i % 2 else F32, 900)


@pytest.mark.parametrize("M,N,K,group,zeros,sdt,epi", [
    (1, 1024, 8192, 128, True, BF16, 0), (16, 8192, 8192, 128, False, BF16, 1), (32, 28672, 8192, 128, False, BF16, 0),
    (64, 28672, 8192, 64, True, BF16, 2), (128, 8192, 8192, 32, True, BF16, 0), (256, 8192, 2752, 128, True, BF16, 0),
    (1024, 8192, 8192, 128, False, BF16, 0), (1024, 2368, 8192, 32, True, F32, 1), (2000, 4096, 2880, 64, True, BF16, 0)])
def test_shapes_of_a_serving_model(ctx, M, N, K, group, zeros, sdt, epi):
    check(ctx, M, N, K, group, zeros, sdt, epi, F32, 200)


@pytest.mark.parametrize("M,N,K", [(1, 300, 8192), (16, 4100, 1000), (24, 100, 4096), (64, 130, 8192), (600, 7000, 1024)])
@pytest.mark.parametrize("group", [32, 128])
def test_x_of_one_sign(ctx, M, N, K, group):
    """What follows an activation: the sums of 16 + code and of x grow, and their difference is what is left."""
    for zeros, sdt in ((True, BF16), (False, F32)):
        check(ctx, M, N, K, group, zeros, sdt, 0, F32, 300, positive=True)
