"""GELU of the integer projection: the same function to the bit in every kernel
that sizes, workspaces and pieces lead to."""
import pytest
import torch

import dense_linear_projection_amd as dlp
from tests import layer_reference as ref
from tests.decode_reference import close
from tests.test_gpu_int import BF16, F32, integers, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("epi", [2, 3])
@pytest.mark.parametrize("M,N,K", [(4, 1024, 256), (1, 2048, 512), (3, 515, 200), (2, 8192, 1024), (4, 300, 8192)])
def test_dynamic_is_the_two_calls(ctx, M, N, K, epi):
    g = torch.Generator().manual_seed(K + M)
    X = torch.randn(M, K, generator=g).to(BF16).cuda()
    W, ws = dlp.proj_quantize_rows(ctx, (torch.randn(N, K, generator=g) / K ** 0.5).to(BF16).cuda())
    bias = torch.randn(N, generator=g).to(BF16).cuda()
    q, s = dlp.proj_quantize_rows(ctx, X)
    two, one = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    dlp.proj_run_int(ctx, q, s, W, ws, bias, epi, two)
    dlp.proj_run_int_dynamic(ctx, X, W, ws, bias, epi, one)
    torch.cuda.synchronize()
    assert torch.equal(one, two)


@pytest.mark.parametrize("room", [1 << 18, 700000, 1 << 20])
def test_pieces_of_a_workspace(ctx, room):
    """Pieces of many rows and a last one of few: other kernels, the same bits."""
    M, N, K = 1030, 8192, 1024
    g = torch.Generator().manual_seed(room)
    X = torch.randn(M, K, generator=g).to(BF16).cuda()
    W, ws = dlp.proj_quantize_rows(ctx, (torch.randn(N, K, generator=g) / K ** 0.5).to(BF16).cuda())
    want, Y = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    dlp.proj_run_int_dynamic(ctx, X, W, ws, None, dlp.EPI_GELU_TANH, want)
    c = dlp.proj_create(0, room)
    dlp.proj_run_int_dynamic(c, X, W, ws, None, dlp.EPI_GELU_TANH, Y)
    torch.cuda.synchronize()
    dlp.proj_destroy(c)
    assert torch.equal(Y, want)


def test_rows_do_not_depend_on_how_many_there_are(ctx):
    """One token alone, in a small batch and in a large one."""
    X, xs, W, ws, bias = integers(2048, 1024, 512, 6)
    ws = ws / 20
    all_rows = run(ctx, X, xs, W, ws, bias, 3, F32)
    for m in (1, 2, 16, 17, 64, 100, 256, 700):
        assert torch.equal(run(ctx, X[:m], xs[:m], W, ws, bias, 3, F32), all_rows[:m])


@pytest.mark.parametrize("M", [1, 40, 600])
def test_gelu_over_the_whole_range(ctx, M):
    """Arguments from the smallest to the largest, of either sign, and infinite ones."""
    K, N = 256, 512
    X = torch.zeros(M, K, dtype=torch.int8)
    X[:, 0] = 1
    W = torch.zeros(N, K, dtype=torch.int8)
    W[:, 0] = torch.where(torch.arange(N) % 2 == 0, 1, -1).to(torch.int8)
    ws = torch.logspace(-45, 38, N, dtype=torch.float64).float()
    xs = torch.ones(M)
    want, tol = ref.product(X, xs, W, ws, None, 2, F32)
    got = run(ctx, X, xs, W, ws, None, 2, F32)
    close(got, want, tol)
    ws[:] = float("inf")
    got = run(ctx, X, xs, W, ws, None, 2, F32).cpu()
    assert bool((got[:, ::2] == float("inf")).all()) and torch.isnan(got[:, 1::2]).all()
