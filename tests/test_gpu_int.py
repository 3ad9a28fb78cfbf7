"""Projection of 8-bit integers and the making of such integers, on the GPU
against their 64-bit forms: sizes that end inside every tile, one row to many,
each epilogue and output type, extreme scales and sums, strided and odd rows,
tokens made integers in a workspace that holds few of them, graphs and streams."""
import pytest
import torch

import dense_linear_projection_amd as dlp
from tests import layer_reference as ref
from tests.decode_reference import close

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------ rows to integers

def check_rows(ctx, X, stream=None):
    q, scales = dlp.proj_quantize_rows(ctx, X.cuda() if not X.is_cuda else X, stream=stream)
    torch.cuda.synchronize()
    want, s = ref.quantize_rows(X.cpu())
    K = X.shape[1]
    assert q.shape[1] % 16 == 0 and q.shape[1] - K < 16
    assert torch.equal(q[:, :K].cpu().long(), want)
    assert not bool(q[:, K:].any())
    assert torch.equal(scales.cpu(), s.float())


@pytest.mark.parametrize("M,K", [(1, 1), (1, 8192), (3, 7), (5, 16), (2, 127), (17, 128), (33, 1000), (9, 1024), (4, 2048), (7, 4100),
                                 (300, 520), (2, 16384), (1, 40000), (1030, 64), (5, 2056), (3, 8200), (70, 4096), (2, 131072)])
def test_rows(ctx, M, K):
    g = torch.Generator().manual_seed(M * 100003 + K)
    check_rows(ctx, (torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-20, 20, (M, 1), generator=g))).to(BF16))


def test_rows_every_quotient(ctx):
    """Every significand over every other, at every distance that leaves a code, exact ties among them: all codes are the
    exact quotient's."""
    tops, rows = torch.arange(128, 256).float(), []
    for j in range(10):  # x = X 2^-j, for a largest value of 128 to 255
        rows.append((torch.arange(128, 256).float() * 2.0 ** -j).repeat(128, 1))
    x = torch.cat(rows, 1)
    x = torch.where(x <= tops[:, None], x, torch.zeros(()))
    x = torch.cat((x, -x, tops[:, None]), 1)
    for scale in (1.0, 2.0 ** -100, 2.0 ** 119, 2.0 ** -126, 2.0 ** -132):
        check_rows(ctx, (x * scale).to(BF16))


def test_rows_that_are_not_numbers(ctx):
    x = torch.randn(6, 300).to(BF16)
    x[0, 5], x[1, 299], x[2, 0], x[3] = float("nan"), float("inf"), -float("inf"), 0
    q, s = dlp.proj_quantize_rows(ctx, x.cuda())
    assert torch.isnan(s[:3]).all() and float(s[3]) == 0 and not bool(q[:4].any())
    want, ws = ref.quantize_rows(x[4:])
    assert torch.equal(q[4:, :300].cpu().long(), want) and torch.equal(s[4:].cpu(), ws.float())
    y = torch.empty(6, 16, dtype=F32, device="cuda")
    w, sw = dlp.proj_quantize_rows(ctx, torch.randn(16, 300).to(BF16).cuda())
    dlp.proj_run_int(ctx, q, s, w, sw, None, dlp.EPI_NONE, y)
    assert torch.isnan(y[:3]).all() and not bool(y[3].any()) and torch.isfinite(y[4:]).all()


@pytest.mark.parametrize("K,wide,first", [(1000, 1008, 0), (1000, 1001, 0), (1000, 1024, 3), (512, 1024, 8), (4096, 4104, 4),
                                          (8, 9, 1), (2048, 2050, 0)])
def test_rows_strided(ctx, K, wide, first):
    big = torch.randn(37, wide + 8).to(BF16).cuda()
    check_rows(ctx, big[:, first:first + K])


# ------------------------------------------------------------------- product

def integers(M, N, K, seed, lo=-127, hi=127):
    g = torch.Generator().manual_seed(seed)
    X, W = (torch.randint(lo, hi + 1, (r, K), generator=g, dtype=torch.int8) for r in (M, N))
    xs, ws = ((torch.rand(r, generator=g) + 0.1) / 100 for r in (M, N))
    return X, xs, W, ws, torch.randn(N, generator=g).to(BF16)


def run(ctx, X, xs, W, ws, bias, epi, out, stream=None):
    M, N = X.shape[0], W.shape[0]
    guard = 64
    flat = torch.full((guard + M * N + guard,), 7.0, dtype=out, device="cuda")
    Y = flat[guard:guard + M * N].view(M, N)
    dlp.proj_run_int(ctx, X.cuda(), xs.cuda(), W.cuda(), ws.cuda(), None if bias is None else bias.cuda(), epi, Y, stream=stream)
    torch.cuda.synchronize()
    assert bool((flat[:guard] == 7).all()) and bool((flat[guard + M * N:] == 7).all())
    return Y


def check(ctx, M, N, K, epi, out, seed=0, **kw):
    print("int", M, N, K, epi, out, flush=True)
    X, xs, W, ws, bias = integers(M, N, K, seed, **kw)
    close(run(ctx, X, xs, W, ws, bias if epi & 1 else None, epi, out),
          *ref.product(X, xs, W, ws, bias, epi, out))


@pytest.mark.parametrize("M", [1, 2, 5, 8, 9, 16, 17, 31, 32, 33, 48, 64, 65, 100, 128, 129, 200, 256, 257, 300, 512, 700])
def test_rows_of_tokens(ctx, M):
    for i, (N, K) in enumerate(((16, 16), (64, 256), (515, 1008), (256, 2048), (1000, 144), (17, 4112), (1025, 640))):
        check(ctx, M, N, K, (i + M) % 4, (BF16, F32)[(i + M // 3) % 2], seed=M + i)


@pytest.mark.parametrize("M,N,K", [(1, 28672, 1024), (16, 8192, 8192), (64, 4096, 2048), (1, 1024, 8192), (4, 1, 131056),
                                   (2048, 2048, 1024), (1024, 512, 8192), (1111, 2222, 1040), (300, 8200, 512), (4096, 1536, 512)])
@pytest.mark.parametrize("out", [BF16, F32])
def test_sizes(ctx, M, N, K, out):
    check(ctx, M, N, K, 3 if out == BF16 else 1, out, seed=5)


@pytest.mark.parametrize("M,N", [(1, 300), (20, 64), (64, 1000), (300, 300), (600, 600), (1100, 520)])
def test_sums_at_the_ends_of_32_bits(ctx, M, N):
    """Sums of K = 131056 products of one sign, the largest there are, are exact."""
    for K in (16, 131056 if M < 300 else 8192):
        for a, b in ((-128, -128), (-128, 127), (127, 127)):
            X, W = torch.full((M, K), a, dtype=torch.int8), torch.full((N, K), b, dtype=torch.int8)
            Y = run(ctx, X, torch.ones(M), W, torch.ones(N), None, 0, F32)
            assert torch.equal(Y, torch.full((M, N), float(a * b * K), device="cuda"))


@pytest.mark.parametrize("M,N,K", [(1, 64, 256), (33, 100, 256), (300, 700, 1024), (1024, 1024, 512)])
def test_extreme_scales(ctx, M, N, K):
    """Scales whose product with the sum, or with each other, passes the ends of fp32 on the way to a result that does not."""
    X, xs, W, ws, _ = integers(M, N, K, 3)
    for a, b in ((2.0 ** 120, 2.0 ** -125), (2.0 ** -130, 2.0 ** 120), (2.0 ** 127, 2.0 ** -149), (2.0 ** -100, 2.0 ** -60), (2.0 ** 120, 2.0 ** 10)):
        sx, sw = torch.full((M,), a), torch.full((N,), b)
        y, tol = ref.product(X, sx, W, sw, None, 0, F32)
        y = torch.where(y.abs() > 3.5e38, torch.copysign(torch.full_like(y, float("inf")), y), y)
        close(run(ctx, X, sx, W, sw, None, 0, F32), y, tol)
    for bad in (float("nan"), float("inf")):
        sx = xs.clone()
        sx[M // 2] = bad
        Y = run(ctx, X, sx, W, ws, None, 0, F32).cpu()
        assert not torch.isfinite(Y[M // 2]).any()
        keep = torch.arange(M) != M // 2
        close(Y[keep], *(t[keep] for t in ref.product(X, xs, W, ws, None, 0, F32)))


def test_empty(ctx):
    X, xs, W, ws, bias = integers(3, 20, 0, 0)
    for epi in range(4):
        want = torch.zeros(3, 20).double() + (bias.double() if epi & 1 else 0)
        if epi & 2:
            want = torch.nn.functional.gelu(want, approximate="tanh")
        close(run(ctx, X, xs, W, ws, bias, epi, F32), want, 1e-5 * want.abs() + 1e-30)
    for M, N in ((0, 5), (5, 0)):
        X, xs, W, ws, bias = integers(M, N, 64, 0)
        dlp.proj_run_int(ctx, X.cuda(), xs.cuda(), W.cuda(), ws.cuda(), None, 0, torch.empty(M, N, device="cuda"))
        dlp.proj_run_int_dynamic(ctx, torch.empty(M, 64, dtype=BF16, device="cuda"), W.cuda(), ws.cuda(), None, 0,
                                 torch.empty(M, N, device="cuda"))
    q, s = dlp.proj_quantize_rows(ctx, torch.empty(4, 0, dtype=BF16, device="cuda"))
    assert q.shape == (4, 0) and not bool(s.any())


def test_every_split_gives_the_same_bits():
    """How far K is split follows from the workspace; the sum is exact, so the result does not."""
    for M, N, K in ((64, 512, 8192), (128, 256, 16384), (300, 300, 4096), (16, 64, 65536)):
        X, xs, W, ws, bias = integers(M, N, K, 9)
        got = []
        for room in (0, 1 << 16, 1 << 18, 1 << 20, 64 << 20):
            c = dlp.proj_create(0, room)
            got.append(run(c, X, xs, W, ws, bias, 3, F32))
            dlp.proj_destroy(c)
        assert all(torch.equal(g, got[0]) for g in got)


# ------------------------------------------------------------- from bf16 tokens

@pytest.mark.parametrize("M,N,K", [(1, 100, 1000), (1, 1, 8), (1, 8200, 32768), (1, 300, 32769), (2, 515, 8192), (3, 40, 2049), (4, 8192, 8192),
                                   (4, 17, 100), (4, 64, 8193), (5, 64, 2048), (7, 515, 1000), (16, 512, 2048), (33, 64, 33), (300, 515, 1000), (1200, 600, 520),
                                   (5, 40, 1), (64, 1024, 4096)])
def test_dynamic_is_the_two_calls(ctx, M, N, K):
    g = torch.Generator().manual_seed(K)
    X = torch.randn(M, K + 8, generator=g).to(BF16).cuda()[:, N % 3:K + N % 3]
    W, ws = dlp.proj_quantize_rows(ctx, torch.randn(N, K, generator=g).to(BF16).cuda())
    bias = torch.randn(N, generator=g).to(BF16).cuda()
    for epi, out in ((0, F32), (3, BF16)):
        q, s = dlp.proj_quantize_rows(ctx, X)
        two, one = (torch.full((M, N), 5.0, dtype=out, device="cuda") for _ in range(2))
        dlp.proj_run_int(ctx, q, s, W, ws, bias, epi, two)
        dlp.proj_run_int_dynamic(ctx, X, W, ws, bias, epi, one)
        assert torch.equal(one, two)
        want, ss = ref.quantize_rows(X.cpu())
        close(one, *ref.product(want, ss.float(), W.cpu()[:, :K], ws.cpu(), bias.cpu(), epi, out))


def test_dynamic_in_a_small_workspace():
    """A workspace that holds a few rows at a time gives the same result; one that holds none is refused."""
    M, N, K = 50, 70, 1000
    X = torch.randn(M, K).to(BF16).cuda()
    big = dlp.proj_create(0)
    W, ws = dlp.proj_quantize_rows(big, torch.randn(N, K).to(BF16).cuda())
    want = torch.empty(M, N, device="cuda")
    dlp.proj_run_int_dynamic(big, X, W, ws, None, 0, want)
    for room in (1012 + 512 + 256, 4096, 9 * 1024, 40 * 1024):
        c = dlp.proj_create(0, room)
        Y = torch.zeros(M, N, device="cuda")
        dlp.proj_run_int_dynamic(c, X, W, ws, None, 0, Y)
        torch.cuda.synchronize()
        assert torch.equal(Y, want)
        dlp.proj_destroy(c)
    for room in (0, 1024):
        c = dlp.proj_create(0, room)
        Y = torch.full((M, N), 3.0, device="cuda")
        with pytest.raises(dlp.ProjError) as e:
            dlp.proj_run_int_dynamic(c, X, W, ws, None, 0, Y)
        torch.cuda.synchronize()
        assert e.value.status == dlp.PROJ_ERR_NO_MEMORY and bool((Y == 3).all())
        dlp.proj_destroy(c)
    dlp.proj_destroy(big)


@pytest.mark.parametrize("M,N,K", [(1, 256, 1024), (40, 300, 1000), (300, 700, 2048), (1100, 1300, 1024)])
def test_graph_replays_follow_their_inputs(ctx, M, N, K):
    W, ws = dlp.proj_quantize_rows(ctx, torch.randn(N, K).to(BF16).cuda())
    X = torch.randn(M, K).to(BF16).cuda()
    Y = torch.empty(M, N, dtype=BF16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dlp.proj_run_int_dynamic(ctx, X, W, ws, None, dlp.EPI_GELU_TANH, Y)
    for i in range(3):
        X.copy_(torch.randn(M, K))
        Y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager = torch.empty_like(Y)
        dlp.proj_run_int_dynamic(ctx, X, W, ws, None, dlp.EPI_GELU_TANH, eager)
        torch.cuda.synchronize()
        assert torch.equal(Y, eager) and bool(Y.any())


def test_another_stream(ctx):
    X, xs, W, ws, bias = integers(70, 900, 2048, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = run(ctx, X, xs, W, ws, bias, 1, F32)
    assert torch.equal(run(ctx, X, xs, W, ws, bias, 1, F32, stream=side), want)
    with torch.cuda.stream(side):
        check_rows(ctx, torch.randn(9, 500).to(BF16).cuda(), stream=side.cuda_stream)


def test_refusals_in_python(ctx):
    X, xs, W, ws, bias = (t.cuda() for t in integers(4, 32, 64, 0))
    Y = torch.empty(4, 32, device="cuda")
    for f in (lambda: dlp.proj_run_int(ctx, X, xs, W[:, :48], ws, None, 0, Y), lambda: dlp.proj_run_int(ctx, X.short(), xs, W, ws, None, 0, Y),
              lambda: dlp.proj_run_int(ctx, X, xs.double(), W, ws, None, 0, Y), lambda: dlp.proj_run_int(ctx, X, xs, W, ws[:31], None, 0, Y),
              lambda: dlp.proj_run_int(ctx, X, xs, W, ws, bias[:31], 1, Y), lambda: dlp.proj_run_int(ctx, X, xs, W, ws, None, 0, Y.t()),
              lambda: dlp.proj_run_int(ctx, X, xs, W, ws, None, 0, Y.half()), lambda: dlp.proj_run_int(ctx, X.cpu(), xs, W, ws, None, 0, Y),
              lambda: dlp.proj_run_int_dynamic(ctx, torch.empty(4, 65, dtype=BF16, device="cuda"), W, ws, None, 0, Y),
              lambda: dlp.proj_quantize_rows(ctx, Y), lambda: dlp.proj_quantize_rows(ctx, bias),
              lambda: dlp.proj_quantize_rows(ctx, torch.empty(4, 60, dtype=BF16, device="cuda"), q=X[:, :60])):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: dlp.proj_run_int(ctx, torch.zeros(4, 40, dtype=torch.int8, device="cuda"), xs, torch.zeros(32, 40, dtype=torch.int8, device="cuda"), ws, None, 0, Y),
              lambda: dlp.proj_run_int(ctx, torch.zeros(4 * 64 + 8, dtype=torch.int8, device="cuda")[8:].view(4, 64), xs, W, ws, None, 0, Y),
              lambda: dlp.proj_run_int(ctx, X, xs, W, ws, None, 1, Y)):
        with pytest.raises(dlp.ProjError) as e:
            f()
        assert e.value.status == dlp.PROJ_ERR_INVALID_ARG
