"""4-bit projection on the GPU against its 64-bit form: every group size, scale
and output type, epilogue, sizes from one to many rows, columns and words,
odd ones among them; exact where sums are whole numbers; its registration
calls; its refusals."""
import pytest
import torch

import dense_linear_projection_amd as dlp
from tests import decode_reference as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def make(M, N, K, group, zeros, sdt, bias, seed):
    g = torch.Generator().manual_seed(seed)
    G = -(-K // group)
    X = torch.randn(M, K, generator=g).to(BF16)
    codes = ref.pack(torch.randint(0, 16, (N, K), generator=g))
    scales = (torch.rand(N, G, generator=g) + 0.5).div(max(1, K) ** 0.5).to(sdt)
    z = torch.randint(0, 16, (N, G), generator=g).to(torch.uint8) if zeros else None
    b = torch.randn(N, generator=g).to(BF16) if bias else None
    return X, codes, scales, z, b


def run(ctx, X, codes, scales, z, group, b, epi, out, offset=0, stream=None):
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    if offset:                                   # X one element past a 16-byte boundary
        flat = torch.zeros(X.numel() + offset, dtype=BF16, device="cuda")
        flat[offset:] = X.cuda().reshape(-1)
        x = flat[offset:].view(X.shape)
    else:
        x = X.cuda()
    Y = torch.full((X.shape[0], codes.shape[0]), float("nan"), dtype=out, device="cuda")
    dlp.proj_run_quant(ctx, x, dev(codes), dev(scales), dev(z), group, dev(b), epi, Y, stream=stream)
    torch.cuda.synchronize()
    return Y


SHAPES = [(1, 1, 8), (1, 16, 32), (1, 1024, 8192), (2, 33, 40), (3, 515, 1000), (5, 100, 1024), (7, 257, 2056),
          (8, 64, 4096), (15, 300, 264), (16, 1000, 1536), (17, 96, 512), (31, 130, 1160), (33, 515, 2048),
          (64, 1029, 1024), (65, 200, 640), (100, 48, 4104), (129, 777, 384), (300, 130, 1000), (513, 1100, 256)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_matches_reference(ctx, M, N, K, group):
    for i, (zeros, sdt, epi, out) in enumerate(((True, BF16, 0, F32), (False, F32, 1, F32), (True, F32, 3, BF16),
                                                (False, BF16, 2, F32))):
        X, codes, scales, z, b = make(M, N, K, group, zeros, sdt, epi & 1, 100 * i + M + N + K)
        want, tol = ref.quant(X, codes, scales, z, group, b, epi, out)
        ref.close(run(ctx, X, codes, scales, z, group, b, epi, out), want, tol)


@pytest.mark.parametrize("M,N,K,group", [(1, 512, 8192, 128), (4, 100, 4096, 32), (16, 640, 8192, 64), (64, 515, 4096, 128),
                                         (200, 300, 2048, 32), (16, 31, 1000, 64), (1024, 256, 1024, 128)])
def test_whole_numbers_are_exact(ctx, M, N, K, group):
    """Whole X, scales that are powers of two: every product and sum is exact
    in fp32 in any order, so the result is the exact one, in every run."""
    g = torch.Generator().manual_seed(M + K)
    X = torch.randint(-3, 4, (M, K), generator=g).to(BF16)
    codes = ref.pack(torch.randint(0, 16, (N, K), generator=g))
    G = -(-K // group)
    scales = 2.0 ** torch.randint(-1, 2, (N, G), generator=g).float()
    z = torch.randint(0, 16, (N, G), generator=g).to(torch.uint8)
    want, _ = ref.quant(X, codes, scales, z, group, None, 0, F32)
    for _ in range(3):
        assert torch.equal(run(ctx, X, codes, scales, z, group, None, 0, F32).cpu().double(), want)


def test_unaligned_operands(ctx):
    for M, K in ((3, 1024), (40, 512)):
        X, codes, scales, z, b = make(M, 70, K, 64, True, BF16, True, 5)
        want, tol = ref.quant(X, codes, scales, z, 64, b, 1, F32)
        ref.close(run(ctx, X, codes, scales, z, 64, b, 1, F32, offset=1), want, tol)
        # codes on a 4-byte boundary only
        flat = torch.zeros(codes.numel() + 1, dtype=torch.int32, device="cuda")
        flat[1:] = codes.cuda().reshape(-1)
        Y = torch.empty(M, 70, device="cuda")
        dlp.proj_run_quant(ctx, X.cuda(), flat[1:].view(codes.shape), scales.cuda(), z.cuda(), 64, b.cuda(), 1, Y)
        ref.close(Y, want, tol)


def test_same_bits_every_run_and_on_another_stream(ctx):
    X, codes, scales, z, b = make(16, 2048, 8192, 128, True, BF16, True, 9)
    first = run(ctx, X, codes, scales, z, 128, b, 1, F32)
    s = torch.cuda.Stream()
    assert torch.equal(run(ctx, X, codes, scales, z, 128, b, 1, F32, stream=s), first)
    assert torch.equal(run(ctx, X, codes, scales, z, 128, b, 1, F32), first)


def test_infinite_and_nan_inputs_reach_their_rows_only(ctx):
    X, codes, scales, z, b = make(20, 100, 1024, 64, True, BF16, False, 11)
    want, tol = ref.quant(X, codes, scales, z, 64, None, 0, F32)
    X[3, 500] = float("nan")
    Y = run(ctx, X, codes, scales, z, 64, None, 0, F32)
    assert torch.isnan(Y[3]).all()
    keep = [i for i in range(20) if i != 3]
    ref.close(Y[keep], want[keep], tol[keep])


def test_no_workspace(ctx):
    """A context without a workspace gives results too (nothing is split)."""
    small = dlp.proj_create(0, 0)
    try:
        X, codes, scales, z, b = make(4, 64, 8192, 128, True, BF16, True, 13)
        want, tol = ref.quant(X, codes, scales, z, 128, b, 1, F32)
        ref.close(run(small, X, codes, scales, z, 128, b, 1, F32), want, tol)
    finally:
        dlp.proj_destroy(small)


def test_empty_sizes(ctx):
    X, codes, scales, z, b = make(4, 30, 64, 32, True, BF16, True, 15)
    assert run(ctx, X[:0], codes, scales, z, 32, b, 1, F32).shape == (0, 30)
    assert run(ctx, X, codes[:0], scales[:0], z[:0], 32, b[:0], 1, F32).shape == (4, 0)
    Y = run(ctx, X[:, :0], codes[:, :0], scales[:, :0], z[:, :0], 32, b, 1, F32)
    assert torch.equal(Y.cpu(), b.float().expand(4, 30))


@pytest.mark.parametrize("M,N,K", [(1, 512, 4096), (16, 1000, 2048), (40, 300, 512), (300, 200, 1024)])
def test_graph_replays(ctx, M, N, K):
    X, codes, scales, z, b = make(M, N, K, 128, True, BF16, True, 17)
    x, args = X.cuda(), [t.cuda() for t in (codes, scales, z)]
    bias, Y = b.cuda(), torch.empty(M, N, device="cuda")
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        dlp.proj_run_quant(ctx, x, *args, 128, bias, 1, Y)
    for i in range(4):
        fresh = make(M, N, K, 128, True, BF16, True, 30 + i)[0]
        x.copy_(fresh)
        Y.fill_(float(i))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, run(ctx, fresh, codes, scales, z, 128, b, 1, F32))


@pytest.mark.parametrize("N,K", [(1, 8), (7, 40), (64, 1024), (33, 1000)])
def test_pack_codes(ctx, N, K):
    q = torch.randint(0, 256, (N, K), dtype=torch.uint8)
    assert torch.equal(dlp.proj_pack_codes(ctx, q.cuda()).cpu(), ref.pack(q & 15))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("sdt", [BF16, F32])
def test_quantize_weights(ctx, group, zeros, sdt):
    """Every weight is within half a scale of its 4-bit form, but for what the
    rounded scale and zero point move: the scale's rounding moves the range's
    ends by 16 times its error, the zero point's shifts them by up to half a
    scale, where codes clamp."""
    g = torch.Generator().manual_seed(group)
    W = (torch.randn(37, 1000, generator=g) * 0.02).to(BF16)
    W[3, :group] = 0
    W[4, :group] = W[4, :group].abs() + 0.01
    codes, scales, z = dlp.proj_quantize_weights(ctx, W.cuda(), group, zeros, sdt)
    assert (z is None) == (not zeros) and scales.dtype == sdt
    got = ref.weights(codes.cpu(), scales.cpu(), None if z is None else z.cpu(), group)
    s = scales.cpu().double()[:, torch.arange(1000) // group]
    assert float(((got - W.double()).abs() - s * (1.0 + 16 * ref.HALF[sdt])).max()) <= 1e-12
    assert float(((got - W.double()).abs() / s.clamp(min=1e-9)).mean()) < 0.3     # a quarter where nothing clamps
    assert torch.equal(got[3, :group], torch.zeros(group).double())
    if not zeros:
        c = ref.unpack(codes.cpu())
        assert int(c[:3].min()) >= 0 and int(c.max()) <= 15


def test_refusals(ctx):
    X, codes, scales, z, b = make(4, 30, 64, 32, True, BF16, True, 19)
    x, c, s, zz, bb = (t.cuda() for t in (X, codes, scales, z, b))
    Y = torch.empty(4, 30, device="cuda")
    ok = dict(X=x, codes=c, scales=s, zeros=zz, group=32, bias=bb, epilogue=1, Y=Y)

    def refused(error=ValueError, **kw):
        with pytest.raises(error):
            dlp.proj_run_quant(ctx, **{**ok, **kw})

    dlp.proj_run_quant(ctx, **ok)
    refused(X=X)
    refused(X=x.float())
    refused(X=x[:, :56].contiguous())
    refused(codes=c[:, ::2])
    refused(scales=s[:, :1].contiguous())
    refused(scales=s.half())
    refused(zeros=zz[:, :1].contiguous())
    refused(zeros=zz.int())
    refused(group=16)
    refused(bias=bb[:4])
    refused(Y=Y[:3])
    refused(Y=Y.half())
    refused(dlp.ProjError, epilogue=4)
    refused(dlp.ProjError, epilogue=1, bias=None)
    refused(ValueError, X=x.t())
    flat = torch.empty(4 * 64 * 2 // 4, device="cuda")
    refused(dlp.ProjError, X=flat.view(BF16).view(4, 64), Y=flat[:120].view(4, 30))
