"""4-bit projection where numbers end: infinities and NaN in X, sums that pass
the largest float on their way, X of one sign, on every kernel and alignment,
against the definition in 64 bits."""
import math

import pytest
import torch

import dense_linear_projection_amd as dlp
from tests import decode_reference as ref
from tests.test_gpu_quant import BF16, F32, make, run

pytestmark = pytest.mark.gpu

# rows, columns, K: waves over K, small tiles, small tiles split over K, large tiles; each with whole and ragged steps
SHAPES = [(1, 70, 1024), (5, 70, 1000), (20, 100, 1024), (40, 300, 512), (40, 70, 2056), (64, 130, 8192), (600, 7000, 264)]


def bound(X, codes, scales, group, K):
    """At most 47 |x| s a term, every one of them rounded on its way, and the sum's own."""
    size = 47.0 * (X.double().abs() @ scales.double().abs()[:, torch.arange(K) // group].t())
    return ref.EPS32 * size


def by_definition(X, codes, scales, z, group):
    """The products summed one by one where X has infinities: torch's product gives those no fixed meaning."""
    W = ref.weights(codes, scales, z, group)
    return torch.stack([(x[None] * W).sum(1) for x in X.double()])


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("offset", [0, 1])
def test_infinities(ctx, M, N, K, group, offset):
    """An infinite x gives infinity, of the sign of its weight, or NaN where the
    weight is zero or a second one has the other sign; its row alone."""
    for zeros, sdt in ((True, BF16), (False, F32)):
        X, codes, scales, z, _ = make(M, N, K, group, zeros, sdt, False, M + N + K + group)
        want, tol = ref.quant(X, codes, scales, z, group, None, 0, F32)
        odd = sorted({0, M // 2, M - 1})
        X[odd[0], K - 3] = math.inf
        X[odd[-1], 5] = -math.inf
        X[odd[len(odd) // 2], K // 2], X[odd[len(odd) // 2], 9] = math.inf, math.inf
        want[odd], tol[odd] = by_definition(X[odd], codes, scales, z, group), 0.0
        got = run(ctx, X, codes, scales, z, group, None, 0, F32, offset=offset)
        assert 0 < int(torch.isinf(want).sum())
        ref.close(got, want, tol)


@pytest.mark.parametrize("M,N,K", SHAPES[:-1])
@pytest.mark.parametrize("offset", [0, 1])
def test_sums_that_pass_the_largest_float(ctx, M, N, K, offset):
    """X of 3e37: times 16 + 15 a code, or a group of them, it is past the
    largest float; times the weights, about 1e-6, it is not."""
    for zeros, sdt, group in ((True, BF16, 64), (False, F32, 32)):
        X, codes, scales, z, _ = make(M, N, K, group, zeros, sdt, False, M + K)
        X = (X.sign() * 3e37).to(BF16)
        scales = (scales.double() * 1e-6).to(sdt)
        want = X.double() @ ref.weights(codes, scales, z, group).t()
        got = run(ctx, X, codes, scales, z, group, None, 0, F32, offset=offset)
        ref.close(got, want, 8 * bound(X, codes, scales, group, K))


@pytest.mark.parametrize("M", [1, 20, 64, 300])
def test_epilogue_of_infinities(ctx, M):
    """Bias and output type apply to an infinity as to a number."""
    X, codes, scales, z, b = make(M, 100, 512, 64, True, BF16, True, M)
    X[0, 77] = math.inf
    want = by_definition(X[:1], codes, scales, z, 64) + b.double()
    for out in (F32, BF16):
        got = run(ctx, X, codes, scales, z, 64, b, 1, out)[:1]
        ref.close(got, want, torch.zeros_like(want))


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("sdt", [BF16, F32])
@pytest.mark.parametrize("odd", [math.nan, math.inf, -math.inf])
def test_quantize_keeps_what_is_not_finite_visible(ctx, zeros, sdt, odd):
    """A group with such a weight is NaN as a whole; the others are as without it."""
    g = torch.Generator().manual_seed(31)
    W = torch.randn(6, 136, generator=g).to(BF16)
    before = [t if t is None else t.cpu() for t in dlp.proj_quantize_weights(ctx, W.cuda(), 64, zeros, sdt)]
    W[1, 3], W[4, 64 + 63], W[5, 135] = odd, odd, odd          # the last in a short group
    after = [t if t is None else t.cpu() for t in dlp.proj_quantize_weights(ctx, W.cuda(), 64, zeros, sdt)]
    want, got = ref.weights(*before, 64), ref.weights(*after, 64)
    want[1, :64] = want[4, 64:128] = want[5, 128:] = math.nan
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got[~torch.isnan(want)], want[~torch.isnan(want)])


@pytest.mark.parametrize("sdt", [BF16, F32])
def test_quantize_weights_at_both_ends(ctx, sdt):
    """A range of twice the largest float: every weight within half a scale, and what the scale's rounding moves."""
    g = torch.Generator().manual_seed(32)
    W = (torch.rand(3, 64, generator=g).double() * 6.6e38 - 3.3e38).to(BF16)
    W[:, 0], W[:, 1] = 3.3e38, -3.3e38
    codes, scales, z = dlp.proj_quantize_weights(ctx, W.cuda(), 64, True, sdt)
    assert torch.isfinite(scales).all()
    got, s = ref.weights(codes.cpu(), scales.cpu(), z.cpu(), 64), scales.cpu().double()
    assert float(((got - W.double()).abs() / s).max()) <= 1.0 + 16 * ref.HALF[sdt]


def stream_of(t):
    """The stream that the allocator keeps a tensor's memory for."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]


@pytest.mark.parametrize("as_handle", [False, True])
def test_registered_weights_belong_to_their_stream(ctx, as_handle):
    """Made on a stream, codes and scales are in its memory: freed, they go to
    later work of that stream, not to another that does not wait for it."""
    s = torch.cuda.Stream()
    stream = s.cuda_stream if as_handle else s
    W = torch.randn(640, 1024, device="cuda").to(BF16)
    q = torch.randint(0, 16, (640, 1024), device="cuda", dtype=torch.uint8)
    s.wait_stream(torch.cuda.current_stream())
    made = [t for t in dlp.proj_quantize_weights(ctx, W, 32, stream=stream)] + [dlp.proj_pack_codes(ctx, q, stream=stream)]
    assert [stream_of(t) for t in made] == [s.cuda_stream] * 4
    assert [stream_of(t) for t in dlp.proj_quantize_weights(ctx, W, 32)] == [torch.cuda.current_stream().cuda_stream] * 3
    with torch.cuda.stream(s):
        assert [stream_of(t) for t in dlp.proj_quantize_weights(ctx, W, 32, stream=0)] == [0] * 3
    s.synchronize()
    for a, b in zip(made, dlp.proj_quantize_weights(ctx, W, 32) + (dlp.proj_pack_codes(ctx, q),)):
        assert torch.equal(a, b)
