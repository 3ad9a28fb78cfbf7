"""Decoding operators beyond what one launch has threads for: more outputs of
unaligned rows, more groups to quantise, more sequences times heads to attend
than 2^24 workgroups or 2^26 waves."""
import pytest
import torch

import dense_linear_projection_amd as dlp
from tests import decode_reference as ref
from tests.test_gpu_quant import BF16, F32

pytestmark = pytest.mark.gpu


def test_unaligned_rows(ctx):
    M, N, K = 8200, 8200, 8
    g = torch.Generator().manual_seed(1)
    X = torch.randint(-3, 4, (M, K), generator=g).to(BF16)
    codes, scales = ref.pack(torch.randint(0, 16, (N, K), generator=g)), 2.0 ** torch.randint(-1, 2, (N, 1), generator=g).float()
    flat = torch.zeros(M * K + 1, dtype=BF16, device="cuda")
    flat[1:] = X.cuda().view(-1)
    Y = torch.full((M, N), float("nan"), device="cuda")
    dlp.proj_run_quant(ctx, flat[1:].view(M, K), codes.cuda(), scales.cuda(), None, 32, None, 0, Y)
    want = X.float().cuda() @ ref.weights(codes, scales, None, 32).float().cuda().t()     # whole halves: exact in fp32
    assert torch.equal(Y, want)


def test_quantize_and_pack(ctx):
    N, tail = (1 << 26) + 9, 70
    W = torch.randn(N, 8, device="cuda", dtype=BF16)
    codes, scales, zeros = dlp.proj_quantize_weights(ctx, W, 32)
    for rows in (slice(0, tail), slice(N - tail, N)):
        few = dlp.proj_quantize_weights(ctx, W[rows].contiguous(), 32)
        for got, want in zip((codes, scales, zeros), few):
            assert torch.equal(got[rows], want)
    assert int((scales == 0).sum()) == 0


def test_many_sequences_of_many_heads(ctx):
    """One token each: every head's result is its value."""
    B, H, D = 20000, 1024, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(3, H, 2, D, generator=g, device="cuda").to(BF16) for _ in range(2))
    q = torch.randn(B, H, D, device="cuda", dtype=BF16)
    tables = torch.randint(0, 3, (B, 1), generator=g, device="cuda", dtype=torch.int32)
    lengths = torch.randint(0, 2, (B,), generator=g, device="cuda", dtype=torch.int32)
    out = torch.full((B, H, D), float("nan"), device="cuda", dtype=BF16)
    dlp.proj_kv_attend(ctx, dlp.kv_cache(k, v), q, tables, lengths, 0.125, out)
    for i in range(0, B, 2000):
        part = slice(i, i + 2000)
        want = torch.where(lengths[part, None, None] > 0, v[tables[part, 0].long(), :, 0], torch.zeros((), device="cuda", dtype=BF16))
        assert torch.equal(out[part], want)
