"""The example's decoding block (4-bit projection, append, attention, 4-bit
projection in one replayed graph) against the same steps in 64 bits on the
CPU, and the large tiles of the 4-bit projection."""
import importlib.util
import os

import pytest
import torch

from tests import decode_reference as ref
from tests.test_gpu_quant import make, run

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_attention.py")
    spec = importlib.util.spec_from_file_location("decode_attention", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("fp8", [False, True])
def test_decoding_steps(fp8):
    batch, hidden, heads, kv, dim, steps = 3, 512, 4, 2, 64, 20
    block = example().DecodeBlock(batch, hidden, heads, kv, dim, steps, page=8, fp8=fp8, seed=1)
    W = [ref.weights(c.cpu(), s.cpu(), z.cpu(), 128) for c, s, z in (block.qkv_weights, block.out_weights)]
    keys = torch.zeros(batch, 0, kv, dim, dtype=torch.float64)
    values = keys.clone()
    g = torch.Generator().manual_seed(2)
    for t in range(steps):
        x = torch.randn(batch, hidden, generator=g).to(BF16)
        got = block.step(x.cuda()).cpu().double()
        qkv = (x.double() @ W[0].t()).view(batch, -1, dim)
        row = block.rope.cpu().double()[t]
        cos, sin = row[:dim // 2], row[dim // 2:]
        turned = ref.rotate(qkv[:, :heads + kv], cos, sin, dim, False)
        keys = torch.cat((keys, turned[:, None, heads:]), 1)
        values = torch.cat((values, qkv[:, None, heads + kv:]), 1)
        q = turned[:, :heads].view(batch, kv, heads // kv, dim)
        w = torch.softmax(torch.einsum("bkhd,btkd->bkht", q, keys) * dim ** -0.5, -1)
        o = torch.einsum("bkht,btkd->bkhd", w, values).reshape(batch, -1)
        want = o @ W[1].t()
        # keys, values, queries and outputs of unit size rounded to bf16 (to e4m3: half a step of 2^-4) on their way;
        # the output sums heads * dim of them with weights of unit norm
        step = (2.0 ** -4 if fp8 else 2.0 ** -8) * 3
        assert float((got - want).norm() / want.norm()) < step, (t, float((got - want).norm() / want.norm()))
    block.close()


@pytest.mark.parametrize("M,N,K", [(600, 7000, 520), (1000, 4200, 264), (130, 17000, 256)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_large_tiles(ctx, M, N, K, group):
    """Enough rows and columns for the 128 x 256 tiles, in sizes that they do not divide."""
    for zeros, sdt, epi, out in ((True, BF16, 1, F32), (False, F32, 0, BF16)):
        X, codes, scales, z, b = make(M, N, K, group, zeros, sdt, epi & 1, M + N + K)
        want, tol = ref.quant(X, codes, scales, z, group, b, epi, out)
        ref.close(run(ctx, X, codes, scales, z, group, b, epi, out), want, tol)
