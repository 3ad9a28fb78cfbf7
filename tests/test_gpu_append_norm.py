"""The append whose query and key heads are normed, on the GPU against its
64-bit form: every head size, pairing and rotation, weights of each type and of
each head, heads near the ends of bf16, places outside, graphs and streams."""
import pytest
import torch

import dense_linear_projection_amd as dlp
from tests import layer_reference as ref
from tests.decode_reference import close
from tests.test_gpu_kv import make_cache

pytestmark = pytest.mark.gpu
BF16, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def weights(Hq, H, D, dtype, per_head, which, g):
    w = [(1 + 0.3 * torch.randn(*((h, D) if per_head else (D,)), generator=g)).to(dtype) for h in (Hq, H)]
    return [w[0] if "q" in which else None, w[1] if "k" in which else None]


def run_append(ctx, T, Hq, H, D, rot, page, dtype, layout, interleaved, seed, wtype=BF16, per_head=False, which="qk", eps=1e-6, pad=0,
               slots=None, positions=None, qkv=None):
    print("append_norm", T, Hq, H, D, rot, page, dtype, layout, interleaved, wtype, per_head, which, flush=True)
    g = torch.Generator().manual_seed(seed)
    scales = (0.05, 0.03125) if dtype == FP8 else (1.0, 1.0)
    pages = -(-T // page) + 2
    k, v, cache = make_cache(pages, H, page, D, dtype, layout, g, scales)
    if qkv is None:
        qkv = (torch.randn(T, Hq + 2 * H, D, generator=g) * torch.exp2(torch.randint(-8, 8, (T, Hq + 2 * H, 1), generator=g))).flatten(1).to(BF16)
    qn, kn = weights(Hq, H, D, wtype, per_head, which, g)
    rope = torch.randn(50, rot, generator=g)
    if positions is None:
        positions = torch.randint(0, 50, (T,), generator=g).to(torch.int32)
    if slots is None:
        slots = torch.randperm(pages * page, generator=g)[:T]
        slots[T - pad:] = -1
    want, tol = ref.append_norm(k, v, qkv, qn, kn, eps, rope, positions, slots, Hq, scales, interleaved)
    wide = torch.zeros(T, qkv.shape[1] + 8, dtype=BF16, device="cuda")
    wide[:, :-8] = qkv.cuda()
    q = torch.full((T, Hq, D), 7.0, dtype=BF16, device="cuda") if Hq else None
    dev = [None if w is None else w.cuda() for w in (qn, kn)]
    dlp.proj_kv_append_norm(ctx, cache, wide[:, :-8], *dev, eps, rope.cuda(), positions.cuda(), slots.cuda(), q, interleaved=interleaved)
    torch.cuda.synchronize()
    if Hq:
        close(q, want[0], tol[0])
    bits = torch.uint8 if dtype == FP8 else torch.int16
    stored = torch.zeros(pages * page, dtype=torch.bool)
    known = (positions >= 0) & (positions < 50) if rot else torch.ones(T, dtype=torch.bool)
    stored[slots[known & (slots >= 0) & (slots < pages * page)]] = True
    for got, before, w, t in ((cache.k, k, want[1], tol[1]), (cache.v, v, want[2], tol[2])):
        close(got, w, t)
        kept = ~stored.view(pages, page)        # slots that no token went to hold what they held, to the bit
        a, b = (x.transpose(1, 2)[kept].contiguous().view(bits) for x in (got.cpu(), before))
        assert torch.equal(a, b)
    return q, cache


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_norm(ctx, dtype, layout, interleaved):
    for i, (T, Hq, H, D, rot, page) in enumerate(((1, 8, 2, 64, 64, 16), (5, 4, 4, 128, 128, 16), (33, 15, 5, 80, 32, 32),
                                                  (70, 6, 1, 96, 96, 16), (9, 0, 3, 192, 64, 64), (17, 5, 1, 256, 256, 128),
                                                  (12, 2, 2, 80, 80, 1), (8, 3, 3, 64, 34, 4), (6, 2, 1, 128, 2, 8),
                                                  (7, 4, 2, 64, 0, 16), (100, 20, 4, 128, 64, 64), (3, 7, 7, 96, 50, 16))):
        run_append(ctx, T, Hq, H, D, rot, page, dtype, layout, interleaved, 10 * i, (BF16, F32)[i % 2], i % 3 == 1,
                   ("qk", "q", "k")[i % 4 % 3] if Hq else "k", (1e-6, 0.0, 1e-2)[i % 3], T // 5)


@pytest.mark.parametrize("rot,interleaved", [(128, False), (64, True), (34, False), (34, True), (0, False)])
def test_many_tokens(ctx, rot, interleaved):
    """Enough tokens that a thread takes several of them, a number that does not divide evenly."""
    run_append(ctx, 5003, 20, 4, 128, rot, 64, FP8, "nhd", interleaved, 77, F32, True, pad=700)
    run_append(ctx, 4999, 20, 4, 80, min(rot, 80), 64, BF16, "hnd", interleaved, 78, BF16, False, pad=7)


def test_heads_at_the_ends_of_bf16(ctx):
    """Heads whose squares or their sum pass the ends of fp32 are normed like any other."""
    T, Hq, H, D = 6, 2, 1, 128
    x = torch.randn(T, Hq + 2 * H, D)
    size = torch.tensor([3e37, 1e25, 1.0, 1e-25, 1e-38, 2e-40])
    qkv = (x.clamp(-5, 5) * size[:, None, None]).flatten(1).to(BF16)
    qkv[:, -D:] = torch.randn(T, D).to(BF16)
    for eps in (0.0, 1e-6, 1e-38):
        run_append(ctx, T, Hq, H, D, 128, 16, BF16, "hnd", False, 5, eps=eps, qkv=qkv)
        run_append(ctx, T, Hq, H, D, 34, 16, BF16, "hnd", True, 5, F32, eps=eps, qkv=qkv)


def test_heads_of_zeros_and_of_no_numbers(ctx):
    T, Hq, H, D = 3, 2, 1, 96
    qkv = torch.randn(T, Hq + 2 * H, D).to(BF16)
    qkv[0, 0], qkv[1, 1, 3], qkv[2, 2, 5] = 0, float("nan"), float("inf")
    k, v, cache = make_cache(1, H, 16, D, BF16, "hnd", torch.Generator().manual_seed(0))
    q = torch.empty(T, Hq, D, dtype=BF16, device="cuda")
    w = torch.ones(D).cuda()
    rope = torch.cat((torch.ones(1, 16), torch.zeros(1, 16)), 1).cuda()
    at = torch.zeros(T, dtype=torch.int32).cuda(), torch.arange(T).cuda()
    dlp.proj_kv_append_norm(ctx, cache, qkv.flatten(1).cuda(), w, w, 1e-6, rope, *at, q)
    assert not bool(q[0, 0].any()) and bool(torch.isnan(q[1, 1]).all()) and bool(torch.isfinite(q[1, 0]).all())
    assert bool(torch.isnan(cache.k[0, 0, 2, 5])) and bool(torch.isfinite(cache.k[0, 0, :2]).all())
    dlp.proj_kv_append_norm(ctx, cache, qkv.flatten(1).cuda(), w, w, 0.0, rope, *at, q)
    assert bool(torch.isnan(q[0, 0]).all()) and bool(torch.isfinite(q[0, 1]).all())


def test_places_outside(ctx):
    T = 9
    slots = torch.tensor([0, 48, 5, 1 << 40, -7, 47, 3, 2 ** 62, 10])       # 3 pages of 16
    positions = torch.tensor([0, 1, 50, 2, 3, -1, 49, 4, 2 ** 31 - 1], dtype=torch.int32)
    for dtype in (BF16, FP8):
        run_append(ctx, T, 4, 2, 128, 128, 16, dtype, "hnd", False, 3, slots=slots, positions=positions)
        run_append(ctx, T, 4, 2, 80, 24, 16, dtype, "nhd", True, 4, slots=slots, positions=positions)


def test_without_weights_it_is_the_plain_append(ctx):
    g = torch.Generator().manual_seed(2)
    qkv, rope = torch.randn(40, 8 * 128, generator=g).to(BF16).cuda(), torch.randn(50, 64, generator=g).cuda()
    pos, slots = torch.randint(0, 50, (40,), generator=g).to(torch.int32).cuda(), torch.randperm(48, generator=g)[:40].cuda()
    got = []
    for f, w in ((dlp.proj_kv_append, ()), (dlp.proj_kv_append_norm, (None, None, 1e-6))):
        _, _, cache = make_cache(3, 2, 16, 128, BF16, "hnd", torch.Generator().manual_seed(1))
        q = torch.empty(40, 4, 128, dtype=BF16, device="cuda")
        f(ctx, cache, qkv, *w, rope, pos, slots, q)
        got.append((q, cache.k, cache.v))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_graph_and_stream(ctx):
    T, Hq, H, D = 20, 8, 2, 128
    g = torch.Generator().manual_seed(3)
    _, _, cache = make_cache(4, H, 16, D, BF16, "hnd", g)
    qkv, rope = torch.randn(T, (Hq + 2 * H) * D, generator=g).to(BF16).cuda(), torch.randn(64, D, generator=g).cuda()
    w = [(1 + 0.1 * torch.randn(D, generator=g)).cuda() for _ in range(2)]
    pos, slots = torch.arange(T, dtype=torch.int32).cuda(), torch.arange(T).cuda()
    q = torch.empty(T, Hq, D, dtype=BF16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dlp.proj_kv_append_norm(ctx, cache, qkv, *w, 1e-6, rope, pos, slots, q)
    for i in range(3):
        qkv.copy_(torch.randn(qkv.shape, generator=g))
        slots.copy_(torch.randperm(64, generator=g)[:T])
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in (q, cache.k, cache.v)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        q.zero_()
        torch.cuda.synchronize()
        dlp.proj_kv_append_norm(ctx, cache, qkv, *w, 1e-6, rope, pos, slots, q, stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, (q, cache.k, cache.v)))


def test_refusals_in_python(ctx):
    _, _, cache = make_cache(2, 2, 16, 64, BF16, "hnd", torch.Generator().manual_seed(0))
    qkv, rope = torch.zeros(3, 8 * 64, dtype=BF16, device="cuda"), torch.zeros(4, 64, device="cuda")
    at = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.arange(3).cuda()
    w = torch.ones(64, device="cuda")
    for qn, kn in ((w, w.bfloat16()), (w, torch.ones(2, 64, device="cuda")), (torch.ones(2, 64, device="cuda"), torch.ones(2, 64, device="cuda")),
                   (w.half(), w.half()), (w[:32], w), (w.cpu(), w), (torch.ones(128, device="cuda")[::2], w)):
        with pytest.raises(ValueError):
            dlp.proj_kv_append_norm(ctx, cache, qkv, qn, kn, 1e-6, rope, *at)
    for qn, eps in ((w, -1.0), (w, float("nan")), (w, float("inf")), (torch.ones(65, device="cuda")[1:], 1e-6)):
        with pytest.raises(dlp.ProjError) as e:
            dlp.proj_kv_append_norm(ctx, cache, qkv, qn, w, eps, rope, *at)
        assert e.value.status == dlp.PROJ_ERR_INVALID_ARG
