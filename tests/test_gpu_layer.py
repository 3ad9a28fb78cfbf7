"""The operators of a decoding layer together, as they are used: tokens made
integers and projected, heads normed, rotated and appended, attention over a
prefix that the batch shares and each sequence's own pages, and the output
projection, captured into one graph and replayed as the sequences grow; every
step against the layer in 64 bits."""
import pytest
import torch

import dense_linear_projection_amd as dlp
from tests import layer_reference as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def rows(x):
    q, s = ref.quantize_rows(x)
    return q.double() * s[:, None]


class Layer64:
    """The same layer on the CPU in 64 bits, rounded where the library stores bf16 or 8 bits."""

    def __init__(self, w_qkv, w_out, norms, rope, heads, kv_heads, dim, prefix_k, prefix_v, fp8, scales):
        self.w_qkv, self.w_out, self.norms, self.rope = rows(w_qkv), rows(w_out), norms, rope.double()
        self.heads, self.kv, self.dim, self.scales = heads, kv_heads, dim, scales
        self.store = torch.float8_e4m3fn if fp8 else BF16
        self.prefix = (prefix_k, prefix_v)
        self.own = None

    def step(self, x, position):
        B = x.shape[0]
        y = (rows(x) @ self.w_qkv.t()).to(BF16).double().view(B, -1, self.dim)
        q, k, v = y.split([self.heads, self.kv, self.kv], 1)
        half = self.dim // 2
        cos, sin = self.rope[position, :half], self.rope[position, half:]

        def turn(t, w):
            t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w.double()
            a, b = t[..., :half], t[..., half:]
            return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        q = turn(q, self.norms[0]).to(BF16).double()
        k = (turn(k, self.norms[1]) / self.scales[0]).clamp(-448, 448) if self.store != BF16 else turn(k, self.norms[1])
        v = (v / self.scales[1]).clamp(-448, 448) if self.store != BF16 else v
        new = [(t.float().to(self.store).double() * s)[:, None] for t, s in ((k, self.scales[0]), (v, self.scales[1]))]
        self.own = new if self.own is None else [torch.cat((a, b), 1) for a, b in zip(self.own, new)]
        out = torch.empty(B, self.heads, self.dim).double()
        per = self.heads // self.kv
        for h in range(self.heads):
            K, V = (torch.cat((p[:, h // per].expand(B, -1, -1), o[:, :, h // per]), 1) for p, o in zip(self.prefix, self.own))
            w = torch.softmax((K @ q[:, h, :, None]).squeeze(-1) * self.dim ** -0.5, 1)
            out[:, h] = (w[:, None] @ V).squeeze(1)
        return rows(out.to(BF16).flatten(1)) @ self.w_out.t()


@pytest.mark.parametrize("B,fp8", [(3, False), (40, False), (21, True)])
def test_layer(ctx, B, fp8):
    hidden, heads, kv, dim, page, L, steps = 512, 8, 2, 64, 16, 70, 6
    g = torch.Generator().manual_seed(B)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    w_qkv, w_out = (rand((heads + 2 * kv) * dim, hidden) / hidden ** 0.5).to(BF16), (rand(hidden, heads * dim) / (heads * dim) ** 0.5).to(BF16)
    norms = [1 + 0.1 * rand(dim) for _ in range(2)]
    angle = torch.outer(torch.arange(L + steps).double(), 1e4 ** (-torch.arange(dim // 2).double() * 2 / dim))
    rope = torch.cat((angle.cos(), angle.sin()), 1).float()
    scales = (0.02, 0.02) if fp8 else (1.0, 1.0)
    store = torch.float8_e4m3fn if fp8 else BF16
    first, each = -(-L // page), -(-steps // page)
    pages = first + B * each
    k, v = (torch.zeros(pages, kv, page, dim, dtype=store) for _ in range(2))
    order = torch.randperm(pages, generator=g)
    held = []
    for c, s in ((k, scales[0]), (v, scales[1])):
        new = (rand(L, kv, dim) / (s if fp8 else 1)).to(store)
        for t in range(L):
            c[order[t // page], :, t % page] = new[t]
        held.append((new.double() * s))
    cache = dlp.kv_cache(k.cuda(), v.cuda(), *scales)
    prefix, tables = order[:first].int().cuda(), order[first:].view(B, each).int().cuda()
    layer = Layer64(w_qkv, w_out, norms, rope, heads, kv, dim, *held, fp8, scales)

    qkv_w, out_w = dlp.proj_quantize_rows(ctx, w_qkv.cuda()), dlp.proj_quantize_rows(ctx, w_out.cuda())
    dev_norms, dev_rope = [n.cuda() for n in norms], rope.cuda()
    x = torch.zeros(B, hidden, dtype=BF16, device="cuda")
    qkv = torch.empty(B, (heads + 2 * kv) * dim, dtype=BF16, device="cuda")
    q, o = (torch.empty(B, heads, dim, dtype=BF16, device="cuda") for _ in range(2))
    y = torch.empty(B, hidden, device="cuda")
    positions, lengths = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    slots = torch.full((B,), -1, dtype=torch.int64, device="cuda")

    def calls():
        xq, xs = dlp.proj_quantize_rows(ctx, x)
        dlp.proj_run_int(ctx, xq, xs, *qkv_w, None, dlp.EPI_NONE, qkv)
        dlp.proj_kv_append_norm(ctx, cache, qkv, *dev_norms, 1e-6, dev_rope, positions, slots, q)
        dlp.proj_kv_attend_shared(ctx, cache, q, prefix, L, tables, lengths, dim ** -0.5, o, max_len=L + steps)
        dlp.proj_run_int_dynamic(ctx, o.flatten(1), *out_w, None, dlp.EPI_NONE, y)

    calls()          # padding places: nothing stored, nothing seen
    torch.cuda.synchronize()
    assert not bool(o.any()) and not bool(y.any()) and torch.equal(cache.k.cpu().view(torch.uint8), k.view(torch.uint8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for t in range(steps):
        x.copy_(rand(B, hidden))
        positions.fill_(L + t)
        lengths.fill_(L + t + 1)
        slots.copy_(tables[:, t // page].long() * page + t % page)
        graph.replay()
        torch.cuda.synchronize()
        want = layer.step(x.cpu(), L + t)
        # Roundings between the calls, bf16 2^-8 and 8-bit codes 2^-8 of a row's largest element, differ where the fp32
        # results before them differ: one step of either in a few of a row's elements, of 512 that add up at random.
        off = (y.cpu().double() - want).norm() / want.norm()
        assert float(off) < 2.0 ** -7, (t, float(off))


def test_two_contexts_at_once():
    """Two contexts on two streams, whose kernels overlap: splits of K, joins and partial results do not meet."""
    g = torch.Generator().manual_seed(7)
    sides = [torch.cuda.Stream() for _ in range(2)]
    contexts = [dlp.proj_create(0) for _ in range(2)]
    calls = []
    for i in range(2):
        X = torch.randn(16, 8192, generator=g).to(BF16).cuda()
        W = dlp.proj_quantize_rows(contexts[0], torch.randn(512, 8192, generator=g).to(BF16).cuda())
        k, v = (torch.randn(40, 2, 16, 64, generator=g).to(BF16).cuda() for _ in range(2))
        q, order = torch.randn(24, 8, 64, generator=g).to(BF16).cuda(), torch.randperm(40, generator=g).int().cuda()
        n = torch.randint(100, 117, (24,), generator=g).int().cuda()
        calls.append((X, W, dlp.kv_cache(k, v), q, order[:7].contiguous(), order[7:31].view(24, 1), n))

    def run(ctx, c, stream):
        X, W, cache, q, prefix, tables, n = c
        with torch.cuda.stream(stream):
            Y, o, lse = torch.empty(16, 512, device="cuda"), torch.empty(24, 8, 64, device="cuda"), torch.empty(24, 8, device="cuda")
            for _ in range(5):
                dlp.proj_run_int_dynamic(ctx, X, *W, None, dlp.EPI_NONE, Y)
                dlp.proj_kv_attend_shared(ctx, cache, q, prefix, 100, tables, n, 0.1, o, lse=lse)
        return Y, o, lse

    torch.cuda.synchronize()
    alone = []
    for i in range(2):
        alone.append(run(contexts[i], calls[i], sides[i]))
        torch.cuda.synchronize()
    both = [run(contexts[i], calls[i], sides[i]) for _ in range(4) for i in range(2)]
    torch.cuda.synchronize()
    for j, got in enumerate(both):
        assert all(torch.equal(a, b) for a, b in zip(got, alone[j % 2]))
    for c in contexts:
        dlp.proj_destroy(c)
