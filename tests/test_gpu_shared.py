"""Attention over a prefix that a batch shares, on the GPU against its 64-bit
form: both cache types and layouts, every head size, rows from one to many
groups, prefixes and own tokens from none to many pages, pages that end inside a
tile, windows, lengths inside the prefix, stale and infinite values, pages and
lengths that are wrong, small workspaces, graphs, streams."""
import math

import pytest
import torch

import dense_linear_projection_amd as dlp
from tests import layer_reference as ref
from tests.decode_reference import close
from tests.test_gpu_kv import make_cache

pytestmark = pytest.mark.gpu
BF16, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def make(B, Hq, H, D, page, dtype, layout, prefix_len, lengths, seed, poison=True):
    """The parts of a call, on the CPU, and the cache on the device; lengths count the prefix."""
    g = torch.Generator().manual_seed(seed)
    scales = (0.125, 0.0625) if dtype == FP8 else (1.0, 1.0)
    first = -(-prefix_len // page)
    need = [-(-max(0, n - prefix_len) // page) for n in lengths]
    pages = first + sum(need) + 3
    k, v, cache = make_cache(pages, H, page, D, dtype, layout, g, scales)
    free, at = torch.randperm(pages, generator=g), first
    prefix = free[:first].int()
    tables = torch.full((B, max(need + [1])), -1, dtype=torch.int32)
    ends = [(free[first - 1], prefix_len % page)] if first else []
    for b, n in enumerate(need):
        tables[b, :n] = free[at:at + n].int()
        at += n
        if n:
            ends.append((free[at - 1], (lengths[b] - prefix_len) % page))
    if poison:
        for i, (p, used) in enumerate(ends):
            if used:
                k[p, :, used:] = float("nan")
                v[p, :, used:] = float("nan") if i % 2 or dtype == FP8 else float("inf")
        k[free[at:]], v[free[at:]] = float("nan"), float("nan")
    cache.k.copy_(k)
    cache.v.copy_(v)
    q = (torch.randn(B, Hq, D, generator=g) * 1.5).to(BF16)
    return k, v, cache, q, prefix, tables, torch.tensor(lengths, dtype=torch.int32), scales


def run(ctx, cache, q, prefix, prefix_len, tables, lengths, scale, out=BF16, window=0, max_len=None, stream=None, lse=True):
    wide = torch.zeros(q.shape[0], q.shape[1] + 1, q.shape[2], dtype=BF16, device="cuda")
    wide[:, 1:] = q.cuda()
    o = torch.full((q.shape[0] + 1,) + tuple(q.shape[1:]), 9.0, dtype=out, device="cuda")
    e = torch.full((q.shape[0] + 1, q.shape[1]), 9.0, device="cuda")
    dlp.proj_kv_attend_shared(ctx, cache, wide[:, 1:], prefix.cuda(), prefix_len, tables.cuda(), lengths.cuda(), scale, o[:-1],
                              lse=e[:-1] if lse else None, window=window, max_len=max_len, stream=stream)
    torch.cuda.synchronize()
    assert bool((o[-1] == 9).all()) and bool((e[-1] == 9).all())     # behind the last sequence
    return o[:-1], e[:-1]


def check(ctx, B, Hq, H, D, page, dtype, layout, prefix_len, lengths, seed, out=BF16, window=0, max_len=None):
    print("shared", B, Hq, H, D, page, dtype, layout, prefix_len, lengths[:6], out, window, flush=True)
    k, v, cache, q, prefix, tables, n, scales = make(B, Hq, H, D, page, dtype, layout, prefix_len, lengths, seed)
    scale = 1 / math.sqrt(D)
    want, tol = ref.attend_shared(k, v, q, prefix, prefix_len, tables, n, scale, window, scales, out)
    o, lse = run(ctx, cache, q, prefix, prefix_len, tables, n, scale, out, window, max_len)
    close(o, want[0], tol[0])
    close(lse, want[1], tol[1])
    return o, lse


def lengths_of(B, prefix, own, seed, empty=False):
    g = torch.Generator().manual_seed(seed)
    n = (prefix + torch.randint(0, own + 1, (B,), generator=g)).tolist()
    return [0 if empty and i % 5 == 2 else x for i, x in enumerate(n)]


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("D", [64, 80, 96, 128, 192, 256])
def test_shapes(ctx, dtype, layout, D):
    for i, (B, Hq, H, page, prefix, own) in enumerate(((1, 1, 1, 16, 1, 3), (4, 8, 2, 16, 100, 40), (3, 12, 4, 32, 333, 5),
                                                       (33, 4, 4, 16, 64, 70), (40, 15, 5, 1, 31, 9), (9, 16, 1, 64, 700, 300),
                                                       (50, 20, 2, 128, 1000, 20), (7, 40, 1, 8, 129, 1))):
        check(ctx, B, Hq, H, D, page, dtype, layout, prefix, lengths_of(B, prefix, own, i, i % 2 == 1), 10 * i + D,
              (BF16, F32)[i % 2])


@pytest.mark.parametrize("prefix", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1000, 2047, 2048, 2049, 4100, 9000])
def test_prefixes(ctx, prefix):
    check(ctx, 3, 8, 2, 128, 16, BF16, "hnd", prefix, [prefix, prefix + 1, prefix + 37], prefix)
    check(ctx, 70, 4, 2, 64, 32, FP8, "nhd", prefix, lengths_of(70, prefix, 3, prefix), prefix, F32)


@pytest.mark.parametrize("B,Hq,H", [(1, 32, 1), (1, 33, 1), (2, 16, 1), (8, 8, 2), (8, 17, 1), (16, 8, 1), (129, 1, 1), (127, 1, 1), (64, 10, 2),
                                    (200, 6, 2), (5, 130, 1)])
def test_rows(ctx, B, Hq, H):
    """Rows that fill groups of 32 and 128 exactly, leave one over, or miss one."""
    check(ctx, B, Hq, H, 128, 16, BF16, "hnd", 300, lengths_of(B, 300, 50, B), B)
    check(ctx, B, Hq, H, 96, 16, FP8, "hnd", 200, lengths_of(B, 200, 50, B, True), B, F32)


def test_long(ctx):
    check(ctx, 20, 16, 2, 128, 64, BF16, "hnd", 30000, lengths_of(20, 30000, 900, 1), 1)
    check(ctx, 2, 4, 2, 64, 16, BF16, "hnd", 70001, [70001, 70500], 2, F32)


@pytest.mark.parametrize("window", [1, 7, 64, 100, 333, 1000, 5000])
def test_windows(ctx, window):
    """Windows that end among the own tokens, inside the prefix and before it."""
    for B, Hq in ((4, 8), (40, 8)):
        lengths = lengths_of(B, 700, 400, window, True)
        check(ctx, B, Hq, 2, 128, 16, BF16, "hnd", 700, lengths, window, window=window)
        check(ctx, B, Hq, 4, 80, 32, FP8, "nhd", 700, lengths, window, F32, window)


@pytest.mark.parametrize("window", [0, 50])
def test_lengths_inside_the_prefix(ctx, window):
    """Sequences that see a part of the prefix only, none of it (a padding place), all of it, or more."""
    lengths = [0, 1, 5, 31, 32, 33, 64, 100, 129, 255, 256, 257, 299, 300, 301, 340, 0, 17]
    check(ctx, len(lengths), 8, 2, 128, 16, BF16, "hnd", 300, lengths, 3, window=window)
    check(ctx, len(lengths), 8, 8, 64, 16, FP8, "nhd", 300, lengths, 4, F32, window, max_len=340)
    check(ctx, 4, 8, 2, 96, 16, BF16, "hnd", 300, [0, 3, 299, 300], 5, F32, window, max_len=300)   # nobody has own tokens
    check(ctx, 3, 8, 2, 96, 16, BF16, "hnd", 300, [0, 0, 0], 6, F32, window)                       # nobody has any


def test_loose_bound_and_no_prefix(ctx):
    check(ctx, 5, 8, 2, 128, 16, BF16, "hnd", 100, [100, 101, 150, 0, 120], 7, max_len=164)
    k, v, cache, q, prefix, tables, n, _ = make(5, 8, 2, 128, 16, BF16, "hnd", 0, [1, 30, 0, 77, 5], 8)
    o, lse = run(ctx, cache, q, prefix, 0, tables, n, 0.1)
    plain, e = torch.empty_like(o), torch.empty_like(lse)
    dlp.proj_kv_attend(ctx, cache, q.cuda(), tables.cuda(), n.cuda(), 0.1, plain, lse=e)
    assert torch.equal(o, plain) and torch.equal(lse, e)


def test_it_is_the_attention_of_whole_tables(ctx):
    """A prefix of whole pages: the same as proj_kv_attend on tables that name its pages for every sequence."""
    B, Hq, H, D, page, L = 24, 16, 4, 128, 16, 512
    lengths = lengths_of(B, L, 200, 5, True)
    _, _, cache, q, prefix, tables, n, _ = make(B, Hq, H, D, page, BF16, "hnd", L, lengths, 5)
    o, lse = run(ctx, cache, q, prefix, L, tables, n, 0.09, F32)
    whole = torch.cat((prefix.expand(B, -1), tables), 1).cuda()
    want, e = torch.empty_like(o), torch.empty_like(lse)
    dlp.proj_kv_attend(ctx, cache, q.cuda(), whole, n.cuda(), 0.09, want, lse=e)
    assert float((o - want).abs().max()) < 2e-5 and torch.equal(torch.isinf(lse), torch.isinf(e))
    assert float((lse - e).nan_to_num(0, 0, 0).abs().max()) < 2e-5
    view = whole[:, L // page:]                   # the own pages as a view of the whole tables
    o2 = torch.empty_like(o)
    dlp.proj_kv_attend_shared(ctx, cache, q.cuda(), prefix.cuda(), L, view, n.cuda(), 0.09, o2, max_len=max(lengths))
    close(o2, want.cpu().double(), torch.full(o.shape, 2e-5).double())


@pytest.mark.parametrize("B,Hq", [(3, 8), (40, 8)])
def test_what_is_wrong_is_not_read(ctx, B, Hq):
    """Bad lengths and own pages make their sequences NaN, a bad page of the prefix those that see a token of it."""
    L, page = 100, 16
    lengths = [L + 5 + b for b in range(B)]
    k, v, cache, q, prefix, tables, n, _ = make(B, Hq, 2, 64, page, BF16, "hnd", L, lengths, 9)
    want = ref.attend_shared(k, v, q, prefix, L, tables, n, 0.1, 0, (1, 1), F32)
    for bad in (1 << 30, -5, cache.pages):
        t = tables.clone()
        t[1, 0] = bad
        o, lse = run(ctx, cache, q, prefix, L, t, n, 0.1, F32)
        assert torch.isnan(o[1]).all() and torch.isnan(lse[1]).all()
        keep = torch.arange(B) != 1
        close(o[keep], want[0][0][keep], want[1][0][keep])
    for bad in (-1, max(lengths) + 1, 2 ** 31 - 1, -2 ** 31):
        m = n.clone()
        m[0] = bad
        o, lse = run(ctx, cache, q, prefix, L, tables, m, 0.1, F32, max_len=max(lengths))
        assert torch.isnan(o[0]).all() and torch.isnan(lse[0]).all()
        close(o[1:], want[0][0][1:], want[1][0][1:])
    for at, bad in ((0, -1), (3, cache.pages), (6, 1 << 30)):
        p = prefix.clone()
        p[at] = bad
        o, lse = run(ctx, cache, q, p, L, tables, n, 0.1, F32)
        assert torch.isnan(o).all() and torch.isnan(lse).all()
        m = n.clone()
        m[B - 1], m[0] = at * page, 0                # sees the prefix up to the bad page
        o, lse = run(ctx, cache, q, p, L, tables, m, 0.1, F32)
        some = ref.attend_shared(k, v, q, prefix, L, tables, m, 0.1, 0, (1, 1), F32)
        for b in (0, B - 1):
            close(o[b], some[0][0][b], some[1][0][b])
        assert torch.isnan(o[1:B - 1]).all()
        w = 20                                       # a window behind the bad page sees nothing of it
        o, lse = run(ctx, cache, q, p, L, tables, n, 0.1, F32, window=w)
        some = ref.attend_shared(k, v, q, prefix, L, tables, n, 0.1, w, (1, 1), F32)
        clear = torch.tensor([max(0, x - w) >= min((at + 1) * page, L) for x in lengths])
        if clear.any():
            close(o[clear], some[0][0][clear], some[1][0][clear])
        assert torch.isnan(o[~clear]).all()


def test_a_cache_without_pages(ctx):
    k = torch.empty(0, 2, 16, 64, dtype=BF16, device="cuda")
    cache = dlp.kv_cache(k, k.clone())
    q = torch.randn(3, 4, 64).to(BF16).cuda()
    o, lse = torch.empty(3, 4, 64, device="cuda"), torch.empty(3, 4, device="cuda")
    dlp.proj_kv_attend_shared(ctx, cache, q, torch.zeros(2, dtype=torch.int32, device="cuda"), 20,
                              torch.zeros(3, 1, dtype=torch.int32, device="cuda"), torch.tensor([0, 7, 25], dtype=torch.int32).cuda(),
                              0.1, o, lse=lse)
    assert not bool(o[0].any()) and torch.isnan(o[1:]).all() and torch.isnan(lse[1:]).all()


@pytest.mark.parametrize("B,Hq", [(2, 8), (40, 8)])
@pytest.mark.parametrize("out", [BF16, F32])
def test_values_that_are_not_numbers(ctx, B, Hq, out):
    """NaN and infinities in keys and values reach the sequences that see them, and no other."""
    L, D, H = 200, 96, 2
    lengths = [L + 3] * B
    lengths[0], lengths[1] = 60, 130
    for where, bad in ((100, float("nan")), (100, float("inf")), (40, -float("inf")), (150, float("nan"))):
        for what in ("v", "k"):
            k, v, cache, q, prefix, tables, n, _ = make(B, Hq, H, D, 16, BF16, "hnd", L, lengths, 11)
            clean = ref.attend_shared(k, v, q, prefix, L, tables, n, 0.1, 0, (1, 1), out)
            at = (int(prefix[where // 16]), 1, where % 16, 33)
            (v if what == "v" else k)[at] = bad
            getattr(cache, what).copy_(v if what == "v" else k)
            o, lse = run(ctx, cache, q, prefix, L, tables, n, 0.1, out)
            o, lse = o.cpu(), lse.cpu()
            rows = slice(Hq // H, Hq)                 # the heads that read key-value head 1
            close(o[:, :Hq // H], clean[0][0][:, :Hq // H], clean[1][0][:, :Hq // H])
            for b in range(B):
                if where >= lengths[b]:
                    close(o[b], clean[0][0][b], clean[1][0][b])
                    close(lse[b], clean[0][1][b], clean[1][1][b])
                elif what == "v":
                    got = o[b, rows, 33]
                    assert torch.isnan(got).all() if math.isnan(bad) else bool((got == bad).all())
                    others = torch.arange(D) != 33
                    close(o[b, rows][:, others], clean[0][0][b, rows][:, others], clean[1][0][b, rows][:, others])
                elif math.isnan(bad):
                    assert torch.isnan(o[b, rows]).all() and torch.isnan(lse[b, rows]).all()


def test_logits_of_minus_infinity(ctx):
    """Rows whose every logit is minus infinity have result 0 and logarithm minus infinity; others do not notice."""
    k, v, cache, q, prefix, tables, n, _ = make(40, 4, 1, 64, 16, BF16, "hnd", 50, [50] * 40, 12, poison=False)
    cache.k[:, :, :, 0] = float("inf")
    q[:, :, 0] = 0.0
    q[3, 2, 0] = -1.0
    kk = cache.k.cpu().clone()
    kk[:, :, :, 0] = 0
    cache.k[:, :, :, 0] = 0
    want, tol = ref.attend_shared(kk, v, q, prefix, 50, tables, n, 0.1, 0, (1, 1), F32)
    cache.k[:, :, :, 0] = 3.0e38
    q[3, 2, 0] = -3.0e38                           # the product passes the largest float
    o, lse = run(ctx, cache, q, prefix, 50, tables, n, 0.1, F32)
    assert not bool(o[3, 2].any()) and float(lse[3, 2]) == -math.inf
    mask = torch.ones(40, 4, dtype=torch.bool)
    mask[3, 2] = False
    close(o[mask], want[0][mask], tol[0][mask])


def test_spread_of_logits(ctx):
    """Logits that rise along the prefix, fall, and lie far apart between prefix and own tokens."""
    for sign in (1, -1):
        for own_up in (-40.0, 0.0, 40.0):
            k, v, cache, q, prefix, tables, n, _ = make(40, 4, 2, 64, 16, BF16, "hnd", 400, [430] * 40, 13, poison=False)
            q[:] = 0
            q[:, :, 0] = 1
            for t in range(400):
                k[prefix[t // 16], :, t % 16, 0] = sign * t * 0.25
            for b in range(40):
                for t in range(30):
                    k[tables[b, t // 16], :, t % 16, 0] = own_up
            cache.k.copy_(k)
            want, tol = ref.attend_shared(k, v, q, prefix, 400, tables, n, 1.0, 0, (1, 1), F32)
            o, lse = run(ctx, cache, q, prefix, 400, tables, n, 1.0, F32)
            close(o, want[0], tol[0])
            close(lse, want[1], tol[1])


@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-30, -1e-42, 2.0, -30.0])
def test_scales(ctx, scale):
    """Scales of either sign, zero, so small that every token counts alike, so large that one does."""
    for B, Hq in ((3, 8), (40, 8)):
        lengths = lengths_of(B, 150, 60, B)
        lengths[0] = 33
        k, v, cache, q, prefix, tables, n, _ = make(B, Hq, 2, 64, 16, BF16, "hnd", 150, lengths, 18)
        want, tol = ref.attend_shared(k, v, q, prefix, 150, tables, n, scale, 0, (1, 1), F32)
        o, lse = run(ctx, cache, q, prefix, 150, tables, n, scale, F32)
        close(o, want[0], tol[0])
        close(lse, want[1], tol[1])


def test_queries_that_are_not_numbers(ctx):
    k, v, cache, q, prefix, tables, n, _ = make(40, 8, 2, 64, 16, BF16, "hnd", 150, [170] * 40, 19)
    want, tol = ref.attend_shared(k, v, q, prefix, 150, tables, n, 0.1, 0, (1, 1), F32)
    q[7, 3, 5], q[9, 0] = float("nan"), float("inf")
    o, lse = run(ctx, cache, q, prefix, 150, tables, n, 0.1, F32)
    keep = torch.ones(40, 8, dtype=torch.bool)
    keep[7, 3] = keep[9, 0] = False
    assert torch.isnan(o[7, 3]).all() and torch.isnan(lse[7, 3])
    close(o[keep], want[0][keep], tol[0][keep])
    close(lse[keep], want[1][keep], tol[1][keep])


def test_workspaces():
    """Whatever the workspace holds, the result is right: fewer parts, fewer sequences at a time, a refusal at last."""
    B, Hq, H, D, L = 30, 16, 2, 64, 600
    lengths = lengths_of(B, L, 300, 3, True)
    k, v, cache, q, prefix, tables, n, _ = make(B, Hq, H, D, 16, BF16, "hnd", L, lengths, 14)
    want, tol = ref.attend_shared(k, v, q, prefix, L, tables, n, 0.1, 0, (1, 1), F32)
    row = Hq * (D + 4) * 4
    for room in (2 * row, 3 * row, 5 * row, 11 * row, 2 * B * row, 5 * B * row, 9 * B * row, 64 << 20):
        c = dlp.proj_create(0, room + 256)
        o, lse = run(c, cache, q, prefix, L, tables, n, 0.1, F32)
        close(o, want[0], tol[0])
        close(lse, want[1], tol[1])
        dlp.proj_destroy(c)
    for room in (0, 2 * row - 256):
        c = dlp.proj_create(0, room)
        with pytest.raises(dlp.ProjError) as e:
            run(c, cache, q[:1], prefix, L, tables[:1], n[:1], 0.1, F32)
        assert e.value.status == dlp.PROJ_ERR_NO_MEMORY
        dlp.proj_destroy(c)


def test_graph_replays_follow_their_inputs(ctx):
    for B, Hq in ((3, 8), (50, 8)):
        lengths = lengths_of(B, 300, 100, 4)
        _, _, cache, q, prefix, tables, n, _ = make(B, Hq, 2, 128, 16, BF16, "hnd", 300, lengths, 15, poison=False)
        dev = [t.cuda() for t in (q, prefix, tables, n)]
        o, lse = torch.empty(B, Hq, 128, dtype=BF16, device="cuda"), torch.empty(B, Hq, device="cuda")

        def call(o, lse):
            dlp.proj_kv_attend_shared(ctx, cache, dev[0], dev[1], 300, dev[2], dev[3], 0.1, o, lse=lse, max_len=max(lengths))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(o, lse)
        for i in range(3):
            dev[0].copy_(torch.randn(q.shape))
            dev[3].copy_(torch.tensor(lengths_of(B, 300, 90, 20 + i, True)).clamp(max=torch.tensor(lengths)))
            graph.replay()
            torch.cuda.synchronize()
            a, b = torch.empty_like(o), torch.empty_like(lse)
            call(a, b)
            torch.cuda.synchronize()
            assert torch.equal(o, a) and torch.equal(lse, b)


def test_another_stream(ctx):
    lengths = lengths_of(9, 300, 100, 4)
    _, _, cache, q, prefix, tables, n, _ = make(9, 8, 2, 128, 16, BF16, "hnd", 300, lengths, 16)
    a = run(ctx, cache, q, prefix, 300, tables, n, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = run(ctx, cache, q, prefix, 300, tables, n, 0.1, stream=side)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_refusals_in_python(ctx):
    _, _, cache, q, prefix, tables, n, _ = make(3, 8, 2, 64, 16, BF16, "hnd", 40, [41, 50, 0], 17)
    q, prefix, tables, n = (t.cuda() for t in (q, prefix, tables, n))
    o = torch.empty(3, 8, 64, device="cuda")
    for f in (lambda: dlp.proj_kv_attend_shared(ctx, cache, q, prefix[:2], 40, tables, n, 0.1, o),
              lambda: dlp.proj_kv_attend_shared(ctx, cache, q, prefix.long(), 40, tables, n, 0.1, o),
              lambda: dlp.proj_kv_attend_shared(ctx, cache, q, prefix, -1, tables, n, 0.1, o),
              lambda: dlp.proj_kv_attend_shared(ctx, cache, q, prefix.view(1, -1), 40, tables, n, 0.1, o),
              lambda: dlp.proj_kv_attend_shared(ctx, cache, q, prefix, 40, tables[:2], n, 0.1, o),
              lambda: dlp.proj_kv_attend_shared(ctx, cache, q, prefix.cpu(), 40, tables, n, 0.1, o),
              lambda: dlp.proj_kv_attend_shared(ctx, cache, q, prefix, 40, tables, n.long(), 0.1, o),
              lambda: dlp.proj_kv_attend_shared(ctx, cache, q, prefix, 40, tables, n, 0.1, o.half())):
        with pytest.raises(ValueError):
            f()
    for kw in (dict(max_len=40 + 16 * tables.shape[1] + 1), dict(window=-1), dict(max_len=-1)):
        with pytest.raises(dlp.ProjError) as e:
            dlp.proj_kv_attend_shared(ctx, cache, q, prefix, 40, tables, n, 0.1, o, **kw)
        assert e.value.status == dlp.PROJ_ERR_INVALID_ARG
