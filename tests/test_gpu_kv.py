"""Rotated append to a paged cache, and attention of one new token over it, on
the GPU against their 64-bit forms: both cache types and layouts, every head
size, groups of query heads from one to more than a tile, lengths from nothing
to many pages, pages that end inside a tile, windows, stale and infinite
values outside a sequence, pages and lengths that are wrong, graphs, streams."""
import math

import pytest
import torch

import dense_linear_projection_amd as dlp
from tests import decode_reference as ref

pytestmark = pytest.mark.gpu
BF16, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def make_cache(pages, heads, page, D, dtype, layout, g, scales=(1.0, 1.0)):
    """(k, v) on the CPU [pages, heads, page, D], and the device cache with the given layout."""
    both = []
    for _ in range(2):
        t = torch.randn(pages, heads, page, D, generator=g)
        both.append((t * 8).to(FP8) if dtype == FP8 else t.to(BF16))
    dev = [t.cuda() if layout == "hnd" else t.transpose(1, 2).contiguous().cuda().transpose(1, 2) for t in both]
    return both[0], both[1], dlp.kv_cache(dev[0], dev[1], *scales)


# ------------------------------------------------------------------ append

def run_append(ctx, T, Hq, H, D, rot, page, dtype, layout, interleaved, seed, pad=0, slots=None, positions=None):
    g = torch.Generator().manual_seed(seed)
    scales = (0.05, 0.03125) if dtype == FP8 else (1.0, 1.0)
    pages = -(-T // page) + 2
    k, v, cache = make_cache(pages, H, page, D, dtype, layout, g, scales)
    qkv = torch.randn(T, (Hq + 2 * H) * D, generator=g).to(BF16)
    rope = torch.randn(50, rot, generator=g)
    if positions is None:
        positions = torch.randint(0, 50, (T,), generator=g).to(torch.int32)
    if slots is None:
        slots = torch.randperm(pages * page, generator=g)[:T]
        slots[T - pad:] = -1
    want, tol = ref.append(k, v, qkv, rope, positions, slots, Hq, scales, interleaved)
    wide = torch.zeros(T, qkv.shape[1] + 8, dtype=BF16, device="cuda")
    wide[:, :-8] = qkv.cuda()
    q = torch.full((T, Hq, D), 7.0, dtype=BF16, device="cuda") if Hq else None
    dlp.proj_kv_append(ctx, cache, wide[:, :-8], rope.cuda(), positions.cuda(), slots.cuda(), q, interleaved=interleaved)
    torch.cuda.synchronize()
    if Hq:
        ref.close(q, want[0], tol[0])
    for got, before, w, t in ((cache.k, k, want[1], tol[1]), (cache.v, v, want[2], tol[2])):
        ref.close(got, w, t)
        kept = t.amax(-1) == 0                   # slots that no token went to hold what they held, to the bit
        bits = torch.uint8 if dtype == FP8 else torch.int16
        assert torch.equal(got.cpu().contiguous().view(bits)[kept], before.view(bits)[kept])


@pytest.mark.parametrize("dtype", [BF16, FP8])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(ctx, dtype, layout, interleaved):
    for i, (T, Hq, H, D, rot, page) in enumerate(((1, 8, 2, 64, 64, 16), (5, 4, 4, 128, 128, 16), (33, 15, 5, 80, 32, 32),
                                                  (70, 6, 1, 96, 96, 16), (9, 0, 3, 192, 64, 64), (17, 5, 1, 256, 256, 128),
                                                  (12, 2, 2, 80, 80, 1), (8, 3, 3, 64, 34, 4), (6, 2, 1, 128, 2, 8),
                                                  (7, 4, 2, 64, 0, 16), (300, 20, 4, 128, 64, 64))):
        print("append", dtype, layout, interleaved, T, Hq, H, D, rot, page, flush=True)
        run_append(ctx, T, Hq, H, D, rot, page, dtype, layout, interleaved, 10 * i, pad=T // 5)


@pytest.mark.parametrize("rot,interleaved", [(128, False), (64, True), (34, False), (34, True), (0, False)])
def test_append_many_tokens(ctx, rot, interleaved):
    """Enough tokens that a thread takes several of them, a number that does not divide evenly."""
    for dtype, layout in ((BF16, "hnd"), (FP8, "nhd")):
        run_append(ctx, 5003, 20, 4, 128, rot, 64, dtype, layout, interleaved, 77, pad=700)


def test_append_ignores_places_outside(ctx):
    """Slots past the cache store nothing; positions outside the table store nothing and give NaN queries."""
    T = 9
    slots = torch.tensor([0, 48, 5, 1 << 40, -7, 47, 3, 2 ** 62, 10])       # 3 pages of 16
    positions = torch.tensor([0, 1, 50, 2, 3, -1, 49, 4, 2 ** 31 - 1], dtype=torch.int32)
    for dtype in (BF16, FP8):
        run_append(ctx, T, 4, 2, 128, 128, 16, dtype, "hnd", False, 3, slots=slots, positions=positions)
        run_append(ctx, T, 4, 2, 80, 24, 16, dtype, "nhd", True, 4, slots=slots, positions=positions)


def test_append_extreme_values(ctx):
    """An 8-bit cache holds what is past its range as its largest value, and NaN as NaN."""
    g = torch.Generator().manual_seed(1)
    k, v, cache = make_cache(2, 1, 16, 64, FP8, "hnd", g, (0.5, 0.25))
    qkv = torch.randn(4, 2 * 64, generator=g).to(BF16)
    qkv[0, 3], qkv[0, 70], qkv[1, 64], qkv[2, 65], qkv[3, 127] = float("nan"), float("nan"), 1e30, -float("inf"), float("inf")
    rope = torch.cat((torch.ones(1, 8), torch.zeros(1, 8)), 1)
    pos, slots = torch.zeros(4, dtype=torch.int32), torch.arange(4)
    want, tol = ref.append(k, v, qkv, rope, pos, slots, 0, (0.5, 0.25), False)
    dlp.proj_kv_append(ctx, cache, qkv.cuda(), rope.cuda(), pos.cuda(), slots.cuda())
    ref.close(cache.v, want[2], tol[2])
    assert float(cache.v[0, 0, 1, 0]) == 448 and float(cache.v[0, 0, 2, 1]) == -448 and float(cache.v[0, 0, 3, 63]) == 448
    assert math.isnan(float(cache.v[0, 0, 0, 6])) and math.isnan(float(cache.k[0, 0, 0, 3]))


# ------------------------------------------------------------------ attend

def make_attend(B, Hq, H, D, page, dtype, layout, lengths, seed, spare=3, poison=True, width=None):
    g = torch.Generator().manual_seed(seed)
    scales = (0.125, 0.0625) if dtype == FP8 else (1.0, 1.0)
    need = [-(-max(0, n) // page) for n in lengths]
    pages = sum(need) + spare
    k, v, cache = make_cache(pages, H, page, D, dtype, layout, g, scales)
    width = max(need + [1]) if width is None else width
    free, tables, at = torch.randperm(pages, generator=g), torch.full((B, width), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        tables[b, :n] = free[at:at + n].int()
        at += n
        if poison and lengths[b] % page and n:
            for t, bad in ((k, float("nan")), (v, float("nan") if b % 2 else -448.0 if dtype == FP8 else float("inf"))):
                t[free[at - 1], :, lengths[b] % page:] = bad
    if poison:
        k[free[at:]], v[free[at:]] = float("nan"), float("nan")
    cache.k.copy_(k)
    cache.v.copy_(v)
    q = (torch.randn(B, Hq, D, generator=g) * 1.5).to(BF16)
    return k, v, cache, q, tables, torch.tensor(lengths, dtype=torch.int32), scales


def run_attend(ctx, cache, q, tables, lengths, scale, out=BF16, window=0, max_len=None, stream=None, lse=True):
    wide = torch.zeros(q.shape[0], q.shape[1] + 1, q.shape[2], dtype=BF16, device="cuda")
    wide[:, 1:] = q.cuda()
    o = torch.full(q.shape, 9.0, dtype=out, device="cuda")
    e = torch.full(q.shape[:2], 9.0, device="cuda") if lse else None
    dlp.proj_kv_attend(ctx, cache, wide[:, 1:], tables.cuda(), lengths.cuda(), scale, o, lse=e, window=window,
                       max_len=max_len, stream=stream)
    torch.cuda.synchronize()
    return o, e


def check_attend(ctx, B, Hq, H, D, page, dtype, layout, lengths, seed, out=BF16, window=0, max_len=None):
    print("attend", B, Hq, H, D, page, dtype, layout, lengths[:6], out, window, flush=True)
    k, v, cache, q, tables, n, scales = make_attend(B, Hq, H, D, page, dtype, layout, lengths, seed)
    scale = 1 / math.sqrt(D)
    want, tol = ref.attend(k, v, q, tables, n, scale, window, scales, out)
    o, e = run_attend(ctx, cache, q, tables, n, scale, out, window, max_len)
    ref.close(o, want[0], tol[0])
    ref.close(e, want[1], tol[1])


@pytest.mark.parametrize("D", [64, 80, 96, 128, 192, 256])
@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_attend_head_sizes(ctx, D, dtype):
    check_attend(ctx, 5, 8, 2, D, 16, dtype, "hnd", [70, 0, 1, 333, 16], D, F32)
    check_attend(ctx, 3, 3, 3, D, 32, dtype, "nhd", [31, 32, 129], D + 1)


@pytest.mark.parametrize("per", [1, 2, 3, 5, 8, 12, 16, 17, 20, 33, 64])
def test_attend_groups(ctx, per):
    check_attend(ctx, 2, 2 * per, 2, 128, 16, BF16, "hnd", [100, 37], per, F32)
    check_attend(ctx, 1, per, 1, 64, 64, FP8, "nhd", [515], per + 100)


@pytest.mark.parametrize("page", [1, 2, 8, 16, 64, 256, 1024])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_attend_pages(ctx, page, layout):
    check_attend(ctx, 4, 8, 2, 128, page, BF16, layout, [1, 300, 64, 65], page, F32)
    check_attend(ctx, 3, 4, 1, 96, page, FP8, layout, [129, 0, 257], page + 1)


def test_attend_lengths(ctx):
    """Every length around the sizes that a tile, a wave's share or a part may end at."""
    lengths = list(range(0, 70)) + [127, 128, 129, 255, 256, 257, 383, 384, 385, 511, 512, 513, 1023, 1024, 1025]
    check_attend(ctx, len(lengths), 4, 2, 64, 16, BF16, "hnd", lengths, 1, F32)
    check_attend(ctx, len(lengths), 5, 1, 128, 32, FP8, "hnd", lengths, 2, F32)


@pytest.mark.parametrize("window", [1, 2, 15, 32, 33, 100, 500, 5000])
def test_attend_window(ctx, window):
    check_attend(ctx, 6, 8, 2, 128, 16, BF16, "hnd", [1, 33, 500, 1040, 0, 777], window, F32, window)
    check_attend(ctx, 2, 5, 1, 64, 64, FP8, "nhd", [2100, 90], window, BF16, window)


@pytest.mark.parametrize("B,Hq,H,D,page,dtype,n", [(1, 16, 2, 128, 64, BF16, 20000), (2, 8, 1, 64, 16, FP8, 9000),
                                                   (1, 4, 1, 256, 32, BF16, 5000), (1, 20, 1, 80, 128, FP8, 12345)])
def test_attend_long(ctx, B, Hq, H, D, page, dtype, n):
    check_attend(ctx, B, Hq, H, D, page, dtype, "hnd", [n] + [n // 3] * (B - 1), n, F32)
    check_attend(ctx, B, Hq, H, D, page, dtype, "nhd", [n] + [n - 1] * (B - 1), n + 1, BF16, n // 2)


def test_attend_many_sequences(ctx):
    g = torch.Generator().manual_seed(3)
    lengths = torch.randint(0, 400, (200,), generator=g).tolist()
    check_attend(ctx, 200, 4, 2, 64, 16, BF16, "hnd", lengths, 5, F32)
    check_attend(ctx, 200, 4, 2, 64, 16, BF16, "hnd", lengths, 6, BF16, 100)


def test_attend_bound_looser_than_lengths(ctx):
    """max_len shapes the launch only: a loose bound gives the same values within rounding."""
    k, v, cache, q, tables, n, scales = make_attend(3, 8, 2, 128, 16, BF16, "hnd", [300, 17, 0], 8, width=4096)
    want, tol = ref.attend(k, v, q, tables, n, 0.1, 0, scales, F32)
    for bound in (300, 1000, 30000, None):
        o, e = run_attend(ctx, cache, q, tables, n, 0.1, F32, max_len=bound)
        ref.close(o, want[0], tol[0])
        ref.close(e, want[1], tol[1])


def test_attend_without_workspace_or_lse(ctx):
    small = dlp.proj_create(0, 0)
    try:
        k, v, cache, q, tables, n, scales = make_attend(1, 8, 1, 128, 16, BF16, "hnd", [3000], 9)
        want, tol = ref.attend(k, v, q, tables, n, 0.1, 0, scales, F32)
        ref.close(run_attend(small, cache, q, tables, n, 0.1, F32)[0], want[0], tol[0])
        ref.close(run_attend(ctx, cache, q, tables, n, 0.1, F32, lse=False)[0], want[0], tol[0])
    finally:
        dlp.proj_destroy(small)


def test_attend_large_logits(ctx):
    """Logits of hundreds: the running maximum keeps every exponential in range, rising or falling along the sequence."""
    k, v, cache, q, tables, n, scales = make_attend(2, 4, 1, 64, 16, BF16, "hnd", [900, 900], 10, poison=False)
    ramp = torch.linspace(-30, 30, 900)
    for b, r in ((0, ramp), (1, -ramp)):
        for t in range(900):
            k[tables[b, t // 16], 0, t % 16] = (q[b, 0].float() / q[b, 0].float().norm() * r[t]).to(BF16)
    cache.k.copy_(k)
    want, tol = ref.attend(k, v, q, tables, n, 1.0, 0, scales, F32)
    assert float(want[1].abs().max()) > 200
    o, e = run_attend(ctx, cache, q, tables, n, 1.0, F32)
    ref.close(o, want[0], tol[0])
    ref.close(e, want[1], tol[1])


def test_attend_infinite_logits(ctx):
    """A key of minus infinity leaves its token out, also where it comes first or alone."""
    k, v, cache, q, tables, n, scales = make_attend(3, 4, 1, 64, 16, BF16, "hnd", [100, 1, 40], 11, poison=False)
    q = q.abs() + 0.5
    for b, t in ((0, 0), (0, 50), (1, 0)) + tuple((2, i) for i in range(40)):
        k[tables[b, t // 16], 0, t % 16] = -float("inf")
    cache.k.copy_(k)
    o, e = run_attend(ctx, cache, q, tables, n, 0.125, F32)
    kk = k.clone()
    kk[kk == -float("inf")] = -1e30
    want, tol = ref.attend(kk, v, q, tables, n, 0.125, 0, scales, F32)
    ref.close(o[:1], want[0][:1], tol[0][:1])
    ref.close(e[:1], want[1][:1], tol[1][:1])
    assert torch.equal(o[1:].cpu(), torch.zeros(2, 4, 64)) and torch.equal(e[1:].cpu(), torch.full((2, 4), -math.inf))


def test_attend_nan_inside(ctx):
    """A NaN value inside a sequence reaches that sequence's heads only."""
    k, v, cache, q, tables, n, scales = make_attend(3, 4, 2, 64, 16, BF16, "hnd", [100, 50, 40], 12)
    want, tol = ref.attend(k, v, q, tables, n, 0.125, 0, scales, F32)
    cache.v[int(tables[1, 2]), 1, 5, 7] = float("nan")
    o, e = run_attend(ctx, cache, q, tables, n, 0.125, F32)
    assert torch.isnan(o[1, 2:, 7]).all()
    o[1, 2:, 7] = want[0][1, 2:, 7].float().cuda()
    ref.close(o, want[0], tol[0] + 1e-6)
    ref.close(e, want[1], tol[1])


def test_attend_wrong_pages_and_lengths(ctx):
    """A page outside the cache, a negative length or one over max_len: NaN for
    that sequence, the others as ever.  Page ids outside the range seen are not used."""
    k, v, cache, q, tables, n, scales = make_attend(7, 8, 2, 128, 16, BF16, "hnd", [300, 300, 300, 40, 300, 300, 64], 13)
    want, tol = ref.attend(k, v, q, tables, n, 0.1, 0, scales, F32)
    pages = k.shape[0]
    bad = tables.clone()
    bad[0, 18], bad[1, 0], bad[2, 7] = pages, -1, 2 ** 31 - 1
    bad[3, 3:], bad[6, 4:] = 2 ** 31 - 1, -2 ** 31
    m = n.clone()
    m[4], m[5] = -1, 305
    o, e = run_attend(ctx, cache, q, bad, m, 0.1, F32, max_len=304)
    for b in (0, 1, 2, 4, 5):
        assert torch.isnan(o[b]).all() and torch.isnan(e[b]).all(), b
    for b in (3, 6):
        ref.close(o[b], want[0][b], tol[0][b])
        ref.close(e[b], want[1][b], tol[1][b])
    # in a window, the pages before it are not used
    want, tol = ref.attend(k, v, q, tables, n, 0.1, 100, scales, F32)
    o, e = run_attend(ctx, cache, q, bad, n, 0.1, F32, window=100)
    assert torch.isnan(o[0]).all()
    for b in (1, 2, 3, 4, 5, 6):
        ref.close(o[b], want[0][b], tol[0][b])


def test_attend_far_offsets(ctx):
    """Pages whose elements sit past 2^32 bytes and 2^31 elements from the cache's start."""
    pages, H, page, D = 300, 2, 16, 128
    stride = 16 << 20                                     # elements from page to page: 300 of them pass 2^32
    base = [torch.zeros(stride * (pages - 1) + H * page * D, dtype=BF16, device="cuda") for _ in range(2)]
    k, v = (torch.as_strided(t, (pages, H, page, D), (stride, page * D, D, 1)) for t in base)
    g = torch.Generator().manual_seed(14)
    cpu = [torch.randn(pages, H, page, D, generator=g).to(BF16) for _ in range(2)]
    k.copy_(cpu[0])
    v.copy_(cpu[1])
    cache = dlp.kv_cache(k, v)
    q = torch.randn(1, 8, D, generator=g).to(BF16)
    tables, n = torch.randperm(pages, generator=g).int().view(1, -1), torch.tensor([pages * page - 5], dtype=torch.int32)
    want, tol = ref.attend(cpu[0], cpu[1], q, tables, n, 0.1, 0, (1., 1.), F32)
    o, e = run_attend(ctx, cache, q, tables, n, 0.1, F32)
    ref.close(o, want[0], tol[0])
    qkv = torch.randn(2, 4 * D, generator=g).to(BF16)
    dlp.proj_kv_append(ctx, cache, qkv.cuda(), torch.zeros(1, 0, device="cuda"), torch.zeros(2, dtype=torch.int32).cuda(),
                       torch.tensor([299 * 16 + 15, 0]).cuda())
    assert torch.equal(v[299, :, 15].cpu(), qkv[0, 2 * D:].view(2, D)) and torch.equal(k[0, :, 0].cpu(), qkv[1, :2 * D].view(2, D))


def test_attend_same_bits_graph_and_stream(ctx):
    k, v, cache, q, tables, n, scales = make_attend(4, 8, 2, 128, 16, BF16, "hnd", [2000, 5, 700, 0], 15, poison=False)
    qd, td, nd = q.cuda(), tables.cuda(), n.cuda()
    first, lse = run_attend(ctx, cache, q, tables, n, 0.1, F32)
    assert torch.equal(run_attend(ctx, cache, q, tables, n, 0.1, F32, stream=torch.cuda.Stream())[0], first)
    o, e = torch.empty_like(first), torch.empty_like(lse)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        dlp.proj_kv_attend(ctx, cache, qd, td, nd, 0.1, o, lse=e)
    for i in range(4):
        m = torch.tensor([2000 - 300 * i, 5 + i, 700, i], dtype=torch.int32)
        m[3] = 0
        fresh = torch.randn(4, 8, 128).to(BF16)
        qd.copy_(fresh)
        nd.copy_(m)
        o.fill_(3.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        again, lse2 = run_attend(ctx, cache, fresh, tables, m, 0.1, F32)
        assert torch.equal(o, again) and torch.equal(e, lse2)


def test_append_then_attend_in_a_graph(ctx):
    """A decoding step's two calls, captured once and replayed as the sequences grow."""
    g0 = torch.Generator().manual_seed(16)
    B, Hq, H, D, page = 3, 8, 2, 128, 16
    k, v, cache, q, tables, n, scales = make_attend(B, Hq, H, D, page, BF16, "hnd", [40, 15, 0], 17, poison=False, spare=6)
    used = {int(x) for x in tables.flatten() if x >= 0}
    spare = [p for p in range(k.shape[0]) if p not in used]
    grown = torch.full((B, 5), -1, dtype=torch.int32)
    grown[:, :tables.shape[1]] = tables
    grown[1, 1], grown[2, 0] = spare[0], spare[1]
    rope = torch.randn(64, D, generator=g0)
    qkv = torch.zeros(B, (Hq + 2 * H) * D, dtype=BF16, device="cuda")
    pos, slots, nd = (torch.zeros(B, dtype=t, device="cuda") for t in (torch.int32, torch.int64, torch.int32))
    qd, td = torch.empty(B, Hq, D, dtype=BF16, device="cuda"), grown.cuda()
    o, rd = torch.empty(B, Hq, D, device="cuda"), rope.cuda()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        dlp.proj_kv_append(ctx, cache, qkv, rd, pos, slots, qd)
        dlp.proj_kv_attend(ctx, cache, qd, td, nd, 0.1, o)
    for step in range(4):
        x = torch.randn(B, (Hq + 2 * H) * D, generator=g0).to(BF16)
        p = n + step
        sl = torch.tensor([int(grown[b, int(p[b]) // page]) * page + int(p[b]) % page for b in range(B)])
        (_, kk, vv), _ = ref.append(k, v, x, rope, p, sl, Hq, scales, False)
        qkv.copy_(x)
        pos.copy_(p)
        slots.copy_(sl)
        nd.copy_(p + 1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        k, v = cache.k.cpu().clone(), cache.v.cpu().clone()
        assert float((k.double() - kk).abs().max()) < 0.1 and torch.equal(v.double(), vv)
        want, tol = ref.attend(k, v, qd.cpu(), grown, p + 1, 0.1, 0, scales, F32)
        ref.close(o, want[0], tol[0])


# ---------------------------------------------------------------- refusals

def test_refusals(ctx):
    k, v, cache, q, tables, n, scales = make_attend(2, 8, 2, 128, 16, BF16, "hnd", [40, 30], 18, poison=False)
    qd, td, nd = q.cuda(), tables.cuda(), n.cuda()
    out = torch.empty(2, 8, 128, device="cuda")
    ok = dict(q=qd, tables=td, lengths=nd, scale=0.1, out=out)
    dlp.proj_kv_attend(ctx, cache, **ok)

    def refused(error=ValueError, c=cache, **kw):
        with pytest.raises(error):
            dlp.proj_kv_attend(ctx, c, **{**ok, **kw})

    refused(q=q)
    refused(q=qd.float())
    refused(q=qd[:, :, :64])
    refused(q=qd.transpose(0, 1))
    refused(tables=td[:1])
    refused(tables=td.long())
    refused(lengths=nd.long())
    refused(lengths=nd[:1])
    refused(out=out[:, :4])
    refused(out=out.half())
    refused(lse=torch.empty(2, 7, device="cuda"))
    refused(dlp.ProjError, max_len=td.shape[1] * 16 + 1)
    refused(dlp.ProjError, window=-1)
    refused(dlp.ProjError, scale=float("nan"))
    refused(dlp.ProjError, q=qd[:, :7], out=torch.empty(2, 7, 128, device="cuda"))
    refused(dlp.ProjError, out=cache.k.view(-1)[:2 * 8 * 128].view(2, 8, 128))
    with pytest.raises(ValueError):
        dlp.kv_cache(cache.k, cache.v[:1])
    with pytest.raises(ValueError):
        dlp.kv_cache(cache.k.transpose(2, 3), cache.v.transpose(2, 3))
    with pytest.raises(ValueError):
        dlp.kv_cache(cache.k.half(), cache.v.half())
    odd = dlp.kv_cache(torch.zeros(2, 1, 16, 72, dtype=BF16, device="cuda"), torch.zeros(2, 1, 16, 72, dtype=BF16, device="cuda"))
    with pytest.raises(dlp.ProjError) as e:
        dlp.proj_kv_attend(ctx, odd, torch.zeros(1, 1, 72, dtype=BF16, device="cuda"), td[:1], nd[:1], 0.1,
                           torch.empty(1, 1, 72, device="cuda"))
    assert e.value.status == dlp.PROJ_ERR_UNSUPPORTED
    three = torch.zeros(2, 1, 3, 64, dtype=BF16, device="cuda")
    with pytest.raises(dlp.ProjError):
        dlp.proj_kv_attend(ctx, dlp.kv_cache(three, three.clone()), torch.zeros(1, 1, 64, dtype=BF16, device="cuda"), td[:1],
                           nd[:1], 0.1, torch.empty(1, 1, 64, device="cuda"))
    scaled = dlp.kv_cache(cache.k, cache.v, 0.5, 1.0)     # a bf16 cache has no scales
    refused(dlp.ProjError, c=scaled)

    qkv = torch.zeros(2, 12 * 128, dtype=BF16, device="cuda")
    good = dict(qkv=qkv, rope=torch.zeros(4, 128, device="cuda"), positions=torch.zeros(2, dtype=torch.int32, device="cuda"),
                slots=torch.zeros(2, dtype=torch.int64, device="cuda"), q_out=torch.empty(2, 8, 128, dtype=BF16, device="cuda"))

    def not_appended(error=ValueError, **kw):
        with pytest.raises(error):
            dlp.proj_kv_append(ctx, cache, **{**good, **kw})

    dlp.proj_kv_append(ctx, cache, **good)
    not_appended(qkv=qkv[:, :-1])
    not_appended(qkv=qkv.float())
    not_appended(qkv=qkv[:, :128])
    not_appended(q_heads=7)
    not_appended(rope=good["rope"].double())
    not_appended(positions=good["positions"].long())
    not_appended(slots=good["slots"].int())
    not_appended(q_out=good["q_out"][:1])
    not_appended(dlp.ProjError, rope=torch.zeros(4, 130, device="cuda"))
    not_appended(dlp.ProjError, rope=torch.zeros(4, 3, device="cuda"))
    not_appended(dlp.ProjError, q_out=qkv[0, :0].new_empty(0).set_(qkv.untyped_storage(), 0, (2, 8, 128), (1024, 128, 1)))
