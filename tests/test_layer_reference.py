"""The 64-bit forms that the GPU tests of a decoding layer compare with, on the
CPU against definitions written out one element at a time, and that a mistake in
them shows."""
import math
from fractions import Fraction

import pytest
import torch

from tests import layer_reference as ref
from tests.decode_reference import close

BF16, F32 = torch.bfloat16, torch.float32


def half_even(x):
    """A Fraction rounded to the nearest integer, ties to even."""
    low = x.numerator // x.denominator
    rest = x - low
    return low + (1 if rest > Fraction(1, 2) or (rest == Fraction(1, 2) and low % 2) else 0)


def test_rows_in_exact_arithmetic():
    g = torch.Generator().manual_seed(0)
    x = (torch.randn(6, 50, generator=g) * torch.tensor([1e-30, 1e-3, 1.0, 7.0, 1e20, 0.0])[:, None]).to(BF16)
    x[2, :4] = torch.tensor([2.0, 1.0, 127 / 128, -1.0])           # ties: 63.5 and its neighbours
    x[2, 4:] = x[2, 4:].clamp(-2, 2)
    q, s = ref.quantize_rows(x)
    for m in range(6):
        row = [Fraction(float(v)) for v in x[m]]
        top = max(abs(v) for v in row)
        assert [int(v) for v in q[m]] == [half_even(127 * v / top) if top else 0 for v in row]
        assert float(s[m]) == pytest.approx(float(top / 127), rel=1e-15)
    assert int(q[2, 1]) == 64 and int(q[2, 3]) == -64


def test_the_rounding_that_the_kernel_relies_on():
    """127 X / (A 2^j), X and A below 2^8, is a half exactly or further from one than 2^-16 of itself."""
    for A in range(128, 256):
        for X in range(128, 256):
            for j in range(0, 10):
                y = Fraction(127 * X, A << j)
                if X > A << j or y < Fraction(1, 4):
                    continue
                near = y.numerator * 2 // y.denominator
                for n in (near, near + 1):
                    if n % 2:
                        assert y == Fraction(n, 2) or abs(y - Fraction(n, 2)) >= y / 65536


def test_product():
    g = torch.Generator().manual_seed(1)
    X, W = (torch.randint(-128, 128, (r, 20), generator=g, dtype=torch.int8) for r in (3, 4))
    xs, ws, b = torch.rand(3, generator=g), torch.rand(4, generator=g), torch.randn(4, generator=g).to(BF16)
    for epi in range(4):
        y, _ = ref.product(X, xs, W, ws, b, epi, F32)
        for m in range(3):
            for n in range(4):
                v = sum(int(X[m, k]) * int(W[n, k]) for k in range(20)) * float(xs[m]) * float(ws[n]) + (float(b[n]) if epi & 1 else 0)
                if epi & 2:
                    v = 0.5 * v * (1 + math.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
                assert float(y[m, n]) == pytest.approx(v, rel=1e-12, abs=1e-300)


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_norm(interleaved):
    g = torch.Generator().manual_seed(2)
    Hq, H, D, rot, page = 2, 1, 8, 4, 4
    k, v = (torch.randn(2, H, page, D, generator=g).to(BF16) for _ in range(2))
    qkv, qn, kn = torch.randn(3, (Hq + 2 * H) * D, generator=g).to(BF16), torch.randn(Hq, D, generator=g), torch.randn(H, D, generator=g)
    rope, pos, slots = torch.randn(5, rot, generator=g), torch.tensor([4, 0, 2], dtype=torch.int32), torch.tensor([5, -1, 0])
    (q, kk, vv), _ = ref.append_norm(k, v, qkv, qn, kn, 1e-3, rope, pos, slots, Hq, (1, 1), interleaved)
    for t in range(3):
        for h in range(Hq + H):
            x = [float(e) for e in qkv[t, h * D:(h + 1) * D]]
            size = math.sqrt(sum(e * e for e in x) / D + 1e-3)
            w = qn[h] if h < Hq else kn[h - Hq]
            x = [e / size * float(w[d]) for d, e in enumerate(x)]
            y = list(x)
            for j in range(rot // 2):
                a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
                c, s = float(rope[pos[t], j]), float(rope[pos[t], rot // 2 + j])
                y[a], y[b] = x[a] * c - x[b] * s, x[b] * c + x[a] * s
            got = q[t, h] if h < Hq else kk[slots[t] // page, h - Hq, slots[t] % page] if slots[t] >= 0 else None
            if got is not None:
                assert [float(e) for e in got] == pytest.approx(y, rel=1e-12, abs=1e-14)
    assert torch.equal(vv[1, 0, 1], qkv[0, -D:].double()) and torch.equal(kk[0, :, 1:], k[0, :, 1:].double())


@pytest.mark.parametrize("window", [0, 4])
def test_attend_shared(window):
    g = torch.Generator().manual_seed(3)
    B, Hq, H, D, page, L = 5, 4, 2, 6, 4, 7
    k, v = (torch.randn(12, H, page, D, generator=g) for _ in range(2))
    q, prefix = torch.randn(B, Hq, D, generator=g), torch.tensor([9, 2])
    tables, lengths = torch.tensor([[0, 1], [3, -1], [-1, -1], [-1, -1], [5, 6]]), torch.tensor([13, 8, 0, 3, 15])
    (o, lse), _ = ref.attend_shared(k, v, q, prefix, L, tables, lengths, 0.4, window, (2.0, 3.0), F32)
    for b in range(B):
        n = int(lengths[b])
        for h in range(Hq):
            ws, vs = [], []
            for t in range(max(0, n - window) if window else 0, n):
                pg, at = (int(prefix[t // page]), t % page) if t < L else (int(tables[b, (t - L) // page]), (t - L) % page)
                ws.append(0.4 * 2 * float(q[b, h].double() @ k[pg, h // 2, at].double()))
                vs.append(3 * v[pg, h // 2, at].double())
            if not ws:
                assert not bool(o[b, h].any()) and float(lse[b, h]) == -math.inf
                continue
            total = sum(math.exp(w) for w in ws)
            want = sum(math.exp(w) / total * x for w, x in zip(ws, vs))
            assert float((o[b, h] - want).abs().max()) < 1e-12 and float(lse[b, h]) == pytest.approx(math.log(total), rel=1e-12)


def test_mistakes_show():
    """What the GPU tests are to catch, planted here: each is beyond the tolerance somewhere."""
    g = torch.Generator().manual_seed(4)
    X, W = (torch.randint(-127, 128, (r, 64), generator=g, dtype=torch.int8) for r in (4, 5))
    xs, ws, b = torch.rand(4, generator=g), torch.rand(5, generator=g), torch.randn(5, generator=g).to(BF16)
    want = ref.product(X, xs, W, ws, b, 1, F32)
    for wrong in ((X, xs, W.roll(1, 1), ws, b), (X, xs.roll(1), W, ws, b), (X, xs, W, ws, b.roll(1)), (X[:, :-1], xs, W[:, :-1], ws, b)):
        with pytest.raises(AssertionError):
            close(ref.product(*wrong, 1, F32)[0], *want)
    k, v = (torch.randn(8, 1, 4, 16, generator=g) for _ in range(2))
    q, prefix, tables, n = torch.randn(2, 2, 16, generator=g), torch.tensor([1, 4]), torch.tensor([[0], [2]]), torch.tensor([8, 10])
    call = lambda q=q, p=prefix, L=7, n=n, w=0: ref.attend_shared(k, v, q, p, L, tables, n, 0.3, w, (1, 1), BF16)  # noqa: E731
    want, tol = call()
    for wrong in (call(p=prefix.flip(0)), call(L=6), call(n=n - 1), call(w=5), call(q=q.roll(1, 1))):
        with pytest.raises(AssertionError):
            close(wrong[0][0], want[0], tol[0])
