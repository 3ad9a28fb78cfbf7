"""Plain 64-bit forms of the decoding operators, on the CPU, with the error
each fp32 kernel may have beside its output's own rounding.  Nothing here is
shared with the library."""
import math

import torch

EPS32 = 2.0 ** -24            # half a step of fp32, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24, torch.float8_e4m3fn: 2.0 ** -4}


def unpack(codes):
    """int32 words [N, K / 8] -> codes [N, K]."""
    w = codes.long() & 0xFFFFFFFF
    parts = [(w >> (4 * (j // 2) + 16 * (j % 2))) & 15 for j in range(8)]
    return torch.stack(parts, -1).reshape(codes.shape[0], -1)


def pack(q):
    q = q.long().reshape(q.shape[0], -1, 8)
    w = sum(q[..., j] << (4 * (j // 2) + 16 * (j % 2)) for j in range(8))
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def weights(codes, scales, zeros, group):
    c = unpack(codes).double()
    g = torch.arange(c.shape[1]) // group
    z = 8.0 if zeros is None else zeros.double()[:, g]
    return (c - z) * scales.double()[:, g]


def quant(X, codes, scales, zeros, group, bias, epilogue, out):
    """(Y, tolerance), for X of zero mean.  The partial sums of K such terms
    grow as sqrt(k), so their K roundings, each 2^-24 of a partial sum, add up
    to about half of 2^-24 times the terms' whole size, sum |term|; 8 covers
    the largest of many outputs.  The terms may be taken as (16 + c) x less
    (16 + z) times the sum of x: at most 47 |x| s each."""
    W = weights(codes, scales, zeros, group)
    K = W.shape[1]
    x = X.double()
    y = x @ W.t()
    g = torch.arange(K) // group
    size = 47.0 * (x.abs() @ scales.double().abs()[:, g].t())
    tol = 8 * EPS32 * size
    if epilogue & 1:
        y = y + bias.double()
        tol = tol + EPS32 * (y.abs() + bias.double().abs())
    if epilogue & 2:
        # slope at most 1.13; the exponential's argument reaches 2^7 before the result vanishes
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
        tol = 1.13 * tol + 2.0 ** -16 * y.abs() + 1e-30
    return y, tol + HALF[out] * (y.abs() + tol)


def rotate(x, cos, sin, rot, interleaved):
    """x [T, H, D] float64 -> rotated."""
    y, h = x.clone(), rot // 2
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :h], x[..., h:rot])
    ya, yb = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = ya, yb
    else:
        y[..., :h], y[..., h:rot] = ya, yb
    return y


def append(k, v, qkv, rope, positions, slots, q_heads, scales, interleaved):
    """(q, k, v) in float64 and their tolerances; k and v [pages, heads, page, D] as stored values."""
    pages, heads, page, D = k.shape
    T, rot = qkv.shape[0], rope.shape[1]
    x = qkv.double().view(T, -1, D)
    known = (positions >= 0) & (positions < rope.shape[0]) if rot else torch.ones(T, dtype=torch.bool)
    row = rope.double()[positions.long().clamp(0, max(0, rope.shape[0] - 1))] if rope.shape[0] else torch.zeros(T, rot).double()
    cos, sin = row[:, None, :rot // 2], row[:, None, rot // 2:]
    y = rotate(x[:, :q_heads + heads], cos, sin, rot, interleaved)
    # two products and a sum in fp32
    size = rotate(x[:, :q_heads + heads].abs(), cos.abs(), -sin.abs(), rot, interleaved).abs() + \
        rotate(x[:, :q_heads + heads].abs(), cos.abs(), sin.abs(), rot, interleaved).abs()
    q, qtol = y[:, :q_heads].clone(), 4 * EPS32 * size[:, :q_heads]
    q[~known] = float("nan")
    out, tol = [], []
    for i, (cache, new, s) in enumerate(((k, y[:, q_heads:], size[:, q_heads:]),
                                         (v, x[:, q_heads + heads:], torch.zeros_like(x[:, :heads])))):
        c, t = cache.double().clone(), torch.zeros_like(cache.double())
        for n in range(T):
            slot = int(slots[n])
            if bool(known[n]) and 0 <= slot < pages * page:
                val, err = new[n], 4 * EPS32 * s[n]
                if cache.dtype == torch.float8_e4m3fn:
                    val, err = (val / scales[i]).clamp(-448, 448), err / scales[i]
                    err = err + 4 * EPS32 * val.abs()
                    err = err + HALF[cache.dtype] * val.abs() + 2.0 ** -10   # e4m3's smallest step is 2^-9
                else:
                    err = err + HALF[cache.dtype] * val.abs()
                c[slot // page, :, slot % page], t[slot // page, :, slot % page] = val, err
        out.append(c)
        tol.append(t)
    return (q, out[0], out[1]), (qtol + HALF[torch.bfloat16] * q.abs(), tol[0], tol[1])


def attend(k, v, q, tables, lengths, scale, window, scales, out):
    """(o, lse) in float64 and their tolerances."""
    B, Hq, D = q.shape
    _, heads, page, _ = k.shape
    per = Hq // heads
    o, lse = torch.zeros(B, Hq, D).double(), torch.full((B, Hq), -math.inf).double()
    otol, ltol = torch.zeros_like(o), torch.zeros_like(lse)
    for b in range(B):
        n = int(lengths[b])
        first = max(0, n - window) if window else 0
        if n <= first:
            continue
        t = torch.arange(first, n)
        pg = tables[b, t // page].long()
        for h in range(heads):
            K, V = k[pg, h, t % page].double() * scales[0], v[pg, h, t % page].double() * scales[1]
            Q = q[b, h * per:(h + 1) * per].double()
            w = scale * (Q @ K.t())
            # a logit's fp32 sum of D terms, the exponential's argument and value, and the fp32 sums over t
            d = EPS32 * (8 * math.sqrt(D) * abs(scale) * (Q.abs() @ K.abs().t()) + 8 * w.abs() + 32).amax(1, keepdim=True)
            p = torch.softmax(w, 1)
            s = slice(h * per, (h + 1) * per)
            o[b, s], lse[b, s] = p @ V, torch.logsumexp(w, 1)
            otol[b, s] = 2 * d * (p @ V.abs()) + 8 * EPS32 * math.sqrt(n) * (p.square() @ V.square()).sqrt()
            ltol[b, s] = 2 * d[:, 0] + 2 * EPS32 * lse[b, s].abs()
    return (o, lse), (otol + HALF[out] * (o.abs() + otol) + 1e-37, ltol)


def close(got, want, tol):
    """Raise unless |got - want| <= tol everywhere, with NaN and infinities in the same places."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)])
    off = (got - want).abs()[fine] - tol[fine]
    if off.numel():
        at = int(off.argmax())
        assert float(off.max()) <= 0, "off by %g beyond the tolerance: got %r, want %r, tolerance %g" % (
            float(off.max()), float(got[fine][at]), float(want[fine][at]), float(tol[fine][at]))
