"""Plain 64-bit forms of a decoding layer's operators in 8-bit integers, of the
normed append and of attention over a shared prefix, on the CPU, with the error
each kernel may have. Nothing here is shared with the library."""
import math

import torch

from tests.decode_reference import EPS32, HALF, rotate

TINY = 2.0 ** -149                # the smallest step of fp32
# Below 2^-126 bf16 has the fixed step 2^-133 (2^-126 over 7 bits), so a result there is rounded by up to half of that, which
# is more than 2^-8 of it: 4.5e-39 lies between multiples of 9.2e-41 and is off by up to 4.6e-41, not 1.8e-41.
TINY_BF16 = 2.0 ** -134


def quantize_rows(X):
    """(q int64 [M, K], scales float64 [M], their fp32 rounding's tolerance): exact, for finite rows."""
    x = X.double()
    top = x.abs().amax(1) if x.shape[1] else torch.zeros(x.shape[0]).double()
    q = torch.round(127 * x / torch.where(top > 0, top, 1.0)[:, None])  # half to even
    return q.long(), top / 127


def product(X, x_scales, W, w_scales, bias, epilogue, out):
    """(Y, tolerance) of integers X and W: the sum is exact, one fp32 rounding after the scales, then those of bias and GELU."""
    y = (X.double() @ W.double().t()) * x_scales.double()[:, None] * w_scales.double()
    tol = 1.0001 * EPS32 * y.abs() + TINY
    if epilogue & 1:
        y = y + bias.double()
        tol = tol + EPS32 * (y.abs() + tol)
    if epilogue & 2:
        # slope at most 1.13; the exponential's argument reaches 2^7 before the result vanishes
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
        tol = 1.13 * tol + 2.0 ** -16 * y.abs() + 1e-30
    return y, tol + HALF[out] * (y.abs() + tol) + (TINY if out == torch.float32 else TINY_BF16)


def append_norm(k, v, qkv, q_norm, k_norm, eps, rope, positions, slots, q_heads, scales, interleaved):
    """(q, k, v) in float64 and their tolerances; k and v [pages, heads, page, D] as stored values. A normed element's roundings
    to fp32, each 2^-24: the head's sum of squares, 16 added in a row and up to 4 such sums (20, halved by the root: 10), the
    mean, two (1, halved), the root itself, good to a step (2), its product with x and that with the weight (2): 15. The
    rotation rounds two products and their sum."""
    pages, heads, page, D = k.shape
    T, rot = qkv.shape[0], rope.shape[1]
    x = qkv.double().view(T, -1, D)
    y, e = x[:, :q_heads + heads].clone(), torch.zeros(T, q_heads + heads, D).double()
    for w, a, b in ((q_norm, 0, q_heads), (k_norm, q_heads, q_heads + heads)):
        if w is not None:
            y[:, a:b] = x[:, a:b] / torch.sqrt((x[:, a:b] ** 2).mean(-1, keepdim=True) + eps) * w.double()
            e[:, a:b] = 15 * EPS32 * y[:, a:b].abs() + TINY
    known = (positions >= 0) & (positions < rope.shape[0]) if rot else torch.ones(T, dtype=torch.bool)
    row = rope.double()[positions.long().clamp(0, max(0, rope.shape[0] - 1))] if rope.shape[0] else torch.zeros(T, rot).double()
    cos, sin = row[:, None, :rot // 2], row[:, None, rot // 2:]
    z = rotate(y, cos, sin, rot, interleaved)
    # |a cos| + |b sin| and |b cos| + |a sin|: the larger of the sum and the difference
    size, err = (torch.maximum(rotate(t, cos.abs(), sin.abs(), rot, interleaved).abs(),
                               rotate(t, cos.abs(), -sin.abs(), rot, interleaved).abs()) for t in (y.abs(), e))
    err = err + 2.001 * EPS32 * (size + err) + TINY
    err[..., rot:] = e[..., rot:]
    q, qtol = z[:, :q_heads].clone(), err[:, :q_heads] + HALF[torch.bfloat16] * (z[:, :q_heads].abs() + err[:, :q_heads]) + TINY_BF16
    q[~known] = float("nan")
    out, tol = [], []
    for i, (cache, new, s) in enumerate(((k, z[:, q_heads:], err[:, q_heads:]),
                                         (v, x[:, q_heads + heads:], torch.zeros(T, heads, D).double()))):
        c, t = cache.double().clone(), torch.zeros_like(cache.double())
        for n in range(T):
            slot = int(slots[n])
            if bool(known[n]) and 0 <= slot < pages * page:
                val, off = new[n], s[n]
                if cache.dtype == torch.float8_e4m3fn:
                    val, off = (val / scales[i]).clamp(-448, 448), off / scales[i]
                    off = off + EPS32 * (val.abs() + off)                          # the quotient
                    off = off + HALF[cache.dtype] * (val.abs() + off) + 2.0 ** -10  # e4m3's smallest step is 2^-9
                else:
                    off = off + HALF[cache.dtype] * (val.abs() + off) + TINY_BF16
                c[slot // page, :, slot % page], t[slot // page, :, slot % page] = val, off
        out.append(c)
        tol.append(t)
    return (q, out[0], out[1]), (qtol, tol[0], tol[1])


def attend_shared(k, v, q, prefix, prefix_len, tables, lengths, scale, window, scales, out):
    """(o, lse) in float64 and their tolerances."""
    B, Hq, D = q.shape
    _, heads, page, _ = k.shape
    per = Hq // heads
    o, lse = torch.zeros(B, Hq, D).double(), torch.full((B, Hq), -math.inf).double()
    otol, ltol = torch.zeros_like(o), torch.zeros_like(lse)
    # terms of a probability in bf16 results: 8 bits cut, 8 more rounded
    terms = 2.0 ** -15 if out == torch.bfloat16 else 0.0
    for b in range(B):
        n = int(lengths[b])
        first = max(0, n - window) if window else 0
        if n <= first:
            continue
        t = torch.arange(first, n)
        shared, own = t[t < prefix_len], t[t >= prefix_len] - prefix_len
        pg = torch.cat((prefix[shared // page].long(), tables[b, own // page].long()))
        at = torch.cat((shared, own)) % page
        for h in range(heads):
            K, V = k[pg, h, at].double() * scales[0], v[pg, h, at].double() * scales[1]
            Q = q[b, h * per:(h + 1) * per].double()
            w = scale * (Q @ K.t())
            # a logit's fp32 sum of D terms, the exponential's argument and value, and the fp32 sums over t
            d = EPS32 * (8 * math.sqrt(D) * abs(scale) * (Q.abs() @ K.abs().t()) + 8 * w.abs() + 32).amax(1, keepdim=True)
            p = torch.softmax(w, 1)
            s = slice(h * per, (h + 1) * per)
            o[b, s], lse[b, s] = p @ V, torch.logsumexp(w, 1)
            otol[b, s] = (2 * d + terms) * (p @ V.abs()) + 8 * EPS32 * math.sqrt(n) * (p.square() @ V.square()).sqrt()
            ltol[b, s] = 2 * d[:, 0] + 2 * EPS32 * lse[b, s].abs()
    return (o, lse), (otol + HALF[out] * (o.abs() + otol) + 1e-37, ltol)
