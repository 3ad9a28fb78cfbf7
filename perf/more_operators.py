"""The operators of a decoding layer in 8-bit integers, in their plain form, and the cases they are measured on.

Three operators:

  int     Y = epilogue(x_scale[m] * w_scale[n] * sum_k xq[m, k] wq[n, k] (+ bias)) with 8-bit integers xq and wq; tokens in bf16
          are first made integers row by row: xq = rint(127 x / max |x|), x_scale = max |x| / 127
  append  an RMS norm of each query and key head of a fused QKV projection's rows, then its rotary position, then keys and
          values stored into a paged cache
  shared  attention of one new token for each sequence of a batch whose first `prefix` tokens are the same pages for all

`run` computes them with elementary torch operations, or, where `own` is true, calls dense_linear_projection_amd.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
KV_TYPES = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
FP8_MAX = 448.0
EPS = 1e-6
_ctx = None


# ------------------------------------------------------------------- cases

def _int(name, M, K, N, tokens, bias=False, gelu=False, out="bf16"):
    c = {"op": "int", "M": M, "K": K, "N": N, "tokens": tokens, "bias": bias, "gelu": gelu, "out": out}
    return dict(c, name=name) if name else c


def _append(name, T, q_heads, kv_heads, dim, rot, page, kv, layout="hnd", interleaved=False, padding=False, weights="bf16",
            per_head=False):
    c = {"op": "append", "T": T, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "rot": rot, "page": page, "kv": kv,
         "layout": layout, "interleaved": interleaved, "padding": padding, "weights": weights, "per_head": per_head}
    return dict(c, name=name) if name else c


def _shared(name, B, q_heads, kv_heads, dim, prefix, own_len, page, kv, layout="hnd", window=0, empty=False, out="bf16"):
    c = {"op": "shared", "B": B, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "prefix": prefix, "own_len": own_len,
         "page": page, "kv": kv, "layout": layout, "window": window, "empty": empty, "out": out}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token through a narrow projection: a single user's decoding, where latency counts
        _int("int_m1_k8192_n1024", 1, 8192, 1024, "bf16"),
        # sixteen decoding sequences through the attention block's square projection
        _int("int_m16_k8192_n8192", 16, 8192, 8192, "bf16", bias=True),
        # sixty-four sequences through a wide projection whose tokens another projection has made integers already
        _int("int_m64_k8192_n28672", 64, 8192, 28672, "int8", gelu=True),
        # a small head with odd sizes: rows of 1000, a ragged edge in every direction, fp32 result
        _int("int_m300_k1000_n515", 300, 1000, 515, "bf16", bias=True, out="f32"),
        # a prompt through the feed-forward layer's first projection
        _int("int_m4096_k8192_n8192", 4096, 8192, 8192, "bf16", bias=True, gelu=True),
        # the new tokens of sixteen sequences in one decoding step
        _append("append_t16", 16, 64, 8, 128, 128, 16, "bf16"),
        # a long prompt stored into an 8-bit cache
        _append("append_t8192_fp8", 8192, 64, 8, 128, 128, 64, "fp8"),
        # a ragged batch padded to its graph's size: partial rotation, neighbouring pairs, token-major pages, weights of each head
        _append("append_t333_odd", 333, 15, 5, 80, 32, 32, "bf16", "nhd", True, True, "f32", True),
        # a few answers sampled from one short prompt
        _shared("shared_b4_p500", 4, 32, 8, 128, 500, 100, 16, "bf16"),
        # a serving batch behind one system prompt
        _shared("shared_b64_p8192", 64, 64, 8, 128, 8192, 1000, 32, "bf16"),
        # a large batch of questions about one long document
        _shared("shared_b256_p32768", 256, 64, 8, 128, 32768, 1000, 64, "bf16"),
        # an 8-bit token-major cache, a prefix that ends inside a page, empty places in the batch, fp32 result
        _shared("shared_b48_fp8_p3001", 48, 20, 4, 96, 3001, 700, 16, "fp8", "nhd", 0, True, "f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("int", "append", "shared"))
    if op == "int":
        while True:
            M, N, K = _log(rng, 1, 4096), _log(rng, 64, 28672), _log(rng, 128, 16384)
            if M * N * K <= 4096 * 8192 * 8192 and N * K <= 28672 * 8192:
                break
        K = K if rng.random() < 0.3 else -(-K // 64) * 64
        return _int(None, M, K, N, rng.choice(("bf16", "bf16", "int8")), rng.random() < 0.5, rng.random() < 0.3,
                    rng.choice(("bf16", "bf16", "f32")))
    dim = rng.choice((64, 64, 80, 96, 128, 128, 128, 192, 256))
    page, kv, layout = rng.choice((16, 32, 64, 128)), rng.choice(("bf16", "bf16", "fp8")), rng.choice(("hnd", "nhd"))
    if op == "append":
        while True:
            T, kv_heads, per = _log(rng, 1, 8192), _log(rng, 1, 16), _log(rng, 1, 12)
            if T * kv_heads * (per + 2) * dim <= 8192 * 80 * 128:
                break
        rot = dim if rng.random() < 0.7 else 2 * rng.randint(1, dim // 2)
        return _append(None, T, kv_heads * per, kv_heads, dim, rot, page, kv, layout, rng.random() < 0.4,
                       rng.random() < 0.4, rng.choice(("bf16", "f32")), rng.random() < 0.3)
    while True:
        B, kv_heads, per = _log(rng, 1, 256), _log(rng, 1, 16), _log(rng, 1, 16)
        prefix, own_len = _log(rng, 16, 65536), _log(rng, 1, 2000)
        if B * kv_heads * per * dim * (prefix + own_len) <= 256 * 64 * 128 * 33000 and \
                kv_heads * dim * (prefix + B * own_len) <= 8 * 128 * 300000:
            break
    window = _log(rng, 1, prefix + own_len) if rng.random() < 0.2 else 0
    return _shared(None, B, kv_heads * per, kv_heads, dim, prefix, own_len, page, kv, layout, window, rng.random() < 0.4,
                   rng.choice(("bf16", "bf16", "f32")))


# ------------------------------------------------------------------ inputs

def _lengths(c):
    """The batch's lengths, prefix and own tokens together: own ones over the range as in a mixed batch, the first the longest."""
    r = random.Random(c["B"] * 1000003 + c["own_len"])
    n = [c["own_len"]] + [int(c["own_len"] * r.random() + 0.5) for _ in range(c["B"] - 1)]
    return [0 if c["empty"] and i % 7 == 5 else c["prefix"] + x for i, x in enumerate(n)]


def _gen(seed):
    return torch.Generator(device=DEVICE).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE)


def _pages(c, count, g, kv):
    """A cache of `count` pages, [pages, heads, page, dim], stored head-major or (layout nhd) token-major."""
    H, P, D = c["kv_heads"], c["page"], c["dim"]
    shape = (count, H, P, D) if c["layout"] == "hnd" else (count, P, H, D)
    t = torch.empty(shape, device=DEVICE, dtype=KV_TYPES[kv])
    step = max(1, (1 << 27) // (H * P * D))
    for i in range(0, count, step):
        part = _randn(g, *((min(step, count - i),) + shape[1:]))
        t[i:i + step] = (part * 8 if kv == "fp8" else part).to(t.dtype)
    return t if c["layout"] == "hnd" else t.transpose(1, 2)


def _codes(g, rows, K, padded):
    """8-bit integers of normally distributed values, rows padded with zeros to a multiple of 16."""
    q = torch.zeros(rows, padded, dtype=torch.int8, device=DEVICE)
    step = max(1, (1 << 27) // K)
    for i in range(0, rows, step):
        q[i:i + step, :K] = (_randn(g, min(step, rows - i), K) * 32).round_().clamp_(-127, 127)
    return q


def _context():
    import dense_linear_projection_amd as dlp
    global _ctx
    if _ctx is None:
        _ctx = dlp.proj_create(torch.cuda.current_device())
    return _ctx


def _epilogue(c):
    return (1 if c["bias"] else 0) | (2 if c["gelu"] else 0)


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"op": c["op"], "c": c}
    out = torch.float32 if c.get("out") == "f32" else torch.bfloat16
    if c["op"] == "int":
        M, K, N = c["M"], c["K"], c["N"]
        padded = -(-K // 16) * 16
        s["W"] = _codes(g, N, K, padded)
        s["w_scales"] = (torch.rand(N, generator=g, device=DEVICE) + 0.5) / (32 * math.sqrt(K))
        if c["tokens"] == "int8":
            s["X"] = _codes(g, M, K, padded)
            s["x_scales"] = (torch.rand(M, generator=g, device=DEVICE) + 0.5) / 32
        else:  # activations: a few channels are much larger than the others
            s["X"] = (_randn(g, M, K) * (1 + 7 * (torch.rand(K, generator=g, device=DEVICE) < 0.01))).bfloat16()
        s["bias"] = (_randn(g, N) * 0.2).bfloat16() if c["bias"] else None
        s["Y"] = torch.empty(M, N, device=DEVICE, dtype=out)
    elif c["op"] == "append":
        T, Hq, Hkv, D, P = c["T"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
        s["qkv"] = (_randn(g, T, Hq + 2 * Hkv, D) * (torch.rand(Hq + 2 * Hkv, 1, generator=g, device=DEVICE) * 3 + 0.2))
        s["qkv"] = s["qkv"].flatten(1).bfloat16()
        for name, heads in (("q_norm", Hq), ("k_norm", Hkv)):
            w = 1 + 0.2 * _randn(g, *((heads, D) if c["per_head"] else (D,)))
            s[name] = w if c["weights"] == "f32" else w.bfloat16()
        pages = -(-T // P) + 8
        s["k"], s["v"] = _pages(c, pages, g, c["kv"]), _pages(c, pages, g, c["kv"])
        s["k_scale"], s["v_scale"] = (0.05, 0.03125) if c["kv"] == "fp8" else (1.0, 1.0)
        top = 16384
        angle = torch.outer(torch.arange(top, dtype=torch.float64),
                            1e4 ** (-torch.arange(c["rot"] // 2, dtype=torch.float64) * 2 / c["rot"])).to(DEVICE)
        s["rope"] = torch.cat((angle.cos(), angle.sin()), 1).float()
        s["positions"] = torch.randint(0, top, (T,), generator=g, device=DEVICE, dtype=torch.int32)
        s["slots"] = torch.randperm(pages * P, generator=g, device=DEVICE)[:T]
        if T > 64:  # a prompt's tokens follow one another
            s["slots"] = s["slots"].sort().values
            s["positions"] = s["positions"].sort().values
        if c["padding"]:
            s["slots"][1 + T - T // 8:] = -1
        s["q"] = torch.empty(T, Hq, D, device=DEVICE, dtype=torch.bfloat16)
    else:
        B, Hq, D, P, L = c["B"], c["q_heads"], c["dim"], c["page"], c["prefix"]
        order = torch.randperm(B, generator=g, device=DEVICE).tolist()
        lengths = [_lengths(c)[i] for i in order]
        need = [-(-max(0, n - L) // P) for n in lengths]
        first, width = -(-L // P), -(-c["own_len"] // P)
        pages = first + sum(need) + 4
        s["k"], s["v"] = _pages(c, pages, g, c["kv"]), _pages(c, pages, g, c["kv"])
        s["k_scale"], s["v_scale"] = (0.125, 0.125) if c["kv"] == "fp8" else (1.0, 1.0)
        s["q_in"] = (_randn(g, B, Hq, D) * 1.5).bfloat16()
        free = torch.randperm(pages, generator=g, device=DEVICE)
        s["prefix"] = free[:first].to(torch.int32)
        ends = [(free[first - 1], L % P)]
        table, at = torch.full((B, width), -1, device=DEVICE, dtype=torch.int32), first
        for b, n in enumerate(need):
            table[b, :n] = free[at:at + n].to(torch.int32)
            at += n
            if n:
                ends.append((free[at - 1], (lengths[b] - L) % P))
        for page, used in ends:  # what an allocator leaves behind a sequence's end
            if used:
                s["k"][page, :, used:] = float("nan")
                s["v"][page, :, used:] = float("nan")
        s["tables"], s["lengths"] = table, torch.tensor(lengths, dtype=torch.int32).to(DEVICE)
        s["scale"] = 1 / math.sqrt(D)
        s["O"] = torch.empty(B, Hq, D, device=DEVICE, dtype=out)
        s["lse"] = torch.empty(B, Hq, device=DEVICE)
    if own:  # the handles that a program keeps
        import dense_linear_projection_amd as dlp
        s["ctx"] = _context()
        if c["op"] != "int":
            s["cache"] = dlp.kv_cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s


# ------------------------------------------------------------- plain forms

def _plain_int(s):
    c = s["c"]
    x, k = s["X"].float(), s["W"].shape[1]
    if c["tokens"] == "bf16":
        top = x.abs().amax(1, keepdim=True)
        scale = (top / 127).squeeze(1)
        # a product of 8 and 7 bits over one of 8: the quotient is a half exactly or far from one
        x = torch.round(x * (127 / 128) / torch.where(top == 0, 1.0, top) * 128)
    else:
        scale = s["x_scales"]
    w, y = s["W"].float(), 0
    for i in range(0, k, 1024):  # 1024 products of integers below 2^7 sum exactly in 32 bits
        part = x[:, i:i + 1024]
        y = y + (part @ w[:, i:i + part.shape[1]].t()).to(torch.int32)
    y = (y.double() * scale.double().unsqueeze(1) * s["w_scales"].double()).float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if c["gelu"]:
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    return y.to(s["Y"].dtype)


def _rotate(x, cos, sin, rot, interleaved):
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y, z = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((y, z), -1).flatten(-2) if interleaved else torch.cat((y, z), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _stored(x, scale, dtype):
    return (x / scale).clamp(-FP8_MAX, FP8_MAX).to(dtype) if dtype == torch.float8_e4m3fn else x.to(dtype)


def _plain_append(s):
    c = s["c"]
    T, Hq, Hkv, D, P, rot = c["T"], c["q_heads"], c["kv_heads"], c["dim"], c["page"], c["rot"]
    x = s["qkv"].float().view(T, Hq + 2 * Hkv, D)
    y = x[:, :Hq + Hkv]
    w = torch.cat([s[name].float().expand(heads, D) for name, heads in (("q_norm", Hq), ("k_norm", Hkv))])
    y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * w
    row = s["rope"][s["positions"].long()].unsqueeze(1)
    y = _rotate(y, row[..., :rot // 2], row[..., rot // 2:], rot, c["interleaved"])
    # padding tokens store the first stored token once more, in its own place
    kept = s["slots"] >= 0
    token = torch.where(kept, torch.arange(T, device=DEVICE), kept.int().argmax())
    slot = s["slots"][token]
    page, place = slot // P, slot % P
    s["k"][page, :, place] = _stored(y[:, Hq:][token], s["k_scale"], s["k"].dtype)
    s["v"][page, :, place] = _stored(x[:, Hq + Hkv:][token], s["v_scale"], s["v"].dtype)
    return {"q": y[:, :Hq].bfloat16(), "k": s["k"], "v": s["v"]}


def _plain_shared(s):
    c = s["c"]
    B, Hq, Hkv, D, P, L, O = c["B"], c["q_heads"], c["kv_heads"], c["dim"], c["page"], c["prefix"], c["own_len"]
    n = s["lengths"].long()
    low = n - c["window"] if c["window"] else torch.zeros_like(n)
    t = torch.arange(L + O, device=DEVICE)
    seen = (t < n[:, None]) & (t >= low[:, None])
    o, lse = [], []
    tp, to = t[:L], t[:O]
    page = s["prefix"].long()[tp // P]
    own_page = s["tables"].long().clamp(min=0)[:, to // P]
    for h in range(Hkv):  # one key-value head at a time
        q = s["q_in"].float().view(B, Hkv, Hq // Hkv, D)[:, h]
        k, v = (s[x][page, h, tp % P].float() * s[x + "_scale"] for x in ("k", "v"))
        k2, v2 = (s[x][own_page, h, to % P].float() * s[x + "_scale"] for x in ("k", "v"))
        v2 = torch.where(seen[:, L:, None], v2, 0.0)
        w = torch.cat(((q.flatten(0, 1) @ k.t()).view(B, -1, L), q @ k2.transpose(1, 2).contiguous()), 2) * s["scale"]
        w = torch.where(seen[:, None], w, -math.inf)
        top = w.amax(-1, keepdim=True)
        w = torch.exp(w - torch.where(top == -math.inf, 0.0, top))
        total = w.sum(-1, keepdim=True)
        a = (w[..., :L].flatten(0, 1) @ v).view(B, -1, D) + w[..., L:] @ v2
        o.append(a / torch.where(total == 0, 1.0, total))
        lse.append((top + torch.log(total)).squeeze(-1))
    return {"o": torch.cat(o, 1).to(s["O"].dtype), "lse": torch.cat(lse, 1)}


def run(state):
    s, c = state, state["c"]
    if own:
        import dense_linear_projection_amd as dlp
        if s["op"] == "int":
            if c["tokens"] == "int8":
                dlp.proj_run_int(s["ctx"], s["X"], s["x_scales"], s["W"], s["w_scales"], s["bias"], _epilogue(c), s["Y"])
            else:
                dlp.proj_run_int_dynamic(s["ctx"], s["X"], s["W"], s["w_scales"], s["bias"], _epilogue(c), s["Y"])
            return s["Y"]
        if s["op"] == "append":
            dlp.proj_kv_append_norm(s["ctx"], s["cache"], s["qkv"], s["q_norm"], s["k_norm"], EPS, s["rope"], s["positions"],
                                    s["slots"], s["q"], interleaved=c["interleaved"])
            return {"q": s["q"], "k": s["k"], "v": s["v"]}
        dlp.proj_kv_attend_shared(s["ctx"], s["cache"], s["q_in"], s["prefix"], c["prefix"], s["tables"], s["lengths"],
                                  s["scale"], s["O"], lse=s["lse"], window=c["window"], max_len=c["prefix"] + c["own_len"])
        return {"o": s["O"], "lse": s["lse"]}
    return {"int": _plain_int, "append": _plain_append, "shared": _plain_shared}[s["op"]](s)


# ----------------------------------------------------------- work and exact

def work(case):
    c = case
    if c["op"] == "int":
        M, K, N = c["M"], c["K"], c["N"]
        b = N * K + 4 * N + M * K * (1 if c["tokens"] == "int8" else 2) + (4 * M if c["tokens"] == "int8" else 0)
        return {"bytes": b + (2 * N if c["bias"] else 0) + M * N * (4 if c["out"] == "f32" else 2), "flops": 2 * M * N * K}
    e = 1 if c["kv"] == "fp8" else 2
    if c["op"] == "append":
        T, D, Hq, Hkv = c["T"], c["dim"], c["q_heads"], c["kv_heads"]
        stored = T - max(0, T // 8 - 1) if c["padding"] else T
        b = T * (Hq + 2 * Hkv) * D * 2 + T * Hq * D * 2 + stored * 2 * Hkv * D * e + T * 12 + min(T, 16384) * c["rot"] * 4
        b += ((Hq + Hkv) if c["per_head"] else 2) * D * (4 if c["weights"] == "f32" else 2)
        return {"bytes": b, "flops": T * (Hq + Hkv) * (3 * c["rot"] + 4 * D)}
    L, n = c["prefix"], _lengths(c)
    low = [max(0, x - c["window"]) if c["window"] else 0 for x in n]
    first = min([L] + [a for a, x in zip(low, n) if x])  # the prefix from here on is seen by a sequence
    tokens = (L - first if any(n) else 0) + sum(x - max(a, L) for a, x in zip(low, n) if x > L)
    rows = c["B"] * c["q_heads"]
    b = tokens * c["kv_heads"] * c["dim"] * 2 * e + rows * c["dim"] * (2 + (4 if c["out"] == "f32" else 2)) + rows * 4
    return {"bytes": b + 4 * (tokens // c["page"]), "flops": 4 * sum(x - a for a, x in zip(low, n)) * c["q_heads"] * c["dim"]}


def _exact_int(s):
    c = s["c"]
    X, scale = s["X"].double(), None
    if c["tokens"] == "bf16":
        peak = torch.linalg.vector_norm(X, ord=math.inf, dim=1)
        scale = peak / 127
        X = torch.round(127 * X / torch.where(peak > 0, peak, 1.0)[:, None])
    else:
        scale = s["x_scales"].double()
    parts, step = [], max(1, (1 << 28) // s["W"].shape[1])
    for i in range(0, c["N"], step):
        W = s["W"][i:i + step, :X.shape[1]].double() * s["w_scales"][i:i + step, None].double()
        parts.append(torch.matmul(W, X.t()).t())
    y = torch.cat(parts, 1) * scale[:, None]
    if s["bias"] is not None:
        y += s["bias"].double()
    if c["gelu"]:
        y = y / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
    return y


def _exact_append(s):
    c = s["c"]
    T, Hq, Hkv, D, P, h = c["T"], c["q_heads"], c["kv_heads"], c["dim"], c["page"], c["rot"] // 2
    heads = s["qkv"].double().view(T, -1, D)
    for name, first, count in (("q_norm", 0, Hq), ("k_norm", Hq, Hkv)):
        part = heads[:, first:first + count]
        size = torch.linalg.vector_norm(part, dim=2, keepdim=True)
        heads[:, first:first + count] = part * s[name].double() * torch.rsqrt(size ** 2 / D + EPS)
    table = s["rope"].double()[s["positions"].long()]
    turn = torch.complex(table[:, :h], table[:, h:])[:, None]
    one, two = (2 * torch.arange(h), 2 * torch.arange(h) + 1) if c["interleaved"] else (torch.arange(h), torch.arange(h) + h)
    turned = torch.complex(heads[..., one], heads[..., two])[:, :Hq + Hkv] * turn
    heads[:, :Hq + Hkv, one], heads[:, :Hq + Hkv, two] = turned.real, turned.imag
    out = {"q": heads[:, :Hq]}
    kept = torch.nonzero(s["slots"] >= 0).flatten()
    for name, first in (("k", Hq), ("v", Hq + Hkv)):
        new = heads[kept, first:first + Hkv]
        if c["kv"] == "fp8":
            new = torch.clip(new / s[name + "_scale"], -FP8_MAX, FP8_MAX)
        cache = s[name].double()
        for i in range(Hkv):
            cache[s["slots"][kept] // P, i, s["slots"][kept] % P] = new[:, i]
        out[name] = cache
    return out


def _exact_shared(s):
    c = s["c"]
    B, Hq, Hkv, D, P, L = c["B"], c["q_heads"], c["kv_heads"], c["dim"], c["page"], c["prefix"]
    o = torch.zeros(B, Hq, D, dtype=torch.float64, device=DEVICE)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=DEVICE)
    lengths = s["lengths"].tolist()
    for h in range(Hkv):
        rows = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
        K, V = (s[x][s["prefix"].long(), h].reshape(-1, D)[:L].double() * s[x + "_scale"] for x in ("k", "v"))
        for b, n in enumerate(lengths):
            if n == 0:
                continue
            first = max(0, n - c["window"]) if c["window"] else 0
            k, v = K[first:n], V[first:n]
            if n > L:
                pages = s["tables"][b, :-(-(n - L) // P)].long()
                k2, v2 = (s[x][pages, h].reshape(-1, D)[:n - L][max(0, first - L):].double() * s[x + "_scale"]
                          for x in ("k", "v"))
                k, v = torch.cat((k, k2)), torch.cat((v, v2))
            w = torch.matmul(s["q_in"][b, rows].double(), k.t()) * s["scale"]
            lse[b, rows] = torch.logsumexp(w, 1)
            o[b, rows] = torch.matmul(torch.softmax(w, 1), v)
    return {"o": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"int": _exact_int, "append": _exact_append, "shared": _exact_shared}[s["op"]](s)
