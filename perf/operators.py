"""The decoding operators in their plain form, and the cases they are measured on.

Three operators, as one decoding step of an attention block meets them:

  quant   Y = epilogue(X . W^T (+ bias)) with 4-bit weights W[n, k] = scales[n, k / group] * (code[n, k] - zeros[n, k / group]);
          eight codes to an int32 word, code j of the eight at bits 4 * (j // 2) + 16 * (j % 2); without zeros the offset is 8
  append  rotary positions applied to the q and k heads of a fused QKV projection's rows, k and v stored into a paged cache
  attend  attention of one new token for each sequence over its pages

`run` computes them with elementary torch operations, or, where `own` is true, calls dense_linear_projection_amd.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
GROUPS = (32, 64, 128)
KV_TYPES = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
FP8_MAX = 448.0
_ctx = None


# ------------------------------------------------------------------- cases

def _quant(name, M, K, N, group, zeros, scales="bf16", bias=False, gelu=False, out="bf16"):
    c = {"op": "quant", "M": M, "K": K, "N": N, "group": group, "zeros": zeros, "scales": scales, "bias": bias,
         "gelu": gelu, "out": out}
    return dict(c, name=name) if name else c


def _append(name, T, q_heads, kv_heads, dim, rot, page, kv, layout="hnd", interleaved=False, padding=False):
    c = {"op": "append", "T": T, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "rot": rot, "page": page, "kv": kv,
         "layout": layout, "interleaved": interleaved, "padding": padding}
    return dict(c, name=name) if name else c


def _attend(name, B, q_heads, kv_heads, dim, max_len, page, kv, layout="hnd", window=0, empty=False, out="bf16"):
    c = {"op": "attend", "B": B, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "max_len": max_len, "page": page,
         "kv": kv, "layout": layout, "window": window, "empty": empty, "out": out}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token through a narrow projection: a single user's decoding, where latency counts
        _quant("quant_m1_k8192_n1024", 1, 8192, 1024, 128, True),
        # sixteen decoding sequences through the attention block's square projection
        _quant("quant_m16_k8192_n8192", 16, 8192, 8192, 128, False, bias=True),
        # sixty-four sequences through the feed-forward layer's first projection, with its activation
        _quant("quant_m64_k8192_n28672", 64, 8192, 28672, 64, True, gelu=True),
        # a small head with odd sizes: a last group that is short, fp32 scales and an fp32 result
        _quant("quant_m7_k1000_n515", 7, 1000, 515, 32, True, scales="f32", bias=True, out="f32"),
        # a prompt through the same 4-bit weights
        _quant("quant_m1024_k8192_n8192", 1024, 8192, 8192, 128, False),
        # the new tokens of sixteen sequences in one decoding step
        _append("append_t16", 16, 64, 8, 128, 128, 16, "bf16"),
        # a long prompt stored into an 8-bit cache
        _append("append_t8192_fp8", 8192, 64, 8, 128, 128, 64, "fp8"),
        # a ragged batch padded to its graph's size: partial rotation, neighbouring pairs, token-major pages
        _append("append_t333_odd", 333, 15, 5, 80, 32, 32, "bf16", "nhd", True, True),
        # one short conversation
        _attend("attend_b1_len500", 1, 32, 8, 128, 500, 16, "bf16"),
        # one very long document
        _attend("attend_b1_len131072", 1, 64, 8, 128, 131072, 64, "bf16"),
        # a serving batch of mixed lengths
        _attend("attend_b32_len16384", 32, 64, 8, 128, 16384, 32, "bf16"),
        # a batch on an 8-bit token-major cache with a sliding window, empty places in the batch, fp32 result
        _attend("attend_b48_fp8_window", 48, 20, 4, 96, 4097, 16, "fp8", "nhd", 1500, True, "f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quant", "append", "attend"))
    if op == "quant":
        while True:
            M, N, K = _log(rng, 1, 1024), _log(rng, 64, 28672), 8 * _log(rng, 16, 1024)
            if M * N * K <= 1024 * 8192 * 8192 and N * K <= 28672 * 8192:
                break
        return _quant(None, M, K, N, rng.choice(GROUPS), rng.random() < 0.5, rng.choice(("bf16", "f32")),
                      rng.random() < 0.5, rng.random() < 0.3, rng.choice(("bf16", "bf16", "f32")))
    dim = rng.choice((64, 64, 80, 96, 128, 128, 128, 192, 256))
    page, kv, layout = rng.choice((16, 32, 64, 128)), rng.choice(("bf16", "bf16", "fp8")), rng.choice(("hnd", "nhd"))
    if op == "append":
        while True:
            T, kv_heads, per = _log(rng, 1, 8192), _log(rng, 1, 16), _log(rng, 1, 12)
            if T * kv_heads * (per + 2) * dim <= 8192 * 80 * 128:
                break
        rot = dim if rng.random() < 0.7 else 2 * rng.randint(1, dim // 2)
        return _append(None, T, kv_heads * per, kv_heads, dim, rot, page, kv, layout, rng.random() < 0.4,
                       rng.random() < 0.4)
    while True:
        B, kv_heads, per, length = _log(rng, 1, 256), _log(rng, 1, 16), _log(rng, 1, 20), _log(rng, 1, 131072)
        if B * kv_heads * dim * length <= 20 * 16384 * 8 * 128:
            break
    window = _log(rng, 1, length) if rng.random() < 0.25 else 0
    return _attend(None, B, kv_heads * per, kv_heads, dim, length, page, kv, layout, window, rng.random() < 0.4,
                   rng.choice(("bf16", "bf16", "f32")))


# ------------------------------------------------------------------ inputs

def _lengths(c):
    """The batch's lengths: the first is the longest, the others fall over the range as a mixed batch's do."""
    r = random.Random(c["B"] * 1000003 + c["max_len"])
    n = [c["max_len"]] + [max(1, int(c["max_len"] * (0.05 + 0.95 * r.random()))) for _ in range(c["B"] - 1)]
    if c["empty"]:
        n = [0 if i % 7 == 5 else x for i, x in enumerate(n)]
    return n


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
    if c["op"] == "quant":
        M, K, N, G = c["M"], c["K"], c["N"], c["group"]
        s["X"] = _randn(g, M, K).bfloat16()
        s["codes"] = torch.zeros(N, K // 8, dtype=torch.int32, device=DEVICE)
        for j in range(8):  # codes of normally distributed weights, centred on the zero point
            code = (_randn(g, N, K // 8) * 2.7 + 7.9).round_().clamp_(0, 15).to(torch.int32)
            s["codes"] |= code << (4 * (j // 2) + 16 * (j % 2))
        groups = -(-K // G)
        s["scales"] = (torch.rand(N, groups, generator=g, device=DEVICE) + 0.5).mul_(0.4 / math.sqrt(K))
        s["scales"] = s["scales"].to(torch.float32 if c["scales"] == "f32" else torch.bfloat16)
        s["zeros"] = torch.randint(6, 11, (N, groups), generator=g, device=DEVICE, dtype=torch.uint8) if c["zeros"] else None
        s["bias"] = (_randn(g, N) * 0.2).bfloat16() if c["bias"] else None
        s["Y"] = torch.empty(M, N, device=DEVICE, dtype=out)
    elif c["op"] == "append":
        T, Hq, Hkv, D, P = c["T"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
        s["qkv"] = _randn(g, T, (Hq + 2 * Hkv) * D).bfloat16()
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
        B, Hq, D, P = c["B"], c["q_heads"], c["dim"], c["page"]
        order = torch.randperm(B, generator=g, device=DEVICE).tolist()
        lengths = [_lengths(c)[i] for i in order]
        need = [-(-n // P) for n in lengths]
        pages, width = sum(need) + 4, -(-c["max_len"] // P)
        s["k"], s["v"] = _pages(c, pages, g, c["kv"]), _pages(c, pages, g, c["kv"])
        s["k_scale"], s["v_scale"] = (0.125, 0.125) if c["kv"] == "fp8" else (1.0, 1.0)
        s["q_in"] = (_randn(g, B, Hq, D) * 1.5).bfloat16()
        free, table = torch.randperm(pages, generator=g, device=DEVICE), torch.full((B, width), -1, device=DEVICE, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            mine = free[at:at + n]
            table[b, :n] = mine.to(torch.int32)
            at += n
            if lengths[b] % P:  # what an allocator leaves behind a sequence's end
                s["k"][mine[-1], :, lengths[b] % P:] = float("nan")
                s["v"][mine[-1], :, lengths[b] % P:] = float("nan")
        s["tables"], s["lengths"] = table, torch.tensor(lengths, dtype=torch.int32).to(DEVICE)
        s["scale"] = 1 / math.sqrt(D)
        s["O"] = torch.empty(B, Hq, D, device=DEVICE, dtype=out)
        s["lse"] = torch.empty(B, Hq, device=DEVICE)
    if own:  # the handles that a program keeps
        import dense_linear_projection_amd as dlp
        s["ctx"] = _context()
        if c["op"] != "quant":
            s["cache"] = dlp.kv_cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s


# ------------------------------------------------------------- plain forms

def _plain_quant(s):
    c, N = s["c"], s["codes"].shape[0]
    at = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=DEVICE, dtype=torch.int32)
    w = (((s["codes"].unsqueeze(2) >> at) & 15).reshape(N, -1)).float()
    K, G = c["K"], c["group"]
    spread = torch.arange(K, device=DEVICE) // G
    zero = 8.0 if s["zeros"] is None else s["zeros"].float()[:, spread]
    w = (w - zero) * s["scales"].float()[:, spread]
    y = s["X"].float() @ w.t()
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
    row = s["rope"][s["positions"].long()].unsqueeze(1)
    y = _rotate(x[:, :Hq + Hkv], row[..., :rot // 2], row[..., rot // 2:], rot, c["interleaved"])
    # padding tokens store the first stored token once more, in its own place
    kept = s["slots"] >= 0
    token = torch.where(kept, torch.arange(T, device=DEVICE), kept.int().argmax())
    slot = s["slots"][token]
    page, place = slot // P, slot % P
    s["k"][page, :, place] = _stored(y[:, Hq:][token], s["k_scale"], s["k"].dtype)
    s["v"][page, :, place] = _stored(x[:, Hq + Hkv:][token], s["v_scale"], s["v"].dtype)
    return {"q": y[:, :Hq].bfloat16(), "k": s["k"], "v": s["v"]}


def _plain_attend(s):
    c = s["c"]
    B, Hq, Hkv, D, P, L = c["B"], c["q_heads"], c["kv_heads"], c["dim"], c["page"], c["max_len"]
    t = torch.arange(L, device=DEVICE)
    page = s["tables"].long().clamp(min=0)[:, t // P]
    n = s["lengths"].long().unsqueeze(1)
    seen = t < n
    if c["window"]:
        seen = seen & (t >= n - c["window"])
    seen = seen[:, None, None]
    q = s["q_in"].float().view(B, Hkv, Hq // Hkv, D)
    k = (s["k"][page, :, t % P].float() * s["k_scale"]).permute(0, 2, 3, 1)
    w = torch.where(seen, (q @ k) * s["scale"], -math.inf)
    top = w.amax(-1, keepdim=True)
    w = torch.exp(w - torch.where(top == -math.inf, 0.0, top))
    total = w.sum(-1, keepdim=True)
    v = (s["v"][page, :, t % P].float() * s["v_scale"]).transpose(1, 2)
    v = torch.where(seen.transpose(2, 3), v, 0.0)
    o = (w @ v) / torch.where(total == 0, 1.0, total)
    return {"o": o.view(B, Hq, D).to(s["O"].dtype), "lse": (top + torch.log(total)).view(B, Hq)}


def run(state):
    s = state
    if own:
        import dense_linear_projection_amd as dlp
        if s["op"] == "quant":
            dlp.proj_run_quant(s["ctx"], s["X"], s["codes"], s["scales"], s["zeros"], s["c"]["group"], s["bias"],
                               _epilogue(s["c"]), s["Y"])
            return s["Y"]
        if s["op"] == "append":
            dlp.proj_kv_append(s["ctx"], s["cache"], s["qkv"], s["rope"], s["positions"], s["slots"], s["q"],
                               interleaved=s["c"]["interleaved"])
            return {"q": s["q"], "k": s["k"], "v": s["v"]}
        dlp.proj_kv_attend(s["ctx"], s["cache"], s["q_in"], s["tables"], s["lengths"], s["scale"], s["O"], lse=s["lse"],
                           window=s["c"]["window"], max_len=s["c"]["max_len"])
        return {"o": s["O"], "lse": s["lse"]}
    return {"quant": _plain_quant, "append": _plain_append, "attend": _plain_attend}[s["op"]](s)


# ----------------------------------------------------------- work and exact

def work(case):
    c = case
    if c["op"] == "quant":
        M, K, N = c["M"], c["K"], c["N"]
        groups = -(-K // c["group"])
        b = N * K // 2 + N * groups * ((4 if c["scales"] == "f32" else 2) + (1 if c["zeros"] else 0))
        b += 2 * M * K + (2 * N if c["bias"] else 0) + M * N * (4 if c["out"] == "f32" else 2)
        return {"bytes": b, "flops": 2 * M * N * K}
    e = 1 if c["kv"] == "fp8" else 2
    if c["op"] == "append":
        T, D, Hq, Hkv = c["T"], c["dim"], c["q_heads"], c["kv_heads"]
        stored = T - max(0, T // 8 - 1) if c["padding"] else T
        b = T * (Hq + 2 * Hkv) * D * 2 + T * Hq * D * 2 + stored * 2 * Hkv * D * e + T * 12 + min(T, 16384) * c["rot"] * 4
        return {"bytes": b, "flops": 3 * T * (Hq + Hkv) * c["rot"]}
    seen = sum(min(n, c["window"]) if c["window"] else n for n in _lengths(c))
    rows = c["B"] * c["q_heads"]
    b = seen * c["kv_heads"] * c["dim"] * 2 * e + rows * c["dim"] * (2 + (4 if c["out"] == "f32" else 2)) + rows * 4
    return {"bytes": b + 4 * (seen // c["page"]), "flops": 4 * seen * c["q_heads"] * c["dim"]}


def _exact_quant(s):
    c = s["c"]
    M, K, N, G = c["M"], c["K"], c["N"], c["group"]
    X, parts, step = s["X"].double(), [], max(1, (1 << 26) // K)
    for n in range(0, N, step):
        word = s["codes"][n:n + step].long() & 0xFFFFFFFF
        W = torch.empty(word.shape[0], K, dtype=torch.float64, device=DEVICE)
        for j in range(8):
            W[:, j::8] = torch.remainder(torch.div(word, 2 ** (4 * (j // 2) + 16 * (j % 2)), rounding_mode="floor"), 16).double()
        for i in range(-(-K // G)):
            part = W[:, i * G:(i + 1) * G]
            part -= 8 if s["zeros"] is None else s["zeros"][n:n + step, i:i + 1].double()
            part *= s["scales"][n:n + step, i:i + 1].double()
        parts.append(torch.matmul(W, X.t()).t())
    y = torch.cat(parts, 1)
    if s["bias"] is not None:
        y += s["bias"].double()
    if c["gelu"]:
        y = y / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
    return y


def _exact_append(s):
    c = s["c"]
    T, Hq, Hkv, D, P, h = c["T"], c["q_heads"], c["kv_heads"], c["dim"], c["page"], c["rot"] // 2
    heads = s["qkv"].double().view(T, -1, D)
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


def _exact_attend(s):
    c = s["c"]
    B, Hq, Hkv, D, P = c["B"], c["q_heads"], c["kv_heads"], c["dim"], c["page"]
    o = torch.zeros(B, Hq, D, dtype=torch.float64, device=DEVICE)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=DEVICE)
    for b, n in enumerate(s["lengths"].tolist()):
        first = max(0, n - c["window"]) if c["window"] else 0
        if n <= first:
            continue
        pages = s["tables"][b, :-(-n // P)].long()
        for h in range(Hkv):
            k = (s["k"][pages, h].reshape(-1, D)[first:n]).double() * s["k_scale"]
            v = (s["v"][pages, h].reshape(-1, D)[first:n]).double() * s["v_scale"]
            rows = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            w = torch.matmul(s["q_in"][b, rows].double(), k.t()) * s["scale"]
            lse[b, rows] = torch.logsumexp(w, 1)
            o[b, rows] = torch.matmul(torch.softmax(w, 1), v)
    return {"o": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"quant": _exact_quant, "append": _exact_append, "attend": _exact_attend}[s["op"]](s)
