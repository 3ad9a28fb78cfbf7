"""One attention block of a decoding model, token by token: a 4-bit QKV
projection, rotary positions and the append to a paged cache, attention over
the pages, and a 4-bit output projection, captured once into a graph and
replayed as the sequences grow.

    python examples/decode_attention.py [--batch 16] [--hidden 4096] [--steps 64] [--fp8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import dense_linear_projection_amd as dlp  # noqa: E402


class PagedSequences:
    """Pages handed out to growing sequences: the host's side of a paged cache."""

    def __init__(self, batch, pages, page, width, device):
        self.page, self.free = page, list(range(pages))
        self.tables = torch.full((batch, width), -1, dtype=torch.int32)
        self.lengths = [0] * batch
        self.device_tables = self.tables.to(device)

    def grow(self):
        """Room for one more token in every sequence: its slots."""
        slots, changed = [], False
        for b, n in enumerate(self.lengths):
            if n % self.page == 0:
                self.tables[b, n // self.page] = self.free.pop()
                changed = True
            slots.append(int(self.tables[b, n // self.page]) * self.page + n % self.page)
            self.lengths[b] = n + 1
        if changed:
            self.device_tables.copy_(self.tables)
        return torch.tensor(slots)


class DecodeBlock:
    """The four calls of a step, with what they keep between steps."""

    def __init__(self, batch, hidden, q_heads, kv_heads, dim, max_len, page=16, fp8=False, group=128, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.ctx = dlp.proj_create(torch.cuda.current_device())
        self.q_heads, self.dim, self.group, self.max_len = q_heads, dim, group, max_len
        wide = (q_heads + 2 * kv_heads) * dim
        self.w_qkv = (rand(wide, hidden) / hidden ** 0.5).bfloat16()
        self.w_out = (rand(hidden, q_heads * dim) / (q_heads * dim) ** 0.5).bfloat16()
        self.qkv_weights = dlp.proj_quantize_weights(self.ctx, self.w_qkv, group)
        self.out_weights = dlp.proj_quantize_weights(self.ctx, self.w_out, group)
        pages_each = -(-max_len // page)
        self.pages = PagedSequences(batch, batch * pages_each, page, pages_each, "cuda")
        store = torch.float8_e4m3fn if fp8 else torch.bfloat16
        k, v = (torch.zeros(batch * pages_each, kv_heads, page, dim, dtype=store, device="cuda") for _ in range(2))
        self.cache = dlp.kv_cache(k, v, *((0.02, 0.02) if fp8 else (1.0, 1.0)))
        angle = torch.outer(torch.arange(max_len, dtype=torch.float64),
                            1e4 ** (-torch.arange(dim // 2, dtype=torch.float64) * 2 / dim))
        self.rope = torch.cat((angle.cos(), angle.sin()), 1).float().cuda()
        self.x = torch.zeros(batch, hidden, dtype=torch.bfloat16, device="cuda")
        self.qkv = torch.empty(batch, wide, dtype=torch.bfloat16, device="cuda")
        self.q, self.o = (torch.empty(batch, q_heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.y = torch.empty(batch, hidden, dtype=torch.bfloat16, device="cuda")
        self.positions, self.lengths = (torch.zeros(batch, dtype=torch.int32, device="cuda") for _ in range(2))
        self.slots = torch.zeros(batch, dtype=torch.int64, device="cuda")
        self.graph = None

    def calls(self):
        dlp.proj_run_quant(self.ctx, self.x, *self.qkv_weights, self.group, None, dlp.EPI_NONE, self.qkv)
        dlp.proj_kv_append(self.ctx, self.cache, self.qkv, self.rope, self.positions, self.slots, self.q)
        dlp.proj_kv_attend(self.ctx, self.cache, self.q, self.pages.device_tables, self.lengths, self.dim ** -0.5, self.o,
                           max_len=self.max_len)
        dlp.proj_run_quant(self.ctx, self.o.flatten(1), *self.out_weights, self.group, None, dlp.EPI_NONE, self.y)

    def step(self, x):
        """Output rows of one token for every sequence; x bf16 [batch, hidden]."""
        self.positions.copy_(torch.tensor(self.pages.lengths, dtype=torch.int32))
        self.slots.copy_(self.pages.grow())
        self.lengths.copy_(torch.tensor(self.pages.lengths, dtype=torch.int32))
        self.x.copy_(x)
        if self.graph is None:
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.calls()
        self.graph.replay()
        return self.y

    def close(self):
        self.graph = None
        dlp.proj_destroy(self.ctx)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--batch", type=int, default=16)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--steps", type=int, default=64)
    p.add_argument("--fp8", action="store_true", help="8-bit cache")
    a = p.parse_args()
    block = DecodeBlock(a.batch, a.hidden, a.hidden // 128, max(1, a.hidden // 512), 128, a.steps + 8, fp8=a.fp8)
    x = torch.randn(a.steps, a.batch, a.hidden, device="cuda").bfloat16()
    block.step(x[0])
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for t in range(1, a.steps):
        y = block.step(x[t])
    end.record()
    torch.cuda.synchronize()
    print("%d sequences of %d tokens: %.1f us a step, output norm %.3f" %
          (a.batch, a.steps, start.elapsed_time(end) * 1e3 / max(1, a.steps - 1), float(y.float().norm())))
    block.close()


if __name__ == "__main__":
    main()
