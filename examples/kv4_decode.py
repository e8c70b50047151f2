"""Decode steps of one attention block on 4-bit weights and a 4-bit key/value
cache (Llama-3-8B-shaped: 32 heads over 8 key/value heads of 128 channels, hidden
size 4096; random weights):

    q | k | v   W4 layer, M rows in one call
    plan        block table, slots and runs of the new tokens
    append      the new keys and values, quantized into their pages
    attention   over all cached tokens, or over the pages chosen for each row
    output      W4 layer

The step is captured into a HIP graph once and replayed; lengths, block table and
page numbers are device data, so the same graph serves a growing cache.

    python examples/kv4_decode.py [--seqs 8] [--prompt 2000] [--steps 100] [--pages 0]
"""

import argparse
import os
import sys
import time

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bit_weight_only_gemv_amd as B  # noqa: E402
from bit_weight_only_gemv_amd.layer import DeviceLayer, pack_host  # noqa: E402


class Block:
    """One attention block and the state of its sequences."""

    def __init__(self, seqs, longest, hidden=4096, heads=32, kv_heads=8, dim=128, seed=0):
        rng = np.random.default_rng(seed)
        self.seqs, self.longest, self.hidden = seqs, longest, hidden
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        rows = (heads + 2 * kv_heads) * dim
        w = (0.02 * rng.standard_normal((rows, hidden))).astype(np.float32)
        o = (0.02 * rng.standard_normal((hidden, heads * dim))).astype(np.float32)
        self.qkv = DeviceLayer(pack_host(B.WQ_FMT_W4, w), tiled=True)
        self.out = DeviceLayer(pack_host(B.WQ_FMT_W4, o), tiled=True)
        width = -(-longest // B.WQ_KV4_PAGE)
        self.cache = B.KV4Cache.empty(seqs * width, kv_heads, dim)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.full((seqs, width), -1, **i32)
        self.free = torch.randperm(seqs * width, generator=torch.Generator().manual_seed(seed)).to(**i32)
        self.lens, self.after = torch.zeros(seqs, **i32), torch.zeros(seqs, **i32)
        self.taken = torch.zeros(1, **i32)

    def place(self, new):
        """Slots and runs of new[b] more tokens of every sequence (a list)."""
        i32 = dict(dtype=torch.int32, device="cuda")
        cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), **i32)
        T = int(sum(new))
        slots, runs = torch.zeros(T, **i32), torch.zeros(B.wq_kv4_max_runs(self.seqs, T), 2, **i32)
        return cu, slots, runs

    def split(self, y):
        """Views of q, k and v in the projection's rows."""
        h, k, d = self.heads, self.kv_heads, self.dim
        y = y.view(torch.float16).view(len(y), h + 2 * k, d)
        return y[:, :h], y[:, h:h + k], y[:, h + k:]

    def write(self, cu, slots, runs, k, v):
        B.wq_kv4_plan(self.lens, cu, self.table, self.free, self.after, slots, runs, self.taken)
        self.cache.append(k, v, slots, runs)

    def advance(self):
        """The new tokens count, and the pages they took leave the free list."""
        self.lens.copy_(self.after)
        at = (torch.arange(self.free.numel(), device="cuda") + self.taken) % self.free.numel()
        self.free.copy_(self.free[at])

    def fill(self, prompt, seed=1):
        """Random keys and values as prompts of the given lengths."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        cu, slots, runs = self.place(prompt)
        kv = torch.randn(2, int(sum(prompt)), self.kv_heads, self.dim, generator=g, device="cuda").half()
        self.write(cu, slots, runs, kv[0], kv[1])
        self.advance()
        return kv

    def stepper(self, pages=0):
        """A step on fixed buffers: x [seqs, hidden] -> y [seqs, hidden]."""
        n = self.seqs
        cu, slots, runs = self.place([1] * n)
        x = torch.zeros(n, self.hidden, dtype=torch.int16, device="cuda")
        proj = torch.zeros(n, self.qkv.N, dtype=torch.int16, device="cuda")
        att = torch.zeros(n, self.heads, self.dim, dtype=torch.float16, device="cuda")
        y = torch.zeros(n, self.hidden, dtype=torch.int16, device="cuda")
        q, k, v = self.split(proj)

        def step():
            for a in range(0, n, B.WQ_GEMM_MAX_M):
                self.qkv.gemm_tiled(x[a:a + B.WQ_GEMM_MAX_M], proj[a:a + B.WQ_GEMM_MAX_M])
            self.write(cu, slots, runs, k, v)
            sel = self.cache.select(q, self.table, self.after, cu, pages) if pages else None
            self.cache.attention(q, self.table, self.after, cu, 1, self.longest, sel=sel, out=att)
            rows = att.view(n, -1).view(torch.int16)
            for a in range(0, n, B.WQ_GEMM_MAX_M):
                self.out.gemm_tiled(rows[a:a + B.WQ_GEMM_MAX_M], y[a:a + B.WQ_GEMM_MAX_M])
            self.advance()

        return step, x, proj, att, y


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--seqs", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=2000)
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--pages", type=int, default=0, help="pages chosen for each row (0: all)")
    a = ap.parse_args(argv)
    block = Block(a.seqs, a.prompt + a.steps + 8)
    block.fill([a.prompt - 7 * b % a.prompt for b in range(a.seqs)])
    step, x, _, _, y = block.stepper(a.pages)
    x.copy_(torch.randn(x.shape, device="cuda").half().view(torch.int16))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                   # loads the kernels
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / a.steps
    what = f"{a.pages} pages a row" if a.pages else "all tokens"
    print(f"{a.seqs} sequences of {int(block.lens.max())} tokens, {what}: {t * 1e6:.1f} us a step, "
          f"|y| {y.view(torch.float16).float().abs().mean():.4f}")


if __name__ == "__main__":
    main()
