"""Decode steps of one attention block on 4-bit weights and a 4-bit or 8-bit
key/value cache (Llama-3-8B-shaped: 32 heads over 8 key/value heads of 128 channels,
hidden size 4096; random weights):

    q | k | v   W4 layer, M rows in one call
    rotation    of queries and keys by position, with their norm (--rotate)
    plan        block table, slots and runs of the new tokens
    append      the new keys and values, quantized into their pages
    attention   over all cached tokens, or over the pages chosen for each row
    accumulate  what the step looked at (--keep)
    output      W4 layer

The step is captured into a HIP graph once and replayed; lengths, block table and
page numbers are device data, so the same graph serves a growing cache.  With --keep,
sequences that have outgrown it keep their last quarter of it and the tokens looked at
most, between the replays.

    python examples/kv4_decode.py [--seqs 8] [--prompt 2000] [--steps 100] [--pages 0]
    python examples/kv4_decode.py --bits 8 --rotate --keep 1500
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

    def __init__(self, seqs, longest, hidden=4096, heads=32, kv_heads=8, dim=128, seed=0, bits=4, rotate=False):
        rng = np.random.default_rng(seed)
        self.seqs, self.longest, self.hidden = seqs, longest, hidden
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        rows = (heads + 2 * kv_heads) * dim
        w = (0.02 * rng.standard_normal((rows, hidden))).astype(np.float32)
        o = (0.02 * rng.standard_normal((hidden, heads * dim))).astype(np.float32)
        self.qkv = DeviceLayer(pack_host(B.WQ_FMT_W4, w), tiled=True)
        self.out = DeviceLayer(pack_host(B.WQ_FMT_W4, o), tiled=True)
        width = -(-longest // B.WQ_KV4_PAGE)
        self.cache = (B.KV4Cache if bits == 4 else B.KV8Cache).empty(seqs * width, kv_heads, dim)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table = torch.full((seqs, width), -1, **i32)
        self.free = torch.randperm(seqs * width, generator=torch.Generator().manual_seed(seed)).to(**i32)
        self.lens, self.after = torch.zeros(seqs, **i32), torch.zeros(seqs, **i32)
        self.taken = torch.zeros(1, **i32)
        self.inv_freq = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim) if rotate else None
        self.at = torch.zeros(seqs, **i32)                   # positions count on behind an eviction
        self.lse = self.mass = None

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
        self.at.add_(self.after - self.lens)
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

    def evict(self, keep):
        """Sequences of more than `keep` tokens keep that many, in fresh pages; their
        old pages are free again."""
        table, lens, mass = self.table.clone(), self.lens.clone(), torch.zeros_like(self.mass)
        free = self.free[:self.free.numel() - int((self.table >= 0).sum())]
        self.cache.evict(self.mass, self.table, self.lens, keep, keep // 4, free, table, lens, mass, self.taken)
        if int(self.taken) > free.numel():
            raise RuntimeError("too few free pages for an eviction")
        self.table.copy_(table)
        self.lens.copy_(lens)
        self.mass.copy_(mass)
        used = torch.zeros(self.free.numel(), dtype=torch.bool, device="cuda")
        used[self.table[self.table >= 0].long()] = True
        order = torch.sort(used[self.free.long()].int(), stable=True).indices    # the free ones first
        self.free.copy_(self.free[order])

    def stepper(self, pages=0, count=False):
        """A step on fixed buffers: x [seqs, hidden] -> y [seqs, hidden].  With `count`
        it accumulates the tokens' softmax weights."""
        n = self.seqs
        cu, slots, runs = self.place([1] * n)
        x = torch.zeros(n, self.hidden, dtype=torch.int16, device="cuda")
        proj = torch.zeros(n, self.qkv.N, dtype=torch.int16, device="cuda")
        att = torch.zeros(n, self.heads, self.dim, dtype=torch.float16, device="cuda")
        y = torch.zeros(n, self.hidden, dtype=torch.int16, device="cuda")
        q, k, v = self.split(proj)
        if count:
            self.lse = torch.zeros(n, self.heads, device="cuda")
            self.mass = torch.zeros(n, self.kv_heads, self.table.shape[1] * B.WQ_KV4_PAGE, device="cuda")

        def step():
            for a in range(0, n, B.WQ_GEMM_MAX_M):
                self.qkv.gemm_tiled(x[a:a + B.WQ_GEMM_MAX_M], proj[a:a + B.WQ_GEMM_MAX_M])
            if self.inv_freq is not None:
                B.wq_qk_norm_rope(q, k, self.at, self.inv_freq, q_out=q, k_out=k)
            self.write(cu, slots, runs, k, v)
            chosen = dict(sel=self.cache.select(q, self.table, self.after, cu, pages)) if pages else {}
            self.cache.attention(q, self.table, self.after, cu, 1, self.longest, out=att, lse=self.lse, **chosen)
            if count:
                self.cache.accumulate(q, self.lse, self.table, self.after, cu, self.lens, self.mass, 1, self.longest)
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
    ap.add_argument("--bits", type=int, default=4, choices=(4, 8), help="of the key/value cache")
    ap.add_argument("--rotate", action="store_true", help="norm and rotate queries and keys")
    ap.add_argument("--keep", type=int, default=0, help="tokens that a sequence keeps, looked at every 32 steps (0: all; 8 bits)")
    a = ap.parse_args(argv)
    if (a.keep and a.bits == 4) or (a.pages and a.bits == 8):
        ap.error("--keep needs --bits 8, --pages needs --bits 4")
    block = Block(a.seqs, 2 * a.prompt + a.steps + 8 if a.keep else a.prompt + a.steps + 8, bits=a.bits, rotate=a.rotate)
    block.fill([a.prompt - 7 * b % a.prompt for b in range(a.seqs)])
    step, x, _, _, y = block.stepper(a.pages, a.keep > 0)
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
    for i in range(a.steps):
        if a.keep and i % 32 == 0:
            block.evict(a.keep)
        graph.replay()
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / a.steps
    what = f"{a.pages} pages a row" if a.pages else "all tokens"
    what += f", {a.bits} bits" + (", rotated" if a.rotate else "") + (f", {a.keep} kept" if a.keep else "")
    print(f"{a.seqs} sequences of {int(block.lens.max())} tokens, {what}: {t * 1e6:.1f} us a step, "
          f"|y| {y.view(torch.float16).float().abs().mean():.4f}")


if __name__ == "__main__":
    main()
