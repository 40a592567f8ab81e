"""One attention layer of a decode or verify step, on block-quantized weights and a 4-bit cache.

    python examples/attention_layer.py [--steps N] [--context N] [--tokens T] [--window W --sinks S]

Each step takes T new tokens (1-8 in all) of a few sequences through
  RMSNorm -> Q8_1 -> query, key and value products -> keys and values appended to the cache ->
  attention over the cache -> output product (its input quantised on the way in)
with the shapes of this package's dense matrices: 24 query and 2 key/value heads of 256, hidden size
2560 (position encodings are the model's own and left out here).  The last step is checked against
plain tensor operations on the values read back from the cache.
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from block_quantized_matvec_gb300 import mmvq, synth  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, PAGE = 2560, 24, 2, 256, 64


class AttentionLayer:
    """Planar Q4_K projections, and everything that is kept from step to step."""

    def __init__(self, n_pages: int, device="cuda", salt: int = 0, window: int = 0, sinks: int = 0):
        def weights(rows, K, n):
            w = torch.from_numpy(synth.q4_k_weights(rows, K, salt=salt + n)).to(device)
            return mmvq.repack_planar(w, rows, K, type_=mmvq.TYPE_Q4_K)
        self.norm = torch.ones(HIDDEN, device=device)
        self.wq = weights(HEADS * DIM, HIDDEN, 1)
        self.wk = weights(KV_HEADS * DIM, HIDDEN, 2)
        self.wv = weights(KV_HEADS * DIM, HIDDEN, 3)
        self.wo = weights(HIDDEN, HEADS * DIM, 4)
        self.cache = mmvq.kv4_cache(n_pages, KV_HEADS, DIM, PAGE, device)
        self.workspace = mmvq.kv4_attention_workspace(DIM, device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.window, self.sinks = window, sinks

    def step(self, x, table, offsets, lens):
        """x [T, HIDDEN] fp32: rows offsets[b]..offsets[b+1]-1 are the last tokens of sequence b, lens[b]
        its length with them.  Returns (layer output [T, HIDDEN], attention output [T, HEADS, DIM], queries)."""
        T, where = x.shape[0], (self.cache, table, offsets, lens)
        xq = mmvq.rmsnorm_quantize_q8_1(x, self.norm, 1e-6)
        project = lambda w, rows: mmvq.gemv(mmvq.TYPE_Q4_K_PLANAR, w, rows, HIDDEN, xq, T)  # noqa: E731
        q = project(self.wq, HEADS * DIM).view(T, HEADS, DIM)
        k = project(self.wk, KV_HEADS * DIM).view(T, KV_HEADS, DIM)
        v = project(self.wv, KV_HEADS * DIM).view(T, KV_HEADS, DIM)
        mmvq.kv4_append(k, v, *where, status=self.status)
        y = mmvq.kv4_attention(q, *where, window=self.window, sinks=self.sinks, scale=1e-4,
                               workspace=self.workspace, status=self.status)
        out, _ = mmvq.gemv_f32(mmvq.TYPE_Q4_K_PLANAR, self.wo, HIDDEN, HEADS * DIM, y.view(T, HEADS * DIM))
        return out, y, q


def plain_attention(q, k, v, new, scale, window, sinks):
    """Attention in 64 bits of a sequence's last `new` queries over its read-back keys and values."""
    n, g = k.shape[0], HEADS // KV_HEADS
    k, v = (t.double().repeat_interleave(g, 1) for t in (k, v))
    x = torch.einsum("thd,nhd->thn", q.double(), k) * scale
    mine = torch.arange(n - new, n, device=q.device)[:, None, None]
    at = torch.arange(n, device=q.device)
    see = at <= mine
    if window:
        see = see & ((at > mine - window) | (at < sinks))
    return torch.einsum("thn,nhd->thd", x.masked_fill(~see, float("-inf")).softmax(-1), v)


def main(argv=None) -> float:
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--steps", type=int, default=8)
    p.add_argument("--context", type=int, default=1000, help="cached tokens before the first step")
    p.add_argument("--tokens", type=int, default=2, help="new tokens of each of the two sequences, 1-4")
    p.add_argument("--window", type=int, default=0)
    p.add_argument("--sinks", type=int, default=0)
    a = p.parse_args(argv)
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(1)
    lens = [a.context, a.context // 2 + 3]
    per = -(-(max(lens) + a.steps * a.tokens) // PAGE)
    layer = AttentionLayer(2 * per, dev, window=a.window, sinks=a.sinks)
    table = torch.randperm(2 * per, device=dev, generator=gen).to(torch.int32).view(2, per)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    # the prompts' keys and values, appended at once
    k = torch.randn((sum(lens), KV_HEADS, DIM), device=dev, generator=gen) * 50
    v = torch.randn((sum(lens), KV_HEADS, DIM), device=dev, generator=gen) * 50
    mmvq.kv4_append(k, v, layer.cache, table, i32([0, lens[0], sum(lens)]), i32(lens), status=layer.status)
    offsets, length = i32([0, a.tokens, 2 * a.tokens]), i32(lens)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for i in range(a.steps):
        if i == min(3, a.steps - 1):
            begin.record()
        x = torch.randn((2 * a.tokens, HIDDEN), device=dev, generator=gen)
        length += a.tokens
        out, y, q = layer.step(x, table, offsets, length)
    end.record()
    lens = [n + a.steps * a.tokens for n in lens]
    kr, vr = mmvq.kv4_read(layer.cache, table, i32([0, lens[0], sum(lens)]), length, sum(lens))
    worst = 0.0
    for b, first in enumerate((0, lens[0])):
        rows = slice(b * a.tokens, (b + 1) * a.tokens)
        want = plain_attention(q[rows], kr[first:first + lens[b]], vr[first:first + lens[b]], a.tokens, 1e-4,
                               a.window, a.sinks)
        worst = max(worst, float((y[rows].double() - want).norm() / want.norm()))
    torch.cuda.synchronize()
    assert int(layer.status[0]) == 0 and bool(torch.isfinite(out).all()) and np.isfinite(worst)
    timed = a.steps - min(3, a.steps - 1)
    print(f"{a.steps} steps of 2 x {a.tokens} tokens over {lens} cached: {begin.elapsed_time(end) / timed * 1e3:.0f} us "
          f"a step, attention within {worst:.1e} of 64 bits")
    return worst


if __name__ == "__main__":
    sys.exit(0 if main() < 1e-4 else 1)
