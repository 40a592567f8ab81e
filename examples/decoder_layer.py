"""One decoder layer and the head of a decode or verify step, on block-quantized weights and a 4-bit cache.

    python examples/decoder_layer.py [--steps N] [--context N] [--tokens T]

Each step takes T new tokens (1-4) of two sequences through
  RMSNorm -> Q8_1 -> query, key and value products -> norm and rotation of queries and keys ->
  keys and values appended to the cache -> attention -> output product, added to the hidden states ->
  RMSNorm -> Q8_1 -> router product -> experts and weights -> expert layer -> experts' rows combined with
  the hidden states -> RMSNorm -> Q8_1 -> head product -> log probabilities, entropy and alternatives,
the layer's matrices shaped as this package's (24 query and 2 key/value heads of 256, a quarter of which turns,
hidden size 2560) with fewer and smaller experts and a shorter vocabulary.  Every operator between the products
is checked against plain tensor operations in 64 bits on its own inputs in the last step.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from block_quantized_matvec_gb300 import mmvq, synth  # noqa: E402
from examples.attention_layer import DIM, HEADS, HIDDEN, KV_HEADS, PAGE, AttentionLayer, plain_attention  # noqa: E402

EXPERTS, CHOSEN, GROUPS, TOP_GROUPS, F, VOCAB, ROT = 32, 4, 8, 4, 256, 8192, 64
EPS = 1e-6


class DecoderLayer(AttentionLayer):
    """AttentionLayer with norms and positions for its heads, a layer of experts and a head."""

    def __init__(self, n_pages: int, device="cuda", salt: int = 0):
        super().__init__(n_pages, device, salt)
        def planar(w, rows, K, type_):  # noqa: E306
            return mmvq.repack_planar(torch.from_numpy(w).to(device), rows, K, type_=type_)
        gen = torch.Generator(device).manual_seed(salt)
        self.q_norm, self.k_norm = (torch.rand(DIM, device=device, generator=gen) + 0.5 for _ in range(2))
        self.frequency = 1e6 ** (-torch.arange(0, ROT, 2, dtype=torch.float64) / ROT)
        self.table = mmvq.rope_table(self.frequency, device=device)
        # the synthetic weights are about a hundred times a trained model's, and not centred
        self.ffn_norm = torch.full((HIDDEN,), 2.0 ** -10, device=device)
        self.router = planar(synth.q6_k_weights(EXPERTS, HIDDEN, salt=salt + 5), EXPERTS, HIDDEN, mmvq.TYPE_Q6_K)
        self.bias = torch.randn(EXPERTS, device=device, generator=gen) * 0.05
        gate_up, down = synth.expert_weights("q4_k", EXPERTS, 2 * F, HIDDEN, salt=salt + 6), synth.expert_weights("q4_k", EXPERTS, HIDDEN, F, salt=salt + 7)
        self.gate_up = torch.cat([planar(w, 2 * F, HIDDEN, mmvq.TYPE_Q4_K) for w in gate_up])
        self.down = torch.cat([planar(w, HIDDEN, F, mmvq.TYPE_Q4_K) for w in down])
        self.head = planar(synth.q6_k_weights(VOCAB, HIDDEN, salt=salt + 8), VOCAB, HIDDEN, mmvq.TYPE_Q6_K)
        self.sync = mmvq.expert_ffn_workspace(torch.device(device))

    def step(self, x, positions, tokens, table, offsets, lens):
        """x [T, HIDDEN] fp32 at positions [T], the rest as in AttentionLayer; tokens [T, m]: whose log probabilities
        are wanted.  Returns a dict of what the operators gave."""
        T, where = x.shape[0], (self.cache, table, offsets, lens)
        xq = mmvq.rmsnorm_quantize_q8_1(x, self.norm, EPS)
        project = lambda w, rows: mmvq.gemv(mmvq.TYPE_Q4_K_PLANAR, w, rows, HIDDEN, xq, T)  # noqa: E731
        q, k, v = (project(w, n * DIM).view(T, n, DIM) for w, n in ((self.wq, HEADS), (self.wk, KV_HEADS), (self.wv, KV_HEADS)))
        r = dict(q=q, k=k)
        r["turned"] = mmvq.norm_rope(q, k, positions, self.table, q_weight=self.q_norm, k_weight=self.k_norm, eps=EPS, status=self.status)
        mmvq.kv4_append(r["turned"][1], v, *where, status=self.status)
        r["y"] = mmvq.kv4_attention(r["turned"][0], *where, workspace=self.workspace, status=self.status)
        out, _ = mmvq.gemv_f32(mmvq.TYPE_Q4_K_PLANAR, self.wo, HIDDEN, HEADS * DIM, r["y"].view(T, HEADS * DIM))
        r["x"] = x = x + out
        h = torch.empty_like(x)
        hq = mmvq.rmsnorm_quantize_q8_1(x, self.ffn_norm, EPS, y_out=h)
        r["logits"] = mmvq.gemv(mmvq.TYPE_Q6_K_PLANAR, self.router, EXPERTS, HIDDEN, hq, T)
        r["chosen"] = mmvq.route_topk(r["logits"], CHOSEN, scoring="sigmoid", bias=self.bias, n_groups=GROUPS, top_groups=TOP_GROUPS, status=self.status)
        topk, weights = r["chosen"]
        r["ffn"] = ffn = mmvq.expert_ffn(mmvq.TYPE_Q4_K_PLANAR, self.gate_up, self.down, EXPERTS, HIDDEN, F, h, topk, sync=self.sync, status=self.status)
        r["out"] = mmvq.combine_experts(ffn["y"], topk, weights, ffn["offsets"], ffn["slot_of"], residual=x, status=self.status)
        r["words"] = mmvq.gemv(mmvq.TYPE_Q6_K_PLANAR, self.head, VOCAB, HIDDEN, mmvq.rmsnorm_quantize_q8_1(r["out"], self.norm, EPS), T)
        r["said"] = mmvq.token_logprobs(r["words"], tokens, top=5, scale=1 / 64, status=self.status)
        return r


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def check(layer, r, positions, tokens, lens, offsets, table, news):
    """The largest relative error of the step's operators against 64 bits."""
    worst = 0.0
    angle = positions.double()[:, None, None] * layer.frequency.to(positions.device)
    for x, w, got in ((r["q"], layer.q_norm, r["turned"][0]), (r["k"], layer.k_norm, r["turned"][1])):
        z = x.double() / (x.double().square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
        a, b = z[..., :ROT // 2], z[..., ROT // 2:ROT]
        want = torch.cat((a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos(), z[..., ROT:]), -1)
        worst = max(worst, off(got, want))
    first = 0
    for b, n in enumerate(lens.tolist()):
        one = torch.tensor([0, n], dtype=torch.int32, device=lens.device)
        k, v = mmvq.kv4_read(layer.cache, table[b:b + 1].contiguous(), one, lens[b:b + 1].contiguous(), n)
        rows = slice(first, first + news)
        worst = max(worst, off(r["y"][rows], plain_attention(r["turned"][0][rows], k, v, news, DIM ** -0.5, 0, 0)))
        first += news
    topk, weights = r["chosen"]
    score = torch.sigmoid(r["logits"].double())
    value = (score + layer.bias.double()).view(len(topk), GROUPS, -1)
    stay = value.topk(2, -1)[0].sum(-1).topk(TOP_GROUPS, -1)[1]
    kept = torch.full_like(value, float("-inf")).scatter(1, stay[..., None].expand(-1, -1, value.shape[-1]), 0.0) + value
    assert torch.equal(kept.flatten(1).topk(CHOSEN, -1)[1].int(), topk)
    w = score.gather(1, topk.long())
    worst = max(worst, off(weights, w / w.sum(-1, keepdim=True)))
    want = r["x"].double()
    for p, slot in enumerate(r["ffn"]["slot_of"].tolist()):
        want[slot // CHOSEN] += weights.flatten()[slot].double() * r["ffn"]["y"][p].double()
    worst = max(worst, off(r["out"], want))
    logp = (r["words"].double() / 64).log_softmax(-1)
    said = r["said"]
    worst = max(worst, off(said["logprobs"], logp.gather(1, tokens.long())), off(said["entropy"], -(logp.exp() * logp).sum(-1)),
                off(said["top_logprobs"], logp.topk(5, -1)[0]))
    return worst


def main(argv=None) -> float:
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--steps", type=int, default=8)
    p.add_argument("--context", type=int, default=500, help="cached tokens before the first step")
    p.add_argument("--tokens", type=int, default=2, help="new tokens of each of the two sequences, 1-4")
    a = p.parse_args(argv)
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(1)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    lens = [a.context, a.context // 2 + 3]
    per = -(-(max(lens) + a.steps * a.tokens) // PAGE)
    layer = DecoderLayer(2 * per, dev)
    table = torch.randperm(2 * per, device=dev, generator=gen).to(torch.int32).view(2, per)
    # the prompts' keys and values: turned and appended at once
    k, v = (torch.randn((sum(lens), KV_HEADS, DIM), device=dev, generator=gen) for _ in range(2))
    at = torch.cat([torch.arange(n, device=dev) for n in lens]).to(torch.int32)
    k, _ = mmvq.norm_rope(k, None, at, layer.table, q_weight=layer.k_norm, eps=EPS)
    mmvq.kv4_append(k, v, layer.cache, table, i32([0, lens[0], sum(lens)]), i32(lens), status=layer.status)
    offsets, length = i32([0, a.tokens, 2 * a.tokens]), i32(lens)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    tokens = torch.randint(0, VOCAB, (2 * a.tokens, 1), dtype=torch.int32, device=dev, generator=gen)
    for i in range(a.steps):
        if i == min(3, a.steps - 1):
            begin.record()
        x = torch.randn((2 * a.tokens, HIDDEN), device=dev, generator=gen)
        positions = (length[:, None] + torch.arange(a.tokens, device=dev)).flatten().to(torch.int32)
        length += a.tokens
        r = layer.step(x, positions, tokens, table, offsets, length)
    end.record()
    worst = check(layer, r, positions, tokens, length, offsets, table, a.tokens)
    assert int(layer.status[0]) == 0 and mmvq.read_device_fault() == 0
    assert all(bool(torch.isfinite(r[name]).all()) for name in ("out", "words"))
    timed = a.steps - min(3, a.steps - 1)
    print(f"{a.steps} steps of 2 x {a.tokens} tokens over {length.tolist()} cached: {begin.elapsed_time(end) / timed * 1e3:.0f} us a step, "
          f"operators within {worst:.1e} of 64 bits; first row: entropy {float(r['said']['entropy'][0]):.3f}, "
          f"likeliest tokens {r['said']['top_ids'][0].tolist()}")
    return worst


if __name__ == "__main__":
    sys.exit(0 if main() < 1e-4 else 1)
