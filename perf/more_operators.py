"""Cases and plain forms of the operators between the products of a layer and after the last one.

Four operators, each next to an operator that this package has already:

* ``mmvq.norm_rope``: RMS norm of every query and key head, then the rotation by the token's position
  (one axis, or several for images and video), between the query and key products and the cache;
* ``mmvq.route_topk``: experts and their weights from router scores, before ``route_groups`` or
  ``expert_ffn``, which take the chosen experts;
* ``mmvq.combine_experts``: the experts' rows weighted and added up for each token, with the residual
  and a gated shared expert, after ``expert_ffn`` or ``grouped``;
* ``mmvq.token_logprobs``: log probabilities of given tokens, entropy and the best alternatives of rows
  of logits, after the LM head.

Definitions.  norm_rope: z = x / sqrt(mean(x^2) + eps) * w over a head's dim values; of the first
``rot`` of them, pair i is (i, i + rot / 2), or (2 i, 2 i + 1) where interleaved, and turns by the angle
position[axis(i)] * frequency(i).  route_topk: scores are the softmax or sigmoid of the logits; experts
are chosen by score + bias, in 64 bits, among the groups whose two best add up to most, ties to the lowest
index; weights are the scores without bias, over their sum where renormalised, times a scale.
token_logprobs: of the softmax of scale * logits; a logit of -inf has no probability and is no alternative
(id -1, log probability -inf); a row of such logits alone has lse -inf and entropy 0.
"""
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------ cases --

def listed():
    """The heads 24 / 2 of 256 (queries next to their gates), the hidden size 2560, 256 experts of which 8 are
    chosen and the vocabulary of 151936 are those of this repository's shapes; the others are generic."""
    r = dict(kind="rope", axes="one", interleaved=False, gated=False, start=0)
    e = dict(kind="route", scoring="softmax", bias=False, groups=1, top_groups=1, renormalize=True)
    c = dict(kind="combine", dropped=False)
    p = dict(kind="logprobs", masked=False)
    return [
        # a decode step of one chat: only latency counts; a quarter of the head turns
        dict(r, name="rope 1 token", dtype="f32", tokens=1, heads=24, kv=2, dim=256, rot=64, gated=True, start=4100),
        # a batch of decoding sequences far into long documents, every head with its own keys, pairs side by side
        dict(r, name="rope 603 far", dtype="f16", tokens=603, heads=12, kv=12, dim=64, rot=64, interleaved=True, start=1000003),
        # a prompt with video frames: time, height and width
        dict(r, name="rope video 16k", dtype="bf16", tokens=16385, heads=32, kv=8, dim=128, rot=128, axes="sections"),
        # one token's experts: latency
        dict(e, name="route 1 token", dtype="f32", tokens=1, experts=256, k=8),
        # a small batch over many experts, an odd count of choices
        dict(e, name="route 301 of 512", dtype="f32", tokens=301, experts=512, k=11, renormalize=False),
        # a prompt's tokens, balanced by a bias, in groups
        dict(e, name="route 8k groups", dtype="bf16", tokens=8192, experts=256, k=8, scoring="sigmoid", bias=True, groups=8, top_groups=4),
        # the layer's end of one token
        dict(c, name="combine 1 token", dtype="f32", tokens=1, experts=256, k=8, hidden=2560, shared=True),
        # the same of a long prompt's chunk
        dict(c, name="combine 4k", dtype="bf16", tokens=4099, experts=256, k=8, hidden=2560, shared=True),
        # a decode step's chosen token with alternatives: latency over one long row
        dict(p, name="logprobs 1 row", dtype="f32", rows=1, vocab=151936, tokens=1, top=20),
        # a verify window of five drafted tokens for each of three chats, some of it under a grammar's mask
        dict(p, name="logprobs 15 rows", dtype="f32", rows=15, vocab=151936, tokens=1, top=5, masked=True),
        # every token of a prompt scored, rows of odd length
        dict(p, name="logprobs 301 odd", dtype="f16", rows=301, vocab=50021, tokens=3, top=8),
        dict(p, name="logprobs 2048 rows", dtype="bf16", rows=2048, vocab=151936, tokens=1, top=20),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))
    c = dict(kind=rng.choice(["rope", "rope", "route", "route", "combine", "logprobs", "logprobs"]),
             dtype=rng.choice(["f32", "bf16", "f16"]))
    if c["kind"] == "rope":
        c.update(kv=rng.choice([1, 2, 3, 4, 8, 12]), dim=rng.choice([64, 128, 256]), axes=rng.choice(["one", "one", "sections", "cycle"]),
                 interleaved=rng.random() < 0.4, gated=rng.random() < 0.3, start=rng.choice([0, 1, 77, 131071, 1000003]))
        c["heads"] = c["kv"] * rng.choice([1, 2, 4, 5, 8, 12])
        c["rot"] = rng.choice([c["dim"], c["dim"], c["dim"] // 2, c["dim"] // 4, 2 * rng.randint(3, c["dim"] // 2)])
        most = 16385 * 40 * 128 * 2 // ((c["heads"] + c["kv"]) * c["dim"] * (4 if c["dtype"] == "f32" else 2))
        c["tokens"] = max(1, min(spread(1, 16384), most))
    elif c["kind"] == "route":
        c["groups"] = rng.choice([1, 1, 4, 8, 16])
        c["experts"] = c["groups"] * max(2, spread(8, 768) // c["groups"])
        c["top_groups"] = rng.choice([1, 2, 4]) if c["groups"] > 4 else c["groups"]
        c["k"] = min(rng.choice([1, 2, 4, 6, 8, 8, 10, 16]), c["top_groups"] * (c["experts"] // c["groups"]))
        c.update(tokens=spread(1, 8192), scoring=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, renormalize=rng.random() < 0.7)
    elif c["kind"] == "combine":
        c.update(experts=spread(8, 512), hidden=rng.choice([1, 2, 4]) * spread(64, 2000), shared=rng.random() < 0.5, dropped=rng.random() < 0.3)
        c["k"] = min(rng.choice([1, 2, 4, 6, 8, 8, 10]), c["experts"])
        c["tokens"] = max(1, min(spread(1, 8192), 4099 * 8 * 2560 // (c["k"] * c["hidden"]) // 2, 65536 // c["k"]))
    else:
        c["vocab"] = spread(1000, 262144)
        most = 2048 * 151936 * 2 // (c["vocab"] * (4 if c["dtype"] == "f32" else 2))
        c.update(rows=max(1, min(spread(1, 4096), most)), tokens=rng.choice([0, 1, 1, 1, 2, 5]), top=rng.choice([0, 1, 5, 8, 20, 32]), masked=rng.random() < 0.3)
    return c


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["kind"] == "rope":
        n = case["tokens"] * (case["heads"] + case["kv"]) * case["dim"]
        axes = 1 if case["axes"] == "one" else 3
        return {"bytes": 2 * n * size + case["tokens"] * 4 * axes + 8 * case["dim"], "flops": 7 * n}
    if case["kind"] == "route":
        n = case["tokens"] * case["experts"]
        return {"bytes": n * size + case["tokens"] * case["k"] * 8 + (4 * case["experts"] if case["bias"] else 0), "flops": 4 * n}
    if case["kind"] == "combine":
        slots, n = case["tokens"] * case["k"], case["tokens"] * case["hidden"]
        sides = 3 if case["shared"] else 2  # the residual in, the result out, the shared expert's rows in
        return {"bytes": slots * (case["hidden"] * 4 + 12) + sides * n * size + 4 * case["experts"], "flops": 2 * (slots * case["hidden"] + 2 * n)}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * size + case["rows"] * (8 * case["tokens"] + 8 * case["top"] + 8), "flops": 5 * n}


# ----------------------------------------------------------------- inputs --

def _axis_of(case):
    n = case["rot"] // 2
    if case["axes"] == "sections":  # time first, then equal shares of height and width
        side = 3 * n // 8
        return [0] * (n - 2 * side) + [1] * side + [2] * side
    return [i % 3 for i in range(n)] if case["axes"] == "cycle" else [0] * n


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case=case)

    def normal(*shape):
        return torch.randn(shape, device=dev, generator=gen)

    def uniform(*shape):
        return torch.rand(shape, device=dev, generator=gen)

    if case["kind"] == "rope":
        n, dim = case["tokens"], case["dim"]
        # products' outputs: heads of different sizes, a few channels far larger than the others
        wide = 2 * dim if case["gated"] else dim
        q = normal(n, case["heads"], wide) * (0.2 + 4 * uniform(1, case["heads"], 1))
        k = normal(n, case["kv"], dim) * (0.2 + 4 * uniform(1, case["kv"], 1))
        k[..., ::dim // 4] *= 8
        s["q"], s["k"] = q.to(dt)[..., :dim], k.to(dt)
        s["q_weight"], s["k_weight"] = 0.5 + uniform(dim), 0.5 + uniform(dim)
        at = torch.arange(n, device=dev, dtype=torch.int32)
        if case["axes"] == "one":
            pos = at[None] + case["start"]
        else:  # frames of 12 x 20 patches
            pos = torch.stack((at // 240, at % 240 // 20, at % 20)) + case["start"]
        s["positions"] = pos.to(torch.int32).contiguous()
        s["frequency"] = 1e6 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])
        s["axis_of"] = _axis_of(case)
        s["axis"] = torch.tensor(s["axis_of"], device=dev)
        s["frequency_gpu"] = s["frequency"].to(dev)
        if own:
            from block_quantized_matvec_gb300 import mmvq
            s["table"] = mmvq.rope_table(s["frequency"], axis_of=s["axis_of"], device=dev)
            s["out"] = (torch.empty((n, case["heads"], dim), dtype=dt, device=dev), torch.empty((n, case["kv"], dim), dtype=dt, device=dev))
    elif case["kind"] == "route":
        n, e = case["tokens"], case["experts"]
        s["logits"] = (normal(n, e) * (0.5 + 2 * uniform(n, 1)) + normal(1, e) * 0.5).to(dt)
        s["bias"] = normal(e) * 0.1 if case["bias"] else None
        if own:
            s["out"] = (torch.empty((n, case["k"]), dtype=torch.int32, device=dev), torch.empty((n, case["k"]), device=dev))
    elif case["kind"] == "combine":
        n, e, k, h = case["tokens"], case["experts"], case["k"], case["hidden"]
        topk = (uniform(n, e) + 0.3 * uniform(1, e)).argsort(1)[:, :k].to(torch.int32)
        if case["dropped"]:  # a few choices that no expert takes
            topk = torch.where(uniform(n, k) < 0.05, torch.full_like(topk, -1), topk)
        # the experts' lists, as route_groups gives them: positions in expert order, then slot order
        flat = topk.flatten().long()
        s["slot_of"] = torch.where(flat < 0, e, flat).argsort(stable=True).to(torch.int32)
        count = torch.zeros(e + 1, dtype=torch.int64, device=dev)
        count.index_add_(0, flat.clamp(min=0) + 1, (flat >= 0).long())
        s["offsets"] = count.cumsum(0).to(torch.int32)
        w = uniform(n, k) + 0.05
        s["topk"], s["weights"] = topk.contiguous(), w / w.sum(1, keepdim=True)
        s["y"] = normal(n * k, h)
        s["residual"] = (normal(n, h) * 3).to(dt)
        s["shared"] = normal(n, h).to(dt) if case["shared"] else None
        s["gate"] = normal(n) if case["shared"] else None
        if own:
            s["out"] = torch.empty((n, h), dtype=dt, device=dev)
    else:
        n, v = case["rows"], case["vocab"]
        x = normal(n, v).mul_(0.8 + 2 * uniform(n, 1))
        sure = (uniform(n) < 0.3).float() * (8 + 12 * uniform(n))  # rows that are all but certain
        best = (uniform(n) * v).long().clamp(max=v - 1)
        at = torch.arange(n, device=dev)
        x[at, best] += 6 + sure
        tokens = (uniform(n, case["tokens"]) * v).to(torch.int32).clamp(max=v - 1)
        if case["tokens"]:
            tokens[:, 0] = torch.where(uniform(n) < 0.6, best.to(torch.int32), tokens[:, 0])
        if case["masked"]:  # a grammar allows a twentieth of the tokens in half of the rows; one row has none
            for i in range(0, n, 2):
                x[i].masked_fill_(uniform(v) > 0.05, float("-inf"))
            if n >= 4:
                x[n // 2] = float("-inf")
        s["logits"], s["tokens"] = x.to(dt), tokens
        s["scale"] = 0.8
        if own:
            f = dict(dtype=torch.float32, device=dev)
            s["out"] = dict(lse=torch.empty(n, **f), entropy=torch.empty(n, **f), logprobs=torch.empty((n, case["tokens"]), **f),
                            top_ids=torch.empty((n, case["top"]), dtype=torch.int32, device=dev), top_logprobs=torch.empty((n, case["top"]), **f))
    return s


# ------------------------------------------------------------ plain forms --

def _turned(x, w, cos, sin, rot, interleaved):
    x = x.float()
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    t = x[..., :rot]
    a, b = (t[..., 0::2], t[..., 1::2]) if interleaved else (t[..., :rot // 2], t[..., rot // 2:])
    a, b = a * cos - b * sin, a * sin + b * cos
    t = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((t, x[..., rot:]), -1)


def _plain_rope(s):
    c = s["case"]
    angle = s["positions"].double().T[:, s["axis"]] * s["frequency_gpu"]  # far positions: in 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    return [_turned(s[x], s[x + "_weight"], cos, sin, c["rot"], c["interleaved"]).to(DTYPES[c["dtype"]]) for x in ("q", "k")]


def _best(x, k):
    """Places of the k largest of each row, the largest first, equal ones by place."""
    x, got = x.clone(), []
    for _ in range(k):
        got.append(x.argmax(-1, keepdim=True))
        x.scatter_(-1, got[-1], float("-inf"))
    return torch.cat(got, -1)


def _plain_route(s):
    c = s["case"]
    x = s["logits"].float()
    wide = x.double()  # values next to one another decide: in 64 bits
    value = torch.softmax(wide, -1) if c["scoring"] == "softmax" else 1 / (1 + torch.exp(-wide))
    if s["bias"] is not None:
        value = value + s["bias"].double()
    elif c["groups"] == c["top_groups"]:
        value = x  # the scores' order is the logits'
    if c["groups"] > c["top_groups"]:
        g = value.unflatten(-1, (c["groups"], -1))
        two = g.gather(-1, _best(g, 2)).sum(-1)
        keep = torch.zeros_like(two, dtype=torch.bool).scatter_(-1, _best(two, c["top_groups"]), True)
        value = g.masked_fill(~keep[..., None], float("-inf")).flatten(-2)
    ids = _best(value, c["k"])
    mine = x.gather(-1, ids)
    if c["scoring"] == "softmax":
        top = x.amax(-1, keepdim=True)
        w = torch.exp(mine - (mine.amax(-1, keepdim=True) if c["renormalize"] else top))
        total = w.sum(-1, keepdim=True) if c["renormalize"] else torch.exp(x - top).sum(-1, keepdim=True)
        w = w / total
    else:
        w = 1 / (1 + torch.exp(-mine))
        if c["renormalize"]:
            w = w / w.sum(-1, keepdim=True)
    return {"topk": ids.to(torch.int32), "weights": w * 2.5}


def _plain_combine(s):
    c = s["case"]
    n, k = s["topk"].shape
    place = torch.empty_like(s["slot_of"], dtype=torch.int64)
    place[s["slot_of"].long()] = torch.arange(n * k, device=place.device)
    w = torch.where(s["topk"] >= 0, s["weights"], torch.zeros_like(s["weights"]))
    out = s["residual"].float()
    for j in range(k):
        out = out + w[:, j:j + 1] * s["y"][place.view(n, k)[:, j]]
    if s["shared"] is not None:
        out = out + s["shared"].float() / (1 + torch.exp(-s["gate"]))[:, None]
    return out.to(DTYPES[c["dtype"]])


def _plain_logprobs(s):
    c = s["case"]
    x = s["logits"].float()
    top = max(1, c["top"])
    ids = _best(x, top)
    best = x.gather(-1, ids)
    none = best[:, :1] == float("-inf")
    far = (x - torch.where(none, torch.zeros_like(best[:, :1]), best[:, :1])) * s["scale"]  # from the largest: 0 and below
    e = torch.exp(far).scatter_(-1, ids[:, :1], 0.0)  # of all but the largest: a sure row keeps its digits
    more = e.sum(-1)
    drop = torch.log1p(more)
    entropy = drop - (e * far.clamp(min=-1e4)).sum(-1) / (1 + more)
    none = none[:, 0]
    minus = torch.full_like(drop, float("-inf"))
    say = far.gather(-1, s["tokens"].long()) - drop[:, None]
    alt = far.gather(-1, ids) - drop[:, None]
    alt = torch.where(best == float("-inf"), minus[:, None], alt)
    ids = torch.where(best == float("-inf"), torch.full_like(ids, -1), ids)
    return {"lse": torch.where(none, minus, best[:, 0] * s["scale"] + drop), "entropy": torch.where(none, torch.zeros_like(drop), entropy),
            "logprobs": torch.where(none[:, None], minus[:, None], say),
            "top_ids": ids[:, :c["top"]].to(torch.int32), "top_logprobs": alt[:, :c["top"]]}


def run(s):
    c = s["case"]
    if not own:
        return {"rope": _plain_rope, "route": _plain_route, "combine": _plain_combine, "logprobs": _plain_logprobs}[c["kind"]](s)
    from block_quantized_matvec_gb300 import mmvq
    if c["kind"] == "rope":
        return list(mmvq.norm_rope(s["q"], s["k"], s["positions"], s["table"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                                   interleaved=c["interleaved"], out=s["out"]))
    if c["kind"] == "route":
        topk, weights = mmvq.route_topk(s["logits"], c["k"], scoring=c["scoring"], bias=s["bias"], n_groups=c["groups"], top_groups=c["top_groups"],
                                        renormalize=c["renormalize"], scale=2.5, out=s["out"])
        return {"topk": topk, "weights": weights}
    if c["kind"] == "combine":
        return mmvq.combine_experts(s["y"], s["topk"], s["weights"], s["offsets"], s["slot_of"], residual=s["residual"], shared=s["shared"],
                                    shared_gate=s["gate"], out=s["out"])
    return mmvq.token_logprobs(s["logits"], s["tokens"], top=c["top"], scale=s["scale"], out=s["out"])


# ---------------------------------------------------- the definition, 64 bits --

def _exact_rope(s):
    c = s["case"]
    n, half = c["tokens"], c["rot"] // 2
    pos = s["positions"].double()
    got = []
    for name in ("q", "k"):
        x, w = s[name].double(), s[name + "_weight"].double()
        z = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        out = z.clone()
        for i in range(half):
            i0, i1 = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
            turn = torch.polar(torch.ones(n, dtype=torch.float64, device=x.device), pos[s["axis_of"][i] if len(pos) > 1 else 0] * float(s["frequency"][i]))
            pair = torch.complex(z[..., i0], z[..., i1]) * turn[:, None]
            out[..., i0], out[..., i1] = pair.real, pair.imag
        got.append(out)
    return got


def _exact_route(s):
    c = s["case"]
    x = s["logits"].double()
    score = (x - torch.logsumexp(x, -1, keepdim=True)).exp() if c["scoring"] == "softmax" else torch.sigmoid(x)
    if s["bias"] is None and c["groups"] == c["top_groups"]:
        order = x.clone()
    else:
        order = score + (0 if s["bias"] is None else s["bias"].double())
    if c["groups"] > c["top_groups"]:
        g = order.view(len(x), c["groups"], -1)
        two = g.sort(-1, descending=True)[0][..., :2].sum(-1)
        out = two.sort(dim=-1, descending=True, stable=True)[1][:, c["top_groups"]:]
        g.scatter_(1, out[..., None].expand(-1, -1, g.shape[-1]), float("-inf"))
    ids = order.sort(dim=-1, descending=True, stable=True)[1][:, :c["k"]]
    w = score.gather(-1, ids)
    if c["renormalize"]:
        w = w / w.sum(-1, keepdim=True)
    return {"topk": ids.to(torch.int32), "weights": 2.5 * w}


def _exact_combine(s):
    c = s["case"]
    out = s["residual"].double()
    if s["shared"] is not None:
        out = out + torch.sigmoid(s["gate"].double())[:, None] * s["shared"].double()
    flat = s["slot_of"].long()[:int(s["offsets"][-1])]  # position by position
    for lo in range(0, len(flat), 8192):
        slots = flat[lo:lo + 8192]
        out.index_add_(0, slots // c["k"], s["y"][lo:lo + len(slots)].double() * s["weights"].flatten()[slots].double()[:, None])
    return out


def _exact_logprobs(s):
    c = s["case"]
    parts = []
    for lo in range(0, c["rows"], 128):
        x = s["logits"][lo:lo + 128].double() * s["scale"]
        lse = torch.logsumexp(x, -1)
        logp = torch.where(lse[:, None] > float("-inf"), x - lse[:, None], torch.full_like(x, float("-inf")))
        p = logp.exp()
        # -sum p log p; the largest term by what the others leave, so that a sure row keeps its digits
        at = x.argmax(-1, keepdim=True)
        rest = p.scatter(-1, at, 0.0).sum(-1)
        sure = torch.where(rest < 0.5, torch.log1p(-rest), logp.gather(-1, at)[:, 0])
        terms = torch.where(p > 0, -p * logp.clamp(min=-1e4), torch.zeros_like(p)).scatter(-1, at, 0.0).sum(-1)
        entropy = torch.where(lse > float("-inf"), terms - (1 - rest) * sure, torch.zeros_like(lse))
        say = logp.gather(-1, s["tokens"][lo:lo + 128].long())
        say = torch.where(s["tokens"][lo:lo + 128].long() == at, sure[:, None], say)
        say = torch.where(lse[:, None] > float("-inf"), say, torch.full_like(say, float("-inf")))
        ids = s["logits"][lo:lo + 128].sort(dim=-1, descending=True, stable=True)[1][:, :c["top"]]
        alt = logp.gather(-1, ids)
        if c["top"]:
            alt[:, 0] = torch.where(lse > float("-inf"), sure, alt[:, 0])
        ids = torch.where(alt == float("-inf"), torch.full_like(ids, -1), ids)
        parts.append((lse, entropy, say, ids.to(torch.int32), alt))
    return dict(zip(("lse", "entropy", "logprobs", "top_ids", "top_logprobs"), (torch.cat(p) for p in zip(*parts))))


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "route": _exact_route, "combine": _exact_combine, "logprobs": _exact_logprobs}[case["kind"]](s)
