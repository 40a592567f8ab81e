"""Cases and plain forms of the operators on a 4-bit paged key/value cache.

Three operators, called next to the block-quantized products of this package
(the query, key and value projections before them, the output projection after):

* ``mmvq.kv4_append``: keys and values quantised as they are written to the
  cache, 4 bits a value in blocks of 32 along the head dimension;
* ``mmvq.kv4_read``: tokens of the cache read back as the values they stand for;
* ``mmvq.kv4_attention``: attention of 1 to 8 query tokens a sequence (a decode
  step, or a window of drafted tokens to verify) over the cache, grouped query
  heads, causal, optionally with a sliding window and a few first tokens (sinks)
  that stay visible.

Format.  A block of 32 values x keeps d = fp16((max - min) / 15), the step, and
z = fp16((max + min) / 2), the midpoint; a code c in 0..15 stands for
z + d * (c - 7.5), and c = round-half-even((x - z) / d + 7.5) clamped to 0..15
(0 where d is 0), every operation in fp32.  Inputs beyond fp16's range are
clamped to +-65504 first.

Layout.  The cache is bytes [pages, kv heads, page / 16, 20 * dim]: a tile of 16
tokens of one head is (nb = dim / 32 blocks, t = token in the tile)

* key codes, 8 * dim bytes: word(j, lane) at 512 * (j / 4) + 16 * lane + 4 * (j % 4);
  j = nb * (t / 8) + b, lane = 4 * (t % 8) + u holds values 32 b + 8 u .. + 7 of
  token t, value i in bits 4 i .. 4 i + 3;
* value codes, 8 * dim bytes, words in the same places: j = nb * (t / 8) + b,
  lane = 4 * g + (t % 8) / 2 holds values 32 b + 4 g .. + 3 of tokens t (even, low
  half) and t + 1 (high half), value i in bits 4 i .. 4 i + 3 of the half;
* key d, then key z: fp16 [token][block];
* value d, then value z: fp16 [(t % 8) / 2][t / 8][block][t % 2].
"""
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TILE = 16  # tokens of a tile


# ------------------------------------------------------------------ cases --

def listed():
    """The heads 24 / 2 of 256 are those of this repository's dense shapes (12288 x 2560 for queries
    with their gates, 512 x 2560 for keys, 2560 x 6144 for the output); the others are generic."""
    a = dict(kind="attention", ragged=False, window=0, sinks=0)
    w = dict(kind="append", ragged=False)
    return [
        # one chat that has just begun: a decode step's attention, where only latency counts
        dict(a, name="decode 1 short", dtype="f32", heads=24, kv=2, dim=256, page=64, seqs=1, tokens=1, context=77),
        # one chat, a verify window of five drafted tokens over a few thousand
        dict(a, name="verify 1x5 4k", dtype="f32", heads=24, kv=2, dim=256, page=64, seqs=1, tokens=5, context=4101),
        # one long document: work is split over the context
        dict(a, name="decode 1 long", dtype="f32", heads=24, kv=2, dim=256, page=256, seqs=1, tokens=1, context=131071),
        # a served batch of mixed lengths, one of them still empty
        dict(a, name="decode 64 ragged", dtype="bf16", heads=32, kv=8, dim=128, page=16, seqs=64, tokens=1, context=8192, ragged=True),
        # drafted tokens verified in a batch: many rows a head
        dict(a, name="verify 8x8 16k", dtype="bf16", heads=24, kv=2, dim=256, page=128, seqs=8, tokens=8, context=16389),
        # sliding-window layers of a long-context batch, four sinks
        dict(a, name="window 32x1 4096", dtype="f16", heads=40, kv=8, dim=128, page=32, seqs=32, tokens=1, context=40000, ragged=True, window=4096, sinks=4),
        # a short window with drafted tokens, every head with its own keys, odd sizes
        dict(a, name="window 12x3 513", dtype="f32", heads=12, kv=12, dim=64, page=16, seqs=12, tokens=3, context=2500, ragged=True, window=513, sinks=5),
        # a decode step's new token of one chat, written and read back: latency
        dict(w, name="write 1x1", dtype="f32", kv=2, dim=256, page=64, seqs=1, tokens=1, context=77),
        # prompts of mixed lengths appended behind 37 cached tokens
        dict(w, name="write 24 ragged", dtype="bf16", kv=8, dim=128, page=32, seqs=24, tokens=1201, context=37, ragged=True),
        # one long prompt
        dict(w, name="write 1x24k", dtype="f32", kv=2, dim=256, page=64, seqs=1, tokens=24575, context=0),
        # cached prefixes read back for a consumer that wants plain values
        dict(kind="read", name="read 6 ragged", dtype="f32", kv=4, dim=64, page=16, seqs=6, context=3001, ragged=True),
        dict(kind="read", name="read 4x16k", dtype="bf16", kv=8, dim=128, page=64, seqs=4, context=16384, ragged=False),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))
    c = dict(kind=rng.choice(["attention", "attention", "attention", "append", "read"]),
             dtype=rng.choice(["f32", "f32", "bf16", "f16"]), dim=rng.choice([64, 128, 256]), kv=rng.choice([1, 2, 3, 4, 8, 12]),
             page=rng.choice([16, 32, 64, 128, 256]), seqs=spread(1, 64), ragged=rng.random() < 0.6)
    cap = 3.0e8 / (c["kv"] * c["dim"] * c["seqs"])  # tokens a sequence, so that the cache stays below the largest listed
    if c["kind"] == "attention":
        c["heads"] = c["kv"] * rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        c["tokens"] = rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
        c["context"] = spread(1, 131072)
        c["window"], c["sinks"] = (spread(16, 8192), rng.choice([0, 1, 4, 16])) if rng.random() < 0.4 else (0, 0)
        rows = c["tokens"] * c["heads"] // c["kv"]
        c["context"] = max(c["tokens"], int(min(c["context"], cap / max(1.0, rows / 8.0))))
    elif c["kind"] == "append":
        c["tokens"] = max(1, int(min(spread(1, 24576), cap / 30)))
        c["context"] = rng.choice([0, 1, 15, 16, 37, 300])
    else:
        c["context"] = max(1, int(min(spread(1, 65536), cap / 6)))
    return c


def shape_of(case):
    """(lengths, new tokens) of each sequence: what the host knows of a case."""
    n = case["seqs"]
    part = [(n - b) / n if case["ragged"] else 1.0 for b in range(n)]
    if case["kind"] == "attention":
        news = [1 + (case["tokens"] - 1 + 3 * b) % case["tokens"] if case["ragged"] else case["tokens"] for b in range(n)]
        lens = [max(t, int(case["context"] * p)) for t, p in zip(news, part)]
        if case["ragged"] and n >= 4:
            lens[n // 2] = 0
    elif case["kind"] == "append":
        news = [max(1, int(case["tokens"] * p)) for p in part]
        lens = [case["context"] + t for t in news]
    else:
        lens = [max(1, int(case["context"] * p)) for p in part]
        news = list(lens)
    return lens, news


def visible(case, n, t):
    """Cached tokens that t queries at the end of n tokens read between them, and their (query, token) pairs."""
    w, s = case["window"], case["sinks"]
    if not w:
        return n, sum(max(0, n - t + i + 1) for i in range(t))
    first = max(0, n - t - w + 1)
    read, pairs = n - first + min(s, first), 0
    for i in range(t):
        p = n - t + i
        if p >= 0:
            lo = max(0, p - w + 1)
            pairs += p - lo + 1 + min(s, lo)
    return read, pairs


def work(case):
    lens, news = shape_of(case)
    size = 4 if case["dtype"] == "f32" else 2
    d, kv = case["dim"], case["kv"]
    token = kv * d * 5 // 4  # cache bytes of a token, keys and values with their d and z
    if case["kind"] == "attention":
        got = [visible(case, n, t) for n, t in zip(lens, news)]
        rows = sum(news) * case["heads"]
        return {"bytes": sum(r for r, _ in got) * token + rows * d * 2 * size + rows * 4, "flops": sum(p for _, p in got) * case["heads"] * 4 * d}
    n = sum(news)
    values = n * kv * 2 * d
    if case["kind"] == "append":  # keys and values in, the cache's bytes, the values back out
        return {"bytes": 2 * values * size + n * token, "flops": values * 8}
    return {"bytes": values * size + n * token, "flops": values * 2}


# ----------------------------------------------------------------- inputs --

def _cache(pages, kv, page, dim, gen, dev):
    """Random codes; steps and midpoints as of keys and values of about unit size, a few blocks larger."""
    c = torch.randint(0, 256, (pages, kv, page // TILE, 20 * dim), dtype=torch.uint8, device=dev, generator=gen)
    shape = (pages, kv, page // TILE, dim // 2)
    half = c.view(torch.float16)
    for at in (8 * dim, 9 * dim):  # in fp16 values: [key d | key z], [value d | value z]
        d = torch.rand(shape, device=dev, generator=gen) * 0.3 + 0.05
        d = torch.where(torch.rand(shape, device=dev, generator=gen) < 0.02, d * 4, d)
        z = (torch.rand(shape, device=dev, generator=gen) - 0.5) * 2 * d
        half[..., at:at + dim // 2] = d.half()
        half[..., at + dim // 2:at + dim] = z.half()
    return c


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    lens, news = shape_of(case)
    page, kv, dim = case["page"], case["kv"], case["dim"]
    need = [-(-n // page) for n in lens]
    pages = max(1, sum(need))
    order = torch.randperm(pages, device=dev, generator=gen, dtype=torch.int64).to(torch.int32)
    table = torch.zeros((len(lens), max(1, max(need))), dtype=torch.int32, device=dev)
    at = torch.arange(table.shape[1], device=dev)[None, :]
    n_pages = torch.tensor(need, device=dev)[:, None]
    table[at < n_pages] = order[:sum(need)]
    offsets = [0]
    for t in news:
        offsets.append(offsets[-1] + t)
    s = dict(case=case, table=table, lens=torch.tensor(lens, dtype=torch.int32, device=dev), total=offsets[-1],
             offsets=torch.tensor(offsets, dtype=torch.int32, device=dev))
    dt = DTYPES[case["dtype"]]
    if case["kind"] == "append":
        s["cache"] = torch.zeros((pages, kv, page // TILE, 20 * dim), dtype=torch.uint8, device=dev)
        k = torch.randn((s["total"], kv, dim), device=dev, generator=gen)
        k[..., ::dim // 4] *= 6  # a few channels of keys are far larger than the others
        s["k"], s["v"] = k.to(dt), torch.randn((s["total"], kv, dim), device=dev, generator=gen).to(dt)
    else:
        s["cache"] = _cache(pages, kv, page, dim, gen, dev)
    if case["kind"] == "attention":
        q = torch.randn((s["total"], case["heads"], dim), device=dev, generator=gen)
        s["q"] = (q * (0.5 + 2.5 * torch.rand((1, case["heads"], 1), device=dev, generator=gen))).to(dt)
        s["scale"] = dim ** -0.5
        if own:  # kept by a program for all of its layers and steps
            from block_quantized_matvec_gb300 import mmvq
            s["workspace"] = mmvq.kv4_attention_workspace(dim, dev)
    # the sequence and the place in it of each new token, and the largest counts: known to a program that made the batch
    t = torch.tensor(news, device=dev)
    s["seq"] = torch.repeat_interleave(torch.arange(len(news), device=dev), t, output_size=s["total"])
    s["nth"] = torch.arange(s["total"], device=dev) - s["offsets"].long()[s["seq"]]
    s["max_new"], s["max_len"] = max(news), max(lens)
    return s


# ------------------------------------------------------------ plain forms --

def _bytes_of(dim, page, table, kv, seq, pos):
    """Places in the flat cache of the bytes of tokens pos of sequences seq: (key codes, value codes)
    [..., kv, dim / 2] in value order, and the fp16 places of (key d, key z, value d, value z) [..., kv, nb]."""
    dev, nb = pos.device, dim // 32
    tile = (table.long()[seq, pos // page][..., None] * kv + torch.arange(kv, device=dev)) * (page // TILE) + (pos % page // TILE)[..., None]
    base = (tile * (20 * dim))[..., None]
    t = (pos % TILE)[..., None, None]
    y = torch.arange(dim // 2, device=dev)
    j = nb * (t // 8) + y // 16
    word = 512 * (j // 4) + 4 * (j % 4)
    key = base + word + 16 * (4 * (t % 8) + y % 16 // 4) + y % 4
    val = base + 8 * dim + word + 16 * (4 * (y % 16 // 2) + t % 8 // 2) + 2 * (t % 2) + y % 2
    b = torch.arange(nb, device=dev)
    ks = base // 2 + 8 * dim + t * nb + b
    vs = base // 2 + 9 * dim + ((t % 8 // 2 * 2 + t // 8) * nb + b) * 2 + t % 2
    return key, val, ks, ks + dim // 2, vs, vs + dim // 2


def _values(codes, d, z, dim):
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], dim).float()
    return (z.float().repeat_interleave(32, -1) + d.float().repeat_interleave(32, -1) * (c - 7.5))


def _gather(s, seq, pos):
    """Keys and values [..., kv, dim] in fp32 of tokens pos of sequences seq."""
    c = s["case"]
    key, val, kd, kz, vd, vz = _bytes_of(c["dim"], c["page"], s["table"], c["kv"], seq, pos)
    flat, half = s["cache"].view(-1), s["cache"].view(-1).view(torch.float16)
    return _values(flat[key], half[kd], half[kz], c["dim"]), _values(flat[val], half[vd], half[vz], c["dim"])


def _quantised(x):
    """Codes (two a byte), d and z of x [..., dim] in blocks of 32."""
    x = x.float().clamp(-65504, 65504).unflatten(-1, (-1, 32))
    hi, lo = x.amax(-1), x.amin(-1)
    d = ((hi - lo) / torch.full((), 15.0, device=x.device)).half()
    z = ((hi + lo) * 0.5).half()
    step = torch.where(d > 0, d, torch.ones_like(d)).float()[..., None]
    c = torch.round((x - z.float()[..., None]) / step + 7.5).clamp(0, 15)
    c = torch.where(d[..., None] > 0, c, torch.zeros_like(c)).to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), d, z


def _plain_append(s):
    c = s["case"]
    pos = s["lens"].long()[s["seq"]] - (s["offsets"][1:] - s["offsets"][:-1]).long()[s["seq"]] + s["nth"]
    key, val, kd, kz, vd, vz = _bytes_of(c["dim"], c["page"], s["table"], c["kv"], s["seq"], pos)
    flat, half = s["cache"].view(-1), s["cache"].view(-1).view(torch.float16)
    flat[key], half[kd], half[kz] = _quantised(s["k"])
    flat[val], half[vd], half[vz] = _quantised(s["v"])


def _plain_read(s):
    pos = s["lens"].long()[s["seq"]] - (s["offsets"][1:] - s["offsets"][:-1]).long()[s["seq"]] + s["nth"]
    k, v = _gather(s, s["seq"], pos)
    dt = DTYPES[s["case"]["dtype"]]
    return {"k": k.to(dt), "v": v.to(dt)}


def _plain_attention(s):
    c = s["case"]
    dev, kv, dim, group, tq = s["q"].device, c["kv"], c["dim"], c["heads"] // c["kv"], s["max_new"]
    n = s["lens"].long()[:, None]
    new = (s["offsets"][1:] - s["offsets"][:-1]).long()[:, None]
    # the positions that any query of the sequence may see: the sinks, then the window (or all)
    w, sinks = c["window"], c["sinks"]
    span = min(s["max_len"], w + tq - 1) if w else s["max_len"]
    first = (n - span).clamp(min=0) if w else torch.zeros_like(n)
    first = torch.maximum(first, torch.full_like(first, min(sinks, s["max_len"])))
    pos = torch.cat((torch.arange(min(sinks, s["max_len"]), device=dev).expand(len(n), -1), first + torch.arange(span, device=dev)), 1)
    inside = pos < n
    at = torch.where(inside, pos, torch.zeros_like(pos))
    k, v = _gather(s, torch.arange(len(n), device=dev)[:, None].expand_as(at), at)
    q = torch.zeros((len(n), tq, kv, group, dim), device=dev)
    q[s["seq"], s["nth"]] = s["q"].float().unflatten(1, (kv, group))
    mine = n - new + torch.arange(tq, device=dev)  # each query's position
    seen = inside[:, None] & (pos[:, None] <= mine[..., None])
    if w:
        seen &= (pos[:, None] > mine[..., None] - w) | (pos[:, None] < sinks)
    seen = seen[:, None, :, None]  # [seqs, 1, queries, 1, positions]
    x = torch.matmul(q.permute(0, 2, 1, 3, 4).flatten(2, 3), k.permute(0, 2, 3, 1)).unflatten(2, (tq, group)) * s["scale"]
    x = x.masked_fill(~seen, float("-inf"))
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top > float("-inf"), top, torch.zeros_like(top)))
    total = e.sum(-1)
    y = torch.matmul(e.flatten(2, 3), (v * inside[..., None, None]).permute(0, 2, 1, 3)).unflatten(2, (tq, group))
    y = torch.where(total[..., None] > 0, y / total[..., None], torch.zeros_like(y))
    lse = torch.where(total > 0, top[..., 0] + torch.log(total), torch.full_like(total, float("-inf")))
    y = y.permute(0, 2, 1, 3, 4)[s["seq"], s["nth"]].flatten(1, 2)
    return {"y": y.to(s["q"].dtype), "lse": lse.permute(0, 2, 1, 3)[s["seq"], s["nth"]].flatten(1, 2)}


def run(s):
    c = s["case"]
    if not own:
        if c["kind"] == "attention":
            return _plain_attention(s)
        if c["kind"] == "append":
            _plain_append(s)
        return _plain_read(s)
    from block_quantized_matvec_gb300 import mmvq
    where = (s["cache"], s["table"], s["offsets"], s["lens"])
    if c["kind"] == "attention":
        y, lse = mmvq.kv4_attention(s["q"], *where, scale=s["scale"], window=c["window"], sinks=c["sinks"], workspace=s["workspace"], with_lse=True)
        return {"y": y, "lse": lse}
    if c["kind"] == "append":
        mmvq.kv4_append(s["k"], s["v"], *where)
    k, v = mmvq.kv4_read(*where, s["total"], dtype=DTYPES[c["dtype"]])
    return {"k": k, "v": v}


# ---------------------------------------------------- the definition, 64 bits --

def _exact_block(x):
    """Values that x [..., 32] stands for once quantised, the format's fp32 and fp16 roundings made one by one on 64-bit numbers."""
    f = lambda t: t.float().double()  # noqa: E731  one correctly rounded fp32 operation, from its 64-bit result
    x = x.double().clamp(-65504, 65504)
    hi, lo = x.amax(-1, keepdim=True), x.amin(-1, keepdim=True)
    d, z = f(f(hi - lo) / 15).half().double(), (f(hi + lo) / 2).half().double()
    c = f(f(f(x - z) / torch.where(d > 0, d, 1.0)) + 7.5).round().clamp(0, 15) * (d > 0)
    return z + d * (c - 7.5)


def _exact_tiles(t, dim):
    """Keys and values [tokens, kv, dim] of whole tiles t [tiles, kv, 20 * dim], by the layout's own order of words."""
    n, kv, nb = t.shape[0], t.shape[1], dim // 32

    def words(part):  # -> [n, kv, half of the tile, block, lane / 4, lane % 4, byte]
        w = part.reshape(n, kv, nb // 2, 8, 4, 4, 4).permute(0, 1, 2, 5, 3, 4, 6)
        return w.reshape(n, kv, 2, nb, 8, 4, 4)

    def nibbles(b):
        return torch.stack((b & 15, b >> 4), -1).flatten(-2).double()

    key = nibbles(words(t[..., :8 * dim]).permute(0, 2, 4, 1, 3, 5, 6).reshape(n * 16, kv, nb, 16))
    val = words(t[..., 8 * dim:16 * dim]).reshape(n, kv, 2, nb, 8, 4, 2, 2).permute(0, 2, 5, 6, 1, 3, 4, 7).reshape(n * 16, kv, nb, 16)
    half = t[..., 16 * dim:].contiguous().view(torch.float16).double().reshape(n, kv, 4, 16 * nb)
    ks = half[:, :, :2].reshape(n, kv, 2, 16, nb).permute(2, 0, 3, 1, 4).reshape(2, n * 16, kv, nb, 1)
    vs = half[:, :, 2:].reshape(n, kv, 2, 4, 2, nb, 2).permute(2, 0, 4, 3, 6, 1, 5).reshape(2, n * 16, kv, nb, 1)
    return (ks[1] + ks[0] * (key - 7.5)).flatten(-2), (vs[1] + vs[0] * (nibbles(val) - 7.5)).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    lens, news = shape_of(case)
    dim, kv = case["dim"], case["kv"]
    if case["kind"] == "append":
        return {x: _exact_block(s[x].unflatten(-1, (-1, 32))).flatten(-2) for x in ("k", "v")}
    ks, vs, ys, ls, done = [], [], [], [], 0
    for b, (n, t) in enumerate(zip(lens, news)):
        pages = s["table"][b, :-(-n // case["page"])].long()
        if case["kind"] == "read":
            k, v = _exact_tiles(s["cache"][pages].transpose(1, 2).flatten(0, 1), dim)
            ks.append(k[:n])
            vs.append(v[:n])
            continue
        q = s["q"][done:done + t].double()
        done += t
        if n == 0:
            ys.append(torch.zeros_like(q))
            ls.append(torch.full(q.shape[:2], float("-inf"), dtype=torch.float64, device=q.device))
            continue
        k, v = _exact_tiles(s["cache"][pages].transpose(1, 2).flatten(0, 1), dim)
        place = torch.arange(n, device=q.device)
        for i in range(t):
            p = n - t + i
            sees = place <= p
            if case["window"]:
                sees &= (place > p - case["window"]) | (place < case["sinks"])
            at = place[sees]
            x = torch.einsum("hgd,nhd->hgn", q[i].reshape(kv, -1, dim), k[at]) * s["scale"]
            ls.append(torch.logsumexp(x, -1).reshape(1, -1))
            ys.append(torch.einsum("hgn,nhd->hgd", torch.softmax(x, -1), v[at]).reshape(1, -1, dim))
    if case["kind"] == "read":
        return {"k": torch.cat(ks), "v": torch.cat(vs)}
    return {"y": torch.cat(ys), "lse": torch.cat(ls)}
