"""A plain 64-bit implementation of the 4-bit key/value cache, byte by byte from the
layout's definition (include/mmvq.h), and batches of sequences to try it on."""
import numpy as np

TILE = 16


def word(j, lane):
    return 512 * (j // 4) + 16 * lane + 4 * (j % 4)


def places(D):
    """For each token of a tile: byte and shift of every key and value code, and the byte of
    every key d and value d (z lies D further)."""
    nb = D // 32
    t, d = np.meshgrid(np.arange(TILE), np.arange(D), indexing="ij")
    b, r = d // 32, d % 32
    kbit = 8 * word(nb * (t // 8) + b, 4 * (t % 8) + r // 8) + 4 * (r % 8)
    vbit = 8 * (8 * D + word(nb * (t // 8) + b, 4 * (r // 4) + (t % 8) // 2)) + 16 * (t % 2) + 4 * (r % 4)
    t, b = np.meshgrid(np.arange(TILE), np.arange(nb), indexing="ij")
    ks = 16 * D + 2 * (t * nb + b)
    vs = 18 * D + 2 * ((((t % 8) // 2 * 2 + t // 8) * nb + b) * 2 + t % 2)
    return kbit // 8, kbit % 8, vbit // 8, vbit % 8, ks, vs


def quantise(x):
    """x [..., D] (exact values in float64) -> codes [..., D], d and z [..., D/32] as float16:
    each fp32 operation of the format is a float64 one rounded to float32."""
    f = lambda v: np.asarray(v, np.float64).astype(np.float32).astype(np.float64)  # noqa: E731
    x = np.where(np.isnan(x), 0.0, np.clip(np.asarray(x, np.float64), -65504, 65504))
    x = x.reshape(*x.shape[:-1], -1, 32)
    hi, lo = x.max(-1), x.min(-1)
    d = f(f(hi - lo) / 15).astype(np.float16)
    z = f(f(hi + lo) * 0.5).astype(np.float16)
    dd, zz = d.astype(np.float64)[..., None], z.astype(np.float64)[..., None]
    c = np.rint(f(f(f(x - zz) / np.where(dd > 0, dd, 1)) + 7.5))
    c = np.where(dd > 0, np.clip(c, 0, 15), 0).astype(np.uint8)
    return c.reshape(*c.shape[:-2], -1), d, z


def values(c, d, z):
    r = lambda a: np.repeat(np.asarray(a, np.float64), 32, -1)  # noqa: E731
    return r(z) + r(d) * (c - 7.5)


def put(tile, t, D, key, value):
    """Writes token t's (codes, d, z) of its key and its value into tile (uint8 [20 D])."""
    kb, ksh, vb, vsh, ks, vs = places(D)
    for (c, d, z), by, sh, sc in ((key, kb[t], ksh[t], ks[t]), (value, vb[t], vsh[t], vs[t])):
        for i in range(D):
            tile[by[i]] = (int(tile[by[i]]) & ~(15 << sh[i])) & 255 | int(c[i]) << sh[i]
        for i in range(D // 32):
            tile[sc[i]:sc[i] + 2] = np.array([d[i]], np.float16).view(np.uint8)
            tile[sc[i] + D:sc[i] + D + 2] = np.array([z[i]], np.float16).view(np.uint8)


def get(tiles, D):
    """(key (codes, d, z), value (codes, d, z)) of tiles [n, 20 D]: arrays [n, 16, ...]."""
    kb, ksh, vb, vsh, ks, vs = places(D)
    two = lambda at: (tiles[:, at].astype(np.uint16) | tiles[:, at + 1].astype(np.uint16) << 8).view(np.float16)  # noqa: E731
    return ((tiles[:, kb] >> ksh & 15, two(ks), two(ks + D)), (tiles[:, vb] >> vsh & 15, two(vs), two(vs + D)))


class Batch:
    """Sequences of the given lengths (the last `news` rows of each are the call's rows) in a
    shuffled paged cache.  `fill`: the byte that unwritten places hold (0xff: fp16 NaN)."""

    def __init__(self, D, kv, page, lens, news, seed=0, fill=0xff, spare=2, table_spare=1):
        self.D, self.kv, self.page, self.lens, self.news = D, kv, page, list(lens), list(news)
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        self.n_pages = sum(need) + spare
        self.table = np.full((len(lens), max(1, max(need)) + table_spare), -7, np.int32)
        order = rng.permutation(self.n_pages)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.offsets = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
        self.n = int(self.offsets[-1])
        self.cache = np.full((self.n_pages, kv, page // TILE, 20 * D), fill, np.uint8)
        self.rng = rng

    def at(self, b, p):
        """(page, tile in it, token in that) of position p of sequence b."""
        return int(self.table[b, p // self.page]), p % self.page // TILE, p % TILE

    def positions(self):
        """(sequence, position) of each row."""
        return [(b, self.lens[b] - self.news[b] + i) for b in range(len(self.lens)) for i in range(self.news[b])]

    def fill_random(self, spread=1.0, offset=0.5):
        """Every cached token of every sequence gets random codes, steps and midpoints; the rest stays."""
        D = self.D
        for b, n in enumerate(self.lens):
            for p0 in range(0, n, TILE):
                pg, ti, _ = self.at(b, p0)
                full = self.rng.integers(0, 256, (self.kv, 20 * D), dtype=np.uint8)
                d = (self.rng.uniform(0.02, 0.3, (self.kv, 2, D // 2)) * spread).astype(np.float16)
                z = (self.rng.uniform(-1, 1, (self.kv, 2, D // 2)) * offset * spread).astype(np.float16)
                sc = np.stack((d, z), 2).reshape(self.kv, 2 * D).view(np.uint8)
                full[:, 16 * D:] = sc
                if n - p0 < TILE:  # keep the unwritten tokens' bytes
                    mine = np.zeros(20 * D, bool)
                    kb, _, vb, _, ks, vs = places(D)
                    for t in range(n - p0):
                        mine[kb[t]] = mine[vb[t]] = True
                        for s in (ks[t], vs[t]):
                            for e in (0, 1):
                                mine[s + e] = mine[s + D + e] = True
                    full = np.where(mine, full, self.cache[pg, :, ti])
                self.cache[pg, :, ti] = full

    def sequence(self, b):
        """Sequence b's keys and values in float64 [n, kv, D], with |z| and d apart: [n, kv, D] each."""
        n, D = self.lens[b], self.D
        if n == 0:
            return [(np.zeros((0, self.kv, D)),) * 4] * 2
        out = []
        tiles = -(-n // TILE)
        ids = [self.at(b, TILE * i)[:2] for i in range(tiles)]
        per = np.stack([self.cache[pg, :, ti] for pg, ti in ids])
        k, v = get(per.reshape(-1, 20 * D), D)
        for c, d, z in (k, v):
            shp = lambda a: a.reshape(tiles, self.kv, TILE, -1).transpose(0, 2, 1, 3).reshape(tiles * TILE, self.kv, -1)[:n]  # noqa: E731
            c, d, z = shp(c), shp(d), shp(z)
            r = lambda a: np.repeat(a.astype(np.float64), 32, -1)  # noqa: E731
            out.append((values(c, d, z), np.abs(r(z)), r(d), np.abs(c - 7.5)))
        return out


def attention(bt, q, scale, window=0, sinks=0):
    """float64 attention of q [rows, heads, D] -> y, lse and, for the error bounds, a [rows, heads, D]
    = sum p (|z| + d |c - 7.5|) of the values and s [rows, heads] = max over the seen tokens of
    scale * sum |q| (|z| + 15 d) of the keys."""
    heads, D = q.shape[1], bt.D
    g = heads // bt.kv
    y = np.zeros(q.shape)
    a = np.zeros(q.shape)
    lse = np.full(q.shape[:2], -np.inf)
    sabs = np.zeros(q.shape[:2])
    seqs = {}
    for r, (b, p) in enumerate(bt.positions()):
        if b not in seqs:
            seqs = {b: bt.sequence(b)}
        (k, kz, kd, _), (v, vz, vd, vc) = seqs[b]
        j = np.arange(bt.lens[b])
        see = j <= p
        if window:
            see &= (j > p - window) | (j < sinks)
        j = j[see]
        if not len(j):
            continue
        qr = q[r].astype(np.float64).reshape(bt.kv, g, D)
        x = scale * np.einsum("hgd,nhd->hgn", qr, k[j])
        sabs[r] = abs(scale) * np.einsum("hgd,nhd->hgn", np.abs(qr), kz[j] + 15 * kd[j]).max(-1).reshape(-1)
        top = x.max(-1, keepdims=True)
        e = np.exp(x - top)
        l = e.sum(-1, keepdims=True)
        y[r] = np.einsum("hgn,nhd->hgd", e / l, v[j]).reshape(heads, D)
        a[r] = np.einsum("hgn,nhd->hgd", e / l, vz[j] + vd[j] * vc[j]).reshape(heads, D)
        lse[r] = (top + np.log(l)).reshape(-1)
    return y, lse, a, sabs
