"""Plain 64-bit implementations of the layer's steps between the products, for the tests: head norm with
rotation, expert routing, the combining of the experts' rows, log probabilities."""
import math
from fractions import Fraction

import numpy as np

# 2 pi to 60 digits: angles of far positions are reduced in whole fractions
TWO_PI = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)


def turns(position, freq):
    """cos and sin of position * freq, the angle reduced exactly."""
    x = Fraction(float(freq)) * int(position)
    x -= TWO_PI * math.floor(x / TWO_PI)
    return math.cos(float(x)), math.sin(float(x))


def norm_rope(x, weight, eps, positions, freqs, axis_of, rot, interleaved):
    """x [n, heads, dim] float64, positions [axes, n]; eps None: no norm.  Returns (values, the size of each
    value's pair, which its error scales with)."""
    x = np.asarray(x, np.float64)
    z = x
    if eps is not None:
        with np.errstate(invalid="ignore", divide="ignore"):
            z = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
            z = z * (1.0 if weight is None else np.asarray(weight, np.float64))
    out, size = z.copy(), np.abs(z)
    half = rot // 2
    a = 2 * np.arange(half) if interleaved else np.arange(half)
    b = a + 1 if interleaved else a + half
    for t in range(x.shape[0]):
        cs = np.array([turns(positions[axis_of[i]][t], freqs[i]) for i in range(half)])
        p, q = z[t][:, a], z[t][:, b]
        out[t][:, a], out[t][:, b] = p * cs[:, 0] - q * cs[:, 1], p * cs[:, 1] + q * cs[:, 0]
        size[t][:, a] = size[t][:, b] = np.abs(p) + np.abs(q)
    return out, size


def route(logits, k, scoring, bias, n_groups, top_groups, renormalize, scale):
    """logits [n, E] float64 -> (topk, weights, the largest distance of a chosen logit from the best)."""
    n, E = logits.shape
    topk, weights = np.full((n, k), -1, np.int32), np.zeros((n, k))
    for t in range(n):
        x = logits[t]
        ok = np.isfinite(x)
        if not ok.any():
            continue
        score = np.zeros(E)
        with np.errstate(over="ignore"):
            if scoring == "softmax":
                score[ok] = np.exp(x[ok] - x[ok].max())
                score /= score.sum()
            else:
                score[ok] = 1 / (1 + np.exp(-x[ok]))
        value = np.where(ok, score, -np.inf)
        if bias is not None:
            value = np.where(ok & ~np.isnan(bias), score + bias, -np.inf)
        elif n_groups == top_groups:
            value = np.where(ok, x, -np.inf)
        if top_groups < n_groups:
            g = value.reshape(n_groups, -1)
            two = []
            for row in g:
                best = sorted((v for v in row if v > -np.inf), reverse=True)[:2]
                two.append(sum(best) if best else -np.inf)
            stay = sorted(range(n_groups), key=lambda i: (-two[i], i))[:top_groups]
            g = np.where(np.isin(np.arange(n_groups), stay)[:, None], g, -np.inf)
            value = g.reshape(-1)
        ids = [i for i in sorted(range(E), key=lambda i: (-value[i], i))[:k] if value[i] > -np.inf]
        topk[t, :len(ids)] = ids
        if renormalize and ids:
            # over the sum, in a form that no score is too small for
            log = x[ids] if scoring == "softmax" else np.minimum(x[ids], 0) - np.log1p(np.exp(-np.abs(x[ids])))
            w = np.exp(log - log.max())
            weights[t, :len(ids)] = w / w.sum() * scale
        else:
            weights[t, :len(ids)] = score[ids] * scale
    return topk, weights


def combine(y, topk, weights, offsets, slot_of, residual, shared, gate, H):
    """(out, sum of the terms' sizes), through the lists position by position."""
    n, k = topk.shape
    out = np.zeros((n, H)) if residual is None else np.array(residual, np.float64)
    size = np.abs(out)
    if shared is not None:
        s = np.asarray(shared, np.float64)
        if gate is not None:
            s = s / (1 + np.exp(-np.asarray(gate, np.float64)))[:, None]
        out, size = out + s, size + np.abs(s)
    for p in range(int(offsets[-1])):
        t, j = divmod(int(slot_of[p]), k)
        term = float(weights[t, j]) * np.asarray(y[p], np.float64)
        out[t] += term
        size[t] += np.abs(term)
    return out, size


def logprobs(logits, tokens, top, scale):
    """A dict as token_logprobs gives it, of logits [n, V] float64."""
    n, V = logits.shape
    got = dict(lse=np.zeros(n), entropy=np.zeros(n), logprobs=np.full(tokens.shape, np.nan),
               top_ids=np.full((n, top), -1, np.int32), top_logprobs=np.full((n, top), -np.inf))
    for r in range(n):
        x = logits[r] * scale
        if np.isnan(x).any() or (x == np.inf).any():
            got["lse"][r] = got["entropy"][r] = np.nan
            got["top_logprobs"][r] = np.nan
            continue
        m = x.max()
        if m == -np.inf:
            got["lse"][r] = -np.inf
            got["logprobs"][r] = np.where((tokens[r] >= 0) & (tokens[r] < V), -np.inf, np.nan)
            continue
        at = int(x.argmax())
        d = x - m
        others = np.delete(d, at)
        others = others[others > -np.inf]
        e = np.exp(others)
        drop = np.log1p(e.sum())
        got["lse"][r] = m + drop
        got["entropy"][r] = drop - (e * np.maximum(others, -1e5)).sum() / (1 + e.sum())
        ok = (tokens[r] >= 0) & (tokens[r] < V)
        got["logprobs"][r][ok] = d[tokens[r][ok]] - drop
        ids = np.argsort(-logits[r], kind="stable")[:top]
        ids = ids[logits[r][ids] > -np.inf]
        got["top_ids"][r, :len(ids)] = ids
        got["top_logprobs"][r, :len(ids)] = d[ids] - drop
    return got
