"""Reference of the transformer block's operators in fp64 (numpy): norms fused
with gate and residual and their gradient, the router's balance loss and its
gradient, and a product's epilogue and its gradient.

Definitions (include/dg_block.h states the same for the library):
* u = y or norm(y) post_weight; r = res_scale h + gate u; x = norm(r) weight +
  bias, with norm(v) = v / sqrt(mean v^2 + eps), or the same of v - mean v;
* balance: f_e = experts c_e / (topk n), loss = coef mean_s sum_e f_e P_e, over
  the tokens in use of each sequence;
* epilogue: z = sum + bias, d = act(z) + residual.

Results of the norms come with the sum of the magnitudes of the terms that they
were formed from, the measure of what float32 can lose in them.

Pinned by tests/test_oracle_block.py: every gradient against central
differences of the function it belongs to.
"""

import math

import numpy as np

from .moe import scores

BLOCK = 128


def _f64(v):
    return None if v is None else np.asarray(v, dtype=np.float64)


def stats(v, kind, eps):
    """(mean or 0, 1 / sqrt(..)) of the rows of v."""
    mean = v.mean(1, keepdims=True) if kind == "layer" else np.zeros((len(v), 1))
    return mean, 1.0 / np.sqrt(((v - mean) ** 2).mean(1, keepdims=True) + eps)


def _norm(v, mag, kind, eps):
    mean, k = stats(v, kind, eps)
    n = (v - mean) * k
    lost = mag + np.abs(mean) + (mag.mean(1, keepdims=True) if kind == "layer" else 0.0)
    # what is lost in v, in its mean and, along n, in k
    return n, k * lost + np.abs(n) * (1.0 + (np.abs(n) * k * mag).mean(1, keepdims=True))


def block_norm(y, h=None, weight=None, bias=None, post=False, post_weight=None, gate=None, res_scale=1.0, kind="rms", eps=1e-6):
    """(r, x, magnitudes of r, of x)."""
    u = _f64(y)
    mag = np.abs(u)
    if post:
        u, mag = _norm(u, mag, kind, eps)
        if post_weight is not None:
            u, mag = u * _f64(post_weight), mag * np.abs(_f64(post_weight))
    if gate is not None:
        u, mag = u * _f64(gate), mag * np.abs(_f64(gate))
    r = u
    if h is not None:
        r = u + res_scale * _f64(h)
        mag = mag + np.abs(res_scale * _f64(h))
    x, xmag = _norm(r, mag, kind, eps)
    if weight is not None:
        x, xmag = x * _f64(weight), xmag * np.abs(_f64(weight))
    if bias is not None:
        x, xmag = x + _f64(bias), xmag + np.abs(_f64(bias))
    return r, x, mag, xmag


def _normed(v, kind, eps):
    """norm(v), its magnitude and 1 / sqrt(..).  A mean is formed from terms of |v| / n: it can be off by what
    float32 loses in their sum where v and the mean are next to 0 themselves (_norm counts that too)."""
    mean, k = stats(v, kind, eps)
    mag = np.abs(v) + np.abs(mean) + (np.abs(v).mean(1, keepdims=True) if kind == "layer" else 0.0)
    return (v - mean) * k, mag * k, k


def _norm_back(g, gmag, v, kind, eps):
    """Gradient of norm(v) from g, its magnitude, norm(v) and its magnitude."""
    n, nmag, k = _normed(v, kind, eps)
    d = g - n * (g * n).mean(1, keepdims=True)
    mag = gmag + nmag * (gmag * nmag).mean(1, keepdims=True)
    if kind == "layer":
        d, mag = d - g.mean(1, keepdims=True), mag + gmag.mean(1, keepdims=True)
    return k * d, k * mag, n, nmag


def block_norm_bwd(dx=None, dr=None, r=None, y=None, weight=None, post=False, post_weight=None, gate=None, res_scale=1.0,
                   kind="rms", eps=1e-6):
    """{name: (value, magnitude)} of dy, dh, dweight, dbias, dpost_weight, dgate
    (those that the arguments define)."""
    out = {}
    t = np.zeros_like(_f64(dr if dx is None else dx))
    tmag = np.zeros_like(t)
    if dx is not None:
        dx = _f64(dx)
        g = dx if weight is None else dx * _f64(weight)
        t, tmag, n, nmag = _norm_back(g, np.abs(g), _f64(r), kind, eps)
        out["dweight"] = (dx * n).sum(0), (np.abs(dx) * nmag).sum(0)
        out["dbias"] = dx.sum(0), np.abs(dx).sum(0)
    if dr is not None:
        t, tmag = t + _f64(dr), tmag + np.abs(_f64(dr))
    out["dh"] = res_scale * t, abs(res_scale) * tmag
    pw = 1.0 if post_weight is None else _f64(post_weight)
    if y is not None:
        y = _f64(y)
        u, umag = y, np.abs(y)
        if post:
            n, nmag, _ = _normed(y, kind, eps)
            u, umag = n * pw, nmag * np.abs(pw)
        if gate is not None:
            axis = 0 if np.ndim(gate) == 1 else 1
            keep = {} if axis == 0 else {"keepdims": True}
            out["dgate"] = (t * u).sum(axis, **keep), (tmag * umag).sum(axis, **keep)
    e, emag = (t, tmag) if gate is None else (t * _f64(gate), tmag * np.abs(_f64(gate)))
    if post:
        n, nmag, _ = _normed(y, kind, eps)
        out["dpost_weight"] = (e * n).sum(0), (emag * nmag).sum(0)
        e, emag, _, _ = _norm_back(e * pw, emag * np.abs(pw), y, kind, eps)
    out["dy"] = e, emag
    return out


def shares(x, score):
    """Shares of the experts of each token; zeros where all are masked."""
    x = _f64(x)
    if score == "softmax":
        return scores(x, "softmax")
    # s / sum s relative to the largest score, so that none leaves the range
    top = x.max(1, keepdims=True)
    log_s = -np.logaddexp(0.0, -x)
    log_top = np.where(np.isneginf(top), 0.0, -np.logaddexp(0.0, -top))
    s = np.where(np.isneginf(x), 0.0, np.exp(log_s - log_top))
    total = s.sum(1, keepdims=True)
    return s / np.where(total == 0, 1.0, total)


def _sequences(x, offsets):
    return [(0, len(x))] if offsets is None else list(zip(offsets[:-1], offsets[1:]))


def balance(x, ids, offsets=None, score="softmax", coef=1.0):
    """(counts [S][E], used [S], loss)."""
    x, ids = _f64(x), np.asarray(ids)
    p, experts, seqs = shares(x, score), x.shape[1], _sequences(x, offsets)
    counts, used, loss = np.zeros((len(seqs), experts), dtype=np.int64), np.zeros(len(seqs), dtype=np.int64), 0.0
    for s, (a, b) in enumerate(seqs):
        live = ~np.isneginf(x[a:b]).all(1)
        chosen = ids[a:b][live].reshape(-1)
        chosen = chosen[(chosen >= 0) & (chosen < experts)]
        counts[s] = np.bincount(chosen, minlength=experts)
        used[s] = live.sum()
        if used[s]:
            f = experts * counts[s] / (ids.shape[1] * used[s])
            loss += (f * p[a:b].sum(0)).sum() / used[s]
    return counts, used, coef * loss / len(seqs)


def balance_bwd(x, counts, used, topk, offsets=None, score="softmax", coef=1.0, dloss=1.0):
    """(dlogits, which tokens are in a sequence, magnitudes)."""
    x = _f64(x)
    p, experts, seqs = shares(x, score), x.shape[1], _sequences(x, offsets)
    dx, mag, inside = np.zeros(x.shape), np.zeros(x.shape), np.zeros(len(x), dtype=bool)
    for s, (a, b) in enumerate(seqs):
        inside[a:b] = True
        if not used[s]:
            continue
        f = experts * counts[s] / (topk * used[s])
        m = p[a:b] @ f
        scale = dloss * coef / (len(seqs) * used[s])
        slope = scores(-x[a:b], "sigmoid") if score == "sigmoid" else 1.0
        dx[a:b] = scale * p[a:b] * slope * (f - m[:, None])
        mag[a:b] = abs(scale) * p[a:b] * slope * (f + m[:, None])
    return dx, inside, mag


def act(z, name):
    z = _f64(z)
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "silu":
        return z * scores(z, "sigmoid")
    if name == "gelu_tanh":
        return z * scores(math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3), "sigmoid")
    return z


def act_slope(z, name):
    z = _f64(z)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        s = scores(z, "sigmoid")
        return s + z * s * scores(-z, "sigmoid")
    if name == "gelu_tanh":
        c = math.sqrt(8.0 / math.pi)
        t = c * (z + 0.044715 * z ** 3)
        s = scores(t, "sigmoid")
        return s + z * s * scores(-t, "sigmoid") * c * (1.0 + 3 * 0.044715 * z ** 2)
    return np.ones_like(z)
