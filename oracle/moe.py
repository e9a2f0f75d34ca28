"""Reference of the mixture-of-experts operators in fp64 (numpy): expert
routing and its gradient, the row plan, combine and its gradient, the gated
unit and its gradient, and the 1x128 scales of real-valued tiles.

Definitions (include/dg_moe.h states the same for the library):
* score: softmax over the experts, or 1 / (1 + exp(-x));
* the choice goes by the logits without a bias and by score + bias with one;
  a group's score is the sum of its group_top best (score + bias); equal
  values go to the lowest index; -inf masks an expert;
* the plan keeps the order of t * topk + j inside each expert;
* tile scale amax / 448 (0 for an all-zero tile, otherwise at least 2^-126).

Pinned by tests/test_oracle_moe.py: gradients against differences, the choice
against a search over all subsets, the plan against its own inverse.
"""

import numpy as np

from . import e4m3

BLOCK = 128
TINY = 2.0 ** -126


def scores(x, score):
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))
        top = x.max(axis=1, keepdims=True)
        e = np.exp(x - np.where(np.isneginf(top), 0.0, top))
        total = e.sum(axis=1, keepdims=True)
        return e / np.where(total == 0, 1.0, total)


def _best(values, n):
    """Indices of the n largest values above -inf, largest first, lowest index first among equals."""
    order = sorted((i for i in range(len(values)) if values[i] > -np.inf), key=lambda i: (-values[i], i))
    return order[:n]


def route(x, topk, score="softmax", bias=None, groups=1, topk_groups=1, group_top=2, renormalize=True, scale=1.0):
    """(ids [T][topk], weights [T][topk]) of logits x [T][E]."""
    x = np.asarray(x, dtype=np.float64)
    s = scores(x, score)
    ids = np.full((x.shape[0], topk), -1, dtype=np.int64)
    weights = np.zeros((x.shape[0], topk))
    per = x.shape[1] // groups
    for t in range(x.shape[0]):
        biased = s[t] + (np.asarray(bias, dtype=np.float64) if bias is not None else 0.0)
        biased = np.where(x[t] > -np.inf, biased, -np.inf)
        key = np.where(x[t] > -np.inf, biased if bias is not None else x[t], -np.inf)
        if groups > 1:
            gs = np.full(groups, -np.inf)
            for g in range(groups):
                part = np.sort(biased[g * per:(g + 1) * per])[::-1][:group_top]
                part = part[part > -np.inf]
                if part.size:
                    gs[g] = part.sum()
            keep = _best(gs, topk_groups)
            allowed = np.isin(np.arange(x.shape[1]) // per, keep)
            key = np.where(allowed, key, -np.inf)
        chosen = _best(key, topk)
        ids[t, :len(chosen)] = chosen
        sel = s[t, chosen]
        if renormalize:
            sel = sel / sel.sum() if sel.sum() > 0 else sel * 0
        weights[t, :len(chosen)] = scale * sel
    return ids, weights


def settled(x, topk, score="softmax", bias=None, groups=1, topk_groups=1, group_top=2, gap=1e-5):
    """Tokens whose choice (and its order) stays when every score moves by up
    to `gap`: the values compared are further apart than that, or equal because
    their logits and biases are."""
    x = np.asarray(x, dtype=np.float64)
    s = scores(x, score)
    biased = np.where(x > -np.inf, s + (0.0 if bias is None else np.asarray(bias, dtype=np.float64)), -np.inf)

    def apart(v, n):
        v = np.sort(v[v > -np.inf])[::-1][:n]
        d = -np.diff(v)
        return bool(np.all((d == 0) | (d > 2 * gap)))

    fine = np.ones(len(x), dtype=bool)
    per = x.shape[1] // groups
    for t in range(len(x)):
        key = biased[t]
        if groups > 1:
            gs = np.full(groups, -np.inf)
            for g in range(groups):
                part = np.sort(key[g * per:(g + 1) * per])[::-1][:group_top]
                if part[0] > -np.inf:
                    gs[g] = part[part > -np.inf].sum()
            fine[t] &= apart(gs, groups)
            key = np.where(np.isin(np.arange(x.shape[1]) // per, _best(gs, topk_groups)), key, -np.inf)
        if bias is not None:
            fine[t] &= apart(key, topk + 1)
    return fine


def weights_of(x, ids, score, renormalize, scale):
    """Routing weights of given ids (the function whose gradient route_bwd is)."""
    s = scores(x, score)
    out = np.zeros(ids.shape)
    for t in range(len(x)):
        live = (ids[t] >= 0) & (ids[t] < s.shape[1])
        sel = s[t, ids[t][live]]
        total = sel.sum()
        out[t, live] = scale * (sel / total if renormalize and total > 0 else sel)
    return out


def route_bwd(x, ids, dw, score="softmax", renormalize=True, scale=1.0):
    s = scores(x, score)
    dx = np.zeros(s.shape)
    for t in range(len(s)):
        live = (ids[t] >= 0) & (ids[t] < s.shape[1])
        e, d = ids[t][live], scale * np.asarray(dw[t], dtype=np.float64)[live]
        sel = s[t, e]
        total = sel.sum()
        g = (d - (d * sel).sum() / total) / total if renormalize and total > 0 else d
        if score == "sigmoid":
            dx[t, e] = g * sel * (1.0 - sel)
        else:
            dx[t] = -s[t] * (g * sel).sum()
            dx[t, e] += sel * g
    return dx


def plan_contiguous(ids, first, groups, m_total):
    """(rows, src, m_indices, k_offsets)."""
    flat = ids.reshape(-1).astype(np.int64) - first
    rows = np.full(flat.size, -1, dtype=np.int32)
    src = np.full(m_total, -1, dtype=np.int32)
    m_indices = np.full(m_total, -1, dtype=np.int32)
    offsets, at = [], 0
    for g in range(groups):
        mine = np.flatnonzero((flat == g) & (ids.reshape(-1) >= 0))
        offsets.append(min(at, m_total))
        for n, i in enumerate(mine):
            if at + n < m_total:
                rows[i] = at + n
                src[at + n] = i
                m_indices[at + n] = g
        at += -(-len(mine) // BLOCK) * BLOCK
    offsets.append(min(at, m_total))
    return rows.reshape(ids.shape), src, m_indices, np.array(offsets, dtype=np.int32)


def plan_masked(ids, first, groups, m_max):
    """(rows, src, masked_m)."""
    flat = ids.reshape(-1).astype(np.int64) - first
    rows = np.full(flat.size, -1, dtype=np.int32)
    src = np.full(groups * m_max, -1, dtype=np.int32)
    count = np.zeros(groups, dtype=np.int32)
    for g in range(groups):
        mine = np.flatnonzero((flat == g) & (ids.reshape(-1) >= 0))[:m_max]
        rows[mine] = g * m_max + np.arange(len(mine))
        src[g * m_max:g * m_max + len(mine)] = mine
        count[g] = len(mine)
    return rows.reshape(ids.shape), src, count


def combine(d, rows, weights=None):
    """(y, sum of |terms|) in fp64; d [M][C]."""
    d = np.asarray(d, dtype=np.float64)
    w = np.ones(rows.shape) if weights is None else np.asarray(weights, dtype=np.float64)
    live = (rows >= 0) & (rows < len(d))
    w = np.where(live, w, 0.0)
    part = d[np.where(live, rows, 0)] if len(d) else np.zeros((*rows.shape, d.shape[1]))
    part = np.where(live[..., None], part, 0.0)
    return (w[..., None] * part).sum(1), (np.abs(w[..., None] * part)).sum(1)


def combine_bwd(dy, d, src, rows, weights):
    """(dd [M][C], dweights [T][k], sum of |terms| of dweights)."""
    dy, d = np.asarray(dy, dtype=np.float64), np.asarray(d, dtype=np.float64)
    topk = rows.shape[1]
    live = src >= 0
    from_ = np.where(live, src, 0)
    dd = np.zeros(d.shape) if not len(d) else np.where(live[:, None], dy[from_ // topk] * np.asarray(weights, dtype=np.float64).reshape(-1)[from_][:, None], 0.0)
    here = (rows >= 0) & (rows < len(d))
    at = d[np.where(here, rows, 0)] if len(d) else np.zeros((*rows.shape, dy.shape[1]))
    terms = np.where(here[..., None], at * dy[:, None, :], 0.0)
    return dd, terms.sum(2), np.abs(terms).sum(2)


def swiglu(h):
    h = np.asarray(h, dtype=np.float64)
    gate, up = np.split(h, 2, axis=-1)
    return gate * scores(gate.reshape(-1, gate.shape[-1]), "sigmoid").reshape(gate.shape) * up


def swiglu_bwd(h, da):
    """d(sum(da * swiglu(h))) / dh."""
    h, da = np.asarray(h, dtype=np.float64), np.asarray(da, dtype=np.float64)
    gate, up = np.split(h, 2, axis=-1)
    sig = scores(gate, "sigmoid")
    return np.concatenate([da * up * (sig + gate * sig * (1.0 - sig)), da * gate * sig], axis=-1)


def dequant_rows(q, sf):
    """Values of codes q [R][C] with scales sf [C/128][ld]."""
    v = e4m3.decode(q).astype(np.float64).reshape(q.shape[0], -1, BLOCK)
    return (v * np.asarray(sf, dtype=np.float64)[:, :q.shape[0]].T[:, :, None]).reshape(q.shape)


def row_scales(v):
    """[C/128][R] scales of real v [R][C]."""
    amax = np.abs(v).reshape(v.shape[0], -1, BLOCK).max(axis=2).T
    return np.where(amax > 0, np.maximum(amax / 448.0, TINY), 0.0)


def column_scales(v):
    """[R/128][C] scales of the 128-row tiles of every column."""
    amax = np.abs(v).reshape(-1, BLOCK, v.shape[1]).max(axis=1)
    return np.where(amax > 0, np.maximum(amax / 448.0, TINY), 0.0)


def half_step(t):
    """Half the distance between e4m3 numbers at t."""
    _, ex = np.frexp(np.abs(t))
    return np.ldexp(1.0, np.maximum(ex - 1, -6) - 3) / 2
