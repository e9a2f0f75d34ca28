"""Binding of the mixture-of-experts operators of libdg (include/dg_moe.h):
expert routing, the exchange between token rows and expert rows, and 8-bit
activation checkpoints of the experts' gated unit.

Argument marshalling only, as for the GEMMs: every function checks devices,
dtypes, shapes and strides and calls the C entry point of the same name on the
current HIP stream.  Outputs are given by the caller and returned.  All names
are also available from the package itself.

Tensor conventions beyond the package's: codes may be torch.uint8 or
torch.float8_e4m3fn, UE8M0 scales torch.uint8 or torch.float8_e8m0fnu.
"""

import ctypes

import torch

from . import _BF, _I, _L, _P, _S, _U8, _check, _contig, _expect, _lib, _ptr, _row_major, _ws

_F = ctypes.c_float

_SIGNATURES = {
    "dg_moe_route": (_I, [_P, _P, _P, _P, _I, _I, _I, _L, _I, _I, _I, _I, _I, _F, _P]),
    "dg_moe_route_bf16": (_I, [_P, _P, _P, _P, _I, _I, _I, _L, _I, _I, _I, _I, _I, _F, _P]),
    "dg_moe_route_bwd": (_I, [_P, _P, _P, _P, _I, _I, _I, _L, _L, _I, _I, _F, _P]),
    "dg_moe_route_bwd_bf16": (_I, [_P, _P, _P, _P, _I, _I, _I, _L, _L, _I, _I, _F, _P]),
    "dg_moe_plan_contiguous": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _S, _P]),
    "dg_moe_plan_masked": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _S, _P]),
    "dg_get_moe_plan_workspace_size": (_S, [_I, _I, _I]),
    "dg_moe_dispatch": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _L, _L, _P]),
    "dg_moe_dispatch_ue8m0": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _L, _L, _P]),
    "dg_moe_combine": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _L, _L, _P]),
    "dg_moe_combine_bwd": (_I, [_P] * 10 + [_I, _I, _I, _I, _L, _L, _L, _L, _P, _S, _P]),
    "dg_get_moe_combine_bwd_workspace_size": (_S, [_I, _I]),
    "dg_swiglu_quant": (_I, [_P] * 7 + [_I, _I, _I, _L, _L, _L, _P]),
    "dg_swiglu_quant_ue8m0": (_I, [_P] * 5 + [_I, _I, _I, _L, _L, _P]),
    "dg_swiglu_bwd": (_I, [_P] * 10 + [_I, _I, _L, _L, _L, _L, _L, _P]),
    "dg_requant_t": (_I, [_P] * 5 + [_I, _I, _L, _L, _P]),
}
_FUNCTIONS = {}
for _name, (_res, _args) in _SIGNATURES.items():
    _fn = _FUNCTIONS[_name] = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_SIGNATURES)

_F32 = (torch.float32,)
_I32 = (torch.int32,)
_E8 = (torch.uint8, torch.float8_e8m0fnu)
_SCORES = {"softmax": 0, "sigmoid": 1}


def _score(score):
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, not {score!r}")
    return _SCORES[score]


# Stream handle of a device's current stream: what torch.cuda.current_stream()
# wraps, without making the wrapper (1.5 us of a call that has 6 us in all).
_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream(t):
    return _raw_stream(t.get_device())


def _shape(t, name, want):
    if tuple(t.shape) != tuple(want):
        raise ValueError(f"{name} must have shape {tuple(want)}, has {tuple(t.shape)}")


def _dense(t, name, dtypes, want):
    """A contiguous tensor of the given shape."""
    if type(t) is torch.Tensor and t.is_cuda and t.dtype in dtypes and t.shape == want and t.is_contiguous():
        return
    _expect(t, name, dtypes, len(want))
    _shape(t, name, want)
    _contig(t, name)


def _topk(t, name, tokens):
    """Slots of an index matrix [tokens][topk]."""
    if type(t) is not torch.Tensor or t.dim() != 2:
        _expect(t, name, _I32, 2)
    topk = t.shape[1]
    _dense(t, name, _I32, (tokens, topk))
    return topk


def _rows_of(t, name, dtypes, ndim=2):
    """A matrix with unit stride in its rows; returns its row stride."""
    if type(t) is torch.Tensor and t.is_cuda and t.dtype in dtypes:
        stride = t.stride()
        if len(stride) == ndim and stride[-1] == 1 and t.numel():
            # (the stride of a single row says nothing)
            return stride[-2] if t.shape[-2] > 1 else (t.shape[-1] + 7) // 8 * 8
    _expect(t, name, dtypes, ndim)
    if t.shape[-2] <= 1 or t.numel() == 0:  # such strides say nothing
        if t.shape[-1] > 1 and t.numel():
            _row_major(t, name)
        return (t.shape[-1] + 7) // 8 * 8
    _row_major(t, name)
    return t.stride(-2)


def _scales(t, name, dtypes, lead, rows):
    """A contiguous scale matrix [*lead][ld] with ld >= rows; returns ld."""
    if type(t) is torch.Tensor and t.is_cuda and t.dtype in dtypes and t.is_contiguous():
        shape = t.shape
        if shape[:-1] == lead and shape[-1] >= rows:
            return shape[-1]
    _expect(t, name, dtypes, len(lead) + 1)
    _shape(t, name, (*lead, t.shape[-1]))
    if t.shape[-1] < rows:
        raise ValueError(f"{name} has {t.shape[-1]} columns, needs {rows}")
    _contig(t, name)
    return t.shape[-1]


def _call(name, *args):
    status = _FUNCTIONS[name](*args)
    if status != 0:
        _check(name, status)


# ---------------------------------------------------------------- routing --

def _route(fn, dtypes, logits, ids, weights, bias, score, expert_groups, topk_groups, group_top, renormalize, scale):
    ld = _rows_of(logits, "logits", dtypes)
    tokens, experts = logits.shape
    topk = _topk(ids, "ids", tokens)
    _dense(weights, "weights", _F32, (tokens, topk))
    if bias is not None:
        _dense(bias, "bias", _F32, (experts,))
    _call(fn, _ptr(logits), _ptr(bias), _ptr(ids), _ptr(weights), tokens, experts, topk, ld, _score(score),
          int(expert_groups), int(topk_groups), int(group_top), int(bool(renormalize)), float(scale), _stream(logits))
    return ids, weights


def dg_moe_route(logits, ids, weights, bias=None, score="softmax", expert_groups=1, topk_groups=1, group_top=2,
                 renormalize=True, scale=1.0):
    """Expert ids [T][k] int32 and weights [T][k] fp32 of logits [T][E] fp32.

    score: "softmax" or "sigmoid"; bias [E] fp32 takes part in the choice only;
    of expert_groups equal groups the topk_groups with the largest sums of
    their group_top (1 or 2) best scores stay; weights are the chosen scores,
    divided by their sum with renormalize, times scale.  Ties go to the lowest
    index; a logit of -inf masks its expert; slots without an expert get id -1
    and weight 0."""
    return _route("dg_moe_route", _F32, logits, ids, weights, bias, score, expert_groups, topk_groups, group_top,
                  renormalize, scale)


def dg_moe_route_bf16(logits, ids, weights, bias=None, score="softmax", expert_groups=1, topk_groups=1, group_top=2,
                      renormalize=True, scale=1.0):
    """dg_moe_route of bf16 logits."""
    return _route("dg_moe_route_bf16", _BF, logits, ids, weights, bias, score, expert_groups, topk_groups, group_top,
                  renormalize, scale)


def _route_bwd(fn, dtypes, logits, ids, dweights, dlogits, score, renormalize, scale):
    ld = _rows_of(logits, "logits", dtypes)
    tokens, experts = logits.shape
    topk = _topk(ids, "ids", tokens)
    _dense(dweights, "dweights", _F32, (tokens, topk))
    ld_d = _rows_of(dlogits, "dlogits", dtypes)
    _shape(dlogits, "dlogits", (tokens, experts))
    _call(fn, _ptr(logits), _ptr(ids), _ptr(dweights), _ptr(dlogits), tokens, experts, topk, ld, ld_d, _score(score),
          int(bool(renormalize)), float(scale), _stream(logits))
    return dlogits


def dg_moe_route_bwd(logits, ids, dweights, dlogits, score="softmax", renormalize=True, scale=1.0):
    """Gradient of the routing weights with respect to the logits, for the
    ids that dg_moe_route chose; fills dlogits [T][E]."""
    return _route_bwd("dg_moe_route_bwd", _F32, logits, ids, dweights, dlogits, score, renormalize, scale)


def dg_moe_route_bwd_bf16(logits, ids, dweights, dlogits, score="softmax", renormalize=True, scale=1.0):
    """dg_moe_route_bwd with bf16 logits and dlogits."""
    return _route_bwd("dg_moe_route_bwd_bf16", _BF, logits, ids, dweights, dlogits, score, renormalize, scale)


# --------------------------------------------------------------- exchange --

def _vector(t, name):
    """Length of a contiguous vector of indices."""
    if not (type(t) is torch.Tensor and t.is_cuda and t.dtype is torch.int32 and t.dim() == 1 and t.is_contiguous()):
        _expect(t, name, _I32, 1)
        _contig(t, name)
    return t.shape[0]


def _entries(ids, rows):
    if type(ids) is not torch.Tensor or ids.dim() != 2:
        _expect(ids, "ids", _I32, 2)
    shape = ids.shape
    _dense(ids, "ids", _I32, shape)
    _dense(rows, "rows", _I32, shape)
    return shape


def dg_get_moe_plan_workspace_size(tokens, topk, num_groups):
    return int(_lib.dg_get_moe_plan_workspace_size(int(tokens), int(topk), int(num_groups)))


def dg_moe_plan_contiguous(ids, rows, src, m_indices, k_offsets, first_expert=0, workspace=None):
    """Row plan of the contiguous layout: ids [T][k] -> rows [T][k], and per
    layout row src (entry t * k + j or -1) and m_indices (group or -1), and
    k_offsets [G+1], all int32.  Group g is expert first_expert + g."""
    tokens, topk = _entries(ids, rows)
    m_total = _vector(src, "src")
    _dense(m_indices, "m_indices", _I32, (m_total,))
    groups = _vector(k_offsets, "k_offsets") - 1
    _call("dg_moe_plan_contiguous", _ptr(ids), _ptr(rows), _ptr(src), _ptr(m_indices), _ptr(k_offsets), tokens, topk,
          int(first_expert), groups, m_total, _ptr(workspace), _ws(workspace), _stream(ids))
    return rows, src, m_indices, k_offsets


def dg_moe_plan_masked(ids, rows, src, masked_m, first_expert=0, workspace=None):
    """Row plan of the masked layout: src holds G * M_max entries, masked_m [G]."""
    tokens, topk = _entries(ids, rows)
    groups, layout_rows = _vector(masked_m, "masked_m"), _vector(src, "src")
    if groups < 1 or layout_rows % groups:
        raise ValueError("src must hold the same number of rows for every group")
    _call("dg_moe_plan_masked", _ptr(ids), _ptr(rows), _ptr(src), _ptr(masked_m), tokens, topk, int(first_expert),
          groups, layout_rows // groups, _ptr(workspace), _ws(workspace), _stream(ids))
    return rows, src, masked_m


def _codes(q, sf, sf_dtypes):
    """(groups, rows, cols, ld) of codes [(G)][rows][cols] and scales [(G)][cols/128][ld]."""
    if not (type(q) is torch.Tensor and q.is_cuda and q.dtype in _U8 and q.is_contiguous()):
        _expect(q, "q", _U8)
        _contig(q, "q")
    shape = q.shape
    if len(shape) == 2:
        rows, cols = shape
        return 1, rows, cols, _scales(sf, "sf", sf_dtypes, (cols // 128,), rows)
    if len(shape) == 3:
        groups, rows, cols = shape
        return groups, rows, cols, _scales(sf, "sf", sf_dtypes, (groups, cols // 128), rows)
    raise ValueError("q must have 2 or 3 dimensions")


def _dispatch(fn, sf_dtypes, x, src, q, sf, topk):
    ld_x = _rows_of(x, "x", _BF)
    groups, rows, cols, ld_sf = _codes(q, sf, sf_dtypes)
    if x.shape[1] != cols:
        raise ValueError("x and q must have the same number of columns")
    _dense(src, "src", _I32, (groups * rows,))
    _call(fn, _ptr(x), _ptr(src), _ptr(q), _ptr(sf), x.shape[0], int(topk), cols, rows, groups, ld_x, ld_sf, _stream(x))
    return q, sf


def dg_moe_dispatch(x, src, q, sf, topk):
    """Quantised expert rows: row r of q [M][C] (or [G][M_max][C]) and its scales
    sf [(G)][C/128][ld] become those of token src[r] // topk of x [T][C] bf16;
    rows with src -1 are not written."""
    return _dispatch("dg_moe_dispatch", _F32, x, src, q, sf, topk)


def dg_moe_dispatch_ue8m0(x, src, q, sf, topk):
    """dg_moe_dispatch with exponent-byte scales."""
    return _dispatch("dg_moe_dispatch_ue8m0", _E8, x, src, q, sf, topk)


def dg_moe_combine(d, rows, y, weights=None):
    """y[t] = sum_j weights[t][j] * d[rows[t][j]] (weights None: ones); d [M][C]
    or [G][M_max][C] bf16, y [T][C] bf16.  Rows outside d add nothing."""
    _expect(d, "d", _BF)
    if d.dim() == 3:
        _contig(d, "d")
        d = d.view(-1, d.shape[-1])
    ld_d, ld_y = _rows_of(d, "d", _BF), _rows_of(y, "y", _BF)
    tokens, cols = y.shape
    if d.shape[1] != cols:
        raise ValueError("d and y must have the same number of columns")
    topk = _topk(rows, "rows", tokens)
    if weights is not None:
        _dense(weights, "weights", _F32, (tokens, topk))
    _call("dg_moe_combine", _ptr(d), _ptr(rows), _ptr(weights), _ptr(y), tokens, topk, cols, d.shape[0], ld_d, ld_y,
          _stream(y))
    return y


def dg_get_moe_combine_bwd_workspace_size(m_total, cols):
    return int(_lib.dg_get_moe_combine_bwd_workspace_size(int(m_total), int(cols)))


def dg_moe_combine_bwd(dy, d, src, rows, weights, dq, dsf, dqt, dsft, dweights, workspace=None):
    """Gradient of dg_moe_combine over a contiguous layout: the expert rows'
    gradient as codes dq [M][C] / dsf [C/128][ld] and transposed dqt [C][M] /
    dsft [M/128][ld] (both None: left out), and dweights [T][k]."""
    ld_dy, ld_d = _rows_of(dy, "dy", _BF), _rows_of(d, "d", _BF)
    tokens, cols = dy.shape
    m_total = d.shape[0]
    _shape(d, "d", (m_total, cols))
    _dense(src, "src", _I32, (m_total,))
    topk = _topk(rows, "rows", tokens)
    _dense(weights, "weights", _F32, (tokens, topk))
    _dense(dweights, "dweights", _F32, (tokens, topk))
    _dense(dq, "dq", _U8, (m_total, cols))
    ld_dsf, ld_dsft = _scales(dsf, "dsf", _F32, (cols // 128,), m_total), 0
    if dqt is not None or dsft is not None:
        _dense(dqt, "dqt", _U8, (cols, m_total))
        ld_dsft = _scales(dsft, "dsft", _F32, (m_total // 128,), cols)
    _call("dg_moe_combine_bwd", _ptr(dy), _ptr(d), _ptr(src), _ptr(rows), _ptr(weights), _ptr(dq), _ptr(dsf), _ptr(dqt),
          _ptr(dsft), _ptr(dweights), tokens, topk, cols, m_total, ld_dy, ld_d, ld_dsf, ld_dsft, _ptr(workspace),
          _ws(workspace), _stream(dy))
    return dq, dsf, dqt, dsft, dweights


# ------------------------------------------------------------ checkpoints --

def _swiglu_args(h, q, sf, sf_dtypes, m_indices, masked_m):
    groups, rows, inter, ld_sf = _codes(q, sf, sf_dtypes)
    ld_h = _rows_of(h, "h", _BF, q.dim())
    if h.shape != ((rows, 2 * inter) if q.dim() == 2 else (groups, rows, 2 * inter)):
        _shape(h, "h", (*q.shape[:-1], 2 * inter))
    if groups > 1 and h.stride(0) != rows * ld_h:
        raise ValueError("h must have its groups one after another")
    if m_indices is not None:
        _dense(m_indices, "m_indices", _I32, (rows,))
    if masked_m is not None:
        _dense(masked_m, "masked_m", _I32, (groups,))
    return groups, rows, inter, ld_h, ld_sf


def dg_swiglu_quant(h, q, sf, m_indices=None, masked_m=None, hq=None, hsf=None):
    """Codes q, sf of silu(gate) * up for h = [gate | up] bf16, [M][2I] or
    [G][M_max][2I]; with hq and hsf also the codes of h, its 8-bit checkpoint.
    Rows with m_indices < 0 (contiguous) or past masked_m[g] (masked) are not
    written."""
    groups, rows, inter, ld_h, ld_sf = _swiglu_args(h, q, sf, _F32, m_indices, masked_m)
    ld_hsf = 0
    if hq is not None or hsf is not None:
        _dense(hq, "hq", _U8, h.shape)
        ld_hsf = _scales(hsf, "hsf", _F32, (*q.shape[:-2], 2 * inter // 128), rows)
    _call("dg_swiglu_quant", _ptr(h), _ptr(m_indices), _ptr(masked_m), _ptr(q), _ptr(sf), _ptr(hq), _ptr(hsf), rows, inter,
          groups, ld_h, ld_sf, ld_hsf, _stream(h))
    return q, sf


def dg_swiglu_quant_ue8m0(h, q, sf, m_indices=None, masked_m=None):
    """dg_swiglu_quant with exponent-byte scales, without a checkpoint."""
    groups, rows, inter, ld_h, ld_sf = _swiglu_args(h, q, sf, _E8, m_indices, masked_m)
    _call("dg_swiglu_quant_ue8m0", _ptr(h), _ptr(m_indices), _ptr(masked_m), _ptr(q), _ptr(sf), rows, inter, groups, ld_h,
          ld_sf, _stream(h))
    return q, sf


def dg_swiglu_bwd(hq, hsf, dact, m_indices, dq, dsf, dqt, dsft, aqt=None, asft=None):
    """Backward of the gated unit from its checkpoint hq [M][2I], hsf and the
    gradient dact [M][I] bf16 of its output: codes of dh by rows (dq, dsf) and
    transposed (dqt [2I][M], dsft [M/128][ld]), and with aqt and asft the
    transposed codes [I][M] of the unit's output."""
    ld_dact = _rows_of(dact, "dact", _BF)
    m_total, inter = dact.shape
    _dense(hq, "hq", _U8, (m_total, 2 * inter))
    _dense(dq, "dq", _U8, (m_total, 2 * inter))
    _dense(dqt, "dqt", _U8, (2 * inter, m_total))
    if m_indices is not None:
        _dense(m_indices, "m_indices", _I32, (m_total,))
    ld_hsf = _scales(hsf, "hsf", _F32, (2 * inter // 128,), m_total)
    ld_dsf = _scales(dsf, "dsf", _F32, (2 * inter // 128,), m_total)
    ld_dsft, ld_asft = _scales(dsft, "dsft", _F32, (m_total // 128,), 2 * inter), 0
    if aqt is not None or asft is not None:
        _dense(aqt, "aqt", _U8, (inter, m_total))
        ld_asft = _scales(asft, "asft", _F32, (m_total // 128,), inter)
    _call("dg_swiglu_bwd", _ptr(hq), _ptr(hsf), _ptr(dact), _ptr(m_indices), _ptr(dq), _ptr(dsf), _ptr(dqt), _ptr(dsft),
          _ptr(aqt), _ptr(asft), m_total, inter, ld_hsf, ld_dact, ld_dsf, ld_dsft, ld_asft, _stream(dact))
    return dq, dsf, dqt, dsft, aqt, asft


def dg_requant_t(q, sf, m_indices, qt, sft):
    """Row-wise codes q [M][C], sf [C/128][ld] -> transposed codes qt [C][M] with
    one scale per column and 128 rows, sft [M/128][ld] (an operand of
    dg_k_grouped_nt); zeros at rows with m_indices < 0 (None: all in use)."""
    _expect(q, "q", _U8, 2)
    rows, cols = q.shape
    _contig(q, "q")
    _dense(qt, "qt", _U8, (cols, rows))
    if m_indices is not None:
        _dense(m_indices, "m_indices", _I32, (rows,))
    ld_sf = _scales(sf, "sf", _F32, (cols // 128,), rows)
    ld_sft = _scales(sft, "sft", _F32, (rows // 128,), cols)
    _call("dg_requant_t", _ptr(q), _ptr(sf), _ptr(m_indices), _ptr(qt), _ptr(sft), rows, cols, ld_sf, ld_sft, _stream(q))
    return qt, sft


__all__ = list(EXPORTED)
