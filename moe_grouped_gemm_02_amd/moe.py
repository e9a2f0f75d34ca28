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

from . import _BF, _I, _L, _P, _S, _U8, _check, _contig, _expect, _lib, _row_major

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
    try:
        return _SCORES[score]
    except (KeyError, TypeError):
        raise ValueError(f"score must be one of {sorted(_SCORES)}, not {score!r}") from None


# Stream handle of a device's current stream: what torch.cuda.current_stream()
# wraps, without making the wrapper (1.5 us of a call that has 6 us in all); a
# torch without that private call has the public one.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw_stream is None:
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


def _stream(t):
    return _raw_stream(t.get_device())


# Sizes are 32-bit numbers in the library, and ctypes would drop the bits above.
_MOST = 2 ** 31 - 1


def _int(value, name):
    if value.__class__ is not int:
        value = int(value)
    if -_MOST <= value <= _MOST:
        return value
    raise ValueError(f"{name}={value} is 2^31 or more")


def _shape(t, name, want):
    if tuple(t.shape) != tuple(want):
        raise ValueError(f"{name} must have shape {tuple(want)}, has {tuple(t.shape)}")


# The checks ask a tensor for as little as they can, since each question costs a
# small call about 0.1 us: what is in order passes on one line, anything else
# goes through the questions one by one for its error.

def _dense(t, name, dtypes, want):
    """Address of a contiguous tensor of the given shape."""
    try:
        if t.is_cuda and t.dtype in dtypes and t.shape == want and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _expect(t, name, dtypes, len(want))
    _shape(t, name, want)
    _contig(t, name)
    return t.data_ptr()


def _dense_or_none(t, name, dtypes, want):
    return None if t is None else _dense(t, name, dtypes, want)


def _topk(t, name, tokens):
    """Address and slots of an index matrix [tokens][topk]."""
    try:
        topk = t.shape[1]
    except (AttributeError, IndexError):
        _expect(t, name, _I32, 2)
        raise
    if topk > _MOST:
        raise ValueError(f"{name} has 2^31 or more columns")
    return _dense(t, name, _I32, (tokens, topk)), topk


def _matrix(t, name, dtypes):
    """Address, rows, columns and row stride of a matrix with unit stride in its
    rows.  (The stride of a single row says nothing.)"""
    try:
        if t.is_cuda and t.dtype in dtypes:
            rows, cols = t.shape
            ld, unit = t.stride()
            if unit == 1 and 0 < rows <= _MOST and 0 < cols <= _MOST:
                return t.data_ptr(), rows, cols, ld if rows > 1 else (cols + 7) // 8 * 8
    except (AttributeError, ValueError):
        pass
    _expect(t, name, dtypes, 2)
    rows, cols = (_int(n, f"size of {name}") for n in t.shape)
    if rows <= 1 or cols == 0:
        if cols > 1 and rows:
            _row_major(t, name)
        return t.data_ptr(), rows, cols, (cols + 7) // 8 * 8
    _row_major(t, name)
    return t.data_ptr(), rows, cols, t.stride(0)


def _dense_groups(t, name, dtypes, want):
    """Address and row stride of matrices [G][rows][cols] one after another, with
    unit stride in their rows."""
    groups, rows, cols = want
    try:
        if t.is_cuda and t.dtype in dtypes and t.shape == want and rows > 1 and cols:
            step, ld, unit = t.stride()
            if unit == 1 and (groups == 1 or step == rows * ld):
                return t.data_ptr(), ld
    except AttributeError:
        pass
    _expect(t, name, dtypes, 3)
    _shape(t, name, want)
    if cols > 1 and t.numel():
        _row_major(t, name)
    ld = t.stride(1) if rows > 1 and t.numel() else (cols + 7) // 8 * 8
    if groups > 1 and t.numel() and t.stride(0) != rows * ld:
        raise ValueError(f"{name} must have its groups one after another")
    return t.data_ptr(), ld


def _scales(t, name, dtypes, lead, rows):
    """Address and ld of a contiguous scale matrix [*lead][ld] with ld >= rows."""
    try:
        if t.is_cuda and t.dtype in dtypes and t.is_contiguous():
            shape = t.shape
            ld = shape[-1]
            if ld >= rows and shape == (*lead, ld):
                return t.data_ptr(), ld
    except (AttributeError, IndexError):
        pass
    _expect(t, name, dtypes, len(lead) + 1)
    _shape(t, name, (*lead, t.shape[-1]))
    if t.shape[-1] < rows:
        raise ValueError(f"{name} has {t.shape[-1]} columns, needs {rows}")
    _contig(t, name)
    return t.data_ptr(), t.shape[-1]


def _workspace(t):
    """Address and bytes of a workspace."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
        _expect(t, "workspace", (getattr(t, "dtype", None),))
        _contig(t, "workspace")
    return t.data_ptr(), t.nbytes


# ---------------------------------------------------------------- routing --

def _route(fn, dtypes, logits, ids, weights, bias, score, expert_groups, topk_groups, group_top, renormalize, scale):
    logits_at, tokens, experts, ld = _matrix(logits, "logits", dtypes)
    ids_at, topk = _topk(ids, "ids", tokens)
    weights_at = _dense(weights, "weights", _F32, (tokens, topk))
    bias_at = _dense_or_none(bias, "bias", _F32, (experts,))
    _check(fn, _FUNCTIONS[fn](
        logits_at, bias_at, ids_at, weights_at, tokens, experts, topk, ld, _score(score),
        _int(expert_groups, "expert_groups"), _int(topk_groups, "topk_groups"), _int(group_top, "group_top"),
        bool(renormalize), scale, _stream(logits)))
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
    logits_at, tokens, experts, ld = _matrix(logits, "logits", dtypes)
    ids_at, topk = _topk(ids, "ids", tokens)
    dweights_at = _dense(dweights, "dweights", _F32, (tokens, topk))
    dlogits_at, rows_d, cols_d, ld_d = _matrix(dlogits, "dlogits", dtypes)
    if rows_d != tokens or cols_d != experts:
        _shape(dlogits, "dlogits", (tokens, experts))
    _check(fn, _FUNCTIONS[fn](
        logits_at, ids_at, dweights_at, dlogits_at, tokens, experts, topk, ld, ld_d, _score(score), bool(renormalize),
        scale, _stream(logits)))
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
    """Address and length of a contiguous vector of indices."""
    try:
        if t.is_cuda and t.dtype is torch.int32 and t.is_contiguous():
            n, = t.shape
            if n <= _MOST:
                return t.data_ptr(), n
    except (AttributeError, ValueError):
        pass
    _expect(t, name, _I32, 1)
    _contig(t, name)
    return t.data_ptr(), _int(t.shape[0], f"size of {name}")


def _entries(ids, rows):
    """Addresses and shape of the routed ids and their rows."""
    try:
        tokens, topk = ids.shape
    except (AttributeError, ValueError):
        _expect(ids, "ids", _I32, 2)
        raise
    if tokens > _MOST or topk > _MOST:
        raise ValueError(f"ids of shape {tuple(ids.shape)} has a size of 2^31 or more")
    shape = tokens, topk
    return _dense(ids, "ids", _I32, shape), _dense(rows, "rows", _I32, shape), tokens, topk


def dg_get_moe_plan_workspace_size(tokens, topk, num_groups):
    return int(_lib.dg_get_moe_plan_workspace_size(
        _int(tokens, "tokens"), _int(topk, "topk"), _int(num_groups, "num_groups")))


def dg_moe_plan_contiguous(ids, rows, src, m_indices, k_offsets, first_expert=0, workspace=None):
    """Row plan of the contiguous layout: ids [T][k] -> rows [T][k], and per
    layout row src (entry t * k + j or -1) and m_indices (group or -1), and
    k_offsets [G+1], all int32.  Group g is expert first_expert + g."""
    ids_at, rows_at, tokens, topk = _entries(ids, rows)
    src_at, m_total = _vector(src, "src")
    m_indices_at = _dense(m_indices, "m_indices", _I32, (m_total,))
    k_offsets_at, ends = _vector(k_offsets, "k_offsets")
    _check("dg_moe_plan_contiguous", _lib.dg_moe_plan_contiguous(
        ids_at, rows_at, src_at, m_indices_at, k_offsets_at, tokens, topk, _int(first_expert, "first_expert"), ends - 1,
        m_total, *_workspace(workspace), _stream(ids)))
    return rows, src, m_indices, k_offsets


def dg_moe_plan_masked(ids, rows, src, masked_m, first_expert=0, workspace=None):
    """Row plan of the masked layout: src holds G * M_max entries, masked_m [G]."""
    ids_at, rows_at, tokens, topk = _entries(ids, rows)
    masked_m_at, groups = _vector(masked_m, "masked_m")
    src_at, layout_rows = _vector(src, "src")
    if groups < 1 or layout_rows % groups:
        raise ValueError("src must hold the same number of rows for every group")
    _check("dg_moe_plan_masked", _lib.dg_moe_plan_masked(
        ids_at, rows_at, src_at, masked_m_at, tokens, topk, _int(first_expert, "first_expert"), groups,
        layout_rows // groups, *_workspace(workspace), _stream(ids)))
    return rows, src, masked_m


def _codes(q, sf, sf_dtypes):
    """Addresses, (groups, rows, cols) and ld of codes [(G)][rows][cols] and
    scales [(G)][cols/128][ld]."""
    try:
        fine = q.is_cuda and q.dtype in _U8 and q.is_contiguous()
    except AttributeError:
        fine = False
    if not fine:
        _expect(q, "q", _U8)
        _contig(q, "q")
    shape = q.shape
    if len(shape) == 2:
        groups, (rows, cols) = 1, shape
        sf_at, ld = _scales(sf, "sf", sf_dtypes, (cols // 128,), rows)
    elif len(shape) == 3:
        groups, rows, cols = shape
        sf_at, ld = _scales(sf, "sf", sf_dtypes, (groups, cols // 128), rows)
    else:
        raise ValueError("q must have 2 or 3 dimensions")
    if groups > _MOST or rows > _MOST or cols > _MOST:
        raise ValueError(f"q of shape {tuple(shape)} has a size of 2^31 or more")
    return q.data_ptr(), sf_at, groups, rows, cols, ld


def _dispatch(fn, sf_dtypes, x, src, q, sf, topk):
    x_at, tokens, x_cols, ld_x = _matrix(x, "x", _BF)
    q_at, sf_at, groups, rows, cols, ld_sf = _codes(q, sf, sf_dtypes)
    if x_cols != cols:
        raise ValueError("x and q must have the same number of columns")
    src_at = _dense(src, "src", _I32, (groups * rows,))
    _check(fn, _FUNCTIONS[fn](
        x_at, src_at, q_at, sf_at, tokens, _int(topk, "topk"), cols, rows, groups, ld_x, ld_sf, _stream(x)))
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
    if isinstance(d, torch.Tensor) and d.dim() == 3:
        _contig(d, "d")
        d = d.view(-1, d.shape[-1])
    d_at, total_rows, d_cols, ld_d = _matrix(d, "d", _BF)
    y_at, tokens, cols, ld_y = _matrix(y, "y", _BF)
    if d_cols != cols:
        raise ValueError("d and y must have the same number of columns")
    rows_at, topk = _topk(rows, "rows", tokens)
    weights_at = _dense_or_none(weights, "weights", _F32, (tokens, topk))
    _check("dg_moe_combine", _lib.dg_moe_combine(
        d_at, rows_at, weights_at, y_at, tokens, topk, cols, total_rows, ld_d, ld_y, _stream(y)))
    return y


def dg_get_moe_combine_bwd_workspace_size(m_total, cols):
    return int(_lib.dg_get_moe_combine_bwd_workspace_size(_int(m_total, "m_total"), _int(cols, "cols")))


def dg_moe_combine_bwd(dy, d, src, rows, weights, dq, dsf, dqt, dsft, dweights, workspace=None):
    """Gradient of dg_moe_combine over a contiguous layout: the expert rows'
    gradient as codes dq [M][C] / dsf [C/128][ld] and transposed dqt [C][M] /
    dsft [M/128][ld] (both None: left out), and dweights [T][k]."""
    dy_at, tokens, cols, ld_dy = _matrix(dy, "dy", _BF)
    d_at, m_total, d_cols, ld_d = _matrix(d, "d", _BF)
    if d_cols != cols:
        _shape(d, "d", (m_total, cols))
    src_at = _dense(src, "src", _I32, (m_total,))
    rows_at, topk = _topk(rows, "rows", tokens)
    entries = tokens, topk
    weights_at = _dense(weights, "weights", _F32, entries)
    dweights_at = _dense(dweights, "dweights", _F32, entries)
    dq_at = _dense(dq, "dq", _U8, (m_total, cols))
    dsf_at, ld_dsf = _scales(dsf, "dsf", _F32, (cols // 128,), m_total)
    dqt_at, dsft_at, ld_dsft = None, None, 0
    if dqt is not None or dsft is not None:
        dqt_at = _dense(dqt, "dqt", _U8, (cols, m_total))
        dsft_at, ld_dsft = _scales(dsft, "dsft", _F32, (m_total // 128,), cols)
    _check("dg_moe_combine_bwd", _lib.dg_moe_combine_bwd(
        dy_at, d_at, src_at, rows_at, weights_at, dq_at, dsf_at, dqt_at, dsft_at, dweights_at, tokens, topk, cols,
        m_total, ld_dy, ld_d, ld_dsf, ld_dsft, *_workspace(workspace), _stream(dy)))
    return dq, dsf, dqt, dsft, dweights


# ------------------------------------------------------------ checkpoints --

def _swiglu_args(h, q, sf, sf_dtypes, m_indices, masked_m):
    q_at, sf_at, groups, rows, inter, ld_sf = _codes(q, sf, sf_dtypes)
    if q.dim() == 2:
        h_at, h_rows, h_cols, ld_h = _matrix(h, "h", _BF)
        if h_rows != rows or h_cols != 2 * inter:
            _shape(h, "h", (rows, 2 * inter))
    else:
        h_at, ld_h = _dense_groups(h, "h", _BF, (groups, rows, 2 * inter))
    m_indices_at = _dense_or_none(m_indices, "m_indices", _I32, (rows,))
    masked_m_at = _dense_or_none(masked_m, "masked_m", _I32, (groups,))
    return h_at, m_indices_at, masked_m_at, q_at, sf_at, groups, rows, inter, ld_h, ld_sf


def dg_swiglu_quant(h, q, sf, m_indices=None, masked_m=None, hq=None, hsf=None):
    """Codes q, sf of silu(gate) * up for h = [gate | up] bf16, [M][2I] or
    [G][M_max][2I]; with hq and hsf also the codes of h, its 8-bit checkpoint.
    Rows with m_indices < 0 (contiguous) or past masked_m[g] (masked) are not
    written."""
    h_at, m_indices_at, masked_m_at, q_at, sf_at, groups, rows, inter, ld_h, ld_sf = _swiglu_args(
        h, q, sf, _F32, m_indices, masked_m)
    hq_at, hsf_at, ld_hsf = None, None, 0
    if hq is not None or hsf is not None:
        hq_at = _dense(hq, "hq", _U8, h.shape)
        hsf_at, ld_hsf = _scales(hsf, "hsf", _F32, (*q.shape[:-2], 2 * inter // 128), rows)
    _check("dg_swiglu_quant", _lib.dg_swiglu_quant(
        h_at, m_indices_at, masked_m_at, q_at, sf_at, hq_at, hsf_at, rows, inter, groups, ld_h, ld_sf, ld_hsf,
        _stream(h)))
    return q, sf


def dg_swiglu_quant_ue8m0(h, q, sf, m_indices=None, masked_m=None):
    """dg_swiglu_quant with exponent-byte scales, without a checkpoint."""
    h_at, m_indices_at, masked_m_at, q_at, sf_at, groups, rows, inter, ld_h, ld_sf = _swiglu_args(
        h, q, sf, _E8, m_indices, masked_m)
    _check("dg_swiglu_quant_ue8m0", _lib.dg_swiglu_quant_ue8m0(
        h_at, m_indices_at, masked_m_at, q_at, sf_at, rows, inter, groups, ld_h, ld_sf, _stream(h)))
    return q, sf


def dg_swiglu_bwd(hq, hsf, dact, m_indices, dq, dsf, dqt, dsft, aqt=None, asft=None):
    """Backward of the gated unit from its checkpoint hq [M][2I], hsf and the
    gradient dact [M][I] bf16 of its output: codes of dh by rows (dq, dsf) and
    transposed (dqt [2I][M], dsft [M/128][ld]), and with aqt and asft the
    transposed codes [I][M] of the unit's output."""
    dact_at, m_total, inter, ld_dact = _matrix(dact, "dact", _BF)
    both = 2 * inter
    hq_at = _dense(hq, "hq", _U8, (m_total, both))
    dq_at = _dense(dq, "dq", _U8, (m_total, both))
    dqt_at = _dense(dqt, "dqt", _U8, (both, m_total))
    m_indices_at = _dense_or_none(m_indices, "m_indices", _I32, (m_total,))
    hsf_at, ld_hsf = _scales(hsf, "hsf", _F32, (both // 128,), m_total)
    dsf_at, ld_dsf = _scales(dsf, "dsf", _F32, (both // 128,), m_total)
    dsft_at, ld_dsft = _scales(dsft, "dsft", _F32, (m_total // 128,), both)
    aqt_at, asft_at, ld_asft = None, None, 0
    if aqt is not None or asft is not None:
        aqt_at = _dense(aqt, "aqt", _U8, (inter, m_total))
        asft_at, ld_asft = _scales(asft, "asft", _F32, (m_total // 128,), inter)
    _check("dg_swiglu_bwd", _lib.dg_swiglu_bwd(
        hq_at, hsf_at, dact_at, m_indices_at, dq_at, dsf_at, dqt_at, dsft_at, aqt_at, asft_at, m_total, inter, ld_hsf,
        ld_dact, ld_dsf, ld_dsft, ld_asft, _stream(dact)))
    return dq, dsf, dqt, dsft, aqt, asft


def dg_requant_t(q, sf, m_indices, qt, sft):
    """Row-wise codes q [M][C], sf [C/128][ld] -> transposed codes qt [C][M] with
    one scale per column and 128 rows, sft [M/128][ld] (an operand of
    dg_k_grouped_nt); zeros at rows with m_indices < 0 (None: all in use)."""
    q_at, rows, cols, ld = _matrix(q, "q", _U8)
    if ld != cols and q.numel():
        _contig(q, "q")
    qt_at = _dense(qt, "qt", _U8, (cols, rows))
    m_indices_at = _dense_or_none(m_indices, "m_indices", _I32, (rows,))
    sf_at, ld_sf = _scales(sf, "sf", _F32, (cols // 128,), rows)
    sft_at, ld_sft = _scales(sft, "sft", _F32, (rows // 128,), cols)
    _check("dg_requant_t", _lib.dg_requant_t(
        q_at, sf_at, m_indices_at, qt_at, sft_at, rows, cols, ld_sf, ld_sft, _stream(q)))
    return qt, sft


__all__ = list(EXPORTED)
