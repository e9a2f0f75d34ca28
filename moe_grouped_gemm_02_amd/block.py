"""Binding of the operators of a transformer block of libdg (include/dg_block.h):
norms fused with gate and residual scale, the router's balance loss, and the
dense GEMM with an epilogue and its gradient.

Argument marshalling only, as for the GEMMs: every function checks devices,
dtypes, shapes and strides and calls the C entry point of the same name on the
current HIP stream.  Outputs are given by the caller and returned.  All names
are also available from the package itself.

Tensor conventions are those of the mixture-of-experts operators: codes may be
torch.uint8 or torch.float8_e4m3fn, UE8M0 scales torch.uint8 or
torch.float8_e8m0fnu.  All tensors of a call are on the current device.
"""

import ctypes

import torch

from . import _BF, _I, _L, _P, _S, _U8, _check, _expect, _lib, _sfb_shape
from .moe import (_E8, _F32, _I32, _dense, _dense_or_none, _int, _matrix, _raw_stream, _scales, _score, _shape, _topk,
                  _workspace)

_F = ctypes.c_float

_SIGNATURES = {
    "dg_block_norm": (_I, [_P] * 10 + [_I, _I] + [_L] * 5 + [_I, _I, _I, _F, _F, _P]),
    "dg_block_norm_ue8m0": (_I, [_P] * 10 + [_I, _I] + [_L] * 5 + [_I, _I, _I, _F, _F, _P]),
    "dg_block_norm_bwd": (_I, [_P] * 13 + [_I, _I] + [_L] * 6 + [_I, _I, _I, _F, _F, _P, _S, _P]),
    "dg_get_block_norm_bwd_workspace_size": (_S, [_I, _I]),
    "dg_moe_balance": (_I, [_P] * 6 + [_I, _I, _I, _I, _L, _I, _F, _P, _S, _P]),
    "dg_moe_balance_bf16": (_I, [_P] * 6 + [_I, _I, _I, _I, _L, _I, _F, _P, _S, _P]),
    "dg_get_moe_balance_workspace_size": (_S, [_I, _I, _I]),
    "dg_moe_balance_bwd": (_I, [_P] * 7 + [_I, _I, _I, _I, _L, _L, _L, _I, _F, _P]),
    "dg_moe_balance_bwd_bf16": (_I, [_P] * 7 + [_I, _I, _I, _I, _L, _L, _L, _I, _F, _P]),
    "dg_fp8_gemm_nt_epilogue": (_I, [_P] * 10 + [_I, _I, _I] + [_L] * 7 + [_I, _P, _S, _P]),
    "dg_fp8_gemm_nt_ue8m0_epilogue": (_I, [_P] * 10 + [_I, _I, _I] + [_L] * 7 + [_I, _P, _S, _P]),
    "dg_epilogue_bwd": (_I, [_P] * 7 + [_I, _I] + [_L] * 4 + [_I, _P, _S, _P]),
    "dg_get_epilogue_bwd_workspace_size": (_S, [_I, _I]),
}
_FUNCTIONS = {}
for _name, (_res, _args) in _SIGNATURES.items():
    _fn = _FUNCTIONS[_name] = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_SIGNATURES)

_KINDS = {"rms": 0, "layer": 1}
_ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu_tanh": 3}


def _choice(table, value, name):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{name} must be one of {sorted(table)}, not {value!r}") from None


# The current device's index: torch.cuda.current_device() without its check that
# CUDA has been initialised, which the tensors answer.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_several = None  # whether there is more than one device, once a call has asked


def _stream(lead, *others):
    """Handle of the current stream of the device that the tensors are on, which must be
    the current one.  The launch goes to the current device, whatever device the default
    stream's handle (0) was taken from, and a kernel may fault on another device's
    addresses.  (Where a process sees one device there is nothing to ask: 0.1 us a
    tensor of a call that has 8 us in all.)"""
    global _several
    index = lead.get_device()
    if _several is None:
        _several = torch.cuda.device_count() > 1
    if _several:
        if index != _current_device():
            raise ValueError(f"the tensors are on cuda:{index}, the current device is cuda:{_current_device()}")
        for t in others:
            if t is not None and t.get_device() != index:
                raise ValueError(f"a tensor on {t.device} beside those on cuda:{index}")
    return _raw_stream(index)


def _rows(t, name, rows, cols):
    """Address and row stride of a bf16 matrix of the given shape, or of none."""
    if t is None:
        return None, 0
    at, r, c, ld = _matrix(t, name, _BF)
    if r != rows or c != cols:
        _shape(t, name, (rows, cols))
    return at, ld


# ------------------------------------------------------------------ norms --

def _gate(gate, name, rows, cols):
    """Address and kind of a gate [cols] or [rows, 1]."""
    if gate is None:
        return None, 0
    if isinstance(gate, torch.Tensor) and gate.dim() == 1:
        return _dense(gate, name, _F32, (cols,)), 1
    return _dense(gate, name, _F32, (rows, 1)), 2


def _block_norm(fn, sf_dtypes, y, h, r, x, q, sf, weight, bias, post, post_weight, gate, res_scale, kind, eps):
    y_at, tokens, cols, ld_y = _matrix(y, "y", _BF)
    h_at, ld_h = _rows(h, "h", tokens, cols)
    r_at, ld_r = _rows(r, "r", tokens, cols)
    x_at, ld_x = _rows(x, "x", tokens, cols)
    q_at, sf_at, ld_sf = None, None, 0
    if q is not None or sf is not None:
        q_at = _dense(q, "q", _U8, (tokens, cols))
        sf_at, ld_sf = _scales(sf, "sf", sf_dtypes, (cols // 128,), tokens)
    shape = (cols,)
    gate_at, gate_kind = _gate(gate, "gate", tokens, cols)
    _check(fn, _FUNCTIONS[fn](
        y_at, h_at, gate_at, _dense_or_none(post_weight, "post_weight", _F32, shape),
        _dense_or_none(weight, "weight", _F32, shape), _dense_or_none(bias, "bias", _F32, shape), r_at, x_at, q_at, sf_at,
        tokens, cols, ld_y, ld_h, ld_r, ld_x, ld_sf, _choice(_KINDS, kind, "kind"), bool(post), gate_kind, res_scale, eps,
        _stream(y, h, r, x, q, sf, weight, bias, post_weight, gate)))
    return r, x, q, sf


def dg_block_norm(y, h=None, r=None, x=None, q=None, sf=None, weight=None, bias=None, post=False, post_weight=None,
                  gate=None, res_scale=1.0, kind="rms", eps=1e-6):
    """The junction of two blocks: u = y [T][C] bf16, or its norm times
    post_weight with post; r = res_scale * h + gate * u; x = norm(r) * weight +
    bias.  gate is [C] or [T, 1] fp32, the parameters [C] fp32.  Fills those of
    r [T][C], x [T][C] (bf16) and q [T][C], sf [C/128][ld] (codes of x) that are
    given; r may be h itself.  kind: "rms" or "layer"."""
    return _block_norm("dg_block_norm", _F32, y, h, r, x, q, sf, weight, bias, post, post_weight, gate, res_scale, kind, eps)


def dg_block_norm_ue8m0(y, h=None, r=None, x=None, q=None, sf=None, weight=None, bias=None, post=False, post_weight=None,
                        gate=None, res_scale=1.0, kind="rms", eps=1e-6):
    """dg_block_norm with exponent-byte scales."""
    return _block_norm("dg_block_norm_ue8m0", _E8, y, h, r, x, q, sf, weight, bias, post, post_weight, gate, res_scale, kind,
                       eps)


def dg_get_block_norm_bwd_workspace_size(tokens, cols):
    return int(_lib.dg_get_block_norm_bwd_workspace_size(_int(tokens, "tokens"), _int(cols, "cols")))


def dg_block_norm_bwd(dy, dx=None, dr=None, r=None, y=None, dh=None, weight=None, dweight=None, dbias=None, post=False,
                      post_weight=None, dpost_weight=None, gate=None, dgate=None, res_scale=1.0, kind="rms", eps=1e-6,
                      workspace=None):
    """Gradient of dg_block_norm: fills dy [T][C] bf16 and those of dh [T][C]
    bf16, dweight, dbias, dpost_weight [C] fp32 and dgate (of the gate's shape)
    that are given, from the gradients dx of x and dr of r (either may be None),
    the forward pass' r (with dx) and y (with post or dgate).  workspace:
    dg_get_block_norm_bwd_workspace_size(T, C) bytes where a [C] result is wanted."""
    dy_at, tokens, cols, ld_dy = _matrix(dy, "dy", _BF)
    dx_at, ld_dx = _rows(dx, "dx", tokens, cols)
    dr_at, ld_dr = _rows(dr, "dr", tokens, cols)
    r_at, ld_r = _rows(r, "r", tokens, cols)
    y_at, ld_y = _rows(y, "y", tokens, cols)
    dh_at, ld_dh = _rows(dh, "dh", tokens, cols)
    shape = (cols,)
    gate_at, gate_kind = _gate(gate, "gate", tokens, cols)
    dgate_at = None
    if dgate is not None:
        if gate is None:
            raise ValueError("dgate without a gate")
        dgate_at = _dense(dgate, "dgate", _F32, gate.shape)
    _check("dg_block_norm_bwd", _lib.dg_block_norm_bwd(
        dx_at, dr_at, r_at, y_at, gate_at, _dense_or_none(post_weight, "post_weight", _F32, shape),
        _dense_or_none(weight, "weight", _F32, shape), dy_at, dh_at, _dense_or_none(dweight, "dweight", _F32, shape),
        _dense_or_none(dbias, "dbias", _F32, shape), _dense_or_none(dpost_weight, "dpost_weight", _F32, shape), dgate_at,
        tokens, cols, ld_dx, ld_dr, ld_r, ld_y, ld_dy, ld_dh, _choice(_KINDS, kind, "kind"), bool(post), gate_kind, res_scale,
        eps, *_workspace(workspace),
        _stream(dy, dx, dr, r, y, dh, weight, dweight, dbias, post_weight, dpost_weight, gate, dgate, workspace)))
    return dy, dh, dweight, dbias, dpost_weight, dgate


# ---------------------------------------------------------------- balance --

def _sequences(seq_offsets):
    """Address of the offsets and the number of sequences."""
    if seq_offsets is None:
        return None, 1
    _expect(seq_offsets, "seq_offsets", _I32, 1)
    ends = _int(seq_offsets.shape[0], "size of seq_offsets")
    return _dense(seq_offsets, "seq_offsets", _I32, (ends,)), ends - 1


def dg_get_moe_balance_workspace_size(tokens, experts, num_seqs=1):
    return int(_lib.dg_get_moe_balance_workspace_size(
        _int(tokens, "tokens"), _int(experts, "experts"), _int(num_seqs, "num_seqs")))


def _balance(fn, dtypes, logits, ids, counts, used, loss, seq_offsets, score, coef, workspace):
    logits_at, tokens, experts, ld = _matrix(logits, "logits", dtypes)
    ids_at, topk = _topk(ids, "ids", tokens)
    offsets_at, seqs = _sequences(seq_offsets)
    _check(fn, _FUNCTIONS[fn](
        logits_at, ids_at, offsets_at, _dense(counts, "counts", _I32, (seqs, experts)), _dense(used, "used", _I32, (seqs,)),
        _dense(loss, "loss", _F32, (1,)), tokens, experts, topk, seqs, ld, _score(score), coef, *_workspace(workspace),
        _stream(logits, ids, counts, used, loss, seq_offsets, workspace)))
    return counts, used, loss


def dg_moe_balance(logits, ids, counts, used, loss, seq_offsets=None, score="softmax", coef=1.0, workspace=None):
    """Per-expert counts [S][E] int32, tokens in use [S] int32 and the balance
    loss [1] fp32 of logits [T][E] fp32 and ids [T][k] int32 over the sequences
    that seq_offsets [S+1] int32 cuts the tokens into (None: one).  score:
    "softmax" or "sigmoid".  workspace: dg_get_moe_balance_workspace_size bytes."""
    return _balance("dg_moe_balance", _F32, logits, ids, counts, used, loss, seq_offsets, score, coef, workspace)


def dg_moe_balance_bf16(logits, ids, counts, used, loss, seq_offsets=None, score="softmax", coef=1.0, workspace=None):
    """dg_moe_balance of bf16 logits."""
    return _balance("dg_moe_balance_bf16", _BF, logits, ids, counts, used, loss, seq_offsets, score, coef, workspace)


def _balance_bwd(fn, dtypes, logits, counts, used, dlogits, topk, seq_offsets, dloss, add, score, coef):
    logits_at, tokens, experts, ld = _matrix(logits, "logits", dtypes)
    dlogits_at, rows_d, cols_d, ld_d = _matrix(dlogits, "dlogits", dtypes)
    if rows_d != tokens or cols_d != experts:
        _shape(dlogits, "dlogits", (tokens, experts))
    add_at, ld_add = None, 0
    if add is not None:
        add_at, rows_a, cols_a, ld_add = _matrix(add, "add", dtypes)
        if rows_a != tokens or cols_a != experts:
            _shape(add, "add", (tokens, experts))
    offsets_at, seqs = _sequences(seq_offsets)
    _check(fn, _FUNCTIONS[fn](
        logits_at, _dense(counts, "counts", _I32, (seqs, experts)), _dense(used, "used", _I32, (seqs,)), offsets_at,
        _dense_or_none(dloss, "dloss", _F32, (1,)), add_at, dlogits_at, tokens, experts, _int(topk, "topk"), seqs, ld, ld_add,
        ld_d, _score(score), coef, _stream(logits, counts, used, dlogits, seq_offsets, dloss, add)))
    return dlogits


def dg_moe_balance_bwd(logits, counts, used, dlogits, topk, seq_offsets=None, dloss=None, add=None, score="softmax",
                       coef=1.0):
    """Gradient of dg_moe_balance's loss times dloss [1] fp32 (None: 1), with the
    counts and used that it gave; fills dlogits [T][E] with it plus add [T][E]
    (None: nothing; dlogits itself: in place)."""
    return _balance_bwd("dg_moe_balance_bwd", _F32, logits, counts, used, dlogits, topk, seq_offsets, dloss, add, score, coef)


def dg_moe_balance_bwd_bf16(logits, counts, used, dlogits, topk, seq_offsets=None, dloss=None, add=None, score="softmax",
                            coef=1.0):
    """dg_moe_balance_bwd with bf16 logits, add and dlogits."""
    return _balance_bwd("dg_moe_balance_bwd_bf16", _BF, logits, counts, used, dlogits, topk, seq_offsets, dloss, add, score,
                        coef)


# --------------------------------------------------------------- epilogue --

def _leading(t, name, dtypes, lead, rows):
    """Address and row stride of scales [lead][ld], ld >= rows."""
    at, r, c, ld = _matrix(t, name, dtypes)
    if r != lead or c < rows:
        raise ValueError(f"{name} must have shape ({lead}, {rows} or more), has {tuple(t.shape)}")
    return at, ld if r > 1 else c


def _gemm_epilogue(fn, ue8m0, a, sfa, b, sfb, d, bias, act, residual, pre, dq, dsf, workspace):
    sf_dtypes = _E8 if ue8m0 else _F32
    a_at, m, k, lda = _matrix(a, "a", _U8)
    b_at, n, k_b, ldb = _matrix(b, "b", _U8)
    if k_b != k:
        raise ValueError("a and b must have the same number of columns")
    lda, ldb = lda if m > 1 else (k + 15) // 16 * 16, ldb if n > 1 else (k + 15) // 16 * 16
    d_at, d_rows, d_cols, ldd = _matrix(d, "d", _BF)
    if d_rows != m or d_cols != n:
        _shape(d, "d", (m, n))
    sfa_at, ld_sfa = _leading(sfa, "sfa", sf_dtypes, k // 128, m)
    sfb_at = _dense(sfb, "sfb", sf_dtypes, _sfb_shape(n, k, ue8m0))
    res_at, ld_res = _rows(residual, "residual", m, n)
    pre_at, ld_pre = _rows(pre, "pre", m, n)
    dq_at, dsf_at, ld_dsf = None, None, 0
    if dq is not None or dsf is not None:
        dq_at = _dense(dq, "dq", _U8, (m, n))
        dsf_at, ld_dsf = _scales(dsf, "dsf", sf_dtypes, (n // 128,), m)
    _check(fn, _FUNCTIONS[fn](
        a_at, sfa_at, b_at, sfb_at, _dense_or_none(bias, "bias", _F32, (n,)), res_at, d_at, pre_at, dq_at, dsf_at, m, n, k, lda,
        ldb, ldd, ld_sfa, ld_res, ld_pre, ld_dsf, _choice(_ACTS, act, "act"), *_workspace(workspace),
        _stream(d, a, sfa, b, sfb, bias, residual, pre, dq, dsf, workspace)))
    return d


def dg_fp8_gemm_nt_epilogue(a, sfa, b, sfb, d, bias=None, act="none", residual=None, pre=None, dq=None, dsf=None,
                            workspace=None):
    """dg_fp8_gemm_nt with an epilogue: z = a b^T + bias [N] fp32, d [M][N] bf16 =
    act(z) + residual [M][N] bf16.  act: "none", "relu", "silu" or "gelu_tanh".
    pre [M][N] bf16 keeps z for dg_epilogue_bwd; dq [M][N] and dsf [N/128][ld] take
    the codes of d.  The workspace is that of dg_fp8_gemm_nt."""
    return _gemm_epilogue("dg_fp8_gemm_nt_epilogue", False, a, sfa, b, sfb, d, bias, act, residual, pre, dq, dsf, workspace)


def dg_fp8_gemm_nt_ue8m0_epilogue(a, sfa, b, sfb, d, bias=None, act="none", residual=None, pre=None, dq=None, dsf=None,
                                  workspace=None):
    """dg_fp8_gemm_nt_epilogue with exponent-byte scales (dsf among them)."""
    return _gemm_epilogue("dg_fp8_gemm_nt_ue8m0_epilogue", True, a, sfa, b, sfb, d, bias, act, residual, pre, dq, dsf,
                          workspace)


def dg_get_epilogue_bwd_workspace_size(rows, cols):
    return int(_lib.dg_get_epilogue_bwd_workspace_size(_int(rows, "rows"), _int(cols, "cols")))


def dg_epilogue_bwd(dd, dq, dsf, pre=None, act="none", dqt=None, dsft=None, dbias=None, workspace=None):
    """Gradient dz = dd * act'(pre) of an epilogue's sum, from dd [M][N] and pre
    [M][N] bf16: codes by rows dq [M][N], dsf [N/128][ld], and those given of the
    transposed codes dqt [N][M up to a multiple of 128], dsft [.../128][ld] (operand
    of dg_k_grouped_nt) and dbias [N] fp32.  workspace:
    dg_get_epilogue_bwd_workspace_size(M, N) bytes with dbias."""
    dd_at, rows, cols, ld_dd = _matrix(dd, "dd", _BF)
    pre_at, ld_pre = _rows(pre, "pre", rows, cols)
    dq_at = _dense(dq, "dq", _U8, (rows, cols))
    dsf_at, ld_dsf = _scales(dsf, "dsf", _F32, (cols // 128,), rows)
    dqt_at, dsft_at, ld_dsft = None, None, 0
    if dqt is not None or dsft is not None:
        tiles = (rows + 127) // 128
        dqt_at = _dense(dqt, "dqt", _U8, (cols, tiles * 128))
        dsft_at, ld_dsft = _scales(dsft, "dsft", _F32, (tiles,), cols)
    _check("dg_epilogue_bwd", _lib.dg_epilogue_bwd(
        dd_at, pre_at, dq_at, dsf_at, dqt_at, dsft_at, _dense_or_none(dbias, "dbias", _F32, (cols,)), rows, cols, ld_dd, ld_pre,
        ld_dsf, ld_dsft, _choice(_ACTS, act, "act"), *_workspace(workspace),
        _stream(dd, dq, dsf, pre, dqt, dsft, dbias, workspace)))
    return dq, dsf, dqt, dsft, dbias


__all__ = list(EXPORTED)
