"""A mixture-of-experts layer on the library's operators: forward and backward
pass with FP8 grouped GEMMs, 8-bit activation checkpoints and no host
synchronisation.

Forward:  route -> plan -> dispatch (quantise) -> grouped GEMM (w1, which also
writes the 8-bit checkpoint of its output) -> gated unit (quantise) -> grouped
GEMM (w2) -> combine.
Backward: combine_bwd -> grouped GEMM (w2^T) -> swiglu_bwd from the checkpoint
-> grouped GEMM (w1^T) -> combine; the weight gradients are two K-grouped GEMMs
over transposed codes, the first layer's input coming from its own forward
operand; route_bwd for the logits.

    python examples/moe_layer.py [--tokens 4096 --hidden 7168 --inter 2048 --experts 16 --topk 8]

prints the error against float32 arithmetic on the same bf16 weights and the
time of a step.  The router's own product (tokens x experts) is the caller's.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_grouped_gemm_02_amd as dg  # noqa: E402

BLOCK = 128


def _codes(*shape):
    return torch.empty(shape, dtype=torch.uint8, device="cuda")


def _f32(*shape):
    return torch.empty(shape, dtype=torch.float32, device="cuda")


def _bf16(*shape):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda")


def _i32(*shape):
    return torch.empty(shape, dtype=torch.int32, device="cuda")


def _quantised_weight(w):
    """128x128 codes and scales of w [E][N][K] bf16."""
    e, n, k = w.shape
    q, sf = _codes(e, n, k), _f32(e, (n + BLOCK - 1) // BLOCK, k // BLOCK)
    dg.dg_quant_128x128(w.contiguous(), q, sf)
    return q, sf


class MoELayer:
    """Experts w1 [E][2 inter][hidden] (gate rows, then up rows) and
    w2 [E][hidden][inter] in bf16.  All buffers are made here, for `tokens`
    tokens and `capacity` expert rows (default: room for every choice).  With
    `balance` (the coefficient of the load-balance loss) the forward pass also
    gives `counts`, `used` and `loss`, and the logits' gradient holds the loss'."""

    def __init__(self, w1, w2, tokens, topk, score="sigmoid", bias=None, expert_groups=1, topk_groups=1, scale=1.0,
                 capacity=None, balance=0.0):
        self.experts, self.inter2, self.hidden = w1.shape
        self.inter, self.topk, self.tokens = self.inter2 // 2, topk, tokens
        self.w1, self.w2 = _quantised_weight(w1), _quantised_weight(w2)
        # The input-gradient GEMMs contract over the other axis of the weights.
        self.w1t, self.w2t = _quantised_weight(w1.transpose(1, 2)), _quantised_weight(w2.transpose(1, 2))
        self.routing = dict(score=score, renormalize=True, scale=scale)
        self.choice = dict(bias=bias, expert_groups=expert_groups, topk_groups=topk_groups)
        if capacity is None:
            capacity = tokens * topk + self.experts * (BLOCK - 1)
        m, h, i = (capacity + BLOCK - 1) // BLOCK * BLOCK, self.hidden, self.inter
        self.rows = m
        self.ids, self.weights = _i32(tokens, topk), _f32(tokens, topk)
        self.row_of, self.src, self.m_indices, self.k_offsets = _i32(tokens, topk), _i32(m), _i32(m), _i32(self.experts + 1)
        self.xq, self.xsf = _codes(m, h), _f32(h // BLOCK, m)
        self.h, self.hq, self.hsf = _bf16(m, 2 * i), _codes(m, 2 * i), _f32(2 * i // BLOCK, m)
        self.aq, self.asf = _codes(m, i), _f32(i // BLOCK, m)
        self.d, self.y = _bf16(m, h), _bf16(tokens, h)
        # backward
        self.dq, self.dsf, self.dqt, self.dsft = _codes(m, h), _f32(h // BLOCK, m), _codes(h, m), _f32(m // BLOCK, h)
        self.dweights, self.dlogits = _f32(tokens, topk), _f32(tokens, self.experts)
        self.dact = _bf16(m, i)
        self.dhq, self.dhsf = _codes(m, 2 * i), _f32(2 * i // BLOCK, m)
        self.dhqt, self.dhsft = _codes(2 * i, m), _f32(m // BLOCK, 2 * i)
        self.aqt, self.asft = _codes(i, m), _f32(m // BLOCK, i)
        self.xqt, self.xsft = _codes(h, m), _f32(m // BLOCK, h)
        self.dxp, self.dx = _bf16(m, h), _bf16(tokens, h)
        self.dw1, self.dw2 = _bf16(self.experts, 2 * i, h), _bf16(self.experts, h, i)
        need = max(dg.dg_get_moe_plan_workspace_size(tokens, topk, self.experts),
                   dg.dg_get_moe_combine_bwd_workspace_size(m, h),
                   *(dg.dg_get_workspace_size(m, n, k, self.experts) for n, k in ((2 * i, h), (h, i), (i, h), (h, 2 * i))))
        self.balance = dict(score=score, coef=balance) if balance else None
        if balance:
            self.counts, self.used, self.loss = _i32(1, self.experts), _i32(1), _f32(1)
            need = max(need, dg.dg_get_moe_balance_workspace_size(tokens, self.experts))
        # The GEMMs want their workspace zero before its first use and leave it so; the others' is their own.
        self.gemm_ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
        self.ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")

    def forward(self, x, logits):
        """x [tokens][hidden] bf16, logits [tokens][experts] float32 -> y [tokens][hidden] bf16."""
        self.logits = logits
        dg.dg_moe_route(logits, self.ids, self.weights, **self.choice, **self.routing)
        if self.balance:
            dg.dg_moe_balance(logits, self.ids, self.counts, self.used, self.loss, workspace=self.ws, **self.balance)
        dg.dg_moe_plan_contiguous(self.ids, self.row_of, self.src, self.m_indices, self.k_offsets, workspace=self.ws)
        dg.dg_moe_dispatch(x, self.src, self.xq, self.xsf, topk=self.topk)
        dg.dg_grouped_contiguous_qout(self.xq, self.xsf, *self.w1, self.h, self.hq, self.hsf, self.m_indices,
                                      workspace=self.gemm_ws)
        dg.dg_swiglu_quant(self.h, self.aq, self.asf, m_indices=self.m_indices)
        dg.dg_grouped_contiguous(self.aq, self.asf, *self.w2, self.d, self.m_indices, workspace=self.gemm_ws)
        return dg.dg_moe_combine(self.d, self.row_of, self.y, weights=self.weights)

    def backward(self, dy):
        """(dx, dw1, dw2, dlogits) for dy [tokens][hidden] bf16 and the last forward pass."""
        dg.dg_moe_combine_bwd(dy, self.d, self.src, self.row_of, self.weights, self.dq, self.dsf, self.dqt, self.dsft,
                              self.dweights, workspace=self.ws)
        dg.dg_grouped_contiguous(self.dq, self.dsf, *self.w2t, self.dact, self.m_indices, workspace=self.gemm_ws)
        dg.dg_swiglu_bwd(self.hq, self.hsf, self.dact, self.m_indices, self.dhq, self.dhsf, self.dhqt, self.dhsft,
                         aqt=self.aqt, asft=self.asft)
        dg.dg_k_grouped_nt(self.dqt, self.dsft, self.aqt, self.asft, self.dw2, self.k_offsets)
        dg.dg_grouped_contiguous(self.dhq, self.dhsf, *self.w1t, self.dxp, self.m_indices, workspace=self.gemm_ws)
        dg.dg_moe_combine(self.dxp, self.row_of, self.dx)
        dg.dg_requant_t(self.xq, self.xsf, self.m_indices, self.xqt, self.xsft)
        dg.dg_k_grouped_nt(self.dhqt, self.dhsft, self.xqt, self.xsft, self.dw1, self.k_offsets)
        dg.dg_moe_route_bwd(self.logits, self.ids, self.dweights, self.dlogits, **self.routing)
        if self.balance:
            dg.dg_moe_balance_bwd(self.logits, self.counts, self.used, self.dlogits, self.topk, add=self.dlogits, **self.balance)
        return self.dx, self.dw1, self.dw2, self.dlogits


def reference(layer, x, logits, w1, w2, dy):
    """(y, dx, dw1, dw2, dlogits) in float32 by autograd, for the experts the layer chose."""
    x, w1, w2 = (t.float().requires_grad_() for t in (x, w1, w2))
    logits = logits.clone().requires_grad_()
    ids = layer.ids.long()
    s = torch.sigmoid(logits) if layer.routing["score"] == "sigmoid" else torch.softmax(logits, 1)
    s = s.gather(1, ids.clamp(min=0)) * (ids >= 0)
    weights = layer.routing["scale"] * s / s.sum(1, keepdim=True).clamp(min=1e-30)
    y = torch.zeros_like(x)
    for e in range(layer.experts):
        t, j = (ids == e).nonzero(as_tuple=True)
        if t.numel():
            gate, up = (x[t] @ w1[e].t()).chunk(2, dim=1)
            y = y.index_add(0, t, weights[t, j, None] * ((torch.nn.functional.silu(gate) * up) @ w2[e].t()))
    (y * dy.float()).sum().backward()
    return y.detach(), x.grad, w1.grad, w2.grad, logits.grad


def make_inputs(tokens, hidden, inter, experts, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    w1 = (normal(experts, 2 * inter, hidden) / hidden ** 0.5).bfloat16()
    w2 = (normal(experts, hidden, inter) / inter ** 0.5).bfloat16()
    return normal(tokens, hidden).bfloat16(), 1.5 * normal(tokens, experts), w1, w2, normal(tokens, hidden).bfloat16()


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 4096), ("hidden", 7168), ("inter", 2048), ("experts", 16), ("topk", 8), ("steps", 10)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    x, logits, w1, w2, dy = make_inputs(a.tokens, a.hidden, a.inter, a.experts)
    layer = MoELayer(w1, w2, a.tokens, a.topk)
    got = (layer.forward(x, logits), *layer.backward(dy))
    for name, u, v in zip(("y", "dx", "dw1", "dw2", "dlogits"), got, reference(layer, x, logits, w1, w2, dy)):
        print(f"{name:8s} relative error against float32: {float((u.float() - v).norm() / v.norm()):.4f}")
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    steps = {"forward": lambda: layer.forward(x, logits),
             "forward and backward": lambda: (layer.forward(x, logits), layer.backward(dy))}
    for name, step in steps.items():
        step()
        begin.record()
        for _ in range(a.steps):
            step()
        end.record()
        torch.cuda.synchronize()
        ms = begin.elapsed_time(end) / a.steps
        print(f"{name}: {ms:.3f} ms, {a.tokens / ms * 1e3:.0f} tokens/s")


if __name__ == "__main__":
    main()
