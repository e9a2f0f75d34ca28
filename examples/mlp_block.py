"""The feed-forward half of a transformer block on the library's operators:
forward and backward pass with dense FP8 GEMMs, norms on both sides and no host
synchronisation.

Forward:  norm (residual add, norm, quantise) -> GEMM with bias and GELU (which
keeps the activation's input and quantises its output) -> GEMM with bias ->
norm after the block, column gate, scaled residual.
Backward: the junction's gradient -> gradient of the second GEMM's epilogue
(codes by rows and transposed, bias) -> GEMM (w2^T) -> gradient of the first
one's -> GEMM (w1^T) -> gradient of the norm; the weight gradients are
K-grouped GEMMs of one group over the transposed codes.

    python examples/mlp_block.py [--tokens 4096 --hidden 4096 --inter 14336]

prints the error against float32 arithmetic on the same bf16 weights and the
time of a step.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_grouped_gemm_02_amd as dg  # noqa: E402

BLOCK = 128
EPS = 1e-6


def _codes(*shape):
    return torch.empty(shape, dtype=torch.uint8, device="cuda")


def _f32(*shape):
    return torch.empty(shape, dtype=torch.float32, device="cuda")


def _bf16(*shape):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda")


def _operand(rows, cols):
    """Buffers of 1x128 codes and scales of a [rows][cols] matrix."""
    return _codes(rows, cols), _f32(cols // BLOCK, dg.dg_get_sf_leading_dim(rows))


def _weight(w):
    q, sf = _codes(*w.shape), _f32((w.shape[0] + BLOCK - 1) // BLOCK, w.shape[1] // BLOCK)
    dg.dg_quant_128x128(w.contiguous(), q, sf)
    return q, sf


class MLPBlock:
    """Weights w1 [inter][hidden], w2 [hidden][inter] bf16; p: norm [hidden],
    b1 [inter], b2 [hidden], post [hidden], gate [hidden] float32.  `tokens` is
    a multiple of 128 (the weight gradients' K)."""

    def __init__(self, w1, w2, p, tokens, res_scale=1.0):
        (i, h), t = w1.shape, tokens
        self.p, self.res_scale = p, res_scale
        self.w1, self.w2, self.w1t, self.w2t = (_weight(w) for w in (w1, w2, w1.t(), w2.t()))
        # forward
        self.r, self.x = _bf16(t, h), _operand(t, h)
        self.z, self.a, self.act = _bf16(t, i), _bf16(t, i), _operand(t, i)
        self.y, self.out = _bf16(t, h), _bf16(t, h)
        # backward
        self.dy, self.dr, self.dyq, self.dyt = _bf16(t, h), _bf16(t, h), _operand(t, h), _operand(h, t)
        self.da, self.dzq, self.dzt = _bf16(t, i), _operand(t, i), _operand(i, t)
        self.dx, self.dinput, self.dstream = _bf16(t, h), _bf16(t, h), _bf16(t, h)
        self.xt, self.at = _operand(h, t), _operand(i, t)
        self.dw1, self.dw2 = _bf16(1, i, h), _bf16(1, h, i)
        self.grads = {k: torch.empty_like(v) for k, v in p.items()}
        self.ends = torch.tensor([0, t], dtype=torch.int32, device="cuda")
        self.gemm_ws = torch.zeros(max(16, *(dg.dg_get_workspace_size(t, n, k) for n, k in ((i, h), (h, i)))),
                                   dtype=torch.uint8, device="cuda")
        self.ws = torch.empty(max(16, dg.dg_get_block_norm_bwd_workspace_size(t, h),
                                  *(dg.dg_get_epilogue_bwd_workspace_size(t, n) for n in (h, i))),
                              dtype=torch.uint8, device="cuda")

    def forward(self, y0, h0):
        """y0: output of the block before, h0: residual stream, [tokens][hidden] bf16 -> the stream after this block."""
        p = self.p
        dg.dg_block_norm(y0, h=h0, r=self.r, q=self.x[0], sf=self.x[1], weight=p["norm"], eps=EPS)
        dg.dg_fp8_gemm_nt_epilogue(*self.x, *self.w1, self.a, bias=p["b1"], act="gelu_tanh", pre=self.z, dq=self.act[0],
                                   dsf=self.act[1], workspace=self.gemm_ws)
        dg.dg_fp8_gemm_nt_epilogue(*self.act, *self.w2, self.y, bias=p["b2"], workspace=self.gemm_ws)
        dg.dg_block_norm(self.y, h=self.r, r=self.out, post=True, post_weight=p["post"], gate=p["gate"],
                         res_scale=self.res_scale, eps=EPS)
        return self.out

    def backward(self, dout):
        """(dy0, dh0, dw1, dw2, gradients of p) for dout [tokens][hidden] bf16 and the last forward pass."""
        p, g = self.p, self.grads
        dg.dg_block_norm_bwd(self.dy, dr=dout, y=self.y, dh=self.dr, post=True, post_weight=p["post"],
                             dpost_weight=g["post"], gate=p["gate"], dgate=g["gate"], res_scale=self.res_scale, eps=EPS,
                             workspace=self.ws)
        dg.dg_epilogue_bwd(self.dy, *self.dyq, dqt=self.dyt[0], dsft=self.dyt[1], dbias=g["b2"], workspace=self.ws)
        dg.dg_fp8_gemm_nt(*self.dyq, *self.w2t, self.da, workspace=self.gemm_ws)
        dg.dg_requant_t(*self.act, None, *self.at)
        dg.dg_k_grouped_nt(*self.dyt, *self.at, self.dw2, self.ends)
        dg.dg_epilogue_bwd(self.da, *self.dzq, pre=self.z, act="gelu_tanh", dqt=self.dzt[0], dsft=self.dzt[1],
                           dbias=g["b1"], workspace=self.ws)
        dg.dg_fp8_gemm_nt(*self.dzq, *self.w1t, self.dx, workspace=self.gemm_ws)
        dg.dg_requant_t(*self.x, None, *self.xt)
        dg.dg_k_grouped_nt(*self.dzt, *self.xt, self.dw1, self.ends)
        dg.dg_block_norm_bwd(self.dinput, dx=self.dx, dr=self.dr, r=self.r, dh=self.dstream, weight=p["norm"],
                             dweight=g["norm"], eps=EPS, workspace=self.ws)
        return self.dinput, self.dstream, self.dw1[0], self.dw2[0], g


def reference(y0, h0, w1, w2, p, dout, res_scale=1.0):
    """The same in float32 by autograd: (out, dy0, dh0, dw1, dw2, gradients of p)."""
    leaves = [t.detach().float().clone().requires_grad_() for t in (y0, h0, w1, w2, *p.values())]
    a, b, u, v = leaves[:4]
    q = dict(zip(p, leaves[4:]))

    def norm(t, weight):
        return t * torch.rsqrt(t.pow(2).mean(1, keepdim=True) + EPS) * weight

    r = a + b
    y = torch.nn.functional.gelu(norm(r, q["norm"]) @ u.t() + q["b1"], approximate="tanh") @ v.t() + q["b2"]
    out = res_scale * r + q["gate"] * norm(y, q["post"])
    out.backward(dout.float())
    return (out.detach(), *(t.grad for t in leaves[:4]), {k: t.grad for k, t in q.items()})


def make_inputs(tokens, hidden, inter, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    w1 = (normal(inter, hidden) / hidden ** 0.5).bfloat16()
    w2 = (normal(hidden, inter) / inter ** 0.5).bfloat16()
    p = dict(norm=1 + 0.1 * normal(hidden), b1=0.1 * normal(inter), b2=0.1 * normal(hidden),
             post=1 + 0.1 * normal(hidden), gate=0.5 + 0.1 * normal(hidden))
    return normal(tokens, hidden).bfloat16(), normal(tokens, hidden).bfloat16(), w1, w2, p, normal(tokens, hidden).bfloat16()


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 4096), ("hidden", 4096), ("inter", 14336), ("steps", 10)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    y0, h0, w1, w2, p, dout = make_inputs(a.tokens, a.hidden, a.inter)
    block = MLPBlock(w1, w2, p, a.tokens)
    out = block.forward(y0, h0)
    got = (out, *block.backward(dout))
    for name, u, v in zip(("out", "dy0", "dh0", "dw1", "dw2"), got, reference(y0, h0, w1, w2, p, dout)):
        print(f"{name:4s} relative error against float32: {float((u.float() - v).norm() / v.norm()):.4f}")
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    steps = {"forward": lambda: block.forward(y0, h0),
             "forward and backward": lambda: (block.forward(y0, h0), block.backward(dout))}
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
