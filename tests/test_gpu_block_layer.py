"""The transformer block's operators together, as examples/mlp_block.py and
examples/moe_layer.py run them: against float32 autograd, on another stream than
the default one, and captured in a graph.

FP8 codes carry a relative rms error of about 2.6 % (3 mantissa bits).  The block's
output passes four quantisations (5.2 %), of which the gate (about 0.5) lets half
into the stream; the gradients pass up to five more, through the activation's slope:
sqrt(9) * 2.6 % = 8 %.  Bounds: 6 % for the output, 12 % for the gradients, and the
same for the parameters', which are sums of them over the tokens.
"""

import importlib.util
import os

import pytest
import torch

from oracle import block as oracle
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _load(name):
    require_gpu()
    spec = importlib.util.spec_from_file_location(f"{name}_example", os.path.join(ROOT, "examples", f"{name}.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _rel(u, v):
    return float((u.float() - v).norm() / v.norm())


@pytest.mark.parametrize("tokens,hidden,inter,res_scale", [(128, 256, 512, 1.0), (384, 512, 1152, 0.7), (1024, 1024, 2048, 1.0)])
def test_block_against_float32(tokens, hidden, inter, res_scale):
    ex = _load("mlp_block")
    y0, h0, w1, w2, p, dout = ex.make_inputs(tokens, hidden, inter, seed=tokens)
    block = ex.MLPBlock(w1, w2, p, tokens, res_scale)
    out = block.forward(y0, h0)
    got = block.backward(dout)
    want = ex.reference(y0, h0, w1, w2, p, dout, res_scale)
    assert _rel(out, want[0]) < 0.06
    for name, u, v in zip(("dy0", "dh0", "dw1", "dw2"), got, want[1:]):
        assert _rel(u, v) < 0.12, name
    for name in p:
        assert _rel(got[4][name], want[5][name]) < 0.12, name


def test_block_on_another_stream_and_in_a_graph():
    ex = _load("mlp_block")
    y0, h0, w1, w2, p, dout = ex.make_inputs(256, 512, 1024, seed=2)
    block = ex.MLPBlock(w1, w2, p, 256)
    sets = [torch.randn(256, 512, device="cuda").bfloat16() for _ in range(3)]

    def step():
        out = block.forward(y0, h0)
        got = block.backward(dout)
        return [t.clone() for t in (out, *got[:4], *got[4].values())]

    want = []
    for v in sets:
        y0.copy_(v)
        want.append(step())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for a, b in zip(step(), want[2]):
            assert torch.equal(a, b)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in (0, 2, 1, 0):
        y0.copy_(sets[i])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want[i]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_layer_with_a_balance_loss(score):
    """The layer's own results stay as they are, and the logits' gradient gains the loss': one float32 addition to
    each, of terms within 2^-16 (tests/test_gpu_block_balance.py)."""
    ex = _load("moe_layer")
    tokens, experts, topk = 300, 16, 4
    x, logits, w1, w2, dy = ex.make_inputs(tokens, 256, 128, experts, seed=7)
    plain, layer = ex.MoELayer(w1, w2, tokens, topk, score=score), ex.MoELayer(w1, w2, tokens, topk, score=score, balance=0.5)
    assert torch.equal(layer.forward(x, logits), plain.forward(x, logits))
    a, b = plain.backward(dy), layer.backward(dy)
    assert all(torch.equal(u, v) for u, v in zip(a[:3], b[:3]))
    counts, used, loss = oracle.balance(logits.cpu().numpy(), layer.ids.cpu().numpy(), None, score, 0.5)
    assert (layer.counts.cpu().numpy() == counts).all() and int(layer.used) == tokens
    assert abs(float(layer.loss) - loss) <= 2.0 ** -16 * loss
    grad, _, mag = oracle.balance_bwd(logits.cpu().numpy(), counts, used, topk, None, score, 0.5)
    base = a[3].double().cpu().numpy()
    off = abs(b[3].double().cpu().numpy() - (base + grad))
    assert (off <= 2.0 ** -16 * mag + 2.0 ** -23 * (abs(base) + abs(grad))).all()
