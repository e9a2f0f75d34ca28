"""GPU calls of more tokens than one grid dimension has threads for (2^32): the
combine from 2^24 tokens on, the routing and its gradient from 2^26 on."""

import pytest
import torch

from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [2 ** 24 - 1, 2 ** 24, 2 ** 24 + 12345])
def test_combine(tokens):
    dg = require_gpu()
    d = torch.arange(64, device="cuda")[:, None].expand(64, 8).to(torch.bfloat16).contiguous()
    rows = (torch.arange(tokens, device="cuda", dtype=torch.int32) % 65 - 1).view(-1, 1)  # -1 .. 63
    y = torch.full((tokens, 8), -1.0, dtype=torch.bfloat16, device="cuda")
    dg.dg_moe_combine(d, rows, y)
    want = rows.clamp(min=0).to(torch.bfloat16).expand(tokens, 8)
    assert torch.equal(y, want)


@pytest.mark.parametrize("tokens", [2 ** 26 - 4, 2 ** 26, 2 ** 26 + 12345])
def test_route_and_gradient(tokens):
    dg = require_gpu()
    x = (torch.arange(2 * tokens, device="cuda", dtype=torch.int32) * 7 % 11).to(torch.float32).view(tokens, 2)
    ids = torch.full((tokens, 1), -7, dtype=torch.int32, device="cuda")
    w = torch.full((tokens, 1), -7.0, device="cuda")
    dg.dg_moe_route(x, ids, w, score="sigmoid", renormalize=True, scale=2.0)
    assert torch.equal(ids.view(-1), (x[:, 1] > x[:, 0]).int()) and bool((w == 2.0).all())
    dx = torch.full_like(x, -7.0)
    dg.dg_moe_route_bwd(x, ids, torch.ones_like(w), dx, score="sigmoid", renormalize=False, scale=1.0)
    s = torch.sigmoid(x)
    want = (s * (1.0 - s)).mul_(torch.nn.functional.one_hot(ids.view(-1).long(), 2))
    # float32 sums and quotients of numbers of about 1, and 1 - s of up to s = 0.99996: 2^-24 / 4e-5
    assert float((dx - want).abs().max()) < 2.0 ** -20
