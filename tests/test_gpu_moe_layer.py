"""The whole layer (examples/moe_layer.py): forward and gradients against a plain
mixture of experts in 64 bits, and its serving form."""
import os
import sys

import pytest
import torch

import combine_ep_get_02_gb300 as ep

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402

pytestmark = pytest.mark.gpu


def plain(layer, x, idx, logits):
    """The layer's output and balance loss for a fixed choice, from 64-bit leaves."""
    up, down = layer.up.double().requires_grad_(True), layer.down.double().requires_grad_(True)
    x = x.double().reshape(-1, layer.hidden).requires_grad_(True)
    l = logits.double().requires_grad_(True)
    p = torch.softmax(l, -1)
    w = torch.softmax(l.gather(1, idx), -1)
    out = torch.zeros_like(x)
    E = up.shape[0]
    for e in range(E):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        a, b = (x[t] @ up[e].T).chunk(2, -1)
        out = out.index_add(0, t, w[t, k, None] * ((torch.nn.functional.silu(a) * b) @ down[e].T))
    B, T, K = layer.ranks, layer.tokens, layer.topk
    count = torch.nn.functional.one_hot(idx, E).double().sum(1).reshape(B, T, E).sum(1)
    loss = ((E * count / (K * T)) * p.reshape(B, T, E).mean(1)).sum(1).mean()
    return out, loss, (x, l, up, down)


def off(got, want):
    want = want.detach()
    return float((got.double().reshape(want.shape) - want).norm() / want.norm())


@pytest.mark.parametrize("size", [dict(ranks=2, tokens=40, hidden=128, inner=64, experts=8, topk=2),
                                  dict(ranks=4, tokens=150, hidden=264, inner=136, experts=12, topk=3),
                                  dict(ranks=1, tokens=1, hidden=256, inner=128, experts=4, topk=4)])
def test_training_step(size):
    layer = moe_layer.MoELayer(**size)
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(size["ranks"], size["tokens"], size["hidden"], device="cuda", generator=g).bfloat16()
    d_out = torch.randn(x.shape, device="cuda", generator=g).bfloat16()
    d_loss = torch.full((1,), 3.0, device="cuda")
    out = layer.forward(x).clone()
    d_x, d_router, d_up, d_down = layer.backward(d_out, d_loss)
    assert layer.check() == ep.EP_OK and ep.ep_check_error(layer.up_grad_ws) == ep.EP_OK
    want, loss, (lx, ll, lup, ldown) = plain(layer, x, layer.route.topk_idx, layer.logits)
    total = (want * d_out.double().reshape(want.shape)).sum() + 3.0 * loss
    gx, gl, gup, gdown = torch.autograd.grad(total, (lx, ll, lup, ldown))
    # every tensor on the way is rounded to bf16 once (2^-9 of its norm at most): z, h, y and out
    # forward, then the gradients of y, h, z and the rows; eight of them are allowed
    tol = 8 * 2 ** -9
    assert off(out, want) <= tol
    loss = float(loss.detach())
    assert abs(float(layer.route.balance_loss) - loss) <= 1e-5 * loss
    assert off(d_up, gup) <= tol and off(d_down, gdown) <= tol
    assert off(layer.d_logits, gl) <= tol
    gx = gx + gl @ layer.router.double()
    assert off(d_x, gx) <= tol


def test_serving_step_from_a_graph():
    """Eight tokens with FP8 rows, captured once and replayed on other inputs."""
    layer = moe_layer.MoELayer(1, 8, 256, 128, 16, 4, fp8=True, grad=False)
    x = torch.randn(1, 8, 256, device="cuda").bfloat16()
    layer.forward(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.forward(x)
    for seed in range(3):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        got = out.clone()
        eager = layer.forward(x)  # its logits are a new tensor
        assert torch.equal(eager, got)
        want, _, _ = plain(layer, x, layer.route.topk_idx, layer.logits)
        # FP8 rows: e4m3 keeps 3 bits after the leading one, 2^-4 of each value at most
        assert off(got, want) <= 2 ** -4
    assert layer.check() == ep.EP_OK
