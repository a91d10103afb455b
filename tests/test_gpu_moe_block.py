"""The blocks around the layer (examples/moe_layer.py): the training step on rows kept in 8 bits, output and
gradients, and the serving step of a few tokens, against 64 bits."""
import os
import sys

import pytest
import torch

import _block_reference as ref
import combine_ep_get_02_gb300 as ep

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402

pytestmark = pytest.mark.gpu
# every tensor on the way is rounded to bf16 once (2^-9 of its norm at most); eight of them are allowed
TOL = 8 * 2 ** -9


def off(got, want):
    want = want.detach()
    return float((got.double().reshape(want.shape) - want).norm() / want.norm())


def lanes_of(layer):
    """Row of every lane in the expanded blocks."""
    d = (layer.idx // (layer.cfg.num_experts // layer.ranks)).long()
    return (layer.layout.exp_pos + layer.layout.exp_region[d]).long().reshape(-1)


@pytest.mark.parametrize("size", [dict(ranks=2, tokens=40, hidden=128, inner=64, experts=8, topk=2),
                                  dict(ranks=4, tokens=150, hidden=256, inner=192, experts=12, topk=3)])
def test_training_step_on_kept_rows(size):
    block = moe_layer.KeptBlock(**size)
    g = torch.Generator(device="cuda").manual_seed(9)
    rnd = lambda: torch.randn(size["ranks"], size["tokens"], size["hidden"], device="cuda", generator=g).bfloat16()  # noqa: E731
    x, residual, d_sum, d_out = rnd(), rnd(), rnd(), rnd()
    block.gamma.copy_(1 + 0.2 * torch.randn(size["hidden"], device="cuda", generator=g))
    total, out = (t.clone() for t in block.forward(x, residual))
    d_x, d_router, d_up, d_down, d_gamma = block.backward(d_sum, d_out, torch.full((1,), 3.0, device="cuda"))
    assert block.check() == ep.EP_OK

    H, K, E, T = size["hidden"], size["topk"], size["experts"], size["tokens"]
    N, idx = size["ranks"] * T, block.route.topk_idx
    s, _, y = ref.norm(x.reshape(N, H), residual.reshape(N, H), block.gamma, 1e-6)
    assert torch.equal(total, (x.float() + residual.float()).bfloat16())
    # what is kept is what was computed, off by the cast alone: 2^-4 of each value at most
    y8 = ref.values(block.codes, block.sf, False)
    assert off(y8, y) <= 2 ** -4 and off(block.y_norm, y) <= TOL
    row, expert, token = lanes_of(block), idx.reshape(-1), torch.arange(N, device="cuda").repeat_interleave(K)
    up, down = block.up.double(), block.down.double()
    z = torch.stack([y8[t] @ up[e].T for t, e in zip(token.tolist(), expert.tolist())])
    z8 = ref.values(block.z_codes, block.z_sf, False)[row]
    assert off(z8, z) <= 2 ** -4
    lanes = lambda h: torch.stack([h[i] @ down[e].T for i, e in enumerate(expert.tolist())])  # noqa: E731
    fwd = lanes(ref.act(z, "swiglu"))
    logits = block.logits.double().requires_grad_(True)
    p = torch.softmax(logits, -1)
    w = torch.softmax(logits.gather(1, idx), -1).reshape(-1, 1)
    assert off(out, torch.zeros(N, H, dtype=torch.float64, device="cuda").index_add(0, token, w.detach() * fwd)) <= TOL
    # gradients: through the kept z for what lies in front of it, the forward's own outputs for the weights
    count = torch.nn.functional.one_hot(idx, E).double().sum(1).reshape(-1, T, E).sum(1)
    loss = ((E * count / (K * T)) * p.reshape(-1, T, E).mean(1)).sum(1).mean()
    do = d_out.double().reshape(N, H)[token]
    (gl,) = torch.autograd.grad((w * fwd * do).sum() + 3.0 * loss, logits)
    leaf = z8.clone().requires_grad_(True)
    h8 = ref.act(leaf, "swiglu")
    dy = w.detach() * do
    (gz,) = torch.autograd.grad((lanes(h8) * dy).sum(), leaf)
    want_up, want_down = torch.zeros_like(up), torch.zeros_like(down)
    rows = torch.stack([gz[i] @ up[e] for i, e in enumerate(expert.tolist())])
    for e in range(E):
        m = expert == e
        want_up[e], want_down[e] = gz[m].T @ y8[token[m]], dy[m].T @ h8.detach()[m]
    assert off(d_up, want_up) <= TOL and off(d_down, want_down) <= TOL and off(block.d_logits, gl) <= TOL
    gy = torch.zeros(N, H, dtype=torch.float64, device="cuda").index_add(0, token, rows) + gl @ block.router.double()
    want_x, want_gamma, _, _ = ref.norm_grad(total.reshape(N, H), block.gamma, None, gy, d_sum.reshape(N, H), 1e-6)
    assert off(d_x, want_x) <= TOL and off(d_gamma, want_gamma) <= TOL
    assert off(d_router, gl.T @ y) <= TOL


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("tokens", [1, 8, 40])
def test_serving_step(tokens, fp8):
    """Against 64 bits for the choice that was made; captured once and replayed on other inputs."""
    E, H, I, K = 16, 512, 256, 4
    g = torch.Generator(device="cuda").manual_seed(tokens)
    rnd = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5).bfloat16()  # noqa: E731
    router, up, down = rnd(E, H), rnd(E, 2 * I, H), rnd(E, H, I)
    gamma = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).bfloat16()
    sf = dict(up_sf=None, down_sf=None)
    plain = up.double(), down.double()
    if fp8:
        packed = []
        for m in (up, down):
            v = m.float().reshape(E, m.shape[1] // 128, 128, m.shape[2] // 128, 128)
            s = v.abs().amax((2, 4)) / 448
            packed.append(((v / s[:, :, None, :, None]).reshape(m.shape).to(torch.float8_e4m3fn).view(torch.uint8), s.contiguous()))
        (up, sf["up_sf"]), (down, sf["down_sf"]) = packed
        plain = ref.unscale(up, sf["up_sf"]), ref.unscale(down, sf["down_sf"])
    block = moe_layer.ServingBlock(tokens, router, up, down, K, gamma, **sf)
    x, residual = (torch.randn(tokens, H, device="cuda").bfloat16() for _ in range(2))
    block.forward(x, residual)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block.forward(x, residual)
    for seed in range(3):
        for t in (x, residual):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        got = out.clone()
        assert torch.equal(block.forward(x, residual), got)
        s, _, y = ref.norm(x, residual, gamma, 1e-6)
        want, _ = ref.layer(block.y, block.route.topk_idx, block.route.topk_weights, plain[0], None, plain[1], None, block.sum,
                            "swiglu", 2.0 ** -17)
        assert off(block.y, y) <= TOL and off(block.sum, s) <= TOL and off(got, want) <= TOL
    assert block.check() == ep.EP_OK
