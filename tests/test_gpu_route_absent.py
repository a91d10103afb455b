"""Gradients of lanes that hold no expert: whatever stands there reaches nothing."""
import math

import pytest
import torch

import combine_ep_get_02_gb300 as ep

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("normalize", [0, 1])
@pytest.mark.parametrize("score", [ep.EP_SCORE_SOFTMAX, ep.EP_SCORE_SIGMOID])
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf])
def test_gradients_of_absent_lanes_are_not_read(score, normalize, junk):
    """Masked tokens, and live tokens with fewer experts available than lanes."""
    g = torch.Generator().manual_seed(3)
    B, T, E, K = 2, 60, 24, 6
    logits = torch.randn(B * T, E, generator=g).cuda()
    logits[::4, 2:] = -math.inf  # two experts are left
    mask = (torch.rand(B * T, generator=g) >= 0.3).to(torch.uint8).cuda()
    cfg = ep.RouteConfig(B, T, E, K, score=score, normalize=normalize, scale=1.5)
    out, ws = ep.alloc_route(cfg), ep.alloc_route_workspace(cfg)
    ep.ep_route(cfg, logits, None, mask, out, ws)
    absent = out.topk_idx < 0
    live = (mask != 0)[:, None] & absent
    assert live.any() and (absent & ~live).any()
    d_weights = torch.randn(B * T, K, generator=g).cuda()
    d_loss = torch.full((1,), 5.0, device="cuda")
    d = []
    for value in (0.0, junk):
        d_weights[absent] = value
        d.append(torch.empty_like(logits))
        ep.ep_route_grad(cfg, logits, mask, out, d_weights, d_loss, d[-1], ws)
    assert ep.ep_check_error(ws) == ep.EP_OK
    assert torch.isfinite(d[1]).all() and torch.equal(d[0], d[1])
    # an index that is no expert's counts as masked, its gradient too
    out.topk_idx[1, 0] = E
    d_weights[1, 0] = junk
    ep.ep_route_grad(cfg, logits, mask, out, d_weights, d_loss, d[1], ws)
    assert ep.ep_check_error(ws) == ep.EP_ERR_BAD_TOPK and torch.isfinite(d[1]).all()
