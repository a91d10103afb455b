"""The most tokens that the router accepts."""
import pytest
import torch

import combine_ep_get_02_gb300 as ep

pytestmark = pytest.mark.gpu


def guarded(n, dtype, fill, guard=1 << 16):
    """n elements between two guards of `guard` elements, all of them `fill`."""
    whole = torch.full((n + 2 * guard,), fill, dtype=dtype, device="cuda")
    return whole, whole[guard:guard + n]


def test_the_most_tokens_of_a_segment():
    """2^31 - 1 tokens with one choice of two experts: every token against the definition, and
    nothing written in front of the buffers or behind them."""
    N, piece, guard = 2 ** 31 - 1, 1 << 27, 1 << 16
    logits = torch.empty(N, 2, dtype=torch.bfloat16, device="cuda")
    for i in range(0, N, piece):
        logits[i:i + piece].normal_(generator=torch.Generator(device="cuda").manual_seed(i))
    cfg = ep.RouteConfig(1, N, 2, 1, ep.EP_DTYPE_BF16, normalize=0)
    out, ws = ep.alloc_route(ep.RouteConfig(1, 1, 2, 1)), ep.alloc_route_workspace(cfg)
    idx, out.topk_idx = guarded(N, torch.int64, 77)
    weights, out.topk_weights = guarded(N, torch.float32, 77.0)
    ep.ep_route(cfg, logits, None, None, out, ws)
    assert ep.ep_check_error(ws) == ep.EP_OK
    for whole in (idx, weights):
        assert (whole[:guard] == 77).all() and (whole[-guard:] == 77).all()
    second = 0
    for i in range(0, N, piece):
        l = logits[i:i + piece].float()
        want = l[:, 1] > l[:, 0]  # a tie goes to the first
        second += int(want.sum())
        assert torch.equal(out.topk_idx[i:i + piece], want.long())
        p = torch.sigmoid((l[:, 0] - l[:, 1]).abs())  # the larger of two softmax values
        assert ((out.topk_weights[i:i + piece] - p).abs() <= 1e-5).all()
    assert out.expert_count.tolist() == [[N - second, second]] and int(out.num_valid) == N
    d_weights = weights.fill_(1.0)[guard:guard + N]
    whole, d_logits = guarded(2 * N, torch.bfloat16, 77.0)
    ep.ep_route_grad(cfg, logits, None, out, d_weights, None, d_logits, ws)
    assert ep.ep_check_error(ws) == ep.EP_OK
    assert (whole[:guard] == 77).all() and (whole[-guard:] == 77).all()
    d_logits = d_logits.view(N, 2)
    for i in range(0, N, piece):
        l = logits[i:i + piece].float()
        d = l[:, 0] - l[:, 1]
        g = torch.sigmoid(d) * torch.sigmoid(-d)  # of the chosen; the other's is its negative
        g = torch.where(l[:, 1] > l[:, 0], -g, g)
        got = d_logits[i:i + piece].float()
        for col, want in ((0, g), (1, -g)):  # one rounding to bf16, and fp32 terms that cancel
            assert ((got[:, col] - want).abs() <= 2 ** -8 * want.abs() + 1e-5).all()
