"""Sigmoid scores far from zero: weights and probabilities are quotients of scores, which stay
of ordinary size when the scores themselves are tiny, and 1 - s stays exact when s is near 1."""
import pytest
import torch

import combine_ep_get_02_gb300 as ep

pytestmark = pytest.mark.gpu

CENTRES = [-1e30, -1000.0, -110.0, -95.0, -88.0, -75.0, -50.0, -20.0, 0.0, 8.0, 12.0, 17.0, 30.0, 100.0]
# a quotient of fast exponentials: each argument (below 90 in magnitude, or the result is 0) is
# rounded twice, which moves e^x by |x| 2^-23 = 1.1e-5; numerator and sum together 2.2e-5, their
# other roundings 1e-6
QUOTIENT = 2.5e-5


def logits_of(dtype, E, seed=0):
    """Rows around every centre, and rows that reach from one end to the other."""
    g = torch.Generator().manual_seed(seed)
    rows = [c + 3 * torch.randn(6, E, generator=g) for c in CENTRES]
    rows.append(torch.linspace(-120, 40, E).expand(4, E))
    rows.append(torch.where(torch.rand(8, E, generator=g) < 0.7, -90.0 + torch.rand(8, E, generator=g), 15.0))
    return torch.cat(rows).to(dtype).cuda()


def run(logits, K, normalize=1, scale=1.0, G=1, keep=1):
    N, E = logits.shape
    kind = ep.EP_DTYPE_BF16 if logits.dtype == torch.bfloat16 else ep.EP_DTYPE_FP32
    cfg = ep.RouteConfig(1, N, E, K, kind, ep.EP_SCORE_SIGMOID, G, keep, normalize, scale)
    out, ws = ep.alloc_route(cfg), ep.alloc_route_workspace(cfg)
    ep.ep_route(cfg, logits, None, None, out, ws)
    assert ep.ep_check_error(ws) == ep.EP_OK and (out.topk_idx >= 0).all()
    return cfg, out, ws


def log_scores(logits):
    return torch.nn.functional.logsigmoid(logits.double())


def quotient(ls):
    """s / sum s of the scores e^ls; 0 where all of them are 0 in 64 bits."""
    return torch.where(ls.amax(-1, keepdim=True) >= -745, torch.softmax(ls, -1), 0.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,K", [(24, 4), (200, 8), (256, 1), (1500, 5)])
def test_quotients_of_tiny_scores(dtype, E, K):
    logits = logits_of(dtype, E)
    _, out, _ = run(logits, K, scale=2.5)
    ls = log_scores(logits)
    want = 2.5 * quotient(ls.gather(1, out.topk_idx))
    assert torch.isfinite(out.topk_weights).all()
    assert ((out.topk_weights.double() - want).abs() <= QUOTIENT * want + 1e-30).all()
    p = quotient(ls).sum(0)
    # fp32 sums of a warp's few tokens, then fixed point of 2^-50 or finer
    assert ((out.prob_sum[0].double() - p).abs() <= QUOTIENT * p + 1e-12).all()
    N = len(logits)
    loss = float((E * out.expert_count[0].double() / (K * N) * p / N).sum())
    assert abs(float(out.balance_loss) - loss) <= QUOTIENT * loss


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("normalize", [0, 1])
@pytest.mark.parametrize("E,K", [(24, 4), (200, 8), (1500, 5)])
def test_gradients_at_both_ends(dtype, normalize, E, K):
    """Each gradient against its own terms, of which 1 - s is a factor."""
    logits = logits_of(dtype, E, seed=1)
    cfg, out, ws = run(logits, K, normalize, scale=1.5)
    N = len(logits)
    g = torch.Generator().manual_seed(2)
    d_weights, d_loss = torch.randn(N, K, generator=g).cuda(), torch.full((1,), 3.0 * N, device="cuda")
    d = torch.empty_like(logits)
    ep.ep_route_grad(cfg, logits, None, out, d_weights, d_loss, d, ws)
    assert ep.ep_check_error(ws) == ep.EP_OK
    l, idx, gw = logits.double(), out.topk_idx, 1.5 * d_weights.double()
    s, c = torch.sigmoid(l), torch.sigmoid(-l)  # c = 1 - s
    p = quotient(log_scores(logits))
    a = float(d_loss) * E / (K * N * N) * out.expert_count[0].double()
    ap = (a * p).sum(-1, keepdim=True)
    sk = s.gather(1, idx)
    if normalize:
        q = quotient(log_scores(logits).gather(1, idx))
        gl = q * (gw - (q * gw).sum(-1, keepdim=True))
        size = q * (gw.abs() + (q * gw.abs()).sum(-1, keepdim=True))
    else:
        gl, size = gw * sk, gw.abs() * sk
    want = c * (p * (a - ap)).scatter_add(1, idx, gl)
    terms = c * (p * (a + ap)).scatter_add(1, idx, size)
    # two quotients and 1 - s multiply in each term
    tol = 3 * QUOTIENT * terms + 1e-35  # what is below the least normal number may be 0
    if dtype == torch.bfloat16:
        tol = tol + 2 ** -8 * want.abs()  # one rounding of the result
    off = (d.double() - want).abs() - tol
    assert torch.isfinite(d.float()).all() and float(off.max()) <= 0, (float(off.max()), int((off > 0).sum()))
