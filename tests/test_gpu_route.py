"""The router, its balance loss and its gradient against the 64-bit definitions."""
import math

import pytest
import torch

import _moe_reference as ref
import combine_ep_get_02_gb300 as ep

pytestmark = pytest.mark.gpu

# fp32 results: fast exponentials are within 2 + 1.2 |x| units of 2^-24 for an argument x
# (|x| <= 40 here), quotients and fixed-order sums add a few more: 1e-5 covers them
RTOL = 1e-5


def close(got, want, rtol=RTOL, atol=None):
    got, want = got.double(), want.double()
    atol = rtol * float(want.abs().max()) * 1e-2 if atol is None else atol
    assert got.shape == want.shape
    assert torch.isfinite(got).all()
    bad = (got - want).abs() > rtol * want.abs() + atol
    assert not bad.any(), f"{int(bad.sum())} off, most {float((got - want).abs().max())}"


class Case:
    def __init__(self, B, T, E, K, dtype="fp32", score="softmax", bias=False, G=1, keep=1, normalize=True, scale=1.0,
                 masked=0.0, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.B, self.T, self.E, self.K, self.score, self.G, self.keep = B, T, E, K, score, G, keep
        self.normalize, self.scale = normalize, scale
        N = B * T
        self.logits = (torch.randn(N, E, generator=g) * 2).to(torch.float32 if dtype == "fp32" else torch.bfloat16).cuda()
        self.bias = (torch.randn(E, generator=g) * 0.1).cuda() if bias else None
        self.mask = (torch.rand(N, generator=g) >= masked).to(torch.uint8).cuda() if masked else None
        self.cfg = ep.RouteConfig(B, T, E, K, ep.EP_DTYPE_FP32 if dtype == "fp32" else ep.EP_DTYPE_BF16,
                                  ep.EP_SCORE_SOFTMAX if score == "softmax" else ep.EP_SCORE_SIGMOID, G, keep,
                                  int(normalize), scale)
        self.ws = ep.alloc_route_workspace(self.cfg)
        self.d_weights = torch.randn(N, K, generator=g).cuda()
        self.d_loss = torch.full((1,), 0.7 * max(N, 1)).cuda()

    def run(self, stats=True):
        out = ep.alloc_route(self.cfg, stats=stats)
        for t in (out.topk_idx, out.topk_weights, out.expert_count, out.prob_sum, out.num_valid, out.balance_loss):
            if t is not None:
                t.fill_(77)
        ep.ep_route(self.cfg, self.logits, self.bias, self.mask, out, self.ws)
        return out

    def want(self):
        return ref.route(self.logits, self.bias, self.mask, self.B, self.T, self.K, self.score, self.G, self.keep,
                         self.normalize, self.scale)

    def grad(self, out, d_weights=True, d_loss=True):
        d = torch.full_like(self.logits, 99)
        ep.ep_route_grad(self.cfg, self.logits, self.mask, out, self.d_weights if d_weights else None,
                         self.d_loss if d_loss else None, d, self.ws)
        return d

    def want_grad(self, want, d_weights=True, d_loss=True):
        idx, _, count, _, valid, _ = want
        l = self.logits.double().requires_grad_(True)
        f = ref.route_objective(l, idx, count, valid, self.mask, self.d_weights.double() * d_weights,
                                self.d_loss.double()[0] * d_loss, self.B, self.T, self.K, self.score, self.normalize, self.scale)
        return torch.autograd.grad(f, l)[0]

    def terms(self, want, d_weights, d_loss):
        """The largest of the terms that a token's gradients are sums of, without their signs."""
        _, _, count, _, valid, _ = want
        a = self.d_loss.double() * self.E / (self.B * self.K) * count / valid.clamp(min=1).double()[:, None] ** 2
        a = a.amax(-1).repeat_interleave(self.T)[:, None] * d_loss  # p <= 1
        w = self.d_weights.double().abs().amax(-1, keepdim=True) * self.scale * d_weights  # q, s <= 1
        return 2 * (a + w)

    def check(self, status=ep.EP_OK):
        out, want = self.run(), self.want()
        assert ep.ep_check_error(self.ws) == status
        assert torch.equal(out.topk_idx, want[0])
        assert torch.equal(out.expert_count.long(), want[2])
        assert torch.equal(out.num_valid.long(), want[4])
        close(out.topk_weights, want[1])
        close(out.prob_sum, want[3])
        close(out.balance_loss, want[5].reshape(1))
        return out, want


SIZES = [
    dict(B=1, T=1, E=1, K=1),
    dict(B=1, T=1, E=256, K=8),
    dict(B=1, T=7, E=5, K=5, score="sigmoid"),
    dict(B=3, T=33, E=31, K=3, masked=0.3),
    dict(B=2, T=100, E=32, K=4, dtype="bf16"),
    dict(B=2, T=65, E=33, K=32, dtype="bf16", normalize=False),
    dict(B=1, T=300, E=64, K=6, score="sigmoid", bias=True, scale=2.5),
    dict(B=5, T=40, E=96, K=8, bias=True, normalize=False, scale=0.5),
    dict(B=2, T=129, E=130, K=2, score="sigmoid", normalize=False, masked=0.1),
    dict(B=4, T=257, E=256, K=8, score="sigmoid", bias=True, G=8, keep=4, scale=2.5),
    dict(B=1, T=64, E=160, K=6, G=8, keep=3),
    dict(B=2, T=50, E=6, K=2, G=3, keep=2, bias=True),
    dict(B=1, T=90, E=64, K=8, G=32, keep=4, dtype="bf16", score="sigmoid"),
    dict(B=7, T=31, E=384, K=16, dtype="bf16", bias=True),
    dict(B=1, T=70, E=512, K=8, masked=0.9),
    dict(B=2, T=20, E=1000, K=10, score="sigmoid", G=4, keep=2, bias=True),
    dict(B=1, T=9, E=4095, K=32),
    dict(B=1, T=9, E=4096, K=32, score="sigmoid", G=16, keep=3),
    dict(B=700, T=3, E=16, K=2),
]


@pytest.mark.parametrize("case", SIZES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_route_and_gradient(case):
    c = Case(**case)
    out, want = c.check()
    for dw, dl in ((True, True), (True, False), (False, True)):
        d, exact = c.grad(out, dw, dl), c.want_grad(want, dw, dl)
        assert ep.ep_check_error(c.ws) == ep.EP_OK
        # differences p (a - sum a p) and q (gw - sum q gw): each of their terms is good to RTOL, and
        # the terms may cancel, so the error is measured by them; bf16 results are rounded once
        terms = c.terms(want, dw, dl)
        tol = 0 if c.logits.dtype == torch.float32 else 2 ** -8
        assert ((d.double() - exact).abs() <= tol * exact.abs() + RTOL * terms).all()


def test_gradient_against_differences():
    for case in (dict(B=2, T=5, E=12, K=3), dict(B=1, T=6, E=16, K=4, score="sigmoid", normalize=False),
                 dict(B=2, T=4, E=9, K=2, score="sigmoid", scale=2.0), dict(B=1, T=7, E=10, K=3, normalize=False)):
        c = Case(**case)
        out, want = c.check()
        d = c.grad(out).double()
        idx, _, count, _, valid, _ = want
        l, h = c.logits.double(), 1e-5
        diff = torch.zeros_like(l)
        for i in range(l.shape[0]):
            for j in range(l.shape[1]):
                f = []
                for s in (h, -h):
                    m = l.clone()
                    m[i, j] += s
                    f.append(ref.route_objective(m, idx, count, valid, c.mask, c.d_weights.double(), c.d_loss.double()[0],
                                                 c.B, c.T, c.K, c.score, c.normalize, c.scale))
                diff[i, j] = (f[0] - f[1]) / (2 * h)
        assert float((d - diff).abs().max()) <= 1e-4 * float(diff.abs().max())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_unavailable_and_broken_logits(score, dtype):
    """-inf logits are never chosen; a row of them alone has no expert, weight or gradient; the type's
    lowest value is an ordinary logit; NaN and +inf count as -inf and are reported."""
    c = Case(2, 16, 40, 4, dtype=dtype, score=score)
    low = torch.finfo(c.logits.dtype).min
    c.logits[0] = -math.inf
    c.logits[1, 3:] = -math.inf
    c.logits[2] = low
    c.logits[3, :-2] = low
    c.logits[4, ::2] = -math.inf
    out, want = c.check()
    assert out.topk_idx[0].tolist() == [-1] * 4 and out.topk_weights[0].tolist() == [0.0] * 4
    assert sorted(out.topk_idx[1].tolist()) == [-1, 0, 1, 2] and out.topk_idx[1, 3] == -1
    assert out.topk_idx[2].tolist() == [0, 1, 2, 3]
    d = c.grad(out)
    assert torch.isfinite(d.float()).all()
    assert (d[0] == 0).all()
    c.logits[5, 7] = math.nan
    c.logits[6, 9] = math.inf
    out, want = c.check(status=ep.EP_ERR_NONFINITE)
    assert not (out.topk_idx[5] == 7).any() and not (out.topk_idx[6] == 9).any()
    assert torch.isfinite(c.grad(out).float()).all()


def test_bias_can_disable_an_expert():
    for score in ("softmax", "sigmoid"):
        c = Case(1, 50, 20, 6, score=score, bias=True)
        c.bias[4] = -math.inf
        out, _ = c.check()
        assert not (out.topk_idx == 4).any()


def test_equal_scores_go_to_the_lowest_expert():
    for score in ("softmax", "sigmoid"):
        c = Case(1, 8, 300, 8, score=score)
        c.logits.fill_(0.25)
        c.logits[1::2, 17] = -0.0
        c.logits[1::2] *= 0.0
        out, _ = c.check()
        assert (out.topk_idx == torch.arange(8, device="cuda")).all()
        c = Case(1, 8, 64, 6, score=score, G=8, keep=2)
        c.logits.fill_(-1.0)
        out, _ = c.check()
        assert (out.topk_idx == torch.arange(6, device="cuda")).all()


def test_masked_tokens_are_not_read():
    c = Case(3, 20, 24, 4, masked=0.5)
    c.logits[c.mask == 0] = math.nan
    c.mask[:20] = 0  # a segment of padding alone
    out, _ = c.check()
    assert (out.topk_idx[c.mask == 0] == -1).all() and out.num_valid[0] == 0 and (out.expert_count[0] == 0).all()
    d = c.grad(out)
    assert torch.isfinite(d).all() and (d[c.mask == 0] == 0).all()


def test_no_tokens():
    c = Case(2, 0, 16, 4)
    out = c.run()
    assert ep.ep_check_error(c.ws) == ep.EP_OK
    assert (out.expert_count == 0).all() and (out.prob_sum == 0).all() and (out.num_valid == 0).all()
    assert out.balance_loss.item() == 0
    c.grad(out)


def test_a_workspace_serves_other_sizes():
    cases = [Case(5, 300, 64, 4), Case(1, 700, 200, 8, score="sigmoid", bias=True), Case(40, 20, 24, 2, dtype="bf16"),
             Case(2, 90, 512, 6)]
    ws = ep.alloc_route_workspace(max((c.cfg for c in cases), key=ep.ep_route_workspace_bytes))
    for c in cases + cases[::-1]:
        c.ws = ws
        c.check()
    assert not ws.any()


def test_offsets_past_32_bits():
    """More than 2^31 logits: the last tokens against the definition, the counts against the choice."""
    T, E, K = 8_400_000, 256, 8
    logits = torch.empty(T, E, device="cuda")
    for i in range(0, T, 1 << 20):
        logits[i:i + (1 << 20)].normal_(generator=torch.Generator(device="cuda").manual_seed(i))
    cfg = ep.RouteConfig(1, T, E, K)
    out, ws = ep.alloc_route(cfg), ep.alloc_route_workspace(cfg)
    ep.ep_route(cfg, logits, None, None, out, ws)
    assert ep.ep_check_error(ws) == ep.EP_OK
    last = slice(T - 1000, T)
    want = ref.route(logits[last], None, None, 1, 1000, K)
    assert torch.equal(out.topk_idx[last], want[0])
    close(out.topk_weights[last], want[1])
    assert int(out.num_valid) == T
    assert torch.equal(out.expert_count[0].long(), torch.bincount(out.topk_idx.reshape(-1), minlength=E))
    close(out.prob_sum.sum(1), torch.full((1,), float(T), device="cuda"))
    d = torch.empty_like(logits)
    g = torch.randn(T, K, device="cuda")
    ep.ep_route_grad(cfg, logits, None, out, g, None, d, ws)
    l = logits[last].double().requires_grad_(True)
    w = torch.softmax(l.gather(1, want[0]), -1)
    exact = torch.autograd.grad((w * g[last].double()).sum(), l)[0]
    assert ((d[last].double() - exact).abs() <= RTOL * 2 * g[last].abs().amax(1, keepdim=True)).all()


def test_without_statistics_and_repeatable():
    c = Case(4, 1111, 256, 8)
    a, b = c.run(), c.run()
    for x, y in zip(vars(a).values(), vars(b).values()):
        if torch.is_tensor(x):
            assert torch.equal(x, y)
    s = c.run(stats=False)
    assert torch.equal(s.topk_idx, a.topk_idx) and torch.equal(s.topk_weights, a.topk_weights)
    assert torch.equal(c.grad(a), c.grad(a))


def test_bad_indices_in_the_gradient_are_masked_and_reported():
    c = Case(1, 12, 16, 3)
    out = c.run()
    clean = c.grad(out)
    out.topk_idx[5, 1] = 16
    out.topk_idx[6, 0] = -7
    d = c.grad(out)
    assert ep.ep_check_error(c.ws) == ep.EP_ERR_BAD_TOPK
    assert torch.equal(d[:5], clean[:5]) and torch.isfinite(d).all()


def test_another_stream_and_feeding_the_dispatch():
    """The router's outputs are what the dispatch layout reads; per-source counts agree."""
    c = Case(4, 64, 32, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = ep.alloc_route(c.cfg)
    cfg = ep.Config(1, 4, 32, 4, 64, 64, 128, expand=1)
    ws, lay = ep.alloc_workspace(cfg), ep.alloc_layout(cfg)
    torch.cuda.synchronize()
    ep.ep_route(c.cfg, c.logits, None, None, out, c.ws, stream=s)
    ep.ep_get_dispatch_layout(cfg, out.topk_idx, lay, ws, stream=s)
    assert ep.ep_check_error(ws, stream=s) == ep.EP_OK
    assert torch.equal(lay.num_tokens_per_expert, out.expert_count)
