"""A mixture-of-experts layer on the library's entry points: one training step (forward,
balance loss, every gradient) and serving steps; and a whole block around it, with its norm and
residual, that trains on rows kept in 8 bits (KeptBlock) and serves a few tokens (ServingBlock).

    python examples/moe_layer.py                 # small sizes, a few training steps
    python examples/moe_layer.py --tokens 4096 --hidden 4096 --inner 2048 --experts 64

The forward is router -> dispatch layout -> dispatch (expanded blocks) -> gated up
product -> down product -> combine; the backward goes the same way back. Between the
calls nothing but the library runs; tensors are allocated once.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_ep_get_02_gb300 as ep  # noqa: E402


class MoELayer:
    """Router matrix [E][H] and experts' matrices [E][2 inner][H] and [E][H][inner]; ranks x tokens
    of hidden size H, K experts each. fp8: rows travel as FP8, which the forward takes; the gradients
    of the experts' matrices need bf16 rows, so backward() refuses it."""

    def __init__(self, ranks, tokens, hidden, inner, experts, topk, seed=0, score=ep.EP_SCORE_SOFTMAX, fp8=False,
                 grad=True):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5).bfloat16()  # noqa: E731
        self.ranks, self.tokens, self.hidden, self.topk, self.grad = ranks, tokens, hidden, topk, grad
        self.router = rnd(experts, hidden)
        self.up, self.down = rnd(experts, 2 * inner, hidden), rnd(experts, hidden, inner)
        self.cfg = ep.Config(1, ranks, experts, topk, tokens, tokens, hidden, expand=1,
                             recv_dtype=ep.EP_DTYPE_FP8_E4M3 if fp8 else ep.EP_DTYPE_BF16)
        rows = ep.ep_recv_rows(self.cfg)
        # the expert outputs and every gradient travel in bf16
        self.back = ep.Config(1, ranks, experts, topk, tokens, tokens, hidden, expand=1)
        self.route_cfg = ep.RouteConfig(ranks, tokens, experts, topk, ep.EP_DTYPE_BF16, score)
        self.up_cfg = ep.ProductConfig(ranks, experts, rows, hidden, inner, ep.EP_ACT_SWIGLU,
                                       ep.EP_DTYPE_FP8_E4M3 if fp8 else ep.EP_DTYPE_BF16)
        self.down_cfg = ep.ProductConfig(ranks, experts, rows, inner, hidden)
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.route, self.layout = ep.alloc_route(self.route_cfg, stats=grad), ep.alloc_layout(self.cfg)
        self.recv = ep.alloc_recv(self.cfg, sidecars=False)
        self.z = torch.empty(rows, 2 * inner, **bf) if grad else None
        self.h, self.y = torch.empty(rows, inner, **bf), torch.empty(rows, hidden, **bf)
        self.out = torch.empty(ranks, tokens, hidden, **bf)
        self.ws, self.route_ws = ep.alloc_workspace(self.cfg), ep.alloc_route_workspace(self.route_cfg)
        self.up_ws = ep.alloc_product_workspace(self.up_cfg)
        self.down_ws = ep.alloc_product_workspace(self.down_cfg)
        if grad:
            self.up_grad_ws = ep.alloc_product_workspace(self.up_cfg, grad=True)
            self.down_grad_ws = ep.alloc_product_workspace(self.down_cfg, grad=True)
            self.d_y, self.d_h, self.d_rows = (torch.empty_like(t) for t in (self.y, self.h, self.y))
            self.d_weights = torch.empty(ranks, tokens, topk, device="cuda")
            self.d_logits = torch.empty(ranks * tokens, experts, **bf)
            self.ones = torch.ones_like(self.d_weights)
            self.d_up, self.d_down = torch.empty_like(self.up), torch.empty_like(self.down)

    def forward(self, x):
        """x bf16 [ranks][tokens][hidden] -> out of the same shape (and route.balance_loss)."""
        shape = (self.ranks, self.tokens, self.topk)
        self.x, self.logits = x, x.reshape(-1, self.hidden) @ self.router.t()
        ep.ep_route(self.route_cfg, self.logits, None, None, self.route, self.route_ws)
        self.idx, self.weights = self.route.topk_idx.view(shape), self.route.topk_weights.view(shape)
        ep.ep_get_dispatch_layout(self.cfg, self.idx, self.layout, self.ws)
        ep.ep_dispatch(self.cfg, self.layout, x, None, self.idx, self.weights, self.recv, self.ws)
        ep.ep_expert_product(self.up_cfg, self.layout, self.recv.recv_x, self.recv.recv_sf, self.up, None, None, self.z,
                             self.h, self.up_ws)
        ep.ep_expert_product(self.down_cfg, self.layout, self.h, None, self.down, None, None, None, self.y, self.down_ws)
        ep.ep_combine(self.back, self.layout, self.y, self.idx, self.weights, self.out, self.ws)
        return self.out

    def backward(self, d_out, d_loss):
        """Gradients of d_out . out + d_loss . balance_loss: (d_x, d_router, d_up, d_down)."""
        ep.ep_combine_grad(self.back, self.layout, self.y, self.idx, self.weights, d_out, self.d_y, self.d_weights, self.ws)
        ep.ep_expert_product_grad(self.down_cfg, self.layout, self.h, self.down, None, self.d_y, self.d_h, self.d_down,
                                  None, self.down_grad_ws)
        ep.ep_expert_product_grad(self.up_cfg, self.layout, self.recv.recv_x, self.up, self.z, self.d_h, self.d_rows,
                                  self.d_up, None, self.up_grad_ws)
        d_x = torch.empty_like(self.x)  # the dispatch's gradient: every lane's row added up
        ep.ep_combine(self.back, self.layout, self.d_rows, self.idx, self.ones, d_x, self.ws)
        ep.ep_route_grad(self.route_cfg, self.logits, None, self.route, self.d_weights.view(-1, self.topk), d_loss,
                         self.d_logits, self.route_ws)
        d_x = d_x + (self.d_logits @ self.router).view_as(d_x)
        return d_x, self.d_logits.t() @ self.x.reshape(-1, self.hidden), self.d_up, self.d_down

    def check(self):
        """First error that the device found since the last call, in the forward or the backward."""
        spaces = [self.ws, self.route_ws, self.up_ws, self.down_ws]
        if self.grad:
            spaces += [self.up_grad_ws, self.down_grad_ws]
        for ws in spaces:
            status = ep.ep_check_error(ws)
            if status != ep.EP_OK:
                return status
        return ep.EP_OK


class KeptBlock(MoELayer):
    """The layer with the norm in front of it and the residual stream around it, in FP8 where rows travel
    or wait: the norm makes the rows that the dispatch sends, they stay as they were received, of z only 8 bits
    are kept, and h is computed again. A row of an expert keeps 3 hidden + 2 inner bytes and the scales (x, y in bf16,
    z) where MoELayer keeps 4 hidden + 6 inner: 4/7 with inner = hidden / 2, half with inner = hidden.

    forward(x, residual) -> (sum, out): sum = x + residual, and out, which the next block adds to sum."""

    def __init__(self, ranks, tokens, hidden, inner, experts, topk, seed=0, score=ep.EP_SCORE_SOFTMAX):
        super().__init__(ranks, tokens, hidden, inner, experts, topk, seed, score, fp8=True)
        n, rows, bf = ranks * tokens, self.h.shape[0], dict(dtype=torch.bfloat16, device="cuda")
        self.cfg.x_dtype = ep.EP_DTYPE_FP8_E4M3  # rows come from the norm as FP8
        self.gamma = torch.ones(hidden, **bf)
        self.norm_cfg = ep.NormConfig(n, hidden)
        self.norm_ws = ep.alloc_norm_workspace(self.norm_cfg)
        self.sum, self.y_norm, self.d_x = (torch.empty(ranks, tokens, hidden, **bf) for _ in range(3))
        self.codes = torch.empty(n, hidden, dtype=torch.uint8, device="cuda")
        self.sf = torch.empty(n, hidden // 128, device="cuda")
        self.d_gamma = torch.empty(hidden, device="cuda")
        self.z_cfg = ep.CheckpointConfig(ranks, experts, rows, 2 * inner, ep.EP_ACT_SWIGLU)
        self.x_cfg = ep.CheckpointConfig(ranks, experts, rows, hidden)
        self.z_ws, self.x_ws = (ep.alloc_checkpoint_workspace(c) for c in (self.z_cfg, self.x_cfg))
        self.z_codes = torch.empty(rows, 2 * inner, dtype=torch.uint8, device="cuda")
        self.z_sf = torch.empty(rows, 2 * inner // 128, device="cuda")
        # behind the activation the up product is a plain one: d_out of 2 inner columns
        self.up_back = ep.ProductConfig(ranks, experts, rows, hidden, 2 * inner)
        self.up_grad_ws = ep.alloc_product_workspace(self.up_back, grad=True)

    def forward(self, x, residual):
        shape = (self.ranks, self.tokens, self.topk)
        ep.ep_norm(self.norm_cfg, x, residual, self.gamma, self.sum, self.y_norm, self.codes, self.sf)
        self.logits = self.y_norm.reshape(-1, self.hidden) @ self.router.t()
        ep.ep_route(self.route_cfg, self.logits, None, None, self.route, self.route_ws)
        self.idx, self.weights = self.route.topk_idx.view(shape), self.route.topk_weights.view(shape)
        ep.ep_get_dispatch_layout(self.cfg, self.idx, self.layout, self.ws)
        ep.ep_dispatch(self.cfg, self.layout, self.codes, self.sf, self.idx, self.weights, self.recv, self.ws)
        ep.ep_expert_product(self.up_cfg, self.layout, self.recv.recv_x, self.recv.recv_sf, self.up, None, None, self.z,
                             self.h, self.up_ws)
        ep.ep_checkpoint(self.z_cfg, self.layout, self.z, self.z_codes, self.z_sf, self.z_ws)
        ep.ep_expert_product(self.down_cfg, self.layout, self.h, None, self.down, None, None, None, self.y, self.down_ws)
        ep.ep_combine(self.back, self.layout, self.y, self.idx, self.weights, self.out, self.ws)
        return self.sum, self.out  # z and h may be another block's from here on

    def backward(self, d_sum, d_out, d_loss):
        """Gradients of d_sum . sum + d_out . out + d_loss . balance_loss:
        (d_x, of the residual too, d_router, d_up, d_down, d_gamma)."""
        ep.ep_combine_grad(self.back, self.layout, self.y, self.idx, self.weights, d_out, self.d_y, self.d_weights, self.ws)
        ep.ep_expert_product_grad(self.down_cfg, self.layout, None, self.down, None, self.d_y, self.d_h, None, None,
                                  self.down_grad_ws)
        ep.ep_checkpoint_grad(self.z_cfg, self.layout, self.z_codes, self.z_sf, self.d_h, self.h, self.z, None, self.z_ws)
        ep.ep_expert_product_grad(self.down_cfg, self.layout, self.h, None, None, self.d_y, None, self.d_down, None,
                                  self.down_grad_ws)
        # z now holds its gradient, and y has done its work: the rows take its place
        ep.ep_checkpoint_rows(self.x_cfg, self.layout, self.recv.recv_x, self.recv.recv_sf, self.y, self.x_ws)
        ep.ep_expert_product_grad(self.up_back, self.layout, self.y, self.up, None, self.z, self.d_rows, self.d_up, None,
                                  self.up_grad_ws)
        d_y = torch.empty_like(self.y_norm)  # of the norm's output: every lane's row added up
        ep.ep_combine(self.back, self.layout, self.d_rows, self.idx, self.ones, d_y, self.ws)
        ep.ep_route_grad(self.route_cfg, self.logits, None, self.route, self.d_weights.view(-1, self.topk), d_loss,
                         self.d_logits, self.route_ws)
        d_y = d_y + (self.d_logits @ self.router).view_as(d_y)
        ep.ep_norm_grad(self.norm_cfg, self.sum, self.gamma, None, d_y, d_sum, self.d_x, self.d_gamma, self.norm_ws)
        return (self.d_x, self.d_logits.t() @ self.y_norm.reshape(-1, self.hidden), self.d_up, self.d_down, self.d_gamma)

    def check(self):
        for ws in (self.norm_ws, self.z_ws, self.x_ws):
            status = ep.ep_check_error(ws)
            if status != ep.EP_OK:
                return status
        return super().check()


class ServingBlock:
    """A block's serving step of up to 64 tokens on one rank: norm, router, and the experts' layer, which adds
    the residual. Matrices as MoELayer's, or FP8 codes with a scale for every 128 x 128."""

    def __init__(self, tokens, router, up, down, topk, gamma=None, up_sf=None, down_sf=None, score=ep.EP_SCORE_SOFTMAX):
        experts, hidden = router.shape
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.router, self.gamma, self.hidden = router, gamma, hidden
        self.matrices = (up, up_sf, None, down, down_sf, None)
        self.norm_cfg = ep.NormConfig(tokens, hidden)
        self.route_cfg = ep.RouteConfig(1, tokens, experts, topk, ep.EP_DTYPE_BF16, score)
        self.layer_cfg = ep.LayerConfig(tokens, experts, topk, hidden, down.shape[2], weight_dtype=(
            ep.EP_DTYPE_BF16 if up_sf is None else ep.EP_DTYPE_FP8_E4M3))
        self.route, self.route_ws = ep.alloc_route(self.route_cfg, stats=False), ep.alloc_route_workspace(self.route_cfg)
        self.layer_ws = ep.alloc_layer_workspace(self.layer_cfg)
        self.sum, self.y, self.out = (torch.empty(tokens, hidden, **bf) for _ in range(3))

    def forward(self, x, residual):
        """(x + residual) + the layer of its norm; x, residual bf16 [tokens][hidden]."""
        ep.ep_norm(self.norm_cfg, x, residual, self.gamma, self.sum, self.y, None, None)
        ep.ep_route(self.route_cfg, self.y @ self.router.t(), None, None, self.route, self.route_ws)
        ep.ep_expert_layer(self.layer_cfg, self.y, self.route.topk_idx, self.route.topk_weights, *self.matrices, self.sum,
                           self.out, self.layer_ws)
        return self.out

    def check(self):
        status = ep.ep_check_error(self.route_ws)
        return status if status != ep.EP_OK else ep.ep_check_error(self.layer_ws)


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("ranks", 4), ("tokens", 256), ("hidden", 1024), ("inner", 512), ("experts", 32), ("topk", 4),
                        ("steps", 5)):
        p.add_argument(f"--{name}", type=int, default=value)
    a = p.parse_args()
    layer = MoELayer(a.ranks, a.tokens, a.hidden, a.inner, a.experts, a.topk)
    x = torch.randn(a.ranks, a.tokens, a.hidden, device="cuda").bfloat16()
    target = torch.randn_like(x)
    coefficient = torch.full((1,), 0.01, device="cuda")
    for step in range(a.steps):
        torch.cuda.synchronize()
        t = time.perf_counter()
        out = layer.forward(x)
        diff = out.float() - target.float()
        grads = layer.backward((diff * (2 / diff.numel())).bfloat16(), coefficient)
        for w, d in zip((layer.router, layer.up, layer.down), grads[1:]):
            w.sub_(d, alpha=50.0)
        torch.cuda.synchronize()
        print(f"step {step}: error {float(diff.square().mean()):.4f}  balance {float(layer.route.balance_loss):.4f}  "
              f"{(time.perf_counter() - t) * 1e3:.2f} ms")
    assert layer.check() == ep.EP_OK
    serve = MoELayer(1, 8, a.hidden, a.inner, a.experts, a.topk, fp8=a.hidden % 128 == 0, grad=False)
    y = serve.forward(x[:1, :8].contiguous())
    assert serve.check() == ep.EP_OK
    print(f"serving step of 8 tokens, FP8 rows: output rms {float(y.float().square().mean().sqrt()):.4f}")
    few = ServingBlock(8, serve.router, serve.up, serve.down, a.topk)
    y = few.forward(x[0, :8].contiguous(), torch.zeros_like(few.sum))
    assert few.check() == ep.EP_OK
    print(f"the same in one block, norm and residual with it: output rms {float(y.float().square().mean().sqrt()):.4f}")
    if a.hidden % 128 == 0 and 2 * a.inner % 128 == 0:
        block = KeptBlock(a.ranks, a.tokens, a.hidden, a.inner, a.experts, a.topk)
        total, out = block.forward(x, torch.zeros_like(x))
        diff = total.float() + out.float() - target.float()
        g = (diff * (2 / diff.numel())).bfloat16()
        grads = block.backward(g, g, coefficient)
        assert block.check() == ep.EP_OK
        print(f"training step on rows kept in 8 bits: error {float(diff.square().mean()):.4f}, "
              f"gradient of the rows {float(grads[0].float().norm()):.3e}")


if __name__ == "__main__":
    main()
