"""Definitions of the router, the combine's gradient and the experts' products in 64
bits, in plain torch operations on the CPU or the GPU."""
from __future__ import annotations

import math

import torch


def order(scores, n):
    """Indices of the n largest of the last dimension, ties to the lowest."""
    return torch.sort(scores, dim=-1, descending=True, stable=True)[1][..., :n]


def route(logits, bias, mask, B, T, K, score="softmax", G=1, keep=1, normalize=True, scale=1.0, choice=None):
    """(idx, weights, count, prob_sum, valid, loss). The choice is made on fp32 scores, as
    defined (`choice` overrides them); what follows is in 64 bits. NaN and +inf logits are -inf."""
    N, E = logits.shape
    l = logits.double()
    l = torch.where(l < math.inf, l, -math.inf)
    s = torch.softmax(l, -1).nan_to_num(0.0) if score == "softmax" else torch.sigmoid(l)
    if choice is None:
        base = l.float() if score == "softmax" else (1.0 / (1.0 + torch.exp(-l.float())))
        choice = base if bias is None else base + bias.float()
    choice = torch.where((choice < math.inf) & (l > -math.inf), choice + 0.0, -math.inf)  # -0 is +0
    if G > 1:
        grouped = choice.reshape(N, G, E // G)
        two = torch.sort(grouped, dim=-1, descending=True)[0][..., :2]
        kept = order(two[..., 0] + two[..., 1], keep)
        off = torch.ones(N, G, dtype=torch.bool, device=l.device).scatter_(1, kept, False)
        choice = grouped.masked_fill(off[..., None], -math.inf).reshape(N, E)
    idx = order(choice, K)
    live = (torch.ones(N, dtype=torch.bool, device=l.device) if mask is None else mask != 0)[:, None]
    idx = torch.where((choice.gather(1, idx) > -math.inf) & live, idx, -1)
    w = torch.where(idx >= 0, s.gather(1, idx.clamp(min=0)), 0.0)
    if normalize:
        if score == "softmax":  # the softmax of the chosen logits
            lk = torch.where(idx >= 0, l.gather(1, idx.clamp(min=0)), -math.inf)
            w = torch.softmax(lk, -1).nan_to_num(0.0)
        else:
            w = w / w.sum(-1, keepdim=True).clamp(min=1e-30)
    w = w * scale
    total = s.sum(-1, keepdim=True)
    p = torch.where(live & (total > 0), s / total.clamp(min=1e-300), 0.0)
    count = torch.zeros(B, E, dtype=torch.int64, device=l.device)
    seg = (torch.arange(N, device=l.device) // max(T, 1))[:, None].expand_as(idx)
    on = idx >= 0
    count.view(-1).index_add_(0, (seg * E + idx.clamp(min=0))[on], torch.ones_like(idx[on]))
    valid = live.reshape(B, T).sum(1) if T else torch.zeros(B, dtype=torch.int64, device=l.device)
    psum = p.reshape(B, T, E).sum(1)
    n = valid.clamp(min=1).double()[:, None]
    loss = ((E * count / (K * n)) * (psum / n)).sum(1).mean()
    return idx, w, count, psum, valid, loss


def route_objective(logits, idx, count, valid, mask, d_weights, d_loss, B, T, K, score, normalize, scale):
    """sum(weights * d_weights) + loss * d_loss for a fixed choice and fixed counts (64 bits)."""
    N, E = logits.shape
    live = (torch.ones(N, dtype=torch.bool, device=logits.device) if mask is None else mask != 0)[:, None]
    s = torch.softmax(logits, -1) if score == "softmax" else torch.sigmoid(logits)
    sel = torch.where(idx >= 0, s.gather(1, idx.clamp(min=0)), 0.0)
    w = sel / sel.sum(-1, keepdim=True).clamp(min=1e-300) if normalize else sel
    p = torch.where(live, s / s.sum(-1, keepdim=True), 0.0)
    n = valid.clamp(min=1).double()[:, None]
    loss = ((E * count / (K * n)) * (p.reshape(B, T, E).sum(1) / n)).sum(1).mean()
    return (torch.where(live, w, 0.0) * scale * d_weights).sum() + loss * d_loss


def combine_grad(row, w, y, d_out):
    """row [N, K] (-1: none), w [N, K], y [rows, H], d_out [N, H] -> (d_y, d_w)."""
    y, g, w = y.double(), d_out.double(), w.double()
    d_w = torch.zeros_like(w)
    d_y = torch.zeros_like(y)
    for k in range(row.shape[1]):
        on = row[:, k] >= 0
        d_w[on, k] = (y[row[on, k]] * g[on]).sum(-1)
        d_y.index_add_(0, row[on, k], w[on, k, None] * g[on])
    return d_y, d_w


def act(z, kind):
    F = torch.nn.functional
    if kind == "swiglu":
        a, b = z.chunk(2, -1)
        return F.silu(a) * b
    return {"none": lambda t: t * 1, "relu": F.relu, "silu": F.silu, "gelu": F.gelu}[kind](z)


def product(blocks, x, weight, bias, residual, kind):
    """blocks: (begin, count) per group -> (out, z), rows of no group NaN."""
    rows = x.shape[0]
    n = weight.shape[1] // (2 if kind == "swiglu" else 1)
    z = torch.full((rows, weight.shape[1]), math.nan, dtype=torch.float64, device=x.device)
    out = torch.full((rows, n), math.nan, dtype=torch.float64, device=x.device)
    for g, (a, c) in enumerate(blocks):
        t = x[a:a + c].double() @ weight[g].double().T
        if bias is not None:
            t = t + bias[g].double()
        z[a:a + c] = t
        out[a:a + c] = act(t, kind) + (residual[a:a + c].double() if residual is not None else 0.0)
    return out, z


def product_grad(blocks, x, weight, z, d_out, kind):
    """-> (d_x, d_weight, d_bias), rows of no group NaN in d_x."""
    d_x = torch.full(x.shape, math.nan, dtype=torch.float64, device=x.device)
    d_w = torch.zeros(weight.shape, dtype=torch.float64, device=x.device)
    d_b = torch.zeros(weight.shape[:2], dtype=torch.float64, device=x.device)
    for g, (a, c) in enumerate(blocks):
        t = z[a:a + c].double().requires_grad_(True)
        with torch.enable_grad():
            (dz,) = torch.autograd.grad(act(t, kind), t, d_out[a:a + c].double())
        d_x[a:a + c] = dz @ weight[g].double()
        d_w[g] = dz.T @ x[a:a + c].double()
        d_b[g] = dz.sum(0)
    return d_x, d_w, d_b
