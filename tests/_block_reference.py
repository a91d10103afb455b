"""Definitions of the norm, of FP8 rows and of the backward pass through kept rows, in 64 bits (the
cast, which is defined in fp32, in fp32), in plain torch operations."""
from __future__ import annotations

import torch

from _moe_reference import act

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative


def norm(x, residual, weight, eps):
    """(s, q, y)"""
    s = x.double() + (0 if residual is None else residual.double())
    q = 1 / torch.sqrt(s.square().mean(-1, keepdim=True) + eps)
    y = s * q
    return s, q, y if weight is None else y * weight.double()


def norm_grad(s, weight, mask, d_y, d_sum, eps):
    """(d_x, d_weight) and, for error bounds, the sums of the magnitudes of what each is a sum of."""
    live = 1.0 if mask is None else (mask != 0).double()[:, None]
    clean = lambda t: torch.where(torch.as_tensor(live, device=t.device) != 0, t.double(), 0.0)  # noqa: E731
    s, d_y = clean(s), clean(d_y)
    q = 1 / torch.sqrt(s.square().mean(-1, keepdim=True) + eps)
    n, t = s * q, d_y if weight is None else d_y * weight.double()
    d = q * (t - n * (t * n).mean(-1, keepdim=True))
    size = q * (t.abs() + n.abs() * (t * n).abs().mean(-1, keepdim=True))
    if d_sum is not None:
        d, size = d + clean(d_sum), size + clean(d_sum).abs()
    return d * live, (d_y * n).sum(0), size, (d_y * n).abs().sum(0)


def cast(x, packed):
    """FP8 rows of bf16 or fp32 rows, as the dispatch's cast is defined: (codes uint8, sf fp32 words)."""
    v = x.float().reshape(x.shape[0], x.shape[1] // 128, 128)
    amax = v.abs().amax(-1).clamp(min=1e-4)
    if packed:
        m, e = torch.frexp(amax.double() / 448)
        e = torch.where(m > 0.5, e, e - 1)
        inv = torch.exp2(-e.double()).float()
        sf = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, -e.shape[1] % 4)).view(torch.float32)
    else:
        # IEEE quotients: by way of 64 bits, as torch divides by a number with its reciprocal
        inv, sf = (448 / amax.double()).float(), (amax.double() / 448).float()
    return (v * inv[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(x.shape), sf


def scales(sf, features, packed):
    """fp32 scale of every column."""
    if packed:
        sf = torch.exp2(sf.view(torch.uint8)[:, :features // 128].double() - 127).float()
    return sf.repeat_interleave(128, 1)


def values(codes, sf, packed):
    """What FP8 rows stand for (64 bits)."""
    return codes.view(torch.float8_e4m3fn).double() * scales(sf, codes.shape[1], packed).double()


def checkpoint_grad(blocks, z, d_h, kind):
    """blocks: (begin, count) per group; z, d_h in 64 bits -> (h, d_z, d_bias), rows of no group NaN."""
    h = torch.full_like(d_h, torch.nan)
    d_z = torch.full_like(z, torch.nan)
    d_bias = torch.zeros(len(blocks), z.shape[1], dtype=torch.float64, device=z.device)
    for g, (a, c) in enumerate(blocks):
        t = z[a:a + c].clone().requires_grad_(True)
        with torch.enable_grad():
            v = act(t, kind)
        (d,) = torch.autograd.grad(v, t, d_h[a:a + c])
        h[a:a + c], d_z[a:a + c], d_bias[g] = v.detach(), d, d.sum(0)
    return h, d_z, d_bias
