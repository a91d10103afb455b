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


def unscale(codes, sf):
    """Matrices of e4m3 codes [E][rows][columns] with a scale for every 128 x 128, in 64 bits."""
    v = codes.view(torch.float8_e4m3fn).double()
    return v * sf.double().repeat_interleave(128, 1)[:, :v.shape[1]].repeat_interleave(128, 2)


def layer(x, idx, w, up, up_bias, down, down_bias, residual, kind, fun):
    """The experts' layer with h rounded to bf16 as defined -> (out, bound of its error before the last rounding).

    Products are exact; a sum of n of them passes through at most n / 128 + 24 additions, of 2^-22 of the sum of
    magnitudes each (the tensor cores cut what they add at 2^-23 of the largest). h of fp32 sums
    lies within such an error, and `fun` for the activation, of h of 64 bits, so its rounding lies
    between the roundings of both ends. Up to 4 tokens h is the sum of two bf16: what the first is off, 2^-8 of h at
    most, the second holds up to 2^-8 of that."""
    T, H = x.shape
    out, bound = (torch.zeros(T, H, dtype=torch.float64, device=x.device) for _ in range(2))
    if residual is not None:
        out += residual.double()
        bound += residual.double().abs() * 2.0 ** -22
    x = x.double()
    for e in torch.unique(idx[(idx >= 0) & (idx < len(up))]).tolist():
        t, k = torch.nonzero(idx == e, as_tuple=True)
        u, d, xe, we = up[e].double(), down[e].double(), x[t], w[t, k].double()[:, None]
        z = xe @ u.T + (0 if up_bias is None else up_bias[e].double())
        ez = (xe.abs() @ u.abs().T) * ((x.shape[1] / 128 + 24) * 2.0 ** -22) + z.abs() * 2.0 ** -23
        h = act(z, kind)
        if kind == "swiglu":
            (a, b), (ea, eb) = z.chunk(2, -1), ez.chunk(2, -1)
            eh = 1.11 * ea * (b.abs() + eb) + torch.nn.functional.silu(a).abs() * eb + a.abs() * b.abs() * fun
        else:
            eh = 1.13 * ez + z.abs() * fun
        low, high = (h - eh).bfloat16().double(), (h + eh).bfloat16().double()
        if T <= 4:
            low, high = h - eh - h.abs() * 2.0 ** -16, h + eh + h.abs() * 2.0 ** -16
        mid = (low + high) / 2
        y = mid @ d.T + (0 if down_bias is None else down_bias[e].double())
        size = mid.abs() @ d.abs().T
        ey = (high - low) / 2 @ d.abs().T + size * ((d.shape[1] / 128 + 24) * 2.0 ** -22) + y.abs() * 2.0 ** -23
        out.index_add_(0, t, we * y)
        bound.index_add_(0, t, we.abs() * (ey + y.abs() * (idx.shape[1] + 8) * 2.0 ** -22))
    return out, bound
