"""The backward pass through SiLU and the gated activation for gates of 2^7 to 2^100, of either sign.

Kept in 8 bits they are 120 or more. There the sigmoid is 1, or below 2^-173: the derivative is 1 within 120 e^-120, or
nothing that bf16 and fp32 hold. So d_z
is d_h, or d_h times the other half, of which the kernel rounds one product to fp32 (2^-24) and once to bf16
(2^-8, half a step); negative gates get 0 (of the smallest numbers of bf16, 2^-133, less than one half)."""
import pytest
import torch

import _block_reference as ref
from test_gpu_checkpoint import blocks_of

pytestmark = pytest.mark.gpu
HALF, FP32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module")
def ep():
    import combine_ep_get_02_gb300 as ep
    ep.lib()
    return ep


def gates(rows, g):
    """A row's groups of 128 columns have values of one power of two each, from 2^7 to 2^100."""
    powers = list(range(7, 100, 4)) + [23, 24, 25, 26, 100]
    size = torch.exp2(torch.tensor(powers, dtype=torch.float64, device="cuda")).repeat_interleave(128)
    x = (1 + torch.rand(rows, len(size), generator=g, device="cuda")).double() * size
    return (x * torch.where(torch.rand(x.shape, generator=g, device="cuda") < 0.5, -1.0, 1.0)).float()


@pytest.mark.parametrize("counts", [[70, 0, 3], [4000, 1]])
@pytest.mark.parametrize("packed", [False, True], ids=["fp32sf", "packed"])
@pytest.mark.parametrize("kind", ["silu", "swiglu"])
def test_far_gates(ep, kind, packed, counts):
    lay, blocks, rows = blocks_of(ep, counts, 1)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = gates(rows, g)
    n = x.shape[1]
    if kind == "swiglu":
        x = torch.cat([x, torch.randn(rows, n, generator=g, device="cuda")], 1)
    codes, sf = ref.cast(x, packed)
    z = ref.values(codes, sf, packed).float().double()  # the product of code and scale is rounded to fp32
    up, other = z[:, :n] > 0, z[:, n:] if kind == "swiglu" else torch.ones_like(z)
    assert z[:, :n].abs().min() >= 2 ** 7 * (1 - 2 ** -4)
    d_h = torch.randn(rows, n, generator=g, device="cuda").bfloat16()
    cfg = ep.CheckpointConfig(1, len(counts), rows, x.shape[1], getattr(ep, f"EP_ACT_{kind.upper()}"), int(packed))
    ws = ep.alloc_checkpoint_workspace(cfg)
    h, d_z = torch.empty_like(d_h), torch.empty(rows, x.shape[1], dtype=torch.bfloat16, device="cuda")
    d_bias = torch.empty(len(counts), x.shape[1], device="cuda")
    ep.ep_checkpoint_grad(cfg, lay, codes, sf, d_h, h, d_z, d_bias, ws)
    d, zero = d_h.double(), torch.zeros_like(d_h).double()
    want_h = torch.where(up, z[:, :n] * other, zero)
    want_z = torch.where(up, d * other, zero)
    if kind == "swiglu":
        want_z = torch.cat([want_z, torch.where(up, d * z[:, :n], zero)], 1)
    near = lambda got, want: ((got.double() - want).abs() <= want.abs() * (HALF + 2 * FP32) + 2.0 ** -133).all()  # noqa: E731
    assert near(h, want_h) and near(d_z, want_z)
    for e, (a, c) in enumerate(blocks):  # terms off by FP32, at most c + 16 additions
        part = want_z[a:a + c]
        assert ((d_bias[e].double() - part.sum(0)).abs() <= part.abs().sum(0) * (c + 18) * FP32 + c * 2.0 ** -133).all()
    assert ep.ep_check_error(ws) == ep.EP_OK


def test_same_gradient_as_of_bf16_rows(ep):
    """Gates that 8 bits hold exactly: the gradient from the kept rows is the products' own gradient, d_bias too (the
    weight's factor is the identity, so ep_expert_product_grad's d_x is d_z)."""
    rows, n = 96, 256
    sign = torch.where(torch.arange(n, device="cuda") % 3 == 0, -1.0, 1.0)
    z = (torch.exp2(torch.arange(rows, device="cuda") % 48 + 7.0)[:, None] * sign).contiguous()
    codes, sf = ref.cast(z, True)
    assert torch.equal(ref.values(codes, sf, True), z.double())
    d_h = torch.randn(rows, n, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    cfg = ep.CheckpointConfig(1, 1, rows, n, ep.EP_ACT_SILU, 1)
    d_z, d_b, far_b = torch.empty_like(d_h), torch.empty(1, n, device="cuda"), torch.empty(1, n, device="cuda")
    ep.ep_checkpoint_grad(cfg, None, codes, sf, d_h, None, d_z, d_b, ep.alloc_checkpoint_workspace(cfg))
    product = ep.ProductConfig(1, 1, rows, n, n, ep.EP_ACT_SILU)
    one = torch.eye(n, device="cuda").bfloat16()[None].contiguous()
    d_x = torch.empty_like(d_h)
    ep.ep_expert_product_grad(product, None, None, one, z.bfloat16(), d_h, d_x, None, far_b,
                              ep.alloc_product_workspace(product, grad=True))
    assert torch.equal(d_z, d_x)
    assert ((d_b - far_b).abs() <= d_h.float().abs().sum(0) * (rows + 16) * FP32).all()
