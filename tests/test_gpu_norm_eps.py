"""The norm with an eps as large as rows whose sum of squares leaves fp32: 1 / sqrt(mean s^2 + eps) counts both. (Error bounds:
test_gpu_norm.)"""
import ctypes as C

import pytest
import torch

import _block_reference as ref

HALF, ROW = ref.HALF, 40 * 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("eps", [1e-6, 1e30, 1e37, 1e38])
@pytest.mark.parametrize("rows,hidden", [(5, 512), (9, 4096), (700, 4096), (170, 16384)])
def test_large_rows_and_eps(rows, hidden, eps, kind):
    import combine_ep_get_02_gb300 as ep
    g = torch.Generator(device="cuda").manual_seed(rows)
    s = (3e18 * torch.randn(rows, hidden, generator=g, device="cuda")).to(kind)
    s[::3] *= 2.0 ** -40  # among rows whose squares fp32 holds
    assert s[1::3].float().square().sum(-1).isinf().all()
    cfg = ep.NormConfig(rows, hidden, ep.EP_DTYPE_FP32 if kind is torch.float32 else ep.EP_DTYPE_BF16, eps=eps)
    y = torch.empty(rows, hidden, dtype=torch.bfloat16, device="cuda")
    ep.ep_norm(cfg, s, None, None, None, y, None, None)
    value = cfg._c().eps  # as rounded to fp32
    want = ref.norm(s, None, None, value)[2]
    assert ((y.double() - want).abs() <= want.abs() * (HALF[torch.bfloat16] + ROW)).all()
    # gradients large enough to be normal numbers behind the division
    d_y = (1e18 * torch.randn(rows, hidden, generator=g, device="cuda")).bfloat16()
    d_x, d_w, ws = torch.empty_like(s), torch.empty(hidden, device="cuda"), ep.alloc_norm_workspace(cfg)
    ep.ep_norm_grad(cfg, s, None, None, d_y, None, d_x, d_w, ws)
    want, want_w, size, size_w = ref.norm_grad(s, None, None, d_y, None, value)
    assert ((d_x.double() - want).abs() <= want.abs() * HALF[kind] + size * 2 * ROW + 2.0 ** -133).all()
    assert ((d_w.double() - want_w).abs() <= size_w * (ROW + (rows + 32) * 2.0 ** -24)).all()
    assert ep.ep_check_error(ws) == ep.EP_OK


def test_an_eps_past_the_sums_is_refused():
    from combine_ep_get_02_gb300 import _build
    _build.build()
    import combine_ep_get_02_gb300 as ep
    ep.lib()
    for eps, code in ((1.01e38, ep.EP_ERR_INVALID_ARG), (3e38, ep.EP_ERR_INVALID_ARG), (1e38, ep.EP_OK), (1e-20, ep.EP_OK)):
        cfg = ep.NormConfig(0, 256, eps=eps)
        assert (ep.ep_norm_workspace_bytes(cfg) != 0) == (code == ep.EP_OK)
        assert ep.lib().ep_norm(C.byref(cfg._c()), *[None] * 8) == code
