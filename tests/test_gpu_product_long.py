"""Matrix gradients that are sums over so many rows that a tile takes seconds: the waits of the
kernel's other warps last as long (here 4.4 seconds)."""
import pytest
import torch

import combine_ep_get_02_gb300 as ep

pytestmark = pytest.mark.gpu


def test_a_billion_rows():
    """One pair of SMs: a group of 2^30 rows, then one of 5, whose tile is the only one that ends inside
    an instruction's 16 rows. A few rows are not zero, so the sums are exact to one rounding."""
    rows, K, N = 2 ** 30 + 5, 8, 8
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    d_out = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    some = torch.tensor([0, 1, 12345, 2 ** 29 + 77, 2 ** 30 - 1] + list(range(2 ** 30, rows)), device="cuda")
    for t in (x, d_out):
        t[some] = torch.randn(len(some), 8, device="cuda", generator=g).bfloat16()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    lay = ep.Layout(*[None] * 6, i32(2 ** 30, 5), i32(0, 2 ** 30, rows), i32(0, rows))
    cfg = ep.ProductConfig(1, 2, rows, K, N, num_sms=2)
    ws = ep.alloc_product_workspace(cfg, grad=True)
    dw = torch.full((2, N, K), 33.0, device="cuda").bfloat16()
    ep.ep_expert_product_grad(cfg, lay, x, None, None, d_out, None, dw, None, ws)
    assert ep.ep_check_error(ws) == ep.EP_OK
    for i, at in enumerate((some[:5], some[5:])):
        want = d_out[at].double().T @ x[at].double()
        size = d_out[at].double().abs().T @ x[at].double().abs()
        assert ((dw[i].double() - want).abs() <= 2 ** -8 * want.abs() + 2 ** -20 * size).all()
