"""Layouts that belong to no configuration: blocks that overlap, and numbers of any kind. Nothing is
written outside the tensors and the workspace, and the caller is told."""
import pytest
import torch

import combine_ep_get_02_gb300 as ep

pytestmark = pytest.mark.gpu

K, N, GUARD = 72, 136, 1 << 16


def run(counts, base, region, rows, act, R):
    """Forward and every gradient with each output and the workspace in front of a guard; the statuses."""
    i32 = lambda t: t.to(torch.int32).cuda().contiguous()  # noqa: E731
    lay = ep.Layout(*[None] * 6, i32(counts), i32(base), i32(region))
    E = counts.numel()
    cfg = ep.ProductConfig(R, E, rows, K, N, act)
    Z = cfg.z_features
    rnd = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    x, w, z, d_out = rnd(rows, K), rnd(E, Z, K), rnd(rows, Z), rnd(rows, N)
    guards = []

    def behind(*shape, dtype=torch.bfloat16):
        n = torch.Size(shape).numel()
        whole = torch.full((n + GUARD,), 33, dtype=dtype, device="cuda")
        guards.append(whole[n:])
        return whole[:n].view(shape)

    def workspace(grad):
        ws = behind(ep.ep_product_workspace_bytes(cfg, grad), dtype=torch.uint8)
        ws[:256] = 0
        return ws

    status = []
    ws = workspace(False)
    ep.ep_expert_product(cfg, lay, x, None, w, None, None, behind(rows, Z), behind(rows, N), ws)
    status.append(ep.ep_check_error(ws))
    ws = workspace(True)
    ep.ep_expert_product_grad(cfg, lay, x, w, z, d_out, behind(rows, K), behind(E, Z, K), behind(E, Z, dtype=torch.float32), ws)
    status.append(ep.ep_check_error(ws))
    for g in guards:
        assert (g == 33).all()
    return status


@pytest.mark.parametrize("act", [ep.EP_ACT_NONE, ep.EP_ACT_SWIGLU])
@pytest.mark.parametrize("E,rows", [(8, 100), (8, 1000), (300, 64), (4096, 300)])
def test_every_block_claims_every_row(E, rows, act):
    R = 4
    status = run(torch.full((R, E // R), rows), torch.zeros(R, E // R + 1), torch.zeros(R + 1), rows, act, R)
    # blocks that lie apart have at most this many tiles (128 rows high, 64 in the gradient)
    for tile, st in zip((128, 64), status):
        needed, most = E * -(-rows // tile), rows // tile + min(E, rows)
        assert st == (ep.EP_ERR_OVERFLOW if needed > most else ep.EP_OK)


@pytest.mark.parametrize("seed", range(6))
def test_any_numbers(seed):
    g = torch.Generator().manual_seed(seed)
    R, E, rows = 4, 64, 500
    high = (600, 2 ** 31 - 1)[seed % 2]
    num = lambda *s: torch.randint(-high, high, s, generator=g)  # noqa: E731
    status = run(num(R, E // R), num(R, E // R + 1), num(R + 1), rows, (ep.EP_ACT_RELU, ep.EP_ACT_SWIGLU)[seed % 2], R)
    assert status == [ep.EP_ERR_OVERFLOW] * 2
