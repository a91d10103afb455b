"""A token's result from a call of its own, and among others: sums are taken in other orders, so both are compared with 64 bits."""
import pytest
import torch

import _block_reference as ref
import combine_ep_get_02_gb300 as ep
from test_gpu_checkpoint import FUN
from test_gpu_layer import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("T,E,K,H,I", [(4, 8, 3, 640, 384), (8, 4, 2, 256, 128), (33, 16, 4, 1024, 256)])
def test_alone_and_among_others(T, E, K, H, I, fp8):
    c = Case(ep, T, E, K, H, I, fp8=fp8, bias=True, residual=True, masked=0.1)
    out = c.check()
    up, down = c.mats["up"], c.mats["down"]
    wide = [ref.unscale(m[0], m[1]) if fp8 else m[0] for m in (up, down)]
    cfg = ep.LayerConfig(1, E, K, H, I, weight_dtype=c.cfg.weight_dtype)
    ws, alone = ep.alloc_layer_workspace(cfg), torch.empty(1, H, dtype=torch.bfloat16, device="cuda")
    c.x[~(c.idx >= 0).any(1)] = 0  # poisoned with NaN, which no token without an expert reads
    for t in range(T):
        x, idx, w, r = (v[t:t + 1].contiguous() for v in (c.x, c.idx, c.w, c.residual))
        ep.ep_expert_layer(cfg, x, idx, w, up[0], up[1], up[2], down[0], down[1], down[2], r, alone, ws)
        want, bound = ref.layer(x, idx, w, wide[0], up[2], wide[1], down[2], r, c.act, FUN)
        near = lambda v: ((v.double() - want).abs() <= want.abs() * 2.0 ** -8 + bound * (1 + 2.0 ** -7)).all()  # noqa: E731
        assert near(alone)
        if T <= 4:  # h is kept alike
            assert near(out[t:t + 1])
    assert ep.ep_check_error(ws) == ep.EP_OK
