"""A call on one SM, whose first kernel takes longer than any wait inside a kernel may."""
import pytest
import torch

import combine_ep_get_02_gb300 as ep

pytestmark = pytest.mark.gpu


def test_first_kernel_of_seconds():
    """All 64 tokens choose all of 8 experts, whose FP8 matrices are zeros: the output is the residual. 32 groups of 16 tokens
    read up matrices of 3.2 GB each, 103 GB through one SM: 3.1 s."""
    T, E, H, I = 64, 8, 8192, 1536 * 128
    cfg = ep.LayerConfig(T, E, E, H, I, weight_dtype=ep.EP_DTYPE_FP8_E4M3, num_sms=1)
    up, down = (torch.zeros(E, *s, dtype=torch.uint8, device="cuda") for s in ((2 * I, H), (H, I)))
    up_sf, down_sf = torch.ones(E, 2 * I // 128, H // 128, device="cuda"), torch.ones(E, H // 128, I // 128, device="cuda")
    x = torch.randn(T, H, device="cuda").bfloat16()
    idx = torch.arange(E, device="cuda").repeat(T, 1)
    w, out, ws = torch.ones(T, E, device="cuda"), torch.empty_like(x), ep.alloc_layer_workspace(cfg)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    ep.ep_expert_layer(cfg, x, idx, w, up, up_sf, None, down, down_sf, None, x, out, ws)
    end.record()
    assert ep.ep_check_error(ws) == ep.EP_OK and torch.equal(out, x)
    # two thirds of it are the first kernel's; a wait gives up after two seconds
    assert start.elapsed_time(end) > 3300, start.elapsed_time(end)
