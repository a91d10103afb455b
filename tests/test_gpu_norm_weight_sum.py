"""d_weight of the norm's gradient where the order of the last sum shows: one row's term is 1, every other's just below
2^-24, half a step of 1, so a chain that adds them to it one by one loses them all.

The rows are as many as the CTAs, one each, of ones, so n = 1 exactly (eps = 1e-20 does not reach 1) and every partial sum is
its row's d_y. Their sum in pairs, of at most 608 partial sums, is off by at most 10 roundings of 2^-24 of the sum of
magnitudes; 12 are allowed. A chain of every eighth of 304 lost 37 of these terms."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("hidden", [256, 2048, 4096, 16384])
@pytest.mark.parametrize("large", [0, 5])
def test_small_terms_beside_a_large_one(hidden, kind, large):
    import combine_ep_get_02_gb300 as ep
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for rows in (sms, 2 * sms, 4 * sms):
        cfg = ep.NormConfig(rows, hidden, ep.EP_DTYPE_FP32 if kind is torch.float32 else ep.EP_DTYPE_BF16, eps=1e-20)
        ws, d_w = ep.alloc_norm_workspace(cfg), torch.empty(hidden, device="cuda")
        s = torch.ones(rows, hidden, dtype=kind, device="cuda")
        d_y = torch.full((rows, hidden), 2.0 ** -24 * (1 - 2.0 ** -8), device="cuda").bfloat16()
        d_y[large] = 1.0
        ep.ep_norm_grad(cfg, s, None, None, d_y, None, None, d_w, ws)
        want = d_y.double().sum(0)
        assert ((d_w.double() - want).abs() <= want * 12 * 2.0 ** -24).all(), ((d_w.double() - want).abs().max() * 2 ** 24)
        first = d_w.clone()
        ep.ep_norm_grad(cfg, s, None, None, d_y, None, None, d_w, ws)
        assert torch.equal(d_w, first) and ep.ep_check_error(ws) == ep.EP_OK
