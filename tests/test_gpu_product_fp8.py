"""Products of dispatched FP8 rows with fp32 scales: nothing is rounded before the results are."""
import pytest
import torch

import _moe_reference as ref
import combine_ep_get_02_gb300 as ep
from test_gpu_product import ACTS, Case

pytestmark = pytest.mark.gpu

SHAPES = {
    "one_row": dict(counts=[1], K=7168, N=256, act="swiglu", dense=True),
    "one_row_few_columns": dict(counts=[1], K=2048, N=72, dense=True),
    "rows_of_a_step": dict(counts=[90], K=2176, N=1104, act="silu", dense=True, bias=True, residual=True),
    "split_wide": dict(counts=[3], K=1152, N=4096, act="relu", dense=True, bias=True),
    "split_groups": dict(counts=[5, 0, 20], K=1152, N=200, act="gelu", bias=True, residual=True),
    "split_gated_groups": dict(counts=[2, 8, 1, 5, 16, 3, 9, 32], K=1024, N=640, R=2, act="swiglu", bias=True),
    "uneven_parts": dict(counts=[7], K=128 * 11, N=136, dense=True),
    "one_scale": dict(counts=[33, 0, 150, 64], K=128, N=200, R=2, act="swiglu", spare=17),
    "short_groups": dict(counts=[(i * 13) % 61 for i in range(24)], K=384, N=1000, act="swiglu", bias=True),
    "short_groups_tall": dict(counts=[300, 129, 128, 1], K=640, N=328, act="none", bias=True, residual=True),
    "many_experts": dict(counts=[(i * 7) % 5 for i in range(600)], K=128, N=16, R=4, act="gelu", bias=True),
    "pairs": dict(counts=[700, 257, 900], K=896, N=264, act="gelu", bias=True, residual=True),
    "pairs_gated": dict(counts=[1000, 0, 513, 400], K=384, N=200, act="swiglu", R=2, align=8, bias=True),
    "pairs_none": dict(counts=[1003], K=1024, N=776, dense=True),
    "pairs_wide": dict(counts=[2000], K=256, N=2048, dense=True, act="relu"),
}


def fp8(case, seed=3):
    """The case's x as codes and scales; scales of a row differ by factors of a hundred."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    G = case.K // 128
    x = case.x.float().nan_to_num(0.0).reshape(case.rows, G, 128)
    spread = torch.exp(torch.randn(case.rows, G, 1, device="cuda", generator=g) * 1.5)
    sf = x.abs().amax(-1, keepdim=True).clamp(min=1e-4) / 448
    codes = (x / sf).reshape(case.rows, case.K).to(torch.float8_e4m3fn)
    sf = (sf * spread)[..., 0].contiguous()
    codes.view(torch.uint8)[~case.live] = 0x7F  # NaN
    return codes, sf, codes.double() * sf.double().repeat_interleave(128, 1)


def make(name, **kw):
    case = Case(**SHAPES[name])
    cfg = ep.ProductConfig(SHAPES[name].get("R", 1), case.E, case.rows, case.K, case.N, ACTS[case.act],
                           ep.EP_DTYPE_FP8_E4M3, **kw)
    return case, cfg, fp8(case)


@pytest.mark.parametrize("name", SHAPES)
def test_only_the_results_are_rounded(name):
    case, cfg, (codes, sf, x) = make(name)
    out, z = case.forward(codes, sf, cfg=cfg)
    want, want_z = ref.product(case.blocks, x, case.w, case.bias, case.res, case.act)
    size = ref.product(case.blocks, x.abs(), case.w.abs(), None if case.bias is None else case.bias.abs(), None, "none")[1]
    m = case.live
    # one rounding to bf16; fp32 sums are off by 2^-20 of their terms' sizes at the very most
    slack = 2 ** -20 * size
    off = (z[m].double() - want_z[m]).abs() - 2 ** -8 * want_z[m].abs() - slack[m]
    assert float(off.max()) <= 0, (float(off.max()), int((off > 0).sum()))
    if case.act == "swiglu":  # |d silu(a) b| <= 1.1 |b| da + |silu(a)| db
        a, b = want_z.chunk(2, -1)
        sa, sb = slack.chunk(2, -1)
        slack = 1.1 * b.abs() * sa + a.abs() * sb
    else:
        slack = 1.2 * slack  # the largest slope of the others
    # the activation's own error: a few units of 2^-23 of its argument
    own = 2 ** -20 * (want_z.abs().amax(-1, keepdim=True) + 1) ** (2 if case.act == "swiglu" else 1)
    off = (out[m].double() - want[m]).abs() - 2 ** -8 * want[m].abs() - slack[m] - own[m]
    assert float(off.max()) <= 0, (float(off.max()), int((off > 0).sum()))


@pytest.mark.parametrize("sms", [1, 2, 5, 40, 100])
@pytest.mark.parametrize("name", SHAPES)
def test_results_do_not_depend_on_the_sms(name, sms):
    case, cfg, (codes, sf, _) = make(name)
    _, few, _ = make(name, num_sms=sms)
    for a, b in zip(case.forward(codes, sf, cfg=cfg), case.forward(codes, sf, cfg=few)):
        assert torch.equal(a[case.live], b[case.live])
