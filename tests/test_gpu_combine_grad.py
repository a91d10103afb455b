"""The combine's gradient against its 64-bit definition, on every receive layout."""
import numpy as np
import pytest
import torch

import _moe_reference as ref
import combine_ep_get_02_gb300 as ep
import oracle
import workloads as W
from _harness import GpuRun

pytestmark = pytest.mark.gpu

BASE = W.Workload("g", 1, 4, 16, 4, 30, 37, 512, routing="zipf", mask_frac=0.1)
CASES = {
    "rows": BASE,
    "rows_hidden8": BASE.replace(hidden=8),
    "rows_one_token": BASE.replace(num_tokens=1, num_max_tokens_per_rank=1, mask_frac=0.0),
    "rows_all_masked": BASE.replace(mask_frac=1.0),
    "rows_one_rank": BASE.replace(n_su=1, num_experts=8),  # every lane of a token shares one row
    "rows_k12": BASE.replace(num_topk=12, hidden=1000),
    "rows_k32": BASE.replace(num_topk=32, num_experts=64, hidden=264),
    "hybrid": BASE.replace(n_so=2, n_su=4, num_experts=32),
    "compact": BASE.replace(compact=1),
    "packed": BASE.replace(compact=2, hidden=7168, num_tokens=9),
    "expanded": BASE.replace(expand=True),
    "expanded_aligned": BASE.replace(expand=True, expert_alignment=16, hidden=2056),
    "expanded_k32": BASE.replace(expand=True, num_topk=32, num_experts=64, hidden=64),
    "expanded_many": BASE.replace(expand=True, num_tokens=900, num_max_tokens_per_rank=900, hidden=256),
}


@pytest.mark.parametrize("name", CASES)
def test_combine_grad(name):
    wl = CASES[name]
    idx, w = W.routing(wl)
    x, _ = W.hidden(wl)
    run = GpuRun(wl, idx, w, x, None).layout()
    st, olay = oracle.layout(wl, idx)
    assert st == 0
    row = torch.from_numpy(oracle.global_rows(wl, olay, idx)).reshape(-1, wl.num_topk).long().cuda()
    rows = ep.ep_recv_rows(run.cfg)
    y = W.expert_outputs(wl, rows, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    d_out = torch.randn(wl.num_ranks, wl.num_tokens, wl.hidden, device="cuda", generator=g).bfloat16()
    used = torch.zeros(rows, dtype=torch.bool, device="cuda")
    used[row[row >= 0]] = True
    y[~used] = float("nan")  # rows that no lane reads
    d_y = torch.full_like(y, 55.0)
    d_w = torch.full(w.shape, 55.0, device="cuda")
    ep.ep_combine_grad(run.cfg, run.lay, y, run.idx, run.w, d_out, d_y, d_w, run.ws)
    assert run.status() == ep.EP_OK
    want_y, want_w = ref.combine_grad(row, run.w.reshape(-1, wl.num_topk), torch.where(used[:, None], y, 0.0),
                                      d_out.reshape(-1, wl.hidden))
    # H products of N(0,1) numbers in fp32: an error of sqrt(H) * H^0.5 * 2^-24 at the very most per lane of 8
    tol = 2 ** -24 * 8 * wl.hidden ** 0.5 + 1e-6
    assert float((d_w.double().reshape(want_w.shape) - want_w).abs().max()) <= tol * 4
    # one fp32 product (and the fp32 sum of at most K weights), rounded once to bf16
    got = d_y[used].double()
    assert ((got - want_y[used]).abs() <= want_y[used].abs() * 2 ** -8 + 1e-30).all()
    assert (d_y[~used] == 55.0).all()

    # each output alone; y is not needed for d_y
    one = torch.full_like(d_y, 55.0)
    ep.ep_combine_grad(run.cfg, run.lay, None, run.idx, run.w, d_out, one, None, run.ws)
    assert torch.equal(one, d_y)
    alone = torch.full_like(d_w, 55.0)
    ep.ep_combine_grad(run.cfg, run.lay, y, run.idx, run.w, d_out, None, alone, run.ws)
    assert torch.equal(alone, d_w)
    assert run.status() == ep.EP_OK


def test_against_differences_of_combine():
    """The combine is linear in y and in the weights: its change equals the gradient's prediction."""
    wl = CASES["expanded"].replace(mask_frac=0.0)
    idx, w = W.routing(wl)
    x, _ = W.hidden(wl)
    run = GpuRun(wl, idx, w, x, None).layout()
    rows = ep.ep_recv_rows(run.cfg)
    y = W.expert_outputs(wl, rows, device="cuda")
    d_out = torch.randn(wl.num_ranks, wl.num_tokens, wl.hidden, device="cuda").bfloat16()
    d_y, d_w = torch.zeros_like(y), torch.zeros_like(run.w)
    ep.ep_combine_grad(run.cfg, run.lay, y, run.idx, run.w, d_out, d_y, d_w, run.ws)

    def value(weights, rows_y):
        out = torch.empty_like(d_out)
        ep.ep_combine(run.cfg, run.lay, rows_y, run.idx, weights, out, run.ws)
        return float((out.double() * d_out.double()).sum())

    f = value(run.w, y)
    # out is rounded to bf16: each of its terms is 2^-9 off at most, with signs that average out
    noise = 2 ** -8 * float((d_out.double() ** 2).sum()) ** 0.5 * 8
    assert abs(f - float((d_w.double() * run.w.double()).sum())) <= noise
    assert abs(f - float((d_y.double() * y.double()).sum())) <= noise


def test_rows_past_a_packed_capacity_are_left_out_and_reported():
    wl = CASES["packed"].replace(hidden=64, recv_capacity=40)
    idx, w = W.routing(wl)
    x, _ = W.hidden(wl)
    run = GpuRun(wl, idx, w, x, None).layout()
    y = torch.randn(40, 64, device="cuda").bfloat16()
    d_out = torch.randn(wl.num_ranks, wl.num_tokens, 64, device="cuda").bfloat16()
    guard = torch.full((64, 64), 7.0, device="cuda").bfloat16()
    d_w = torch.zeros_like(run.w)
    ep.ep_combine_grad(run.cfg, run.lay, y, run.idx, run.w, d_out, guard[:40], d_w, run.ws)
    assert run.status() == ep.EP_ERR_OVERFLOW
    assert (guard[40:] == 7.0).all()
    st, olay = oracle.layout(wl.replace(recv_capacity=0), idx)
    row = torch.from_numpy(oracle.global_rows(wl.replace(recv_capacity=0), olay, idx)).reshape(d_w.shape)
    assert (d_w.cpu()[row >= 40] == 0).all() and np.count_nonzero(d_w.cpu()[(row >= 0) & (row < 40)].numpy())
