"""A NaN among a row's inputs shows in that row's results, under every activation."""
import math

import pytest
import torch

from test_gpu_product import ACTS, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ACTS)
def test_nan_reaches_the_results(act):
    c = Case([20, 40], 72, 136, act=act, bias=True, residual=True)
    want, want_z = c.forward()
    dx, dw, db = c.grads()
    rest = torch.ones(c.rows, dtype=torch.bool, device="cuda")
    rest[[7, 33]] = False
    c.x[7, 5] = math.nan
    c.x[33, 71] = math.nan
    out, z = c.forward()
    assert torch.isnan(z[~rest]).all() and torch.isnan(out[~rest]).all()
    assert torch.equal(out[rest], want[rest]) and torch.equal(z[rest], want_z[rest])
    c = Case([20, 40], 72, 136, act=act, bias=True, residual=True)
    if act == "none":  # z is not read
        return
    c.z_in[7, 3] = math.nan
    c.z_in[33, -1] = math.nan
    gx, gw, gb = c.grads()
    assert torch.isnan(gx[~rest]).all() and torch.equal(gx[rest], dx[rest])
    # gated: a gate reaches both halves of dz, a factor the gate's half alone
    where = ((0, 3), (0, c.N + 3), (1, c.N - 1)) if act == "swiglu" else ((0, 3), (1, c.Z - 1))
    hit = torch.zeros_like(gb, dtype=torch.bool)
    for g, column in where:
        hit[g, column] = True
    assert torch.equal(torch.isnan(gb), hit) and torch.isnan(gw[hit]).all()
    assert torch.equal(gb[~hit], db[~hit]) and torch.equal(gw[~hit], dw[~hit])
