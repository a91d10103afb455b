"""The smoke run's comparison of the example layer covers everything that it claims (on the CPU, with a
layer's results computed by another plain form)."""
import os
import sys
from types import SimpleNamespace

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import __graft_entry__ as entry  # noqa: E402


def layer_and_inputs():
    g = torch.Generator().manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g) * s[-1] ** -0.5  # noqa: E731
    R, T, H, I, E, K = 2, 10, 16, 8, 6, 2
    layer = SimpleNamespace(ranks=R, tokens=T, topk=K, up=rnd(E, 2 * I, H), down=rnd(E, H, I), router=rnd(E, H))
    x = torch.randn(R, T, H, generator=g)
    layer.logits = x.reshape(-1, H) @ layer.router.T
    layer.route = SimpleNamespace(topk_idx=layer.logits.topk(K, -1)[1])
    return layer, x, torch.randn(R, T, H, generator=g)


def test_against_differences():
    """Each gradient's product with a direction against the objective's central difference along it."""
    layer, x, d_out = layer_and_inputs()
    names = dict(d_x="x", d_router="router", d_up="up", d_down="down")
    base = dict(x=x.double(), router=layer.router.double(), up=layer.up.double(), down=layer.down.double())

    def objective(v):
        xs = v["x"].reshape(-1, x.shape[-1])
        l = xs @ v["router"].T
        p, sel = l.softmax(-1), l.gather(1, layer.route.topk_idx).softmax(-1)
        dense = torch.zeros_like(l).scatter(1, layer.route.topk_idx, sel)
        a, b = torch.einsum("nh,eih->nei", xs, v["up"]).chunk(2, -1)
        out = torch.einsum("ne,nei,ehi->nh", dense, a * torch.sigmoid(a) * b, v["down"])
        E, n = l.shape[1], layer.tokens
        count = (dense != 0).double().reshape(layer.ranks, n, E).sum(1)
        loss = (E * count / (layer.topk * n) * p.reshape(layer.ranks, n, E).mean(1)).sum(1).mean()
        return float((out * d_out.double().reshape(out.shape)).sum() + loss)

    layer.logits = (base["x"].reshape(-1, x.shape[-1]) @ base["router"].T)
    want = entry._layer_in_64_bits(layer, x, d_out)
    g = torch.Generator().manual_seed(1)
    for name, key in names.items():
        v = torch.randn(base[key].shape, generator=g, dtype=torch.float64)
        f = [objective({**base, key: base[key] + s * v}) for s in (1e-5, -1e-5)]
        slope = float((want[name].reshape(v.shape) * v).sum())
        # third derivatives times 1e-10, and 1e-16 of the objective over 1e-5
        assert abs((f[0] - f[1]) / 2e-5 - slope) <= 1e-6 * (1 + abs(slope)), name


@pytest.mark.parametrize("name", ["out", "d_x", "d_router", "d_up", "d_down"])
def test_every_result_is_compared(name):
    layer, x, d_out = layer_and_inputs()
    want = entry._layer_in_64_bits(layer, x, d_out)
    entry._compare_layer({k: t.bfloat16() for k, t in want.items()}, want)
    for wrong in (want[name] * 1.03, torch.zeros_like(want[name]), want[name] * float("nan")):
        with pytest.raises(AssertionError, match=f"the layer's {name} "):
            entry._compare_layer({**want, name: wrong}, want)
    with pytest.raises(AssertionError):
        entry._compare_layer({k: t for k, t in want.items() if k != name}, want)
