"""One workspace, zeroed once, under layers of different sizes in turn: each call's result is that of a workspace
of its own. Tiles of the second product whose sums are split among CTAs are ended by the last of them, which counters in the
workspace find; what another size's call left in their place must not count."""
import pytest
import torch

import combine_ep_get_02_gb300 as ep
from test_gpu_layer import Case

pytestmark = pytest.mark.gpu

# (tokens, experts, lanes, hidden, inner, FP8 matrices)
WIDE = (12, 16, 8, 2560, 1024, False)   # 80 tiles of 32 rows, split: counters up to byte 576
FEW = (8, 16, 8, 4096, 2048, False)     # 256 tiles of 16 rows, split
CODES = (12, 8, 4, 3584, 2048, True)    # 112 tiles of 32 rows, split
NARROW = (12, 16, 8, 1024, 512, False)  # their first kernels write from byte 512 on
ONE = (1, 16, 4, 256, 512, False)


def space(cases):
    return torch.zeros(max(c.ws.numel() for c in cases), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("sizes", [(NARROW, WIDE), (ONE, FEW), (NARROW, CODES), (FEW, NARROW, CODES, ONE, WIDE)])
def test_sizes_in_turn(sizes):
    cases = [Case(ep, *s[:5], fp8=s[5], residual=True, seed=i) for i, s in enumerate(sizes)]
    want = [c.run() for c in cases]
    ws = space(cases)
    for c in cases:
        assert ep.ep_check_error(c.ws) == ep.EP_OK
        c.ws = ws
    for _ in range(2):
        for c, w in zip(cases, want):
            assert torch.equal(c.run(), w)
    assert ep.ep_check_error(ws) == ep.EP_OK


def test_other_operators_on_the_same_workspace():
    """The norm's gradient and the rows kept in 8 bits leave their own sums there."""
    c = Case(ep, *WIDE[:5], residual=True, seed=7)
    want = c.run()
    norm, kept = ep.NormConfig(700, 2048), ep.CheckpointConfig(1, 1, 700, 2048)
    c.ws = torch.zeros(max(c.ws.numel(), ep.ep_norm_workspace_bytes(norm), ep.ep_checkpoint_workspace_bytes(kept)),
                       dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    x, d_y = (torch.randn(700, 2048, generator=g, device="cuda").bfloat16() for _ in range(2))
    codes, sf = torch.empty(700, 2048, dtype=torch.uint8, device="cuda"), torch.empty(700, 16, device="cuda")
    for _ in range(2):
        ep.ep_norm_grad(norm, x, None, None, d_y, None, None, torch.empty(2048, device="cuda"), c.ws)
        assert torch.equal(c.run(), want)
        ep.ep_checkpoint(kept, None, x, codes, sf, c.ws)
        ep.ep_checkpoint_grad(kept, None, codes, sf, d_y, None, None, torch.empty(1, 2048, device="cuda"), c.ws)
        assert torch.equal(c.run(), want)
    assert ep.ep_check_error(c.ws) == ep.EP_OK


def test_only_the_header_need_be_zero():
    c = Case(ep, *WIDE[:5], seed=3)
    want = c.run()
    c.ws[256:] = 0xFF
    assert torch.equal(c.run(), want)


def test_two_sizes_captured():
    """Graphs of two sizes on one workspace, replayed in turn."""
    cases = [Case(ep, *s[:5], residual=True, seed=9) for s in (NARROW, WIDE)]
    want = [c.run() for c in cases]
    ws, graphs, outs = space(cases), [], [torch.empty_like(w) for w in want]
    for c, o in zip(cases, outs):
        c.ws = ws
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.run(out=o)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for graph in graphs:
            graph.replay()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
