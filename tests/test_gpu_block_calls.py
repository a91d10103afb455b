"""Calls that the documentation allows around the norm, the kept rows and the experts' layer: tensors that begin
16 bytes into a sector, two calls at once, and a run of them all in one graph."""
import pytest
import torch

import _block_reference as ref
import combine_ep_get_02_gb300 as ep
from test_gpu_checkpoint import blocks_of
from test_gpu_layer import Case

pytestmark = pytest.mark.gpu


def shifted(t):
    """A copy of t that begins 16 bytes behind a 32-byte boundary."""
    pad = 16 // t.element_size()
    flat = torch.empty(t.numel() + 2 * pad, dtype=t.dtype, device=t.device)
    off = pad if flat.data_ptr() % 32 == 0 else 0
    out = flat[off:off + t.numel()].view(t.shape)
    assert out.data_ptr() % 32 == 16
    return out.copy_(t)


def test_tensors_that_begin_inside_a_sector():
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    n, h = 700, 1152
    cfg = ep.NormConfig(n, h)
    x, r, w, d_y = rnd(n, h), rnd(n, h), rnd(h), rnd(n, h)
    made = []
    for place in (lambda t: t.clone(), shifted):
        a, b, c, d = (place(t) for t in (x, r, w, d_y))
        total, y, d_x = (place(torch.zeros_like(x)) for _ in range(3))
        codes, sf, d_w = place(torch.zeros(n, h, dtype=torch.uint8, device="cuda")), place(torch.zeros(n, h // 128, device="cuda")), \
            place(torch.zeros(h, device="cuda"))
        ep.ep_norm(cfg, a, b, c, total, y, codes, sf)
        ep.ep_norm_grad(cfg, total, c, None, d, None, d_x, d_w, ep.alloc_norm_workspace(cfg))
        lay, _, rows = blocks_of(ep, [n - 9, 3], 1, 1, 6)
        ck = ep.CheckpointConfig(1, 2, rows, h, ep.EP_ACT_SWIGLU)
        ws = ep.alloc_checkpoint_workspace(ck)
        q, qs = place(torch.zeros(n, h, dtype=torch.uint8, device="cuda")), place(torch.zeros(n, h // 128, device="cuda"))
        back, h_again, d_z = place(torch.zeros_like(x)), place(torch.zeros(n, h // 2, device="cuda").bfloat16()), place(torch.zeros_like(x))
        ep.ep_checkpoint(ck, lay, a, q, qs, ws)
        ep.ep_checkpoint_rows(ck, lay, q, qs, back, ws)
        ep.ep_checkpoint_grad(ck, lay, q, qs, place(d_y[:, :h // 2].contiguous()), h_again, d_z, None, ws)
        made.append((total, y, codes, sf, d_x, d_w, q, qs, back, h_again, d_z))
    for a, b in zip(*made):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("T", [1, 6, 24, 64])
def test_layer_on_tensors_inside_a_sector(T, fp8):
    c = Case(ep, T, 8, 2, 384, 256, fp8=fp8, bias=True, residual=True)
    want = c.run()
    c.mats = {k: tuple(None if t is None else shifted(t) for t in v) for k, v in c.mats.items()}
    c.x, c.residual, c.w = shifted(c.x), shifted(c.residual), shifted(c.w) if c.w.numel() > 3 else c.w
    assert torch.equal(c.run(out=shifted(torch.zeros_like(c.x))), want)
    assert ep.ep_check_error(c.ws) == ep.EP_OK


def test_two_calls_at_once():
    """On two streams, each with its own workspace, long and short calls among each other."""
    cases = [Case(ep, 64, 16, 4, 1024, 512, seed=1), Case(ep, 2, 16, 4, 1024, 512, seed=2, residual=True),
             Case(ep, 8, 16, 4, 1024, 512, fp8=True, seed=3), Case(ep, 1, 16, 4, 1024, 512, seed=4)]
    want = [c.run() for c in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(40):
        for k, c in enumerate(cases):
            with torch.cuda.stream(streams[k % 2]):
                got.append((k, c.run()))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[k]) for k, o in got)
    assert all(ep.ep_check_error(c.ws) == ep.EP_OK for c in cases)


def test_matrices_written_just_before():
    """The second kernel fetches its matrices before the first has ended: an update in front of the call is seen."""
    c = Case(ep, 4, 8, 2, 1024, 512)
    up, down = c.mats["up"][0], c.mats["down"][0]
    base = up.clone(), down.clone()
    want = []
    for i in range(4):
        torch.mul(base[0], 1.0 + i, out=up)
        torch.mul(base[1], 2.0 - i, out=down)
        torch.cuda.synchronize()
        want.append(c.run())
        torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for i in range(4):
            torch.mul(base[0], 1.0 + i, out=up)
            torch.mul(base[1], 2.0 - i, out=down)
            got.append(c.run())
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_choice_and_rows_of_the_kernels_in_front():
    """Norm, router and layer back to back and in a graph: each reads what the one before it wrote."""
    T, E, K, H = 12, 16, 4, 512
    c = Case(ep, T, E, K, H, 256)
    norm, route = ep.NormConfig(T, H), ep.RouteConfig(1, T, E, K)
    out, ws = ep.alloc_route(route, stats=False), ep.alloc_route_workspace(route)
    y, logits, x = torch.empty_like(c.x), torch.empty(T, E, device="cuda"), c.x
    router = torch.randn(E, H, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") * H ** -0.5
    c.idx, c.w = out.topk_idx, out.topk_weights

    def step():
        ep.ep_norm(norm, x, None, None, None, y, None, None)
        torch.matmul(y.float(), router.t(), out=logits)
        ep.ep_route(route, logits, None, None, out, ws)
        return c.run(x=y)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        result = step()
    for seed in range(5):
        x.copy_(torch.randn(T, H, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        got = result.clone()
        assert torch.equal(step(), got)
        want, bound = ref.layer(y, out.topk_idx, out.topk_weights, c.mats["up"][0], None, c.mats["down"][0], None, None, "swiglu",
                                2.0 ** -17)
        assert ((got.double() - want).abs() <= want.abs() * 2.0 ** -8 + bound * (1 + 2.0 ** -7)).all()
