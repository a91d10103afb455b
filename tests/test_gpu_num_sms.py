"""num_sms bounds the CTAs of the products, and the results do not depend on it."""
import ctypes as C

import pytest
import torch

import combine_ep_get_02_gb300 as ep
from test_gpu_product import Case

pytestmark = pytest.mark.gpu


def grids(call):
    """CTAs of every kernel that call(stream) launches, from a capture that is not run."""
    driver = C.CDLL("libcuda.so.1")
    s = torch.cuda.Stream()
    stream, graph = C.c_void_p(s.cuda_stream), C.c_void_p()
    assert driver.cuStreamBeginCapture_v2(stream, 2) == 0
    try:
        call(s)
    finally:
        ended = driver.cuStreamEndCapture(stream, C.byref(graph))
    assert ended == 0
    n = C.c_size_t()
    assert driver.cuGraphGetNodes(graph, None, C.byref(n)) == 0
    nodes = (C.c_void_p * n.value)()
    assert driver.cuGraphGetNodes(graph, nodes, C.byref(n)) == 0
    out = []
    for node in nodes:
        kind, params = C.c_int(), (C.c_uint32 * 64)()
        assert driver.cuGraphNodeGetType(C.c_void_p(node), C.byref(kind)) == 0
        if kind.value == 0:  # a kernel: function address, grid, block, ...
            assert driver.cuGraphKernelNodeGetParams_v2(C.c_void_p(node), params) == 0
            out.append(params[2] * params[3] * params[4])
    assert driver.cuGraphDestroy(graph) == 0
    return out


SHAPES = {
    "one_token": dict(counts=[1], K=7168, N=2048, act="swiglu", dense=True),
    "rows_of_a_step": dict(counts=[90], K=2120, N=1104, act="silu", dense=True, bias=True, residual=True),
    "groups": dict(counts=[5, 0, 20], K=1096, N=200, act="gelu", bias=True, residual=True),
    "gated_groups": dict(counts=[2, 8, 1, 5, 16, 3, 9, 32], K=1024, N=640, R=2, act="swiglu", bias=True),
    "narrow": dict(counts=[17], K=2056, N=72, dense=True),
    "no_split": dict(counts=[50, 0, 200], K=256, N=136, act="swiglu", bias=True),
    "pairs": dict(counts=[700, 257, 900], K=392, N=264, act="gelu", bias=True),
}


@pytest.mark.parametrize("sms", [1, 2, 3, 7, 8, 40, 100, 151])
@pytest.mark.parametrize("name", SHAPES)
def test_products_keep_to_num_sms(name, sms):
    a, b = Case(**SHAPES[name]), Case(**SHAPES[name], num_sms=sms)
    ws = ep.alloc_product_workspace(b.cfg, grad=True)
    out, dx, dw = torch.empty_like(b.d_out), torch.empty_like(b.x), torch.empty_like(b.w)
    fwd = grids(lambda s: ep.ep_expert_product(b.cfg, b.lay, b.x, None, b.w, b.bias, b.res, None, out, ws, stream=s))
    rows = grids(lambda s: ep.ep_expert_product_grad(b.cfg, b.lay, b.x, b.w, b.z_in, b.d_out, dx, None, None, ws, stream=s))
    both = grids(lambda s: ep.ep_expert_product_grad(b.cfg, b.lay, b.x, b.w, b.z_in, b.d_out, dx, dw, None, ws, stream=s))
    assert max(fwd) <= sms
    assert rows[-1] <= sms  # after the elementwise kernel, which runs several CTAs on an SM
    assert both[-1] <= max(sms, 2)  # matrix gradients take a pair of SMs at least
    for x, y in zip(a.forward(), b.forward()):
        assert torch.equal(x[a.live], y[a.live])
    dx, dw, db = a.grads()
    for x, y in zip((dx[a.live], dw, db), (lambda g: (g[0][a.live], g[1], g[2]))(b.grads())):
        assert torch.equal(x, y)
