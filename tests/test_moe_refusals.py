"""Arguments that the router, the combine's gradient and the experts' products refuse before
touching the device (CPU: a call that got as far as CUDA would answer EP_ERR_CUDA)."""
import ctypes as C

import pytest
import torch

P = C.c_void_p
WS = P(0x10000)


@pytest.fixture(scope="module")
def ep():
    from combine_ep_get_02_gb300 import _build
    _build.build()
    import combine_ep_get_02_gb300 as ep
    ep.lib()
    return ep


def route_cfg(ep, **kw):
    return ep.RouteConfig(**{**dict(num_segments=2, num_tokens=64, num_experts=32, num_topk=4), **kw})


def product_cfg(ep, **kw):
    return ep.ProductConfig(**{**dict(num_ranks=2, num_experts=8, rows=100, in_features=128, out_features=64), **kw})


@pytest.mark.parametrize("bad,code", [
    (dict(num_segments=0), -1), (dict(num_tokens=-1), -1), (dict(num_experts=0), -1), (dict(num_experts=4097), -2),
    (dict(num_topk=0), -1), (dict(num_topk=33), -1), (dict(num_experts=3), -1), (dict(logits_dtype=1), -1),
    (dict(score=2), -1), (dict(normalize=2), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(num_groups=-1), -1), (dict(num_groups=5), -1), (dict(num_groups=32), -1),
    (dict(num_groups=64, num_experts=128), -2), (dict(num_groups=4, topk_groups=0), -1),
    (dict(num_groups=4, topk_groups=5), -1), (dict(num_groups=16, topk_groups=1), -1),
    (dict(num_tokens=1 << 30), -2),
])
def test_route_configs(ep, bad, code):
    cfg = route_cfg(ep, **bad)
    assert ep.ep_route_workspace_bytes(cfg) == 0
    out = ep._Route()
    assert ep.lib().ep_route(C.byref(cfg._c()), None, None, None, C.byref(out), None, 0, None) == code
    assert ep.lib().ep_route_grad(C.byref(cfg._c()), None, None, C.byref(out), None, None, None, None, 0, None) == code
    with pytest.raises(ep.EpError):
        ep.alloc_route_workspace(cfg)


def test_route_arguments(ep):
    L, cfg = ep.lib(), route_cfg(ep)
    n, c = ep.ep_route_workspace_bytes(cfg), route_cfg(ep)._c()
    full = ep._Route(*[P(0x20000)] * 6)
    call = lambda logits=P(0x30000), out=full, ws=WS, size=n, bias=None: L.ep_route(  # noqa: E731
        C.byref(c), logits, bias, None, None if out is None else C.byref(out), ws, size, None)
    assert call(ws=None) == ep.EP_ERR_WORKSPACE and call(ws=P(0x10010)) == ep.EP_ERR_WORKSPACE
    assert call(size=n - 1) == ep.EP_ERR_WORKSPACE
    assert call(logits=None) == ep.EP_ERR_INVALID_ARG and call(out=None) == ep.EP_ERR_INVALID_ARG
    assert call(logits=P(0x30004)) == ep.EP_ERR_INVALID_ARG and call(bias=P(0x30002)) == ep.EP_ERR_INVALID_ARG
    for i in range(6):  # idx and weights always; the statistics all or none
        some = ep._Route(*[None if k == i else P(0x20000) for k in range(6)])
        assert call(out=some) == ep.EP_ERR_INVALID_ARG
    grad = lambda logits=P(0x30000), d=P(0x40000), out=full, loss=P(0x50000): L.ep_route_grad(  # noqa: E731
        C.byref(c), logits, None, C.byref(out), None, loss, d, WS, n, None)
    assert grad(logits=None) == grad(d=None) == grad(d=P(0x40008)) == ep.EP_ERR_INVALID_ARG
    assert grad(out=ep._Route(P(0x20000))) == ep.EP_ERR_INVALID_ARG  # a loss without its counts
    assert grad(out=ep._Route(None, P(0x20000))) == ep.EP_ERR_INVALID_ARG


def test_combine_grad_arguments(ep):
    L = ep.lib()
    cfg = ep.Config(1, 4, 16, 4, 8, 8, 64)
    n, c = ep.ep_workspace_bytes(cfg), cfg._c()
    lay = ep._Layout(*[P(0x20000)] * 11)
    call = lambda y=P(0x30000), g=P(0x40000), dy=P(0x50000), dw=P(0x60000), l=lay, ws=WS, w=P(0x70000): L.ep_combine_grad(  # noqa: E731
        C.byref(c), None if l is None else C.byref(l), y, P(0x80000), w, g, dy, dw, ws, n, None)
    assert call(ws=None) == ep.EP_ERR_WORKSPACE
    assert call(l=None) == call(l=ep._Layout()) == call(y=None) == call(g=None) == call(w=None) == ep.EP_ERR_INVALID_ARG
    assert call(y=P(0x30008)) == call(g=P(0x40002)) == call(dy=P(0x50008)) == call(dw=P(0x60002)) == ep.EP_ERR_INVALID_ARG
    assert call(dy=None, dw=None) == ep.EP_OK  # nothing asked for
    bad = ep.Config(1, 4, 15, 4, 8, 8, 64)._c()
    assert L.ep_combine_grad(C.byref(bad), C.byref(lay), *[P(0x30000)] * 6, WS, n, None) == ep.EP_ERR_INVALID_ARG


@pytest.mark.parametrize("bad,code", [
    (dict(num_ranks=0), -1), (dict(num_experts=0), -1), (dict(num_experts=9), -1), (dict(num_experts=8192), -2),
    (dict(rows=-1), -1), (dict(rows=1 << 31), -2), (dict(in_features=0), -1), (dict(in_features=100), -1),
    (dict(out_features=4), -1), (dict(out_features=68), -1), (dict(in_features=1 << 21), -2), (dict(activation=5), -1),
    (dict(activation=-1), -1), (dict(x_dtype=2), -1), (dict(x_dtype=1, in_features=136), -1), (dict(sf_pack=1), -2),
    (dict(sf_pack=2), -1), (dict(num_sms=-1), -1),
])
def test_product_configs(ep, bad, code):
    cfg = product_cfg(ep, **bad)
    assert ep.ep_product_workspace_bytes(cfg) == 0 and ep.ep_product_workspace_bytes(cfg, True) == 0
    none = [None] * 7
    assert ep.lib().ep_expert_product(C.byref(cfg._c()), None, *none, None, 0, None) == code
    assert ep.lib().ep_expert_product_grad(C.byref(cfg._c()), None, *none, None, 0, None) == code
    with pytest.raises(ep.EpError):
        ep.alloc_product_workspace(cfg)


def test_product_workspace_closed_forms(ep):
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    assert ep.ep_product_workspace_bytes(product_cfg(ep)) == 256
    assert ep.ep_product_workspace_bytes(product_cfg(ep, x_dtype=1)) == 256 + up(100 * 128 * 2)
    tiles = 100 // 64 + 8
    assert ep.ep_product_workspace_bytes(product_cfg(ep), True) == 256 + up(4 * tiles * 64)
    assert ep.ep_product_workspace_bytes(product_cfg(ep, activation=4), True) == 256 + up(100 * 128 * 2) + up(4 * tiles * 128)


def test_product_arguments(ep):
    L, cfg = ep.lib(), product_cfg(ep)
    n, c = ep.ep_product_workspace_bytes(cfg, True), cfg._c()
    lay = ep._Layout(*[None] * 6, P(0x20000), P(0x20000), P(0x20000))
    A = P(0x40000)

    def call(l=lay, x=A, sf=None, w=A, bias=None, res=None, z=None, out=A, ws=WS, size=n):
        return L.ep_expert_product(C.byref(c), None if l is None else C.byref(l), x, sf, w, bias, res, z, out, ws, size, None)

    def grad(l=lay, x=A, w=A, z=A, g=A, dx=A, dw=A, db=A, cc=c):
        return L.ep_expert_product_grad(C.byref(cc), None if l is None else C.byref(l), x, w, z, g, dx, dw, db, WS, 1 << 30, None)

    bad = ep.EP_ERR_INVALID_ARG
    assert call(ws=None) == call(size=255) == call(ws=P(0x10008)) == ep.EP_ERR_WORKSPACE
    assert call(l=None) == bad and grad(l=None) == bad  # several experts need a layout
    assert call(l=ep._Layout()) == bad
    assert call(x=None) == call(w=None) == call(out=None) == call(sf=A) == bad
    for k in ("x", "w", "bias", "res", "z", "out"):
        assert call(**{k: P(0x40008)}) == bad, k
    assert grad(x=None) == grad(w=None) == grad(g=None) == bad
    for k in ("x", "w", "z", "g", "dx", "dw"):
        assert grad(**{k: P(0x40008)}) == bad, k
    assert grad(z=None, cc=product_cfg(ep, activation=2, rows=8)._c()) == bad  # act' needs z
    assert grad(cc=product_cfg(ep, x_dtype=1)._c()) == ep.EP_ERR_UNSUPPORTED


def test_tensors_that_the_abi_would_misread_are_refused(ep):
    """The binding looks at types, order and sizes (the C ABI sees addresses alone)."""
    cfg = product_cfg(ep, num_ranks=1, num_experts=1)
    bf = dict(dtype=torch.bfloat16)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    good = dict(x=torch.zeros(100, 128, **bf), w=torch.zeros(1, 64, 128, **bf), out=torch.zeros(100, 64, **bf))

    def call(**kw):
        t = {**good, **kw}
        ep.ep_expert_product(cfg, None, t["x"], None, t["w"], None, None, None, t["out"], ws, stream=0)

    for kw, word in ((dict(x=torch.zeros(100, 128)), "float32"), (dict(x=torch.zeros(128, 100, **bf).t()), "contiguous"),
                     (dict(x=torch.zeros(99, 128, **bf)), "elements"), (dict(x=None), "missing"), ({}, "GPU")):
        with pytest.raises(ep.EpError, match=word) as e:
            call(**kw)
        assert e.value.status == ep.EP_ERR_INVALID_ARG


def test_outputs_too_small_for_another_configuration_are_refused(ep):
    """What was checked with one configuration is held against the next one's sizes."""
    small, large = route_cfg(ep), route_cfg(ep, num_tokens=65)
    out = ep.Route(torch.zeros(128, 4, dtype=torch.int64), torch.zeros(128, 4))
    object.__setattr__(out, "_sizes", [512, 512, -1, -1, -1, -1])  # as a call with `small` on the GPU leaves it
    with pytest.raises(ep.EpError, match="logits .*GPU"):
        ep.ep_route(small, torch.zeros(128, 32), None, None, out, torch.zeros(1), stream=0)
    with pytest.raises(ep.EpError, match="topk_idx has 512 elements, 520 needed"):
        ep.ep_route(large, torch.zeros(130, 32), None, None, out, torch.zeros(1), stream=0)
    with pytest.raises(ep.EpError, match="topk_idx is not on the GPU"):
        out.topk_weights = torch.zeros(128, 4)  # an assignment: looked at again
        ep.ep_route(small, torch.zeros(128, 32), None, None, out, torch.zeros(1), stream=0)
