"""What the binding of the router, the combine's gradient and the products refuses before the
library is called: the library is a stub here, so nothing reaches a device."""
import pytest
import torch

import combine_ep_get_02_gb300 as ep


class Device:
    """Stands for a dense GPU tensor of this type and shape."""

    is_cuda = True

    def __init__(self, *shape, dtype=torch.float32):
        self.shape, self.dtype, self.n = shape, dtype, torch.Size(shape).numel()

    def is_contiguous(self):
        return True

    def numel(self):
        return self.n

    def data_ptr(self):
        return 0x100000

    @property
    def nbytes(self):
        return self.n * self.dtype.itemsize


class Stub:
    """Counts the calls that get as far as the library."""

    def __init__(self, real):
        self.real, self.calls = real, 0

    def __getattr__(self, name):
        if name in ("ep_recv_rows", "ep_status_string"):  # these only read their arguments
            return getattr(self.real, name)

        def call(*a):
            self.calls += 1
            return 0
        return call


@pytest.fixture
def stub(monkeypatch):
    from combine_ep_get_02_gb300 import _build
    _build.build()
    s = Stub(ep.lib())
    monkeypatch.setattr(ep, "_lib", s)
    return s


BF, I32, I64, U8 = torch.bfloat16, torch.int32, torch.int64, torch.uint8


def calls():
    """Each entry point with arguments that pass every check, but for the workspace."""
    rc = ep.RouteConfig(2, 8, 16, 4)
    route = lambda: ep.Route(Device(16, 4, dtype=I64), Device(16, 4), Device(2, 16, dtype=I32), Device(2, 16),  # noqa: E731
                             Device(2, dtype=I32), Device(1))
    pc = ep.ProductConfig(1, 1, 10, 64, 32)
    x, w, out = Device(10, 64, dtype=BF), Device(1, 32, 64, dtype=BF), Device(10, 32, dtype=BF)
    cc = ep.Config(1, 2, 16, 4, 8, 8, 64)
    lay = ep.Layout(*[None] * 3, Device(2, 8, 4, dtype=I32), None, None)
    y, tok = Device(ep.ep_recv_rows(cc), 64, dtype=BF), Device(2, 8, 64, dtype=BF)
    idx, wt = Device(2, 8, 4, dtype=I64), Device(2, 8, 4)
    return {
        "ep_route": lambda ws: ep.ep_route(rc, Device(16, 16), None, None, route(), ws, stream=0),
        "ep_route_grad": lambda ws: ep.ep_route_grad(rc, Device(16, 16), None, route(), None, None, Device(16, 16), ws, stream=0),
        "ep_combine_grad": lambda ws: ep.ep_combine_grad(cc, lay, y, idx, wt, tok, y, wt, ws, stream=0),
        "ep_expert_product": lambda ws: ep.ep_expert_product(pc, None, x, None, w, None, None, None, out, ws, stream=0),
        "ep_expert_product_grad": lambda ws: ep.ep_expert_product_grad(pc, None, x, w, None, out, x, w, None, ws, stream=0),
    }


@pytest.mark.parametrize("name", ["ep_route", "ep_route_grad", "ep_combine_grad", "ep_expert_product",
                                  "ep_expert_product_grad"])
def test_workspaces_outside_the_gpu(stub, name):
    call = calls()[name]
    for ws, why in ((torch.zeros(1 << 20, dtype=U8), "not on the GPU"), (None, "missing")):
        with pytest.raises(ep.EpError, match=why) as e:
            call(ws)
        assert e.value.status == ep.EP_ERR_WORKSPACE
    strided = Device(1 << 20, dtype=U8)
    strided.is_contiguous = lambda: False
    with pytest.raises(ep.EpError, match="not contiguous"):
        call(strided)
    assert stub.calls == 0
    call(Device(1 << 20, dtype=U8))
    assert stub.calls == 1


@pytest.mark.parametrize("mode,names", [
    (dict(), ("slot_map",)), (dict(compact_recv=1), ("slot_map", "recv_psum")),
    (dict(compact_recv=2), ("slot_map", "recv_psum", "recv_region")), (dict(expand=1), ("exp_pos", "exp_region"))])
def test_layouts_of_a_smaller_configuration(stub, mode, names):
    """The combine's gradient reads a row's place from these and writes there."""
    R, T, K, H = 4, 8, 4, 64
    cfg = ep.Config(1, R, 16, K, T, T, H, **mode)
    full = dict(slot_map=R * T * K, exp_pos=R * T * K, recv_psum=R * R, recv_region=R, exp_region=R)
    lay = ep.Layout(*[None] * 6)
    for name in names:
        setattr(lay, name, Device(full[name], dtype=I32))
    y, tok = Device(ep.ep_recv_rows(cfg), H, dtype=BF), Device(R, T, H, dtype=BF)
    idx, wt, ws = Device(R, T, K, dtype=I64), Device(R, T, K), Device(1 << 20, dtype=U8)
    call = lambda: ep.ep_combine_grad(cfg, lay, y, idx, wt, tok, y, wt, ws, stream=0)  # noqa: E731
    call()
    assert stub.calls == 1
    for name in names:
        for t, why in ((Device(full[name] - 1, dtype=I32), f"{full[name] - 1} elements, {full[name]} needed"),
                       (Device(full[name], dtype=I64), "int64"), (torch.zeros(full[name], dtype=I32), "not on the GPU")):
            setattr(lay, name, t)
            with pytest.raises(ep.EpError, match=f"{name} .*{why}") as e:
                call()
            assert e.value.status == ep.EP_ERR_INVALID_ARG
        setattr(lay, name, Device(full[name], dtype=I32))
    assert stub.calls == 1
    call()
    assert stub.calls == 2
    cfg.num_tokens = T + 1  # the layout was looked at with the smaller configuration
    more = dict(y=Device(ep.ep_recv_rows(cfg), H, dtype=BF), tok=Device(R, T + 1, H, dtype=BF),
                idx=Device(R, T + 1, K, dtype=I64), wt=Device(R, T + 1, K))
    with pytest.raises(ep.EpError, match=f"{names[0]} has"):
        ep.ep_combine_grad(cfg, lay, more["y"], more["idx"], more["wt"], more["tok"], more["y"], more["wt"], ws, stream=0)
    assert stub.calls == 2
