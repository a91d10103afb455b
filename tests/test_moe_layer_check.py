"""check() of the example layer looks at every workspace that its calls report into (no GPU: the
workspaces are names here)."""
import os
import sys

import pytest

import combine_ep_get_02_gb300 as ep

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402

FORWARD = ("ws", "route_ws", "up_ws", "down_ws")
BACKWARD = ("up_grad_ws", "down_grad_ws")


@pytest.mark.parametrize("grad", [False, True])
def test_every_workspace_is_looked_at(monkeypatch, grad):
    layer = moe_layer.MoELayer.__new__(moe_layer.MoELayer)
    names = FORWARD + (BACKWARD if grad else ())
    for name in names:
        setattr(layer, name, name)
    layer.grad = grad
    broken = None
    monkeypatch.setattr(ep, "ep_check_error", lambda ws, stream=None: ep.EP_ERR_TIMEOUT if ws == broken else ep.EP_OK)
    assert layer.check() == ep.EP_OK
    for broken in names:
        assert layer.check() == ep.EP_ERR_TIMEOUT, broken
