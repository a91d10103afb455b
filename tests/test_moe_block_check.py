"""check() of the example's blocks looks at every workspace that their calls report into (no GPU: the
workspaces are names here)."""
import os
import sys

import pytest

import combine_ep_get_02_gb300 as ep

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402


@pytest.mark.parametrize("kind,names", [
    ("KeptBlock", ("norm_ws", "z_ws", "x_ws", "ws", "route_ws", "up_ws", "down_ws", "up_grad_ws", "down_grad_ws")),
    ("ServingBlock", ("route_ws", "layer_ws")),
])
def test_every_workspace_is_looked_at(monkeypatch, kind, names):
    kind = getattr(moe_layer, kind)
    block = kind.__new__(kind)
    for name in names:
        setattr(block, name, name)
    block.grad = True
    broken = None
    monkeypatch.setattr(ep, "ep_check_error", lambda ws, stream=None: ep.EP_ERR_TIMEOUT if ws == broken else ep.EP_OK)
    assert block.check() == ep.EP_OK
    for broken in names:
        assert block.check() == ep.EP_ERR_TIMEOUT, broken
