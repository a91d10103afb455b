"""What the binding keeps in its configuration and tensor bundles does not keep them from being
copied, pickled or sent to another process."""
import copy
import dataclasses
import os
import pickle
import subprocess
import sys

import pytest
import torch

import combine_ep_get_02_gb300 as ep


def used(obj):
    """As a call leaves it: struct, reference to it and element counts kept."""
    obj._ref()
    object.__setattr__(obj, "_sizes", [1, 2, 3])
    object.__setattr__(obj, "_lanes", ((), [1]))
    return obj


CONFIGS = [ep.Config(1, 4, 16, 4, 8, 8, 64), ep.RouteConfig(2, 8, 16, 4, scale=2.5), ep.ProductConfig(2, 8, 100, 128, 64)]


@pytest.mark.parametrize("cfg", CONFIGS, ids=lambda c: type(c).__name__)
@pytest.mark.parametrize("twin", [copy.copy, copy.deepcopy, lambda c: pickle.loads(pickle.dumps(c)), dataclasses.replace],
                         ids=["copy", "deepcopy", "pickle", "replace"])
def test_configurations_after_a_call(cfg, twin):
    used(cfg)
    other = twin(cfg)
    assert other == cfg and other._sizes is None and other._lanes is None
    assert bytes(other._c()) == bytes(cfg._c())
    other.num_experts = 2 * cfg.num_experts
    assert other._c().num_experts == 2 * cfg.num_experts == 2 * cfg._c().num_experts


@pytest.mark.parametrize("twin", [copy.deepcopy, lambda c: pickle.loads(pickle.dumps(c))], ids=["deepcopy", "pickle"])
def test_tensors_after_a_call(twin):
    lay = used(ep.Layout(*(torch.full((4,), i) for i in range(6))))
    other = twin(lay)
    assert torch.equal(other.slot_map, lay.slot_map)
    assert other._c().slot_map == other.slot_map.data_ptr() != lay.slot_map.data_ptr()
    assert other._sizes is None and other._lanes is None


def test_import_without_the_cuda_part_of_torch():
    """A build of torch for the CPU has no current stream; the package still imports there."""
    code = ("import torch\n"
            "for name in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, name): delattr(torch._C, name)\n"
            "import combine_ep_get_02_gb300 as ep\n"
            "assert ep._raw_stream(7) == 7\n"
            "assert ep.RouteConfig(1, 1, 8, 2).num_topk == 2\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
