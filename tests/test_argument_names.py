"""Refusals of the layer norm's parameters name the argument that is at fault (no
GPU needed: the tensors are host ones, taken to be on the device that the call runs on)."""
import pytest
import torch

import combine_ep_layout_09_amd as ep

T, H = 4, 64


@pytest.fixture(autouse=True)
def host_tensors_pass(monkeypatch):
    monkeypatch.setattr(ep, "_device_of", lambda t, name: -1)


def rows():
    return torch.zeros((T, H), dtype=torch.bfloat16)


def stat():
    return torch.ones(T)


@pytest.mark.parametrize("name", ["weight", "bias"])
def test_layer_norm(name):
    args = dict(weight=None, bias=None)
    args[name] = torch.ones(H, dtype=torch.float16)
    with pytest.raises(TypeError, match=f"^{name} has dtype torch.float16"):
        ep.ep_layer_norm(ep.Norm(T, H), rows(), args["weight"], args["bias"], rows())


@pytest.mark.parametrize("name", ["weight", "d_weight", "d_bias"])
def test_layer_norm_backward(name):
    args = dict(weight=None, d_weight=None, d_bias=None)
    args[name] = torch.ones(H, dtype=torch.float16)
    with pytest.raises(TypeError, match=f"^{name} has dtype torch.float16"):
        ep.ep_layer_norm_backward(ep.Norm(T, H), rows(), rows(), args["weight"], stat(), stat(),
                                  rows(), args["d_weight"], args["d_bias"])
