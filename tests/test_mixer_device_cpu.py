"""Calls on tensors of a device that is not the current one: the workspace is
planned on the tensors' device too (the plan goes by its number of SMs)."""
import contextlib

import pytest
import torch

import gated_delta_rule_72_b200 as gdn
from gated_delta_rule_72_b200 import _lib, api


class _Cuda1:
    """A CPU tensor that says it is on cuda:1."""

    is_cuda = True
    device = torch.device("cuda", 1)

    def __init__(self, t):
        self._t = t

    def __getattr__(self, name):
        return getattr(self._t, name)

    def new_empty(self, shape):
        return _Cuda1(self._t.new_empty(shape))


@pytest.fixture
def devices(monkeypatch):
    current = [0]
    seen = []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d.index
        yield
        current[0] = before

    class Lib:
        def gdn_ssm_workspace_size(self, *a):
            seen.append(("size", current[0]))
            return 512 * (1 + current[0])

        def gdn_ssm_scan(self, *a):
            seen.append(("scan", current[0], a[-2]))
            return 0

    class Stream:
        cuda_stream = None

    lib = Lib()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: None, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: Stream)
    monkeypatch.setattr(_lib, "load", lambda: lib)
    monkeypatch.setattr(api, "_workspace", lambda n, d, w: (torch.empty(n, dtype=torch.uint8), n))
    return seen


def test_scan_plans_its_workspace_on_the_tensors_device(devices):
    q = _Cuda1(torch.zeros(1, 200, 1, 64, dtype=torch.bfloat16))
    dt, A = _Cuda1(torch.zeros(1, 200, 1)), _Cuda1(torch.zeros(1))
    gdn.ssm_scan(q, q, q, dt, A)
    assert devices == [("size", 1), ("scan", 1, 1024)]


def test_workspace_size_of_a_given_device(devices):
    assert gdn.ssm_workspace_size(1, 200, 1, 1, 64, 64) == 512
    assert gdn.ssm_workspace_size(1, 200, 1, 1, 64, 64, device="cuda:1") == 1024
    assert gdn.ssm_workspace_size(1, 200, 1, 1, 64, 64, device="cuda:0") == 512
    assert gdn.ssm_workspace_size(1, 200, 1, 1, 64, 64, device="cuda") == 512
    with pytest.raises(ValueError):
        gdn.ssm_workspace_size(1, 200, 1, 1, 64, 64, device="cpu")
