"""The wrappers launch with the tensors' device as the current one (CPU: the
device calls are stand-ins)."""

import contextlib
import inspect
import re

import pytest
import torch

from kolmogorov_arnold_network_amd import _lib as L
from kolmogorov_arnold_network_amd import functional as F


@pytest.fixture
def devices(monkeypatch):
    now = [0]

    @contextlib.contextmanager
    def device(k):
        was, now[0] = now[0], k
        try:
            yield
        finally:
            now[0] = was

    monkeypatch.setattr(F, "_current", lambda: now[0])
    monkeypatch.setattr(F, "_raw_stream", lambda k: 1000 + k)
    monkeypatch.setattr(torch.cuda, "device", device)
    return now


@pytest.mark.parametrize("dev", [0, 1])
def test_launches_on_the_tensors_device(devices, dev):
    seen = []

    def entry(*args):
        seen.append((devices[0], args))
        return L.KAN_OK

    F._launch("entry", dev, entry, 7, None)
    assert seen == [(dev, (7, None, 1000 + dev))] and devices == [0]


def test_errors_leave_the_device_as_it_was(devices):
    with pytest.raises(L.KanError):
        F._launch("entry", 1, lambda *a: L.KAN_ERR_SHAPE, 7)
    assert devices == [0]


def test_every_launch_of_the_wrappers_does_one_of_both():
    for name in L.EXPORTS:
        if re.search("workspace_size|abi_version|status_string", name):
            continue
        text = inspect.getsource(F._basis if name.startswith("kan_basis") else getattr(F, name))
        assert ("_launch(" in text and "L.check(" not in text) or (
            "with torch.cuda.device(dev):\n            return %s(" % name in text
            and "& 15 or dev != _current():\n" in text), name
