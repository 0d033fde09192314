"""The binding refuses tokens of another device than the current one, and keeps a workspace to a
thread's own calls on the default stream."""
import threading

import pytest
import torch

from gated_deltanet_recurrence_02_gb300 import gdn


class Tokens:
    """As much of a device tensor as is looked at before a call."""
    shape = torch.Size((4, 2, 64))
    dtype = torch.bfloat16
    is_cuda = True

    def __init__(self, device):
        self.on = device

    def stride(self):
        return 128, 64, 1

    def get_device(self):
        return self.on

    def data_ptr(self):
        return 1 << 20


def test_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(gdn, "_device", lambda: 0)
    assert gdn._heads(Tokens(0), 4, 2, 64) == (1 << 20, 128)
    with pytest.raises(ValueError, match="current device"):
        gdn._heads(Tokens(1), 4, 2, 64)


def test_kept_workspaces_are_a_threads_own(monkeypatch):
    monkeypatch.setattr(gdn, "_device", lambda: 0)
    monkeypatch.setattr(gdn, "_kept", threading.local())
    mine = gdn._keep(1000, "cpu")
    assert gdn._kept.__dict__[0] is mine and mine[1] == mine[0].data_ptr() and mine[2] == mine[0].numel() == 1000
    others = []
    t = threading.Thread(target=lambda: others.append(gdn._kept.__dict__.get(0)))
    t.start()
    t.join()
    assert others == [None]
    assert gdn._keep(2000, "cpu") is gdn._kept.__dict__[0]  # a larger one takes its place
