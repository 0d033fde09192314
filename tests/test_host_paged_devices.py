"""The rotary, append and attention bindings refuse each tensor that is not on the current
device (stand-ins for device tensors and for the library, so no GPU is needed)."""
import types

import pytest
import torch

from gated_deltanet_recurrence_02_gb300 import gdn


class On:
    """A tensor that says it is on a device."""

    def __init__(self, t, device=0):
        self.t, self.on = t, device

    is_cuda = True

    def get_device(self):
        return self.on

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.fixture
def calls(monkeypatch):
    seen = []

    def fn(name):
        def call(*args):
            seen.append((name, args))
            return 0
        return call

    names = ("gdn_rotary", "gdn_paged_append", "gdn_paged_attention")
    L = types.SimpleNamespace(**{n: fn(n) for n in names}, gdn_paged_attention_workspace_size=lambda *a: 64)
    monkeypatch.setattr(gdn, "lib", lambda: L)
    monkeypatch.setattr(gdn, "_device", lambda: 0)
    monkeypatch.setattr(gdn, "_stream", lambda stream: 5)
    monkeypatch.setattr(gdn, "_empty", lambda shape, dtype, device, stream, scratch=False: torch.empty(shape, dtype=dtype))
    return seen


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def tokens(h):
    return torch.zeros(6, h, 64)


def pages():
    return torch.zeros(3, 16, 2, 64)


CALLS = {
    "gdn_rotary": (dict(x=tokens(4), positions=ints(3, 6), inv_freq=torch.zeros(32), axes=ints(32), out=tokens(4)), {}),
    "gdn_paged_append": (dict(k=tokens(2), v=tokens(2), k_pages=pages(), v_pages=pages(), page_table=ints(2, 4),
                              kv_lens=ints(2), cu_seqlens=ints(3), q=tokens(4), q_out=tokens(4),
                              inv_freq=torch.zeros(32), positions=ints(3, 6), axes=ints(32)), dict(B=2)),
    "gdn_paged_attention": (dict(q=tokens(4), k_pages=pages(), v_pages=pages(), page_table=ints(2, 4), kv_lens=ints(2),
                                 cu_seqlens=ints(3), out=tokens(4), lse=torch.zeros(6, 4),
                                 workspace=torch.zeros(64, dtype=torch.uint8)), dict(B=2)),
}


@pytest.mark.parametrize("name,which", [(n, w) for n, (tensors, _) in CALLS.items() for w in (None, *tensors)])
def test_each_tensor_is_on_the_current_device(calls, name, which):
    tensors, kw = CALLS[name]
    args = {n: On(t, int(n == which)) for n, t in tensors.items()}
    if which is None:
        getattr(gdn, name)(**args, **kw)
        assert [n for n, _ in calls] == [name]
        return
    with pytest.raises(ValueError, match="current device"):
        getattr(gdn, name)(**args, **kw)
    assert not calls


class Long(On):
    """More tokens, heads or pages than 32 bits count, as the shape has it."""

    def __init__(self, t, **sizes):
        super().__init__(t)
        shape = list(t.shape)
        for at, n in sizes.items():
            shape[int(at[1:])] = n
        self.shape = torch.Size(shape)

    def stride(self):
        return self.t.stride()

    def is_contiguous(self):
        return True


BIG = 2**32 + 3  # the 32 bits of a C int would be 3


@pytest.mark.parametrize("name,change,kw", [
    ("gdn_rotary", dict(x=dict(_1=BIG), out=dict(_1=BIG)), {}),
    ("gdn_rotary", dict(positions=dict(_0=BIG)), {}),
    ("gdn_paged_append", dict(k=dict(_0=BIG), v=dict(_0=BIG), q=dict(_0=BIG), q_out=dict(_0=BIG), positions=dict(_1=BIG)), {}),
    ("gdn_paged_append", dict(q=dict(_1=BIG), q_out=dict(_1=BIG)), {}),
    ("gdn_paged_append", dict(k_pages=dict(_0=BIG), v_pages=dict(_0=BIG)), {}),
    ("gdn_paged_append", dict(k_pages=dict(_1=BIG), v_pages=dict(_1=BIG)), {}),
    ("gdn_paged_append", dict(page_table=dict(_1=BIG)), {}),
    ("gdn_paged_append", dict(positions=dict(_0=BIG)), {}),
    ("gdn_paged_attention", dict(q=dict(_0=BIG), out=dict(_0=BIG), lse=dict(_0=BIG)), {}),
    ("gdn_paged_attention", dict(q=dict(_1=BIG), out=dict(_1=BIG), lse=dict(_1=BIG)), {}),
    ("gdn_paged_attention", dict(k_pages=dict(_0=BIG), v_pages=dict(_0=BIG)), {}),
    ("gdn_paged_attention", dict(page_table=dict(_1=BIG)), {}),
    ("gdn_paged_attention", {}, dict(window=BIG)),
    ("gdn_paged_attention", {}, dict(window=2**31)),
])
def test_sizes_that_a_c_int_does_not_hold(calls, name, change, kw):
    """They are refused, not cut to their lower 32 bits."""
    tensors, rest = CALLS[name]
    args = {n: Long(t, **change[n]) if n in change else On(t) for n, t in tensors.items()}
    with pytest.raises(ValueError, match="2\\^31"):
        getattr(gdn, name)(**args, **rest, **kw)
    assert not calls
