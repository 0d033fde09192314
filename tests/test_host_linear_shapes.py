"""Shapes and dtypes that the binding of the linear-attention calls refuses before the
library sees an address.  No GPU is needed: the tensors lie on the host, and a call whose
shapes are right is refused for that alone."""
import pytest
import torch

from gated_deltanet_recurrence_02_gb300 import gdn

B, T, Hk, Hv, dk, dv = 2, 5, 1, 2, 32, 64
F32, I32 = torch.float32, torch.int32


def call(fn, **kw):
    n = B * T
    a = dict(q=torch.zeros(n, Hk, dk), k=torch.zeros(n, Hk, dk), v=torch.zeros(n, Hv, dv),
             alpha=torch.zeros(n, Hv), B=B, T=T)
    a.update(kw)
    return fn(a.pop("q"), a.pop("k"), a.pop("v"), a.pop("alpha"), **a)


WRONG = [
    (dict(alpha=torch.zeros(Hv)), "alpha"),
    (dict(alpha=torch.zeros(B * T, Hv), conventions=gdn.GDN_ALPHA_PER_HEAD), "alpha"),
    (dict(alpha=torch.zeros(B * T - 1, Hv)), "alpha"),
    (dict(alpha=torch.zeros(Hv, B * T)), "alpha"),
    (dict(alpha=torch.zeros(Hk), conventions=gdn.GDN_ALPHA_PER_HEAD), "alpha"),
    (dict(k=torch.zeros(B * T - 1, Hk, dk)), "q and k"),
    (dict(k=torch.zeros(B * T, Hk, dk).half()), "one dtype"),
    (dict(v=torch.zeros(B * T - 1, Hv, dv)), "v "),
    (dict(T=T + 1), "B rows of T tokens"),
    (dict(cu_seqlens=torch.zeros(B, dtype=I32)), "cu_seqlens"),
    (dict(cu_seqlens=torch.zeros(B + 1, dtype=torch.int64)), "cu_seqlens"),
    (dict(initial_state=torch.zeros(B, Hv, dk, dv)), "initial_state"),
    (dict(initial_state=torch.zeros(B, Hv, dv, dk).half()), "initial_state"),
    (dict(initial_state=torch.zeros(Hv, dv, dk)), "initial_state"),
    (dict(initial_state=torch.zeros(3, Hv, dv, dk), initial_state_indices=torch.zeros(1, dtype=I32)), "indices"),
    (dict(initial_state=torch.zeros(3, Hv, dv, dk), initial_state_indices=torch.zeros(B, dtype=torch.int64)), "indices"),
    (dict(final_state=torch.zeros(1, Hv, dv, dk)), "final_state"),
    (dict(final_state=torch.zeros(B, Hv, dv, dk).double()), "final_state"),
    (dict(out=torch.zeros(B * T - 1, Hv, dv)), "out"),
    (dict(out=torch.zeros(B * T, Hv, dv).half()), "out"),
]


@pytest.mark.parametrize("fn", [gdn.gdn_linear_prefill, gdn.gdn_linear_recurrent], ids=["prefill", "recurrent"])
@pytest.mark.parametrize("kw,what", WRONG, ids=lambda x: x if isinstance(x, str) else ",".join(x))
def test_refused(fn, kw, what):
    with pytest.raises(ValueError, match=what):
        call(fn, **kw)


@pytest.mark.parametrize("kw,what", [
    (dict(capture_count=torch.zeros(1, dtype=I32)), "capture_count"),
    (dict(capture_count=torch.zeros(B)), "capture_count"),
    (dict(state_update=torch.zeros(B, 2, gdn.slot_width(Hk, Hv, dk, dv))), "state_update"),
    (dict(state_update=torch.zeros(B, 3, gdn.slot_width(Hk, Hv, dk, dv)).half()), "state_update"),
    (dict(state_update_active=torch.zeros(1)), "state_update_active"),
    (dict(state_update_active=torch.zeros(0, dtype=I32)), "state_update_active"),
])
def test_capture_refused(kw, what):
    kw = {"capture_count": torch.zeros(B, dtype=I32), **kw}
    with pytest.raises(ValueError, match=what):
        call(gdn.gdn_linear_recurrent, state_update_capacity=3, **kw)


@pytest.mark.parametrize("fn", [gdn.gdn_linear_prefill, gdn.gdn_linear_recurrent], ids=["prefill", "recurrent"])
@pytest.mark.parametrize("kw", [
    {}, dict(T=None), dict(T=T - 1), dict(alpha=torch.zeros(Hv), conventions=gdn.GDN_ALPHA_PER_HEAD),
    dict(T=None, cu_seqlens=torch.zeros(B + 1, dtype=I32)),
    dict(initial_state=torch.zeros(3, Hv, dv, dk), initial_state_indices=torch.zeros(B, dtype=I32)),
    dict(final_state=torch.zeros(B, Hv, dv, dk), out=torch.zeros(B * T, Hv, dv)),
])
def test_right_shapes_on_the_host(fn, kw):
    from gated_deltanet_recurrence_02_gb300 import build
    build.build()
    with pytest.raises(ValueError, match="device tensors"):
        call(fn, **kw)
