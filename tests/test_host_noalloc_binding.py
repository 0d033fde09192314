"""The binding of the allocation-free prefill hands its arguments on in the C order (a
stand-in for the library records them, so no GPU is needed)."""
import ctypes
import types

import torch

from gated_deltanet_recurrence_02_gb300 import gdn


def test_noalloc_binding_passes_the_number_of_states(monkeypatch):
    seen = []

    def fn(*args):
        seen.append(args)
        return 0

    fn.restype, fn.argtypes = ctypes.c_int, [ctypes.c_void_p]
    monkeypatch.setattr(gdn, "lib", lambda: types.SimpleNamespace(gdn_prefill_chunked_noalloc=fn))
    monkeypatch.setattr(gdn, "_p", lambda t: t)
    q, v = torch.zeros(6, 1, 32), torch.zeros(6, 2, 32)
    gate, state, out = torch.zeros(6, 2), torch.zeros(5, 2, 32, 32), torch.empty(6, 2, 32)
    kw = dict(B=2, T=3, final_state=None, out=out, stream=7)
    assert gdn.gdn_prefill_chunked_noalloc(q, q, v, gate, gate, initial_state=state, **kw) == (out, None)
    gdn.gdn_prefill_chunked_noalloc(q, q, v, gate, gate, **kw)
    assert [a[8] for a in seen] == [5, 0] and seen[0][6] is state
    assert seen[0][11:21] == (2, 3, 1, 1, 2, 32, 32, 64, 1.0, 0) and seen[0][-1] == 7
