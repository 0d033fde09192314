"""Decays that drop the state: whatever stood in front of one, however large, leaves
nothing behind it; and decays that are strong but not zero keep their share.

Element by element: with u = 2^-8 (bf16), 2^-11 (fp16) the scores, the state's image
and the result are rounded once each where the tensor cores take them, relative to the
terms of the sum, so |error| <= 2 u (sum of the terms' magnitudes), and 2^-10 of it more
for the exponents of strong decays (sums of up to 32 x 127 in fp32); fp32: 1e-5."""
import pytest
import torch

from gated_deltanet_recurrence_02_gb300 import gdn
from gated_deltanet_recurrence_02_gb300.inputs import make_inputs
from test_gpu_linear import call

pytestmark = pytest.mark.gpu

TOL = {"f32": 1e-5, "f16": 2.0 ** -10 + 2.0 ** -10, "bf16": 2.0 ** -7 + 2.0 ** -10}


def recurrence(q, k, v, alpha, state):
    """Outputs and last state of one row [T, H, d] in 64 bits."""
    S = state.clone()
    out = torch.empty_like(v)
    for t in range(q.shape[0]):
        S = alpha[t, :, None, None] * S + v[t, :, :, None] * k[t, :, None, :]
        out[t] = (S @ q[t, :, :, None]).squeeze(-1)
    return out, S


@pytest.mark.parametrize("dtype,front", [("bf16", 2.0 ** 60), ("bf16", 2.0 ** 45), ("f16", 2.0 ** 13), ("f32", 2.0 ** 60)])
@pytest.mark.parametrize("resets", [[40], [31, 32], [5, 20, 50, 70, 100, 131], [1100]],
                         ids=["one", "halves", "many", "segments"])
@pytest.mark.parametrize("drop", [0.0, 2.0 ** -60, 2.0 ** -100.5], ids=["zero", "60", "100"])
@pytest.mark.parametrize("log", [False, True], ids=["factor", "log"])
def test_nothing_comes_through(dtype, front, resets, drop, log):
    T = 1500 if resets[0] > 1000 else 150
    x = make_inputs(61, lengths=[T], Hk=1, Hv=2, dk=64, dv=64, dtype_qkv=dtype, dtype_gate="f32")
    v = x.v.float()
    v[:resets[-1]] *= front  # in front of the last reset
    x.v = v.to(x.v.dtype)
    alpha = x.alpha.clone()
    alpha[resets] = drop
    given = torch.log(alpha) if log else alpha
    out, last, _ = call(x, given, gdn.gdn_linear_prefill, state=x.initial_state,
                        conventions=gdn.GDN_ALPHA_LOG if log else 0)
    q, k, v, a = (t.cuda().double() for t in (x.q, x.k, x.v, torch.exp(given.double()) if log else alpha))
    q, k = (t.repeat_interleave(2, 1) for t in (q, k))
    S0 = x.initial_state[0].cuda().double()
    want, state = recurrence(q, k, v, a, S0)
    terms, held = recurrence(q.abs(), k.abs(), v.abs(), a, S0.abs())
    assert torch.isfinite(out).all() and torch.isfinite(last).all()
    over = (out.double() - want).abs() - TOL[dtype] * terms - (2.0 ** -24 if dtype == "f16" else 1e-30)
    assert float(over.max()) <= 0, (float(over.max()), int(over.flatten(1).amax(1).argmax()))
    over = (last[0].double() - state).abs() - 1e-5 * held - 1e-30
    assert float(over.max()) <= 0, float(over.max())
