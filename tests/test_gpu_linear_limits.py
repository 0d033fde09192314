"""Waits of the linear-attention prefill that run out, and what ragged rows leave behind.

A limit of a nanosecond gives up at the first hand-off that is not complete; limits of
some microseconds give up somewhere on the way, each role of a CTA on its own.  Every
such call has to end by itself, to say so where its results are not whole, and to
leave the context usable: the same call with the limit restored is right."""
import ctypes

import pytest
import torch

from gated_deltanet_recurrence_02_gb300 import gdn
from gated_deltanet_recurrence_02_gb300.inputs import make_inputs
from test_gpu_linear import call, check

pytestmark = pytest.mark.gpu

LIMITS = [1, 2000, 8000, 30000]  # ns


def errors():
    flags = ctypes.c_uint32(0)
    gdn.lib().gdn_device_errors(torch.cuda.current_stream().cuda_stream, ctypes.byref(flags))
    return flags.value


def runs_out(x, dtype, limits=LIMITS, turns=5):
    """Calls with short limits; each one without an error bit has the whole result."""
    whole, last, _ = call(x, x.alpha, gdn.gdn_linear_prefill, state=x.initial_state, packed=True)
    whole, last = whole.clone(), last.clone()
    assert errors() == 0
    try:
        for ns in limits:
            gdn.gdn_set_wait_limit_ns(ns)
            for _ in range(turns):
                out, end, _ = call(x, x.alpha, gdn.gdn_linear_prefill, state=x.initial_state, packed=True)
                flags = errors()
                assert flags in (0, gdn.GDN_DEVERR_TIMEOUT)
                assert ns > 1 or flags
                if not flags:
                    assert torch.equal(out, whole) and torch.equal(end, last)
    finally:
        gdn.gdn_set_wait_limit_ns(0)
    out, end, _ = call(x, x.alpha, gdn.gdn_linear_prefill, state=x.initial_state, packed=True)
    check(x, x.alpha, out, end, dtype, state=x.initial_state)
    assert errors() == 0


@pytest.mark.parametrize("lengths", [[90, 1, 65, 130, 63, 7], [1000, 333]], ids=["rows", "segments"])
def test_ragged_rows_bf16(lengths):
    x = make_inputs(51, lengths=lengths, Hk=1, Hv=2, dk=128, dv=128, dtype_qkv="bf16", dtype_gate="f32")
    runs_out(x, "bf16")


@pytest.mark.parametrize("lengths", [[64] * 12, [90, 1, 65, 130, 63, 7], [1000, 333]],
                         ids=["chunks", "rows", "segments"])
def test_fp16(lengths):
    """Two warps share the scales of P's later rows."""
    x = make_inputs(53, lengths=lengths, Hk=1, Hv=2, dk=128, dv=64, dtype_qkv="f16", dtype_gate="f32")
    runs_out(x, "f16")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_few_chunks(dtype):
    """CTAs whose tiles are all on their way at once, and calls that follow at once."""
    x = make_inputs(54, lengths=[64, 40, 200, 129] * 40, Hk=2, Hv=4, dk=128, dv=128, dtype_qkv=dtype, dtype_gate="f32")
    g = [t.cuda() for t in (x.q, x.k, x.v, x.alpha)]
    how = dict(B=x.B, cu_seqlens=x.cu_seqlens.cuda(), initial_state=x.initial_state.cuda())
    whole, last = gdn.gdn_linear_prefill(*g, **how)
    assert errors() == 0
    for _ in range(5):
        gdn.gdn_set_wait_limit_ns(1)
        try:
            gdn.gdn_linear_prefill(*g, **how)
        finally:
            gdn.gdn_set_wait_limit_ns(0)
        out, end = gdn.gdn_linear_prefill(*g, **how)  # on the same SMs, right behind it
        assert errors() == gdn.GDN_DEVERR_TIMEOUT
        assert torch.equal(out, whole) and torch.equal(end, last)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 32), (32, 64)])
@pytest.mark.parametrize("n", [5, 63, 97])
def test_the_next_row_stays_out(dtype, dk, dv, n):
    """Keys, queries and values that are not finite right behind a row's end."""
    x = make_inputs(52, lengths=[n, 70], Hk=1, Hv=2, dk=dk, dv=dv, dtype_qkv=dtype, dtype_gate="f32")
    out, last, _ = call(x, x.alpha, gdn.gdn_linear_prefill, state=x.initial_state, packed=True)
    out, last = out[:n].clone(), last[0].clone()
    x.q[n:], x.k[n:], x.v[n:] = float("nan"), float("inf"), float("nan")
    dirty, end, _ = call(x, x.alpha, gdn.gdn_linear_prefill, state=x.initial_state, packed=True)
    assert torch.equal(dirty[:n], out) and torch.equal(end[0], last)
