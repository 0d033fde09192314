"""Waits of the residual norm's long rows that run out.

A call with a short limit ends by itself; where a row's copy came too late it says so,
and a call without an error bit has the whole result.  The rows of a CTA that gives up
are not written from the late one on, never from a stage that has not come."""
import ctypes

import pytest
import torch

from gated_deltanet_recurrence_02_gb300 import gdn

pytestmark = pytest.mark.gpu


def errors():
    flags = ctypes.c_uint32(0)
    gdn.lib().gdn_device_errors(torch.cuda.current_stream().cuda_stream, ctypes.byref(flags))
    return flags.value


@pytest.mark.parametrize("post", [False, True], ids=["plain", "post"])
@pytest.mark.parametrize("dtype,res,D", [(torch.bfloat16, torch.float32, 2048), (torch.float32, torch.float32, 4096),
                                         (torch.float16, torch.float16, 8192)], ids=["2048", "f32", "8192"])
def test_rows_that_come_late(dtype, res, D, post):
    N = 3001
    g = torch.Generator("cuda").manual_seed(D)
    y, z = (torch.randn(N, D, device="cuda", generator=g).to(dtype) for _ in range(2))
    x = torch.randn(N, D, device="cuda", generator=g).to(res)
    w = (1 + 0.1 * torch.randn(D, device="cuda", generator=g)).to(dtype)
    how = dict(post_weight=w if post else None, pre_weight=w, gate=z, res_scale=0.5)
    whole, normed = gdn.gdn_residual_norm(y, x, **how)
    assert errors() == 0
    try:
        for ns in (1, 1000, 3000, 10000):
            gdn.gdn_set_wait_limit_ns(ns)
            for _ in range(5):
                a, b = torch.full_like(whole, -7.0), torch.full_like(normed, -7.0)
                gdn.gdn_residual_norm(y, x, residual_out=a, out=b, **how)
                flags = errors()
                assert flags in (0, gdn.GDN_DEVERR_TIMEOUT)
                assert ns > 1 or flags  # (the first row's copy has only just been asked for)
                bad = ((a != whole).any(1) | (b != normed).any(1)).nonzero().flatten()
                assert flags or bad.numel() == 0
                # a row that was given up was not touched
                assert bool((a[bad] == -7).all()) and bool((b[bad] == -7).all())
    finally:
        gdn.gdn_set_wait_limit_ns(0)
    a, b = gdn.gdn_residual_norm(y, x, **how)
    assert torch.equal(a, whole) and torch.equal(b, normed) and errors() == 0
