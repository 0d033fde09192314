"""Refusals of the linear-attention, norm and draft-verification entry points:
each call fails validation before anything is launched, so no GPU is needed and
the fake device addresses are never dereferenced."""
import inspect

import pytest
import torch

INVALID, UNSUPPORTED, ALIAS, ALIGN, WORKSPACE = 1, 2, 3, 4, 7
A, GiB = 1 << 32, 1 << 30


@pytest.fixture(scope="module")
def L():
    from gated_deltanet_recurrence_02_gb300 import build, gdn
    build.build()
    return gdn.lib()


LINEAR = dict(q=A, k=A + GiB, v=A + 2 * GiB, alpha=A + 3 * GiB, cu=None, s0=A + 5 * GiB, idx=None, n0=2,
              sf=A + 6 * GiB, out=A + 7 * GiB, B=2, T=300, Hq=2, Hk=2, Hv=6, dk=128, dv=128, scale=1.0, dtq=2, dtg=0)


def prefill(L, **kw):
    a = {**LINEAR, "ws": A + 8 * GiB, "wsb": GiB, **kw}
    return L.gdn_linear_prefill(*a.values(), None)


def recurrent(L, **kw):
    a = {**LINEAR, "cap": 4, "cc": A + 8 * GiB, "act": None, "su": A + 9 * GiB, **kw}
    return L.gdn_linear_recurrent(*a.values(), None)


COMMON = [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(Hq=1), INVALID), (dict(Hv=5), INVALID),
    (dict(q=None), INVALID), (dict(alpha=None), INVALID), (dict(out=None), INVALID),
    (dict(dk=48), UNSUPPORTED), (dict(dv=256), UNSUPPORTED), (dict(dtq=3), INVALID), (dict(dtg=7), INVALID),
    (dict(dtq=2 | 0x100), INVALID),   # no normalisation of q and k here
    (dict(dtg=0 | 0x400), INVALID),   # no beta here
    (dict(n0=1), INVALID), (dict(s0=None, idx=A + 4 * GiB), INVALID),
    (dict(v=A + 2 * GiB + 2), ALIGN), (dict(cu=A + 4 * GiB + 2), ALIGN),
    (dict(out=A), ALIAS), (dict(sf=A + 5 * GiB, idx=A + 4 * GiB), ALIAS), (dict(out=A + 6 * GiB), ALIAS),
    (dict(sf=A + 5 * GiB + 4096), ALIAS),
]


@pytest.mark.parametrize("kw,code", COMMON)
def test_linear_rejects(L, kw, code):
    assert prefill(L, **kw) == code
    assert recurrent(L, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(cap=-1), INVALID), (dict(cc=None), INVALID), (dict(su=None), INVALID),
    (dict(su=A + 9 * GiB + 4), ALIGN), (dict(cc=A + 8 * GiB + 1), ALIGN), (dict(su=A + 7 * GiB), ALIAS)])
def test_linear_recurrent_rejects_capture(L, kw, code):
    assert recurrent(L, **kw) == code


def test_linear_workspace_and_empty(L):
    size = L.gdn_linear_prefill_workspace_size
    bad = (1 << 64) - 1
    assert size(-1, 1, 1, 1, 64, 64, 2, 0) == bad and size(1, 1, 1, 1, 64, 64, 9, 0) == bad
    need = size(1, 4100, 16, 32, 128, 128, 2, 0)
    if need > 0:
        kw = dict(B=1, T=4100, Hq=16, Hk=16, Hv=32)
        assert prefill(L, **kw, wsb=need - 1) == WORKSPACE
        assert prefill(L, **kw, ws=None) == WORKSPACE
    assert prefill(L, B=0) == 0 and recurrent(L, B=0) == 0


def gated(L, **kw):
    a = dict(x=A, z=A + GiB, w=A + 2 * GiB, out=A + 3 * GiB, N=4, H=2, d=64, xs=128, zs=128, os=128, eps=1e-6,
             gate=1, dtx=2, dtw=0)
    a.update(kw)
    return L.gdn_gated_norm(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), INVALID), (dict(H=0), INVALID), (dict(d=0), INVALID), (dict(d=16385, xs=1 << 16, zs=1 << 16, os=1 << 16), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(z=None), INVALID), (dict(gate=0), INVALID),
    (dict(gate=3), INVALID), (dict(gate=0x41), INVALID), (dict(dtx=5), INVALID), (dict(dtw=5), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(xs=127), INVALID), (dict(zs=1), INVALID), (dict(os=0), INVALID),
    (dict(x=A + 1), ALIGN), (dict(w=A + 2 * GiB + 2), ALIGN), (dict(N=1 << 31), UNSUPPORTED),
    (dict(out=A + 64), ALIAS), (dict(out=A + GiB), ALIAS), (dict(out=A, os=256), ALIAS), (dict(N=0), 0)])
def test_gated_norm_rejects(L, kw, code):
    assert gated(L, **kw) == code


def residual(L, **kw):
    a = dict(y=A, x=A + GiB, z=A + 2 * GiB, w1=A + 3 * GiB, w2=A + 4 * GiB, xo=A + 5 * GiB, out=A + 6 * GiB, N=4,
             D=128, ys=128, zs=128, scale=1.0, eps=1e-6, flags=1, dtx=2, dtr=0, dtw=0)
    a.update(kw)
    return L.gdn_residual_norm(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), INVALID), (dict(D=0), INVALID), (dict(D=16385, ys=1 << 16, zs=1 << 16), UNSUPPORTED), (dict(y=None), INVALID),
    (dict(xo=None, out=None), INVALID), (dict(z=None), INVALID), (dict(flags=0), INVALID), (dict(flags=0x10), INVALID),
    (dict(dtr=1), UNSUPPORTED), (dict(dtx=0, dtr=2), UNSUPPORTED), (dict(dtr=8), INVALID), (dict(ys=127), INVALID),
    (dict(zs=4), INVALID), (dict(eps=-1.0), INVALID), (dict(x=A + GiB + 2), ALIGN), (dict(out=A + 6 * GiB + 1), ALIGN),
    (dict(xo=A), ALIAS), (dict(xo=A + GiB + 64), ALIAS), (dict(out=A + 5 * GiB), ALIAS), (dict(out=A), ALIAS), (dict(N=0), 0)])
def test_residual_norm_rejects(L, kw, code):
    assert residual(L, **kw) == code


def accept(L, **kw):
    a = dict(p=A, q=A + GiB, x=A + 2 * GiB, u=A + 3 * GiB, count=None, tokens=A + 4 * GiB, n=A + 5 * GiB, B=2, K=4,
             V=1000, ps=1000, qs=1000, dt=0)
    a.update(kw)
    return L.gdn_accept_drafts(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(K=-1), INVALID), (dict(V=0), INVALID), (dict(dt=4), INVALID), (dict(ps=999), INVALID),
    (dict(qs=10), INVALID), (dict(p=None), INVALID), (dict(x=None), INVALID), (dict(u=None), INVALID),
    (dict(tokens=None), INVALID), (dict(n=None), INVALID), (dict(V=(1 << 22) + 1, ps=1 << 23, qs=1 << 23), UNSUPPORTED),
    (dict(K=1025), UNSUPPORTED), (dict(B=65536), UNSUPPORTED), (dict(p=A + 2), ALIGN), (dict(u=A + 3 * GiB + 2), ALIGN),
    (dict(tokens=A + 3 * GiB), ALIAS), (dict(n=A + 4 * GiB + 4), ALIAS), (dict(B=0), 0)])
def test_accept_drafts_rejects(L, kw, code):
    assert accept(L, **kw) == code


def test_binding_checks_shapes_before_the_call():
    from gated_deltanet_recurrence_02_gb300 import gdn
    x = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError):
        gdn.gdn_gated_norm(x, x[:, :2], None)
    with pytest.raises(ValueError):
        gdn.gdn_gated_norm(x, x, None)            # not on a device
    with pytest.raises(ValueError):
        gdn.gdn_gated_norm(x, x, torch.zeros(7))
    with pytest.raises(ValueError):
        gdn.gdn_residual_norm(x[0], x[0, :2])
    with pytest.raises(ValueError):
        gdn.gdn_residual_norm(x[0], x[0], post_weight=torch.zeros(8), pre_weight=torch.zeros(8).half())
    p = torch.zeros(2, 3, 10)
    with pytest.raises(ValueError):
        gdn.gdn_accept_drafts(p, None, torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3))
    with pytest.raises(ValueError):
        gdn.gdn_accept_drafts(p, None, torch.zeros(2, 2), torch.zeros(2, 3))
    for fn in (gdn.gdn_linear_prefill, gdn.gdn_linear_recurrent, gdn.gdn_gated_norm, gdn.gdn_residual_norm,
               gdn.gdn_accept_drafts):
        assert "stream" in inspect.signature(fn).parameters
