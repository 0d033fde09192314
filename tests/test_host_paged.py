"""Refusals of the rotary, append and attention entry points: each call fails validation
before anything is launched, so no GPU is needed and the fake addresses are never read."""
import inspect

import pytest
import torch

INVALID, UNSUPPORTED, ALIAS, ALIGN, WORKSPACE = 1, 2, 3, 4, 7
A, GiB = 1 << 36, 1 << 30


@pytest.fixture(scope="module")
def L():
    from gated_deltanet_recurrence_02_gb300 import build, gdn
    build.build()
    return gdn.lib()


def rotary(L, **kw):
    a = dict(x=A, out=A + GiB, pos=A + 2 * GiB, axes=A + 3 * GiB, f=A + 4 * GiB, N=10, H=4, d=64, R=64, axes_n=3,
             xs=256, os=256, flags=0, dt=2)
    a.update(kw)
    return L.gdn_rotary(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), INVALID), (dict(H=0), INVALID), (dict(d=0), INVALID), (dict(R=63), INVALID), (dict(R=66), INVALID),
    (dict(R=-2), INVALID), (dict(axes_n=0), INVALID), (dict(xs=255), INVALID), (dict(os=0), INVALID),
    (dict(flags=4), INVALID), (dict(dt=3), INVALID), (dict(dt=0x102), INVALID), (dict(x=None), INVALID),
    (dict(out=None), INVALID), (dict(pos=None), INVALID), (dict(f=None), INVALID),
    (dict(d=1025, xs=4100, os=4100), UNSUPPORTED), (dict(H=16385, xs=1 << 21, os=1 << 21), UNSUPPORTED),
    (dict(N=1 << 31), UNSUPPORTED), (dict(x=A + 1), ALIGN), (dict(dt=0, out=A + GiB + 2), ALIGN),
    (dict(pos=A + 2 * GiB + 2), ALIGN), (dict(axes=A + 3 * GiB + 1), ALIGN), (dict(f=A + 4 * GiB + 2), ALIGN),
    (dict(out=A + 2), ALIAS), (dict(out=A, os=512), ALIAS), (dict(out=A + 256, xs=384, os=384), ALIAS),
    (dict(out=A + 2 * GiB), ALIAS), (dict(out=A + 4 * GiB + 128 - 512), ALIAS), (dict(N=0), 0),
    (dict(N=0, x=None, out=None), 0)])
def test_rotary_rejects(L, kw, code):
    assert rotary(L, **kw) == code


def append(L, **kw):
    a = dict(q=A, k=A + 512, v=A + 768, q_out=A + GiB, kp=A + 2 * GiB, vp=A + 3 * GiB, table=A + 4 * GiB,
             lens=A + 5 * GiB, cu=None, pos=A + 6 * GiB, axes=None, f=A + 7 * GiB, B=2, T=5, Hq=4, Hk=2, d=64, R=64,
             axes_n=1, qs=512, ks=512, vs=512, os=256, pages=8, page=16, width=4, ps=2048, ss=128, hs=64, flags=0, dt=2)
    a.update(kw)
    return L.gdn_paged_append(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(Hq=-1), INVALID), (dict(Hk=0), INVALID), (dict(d=0), INVALID),
    (dict(R=1), INVALID), (dict(R=128), INVALID), (dict(axes_n=0), INVALID), (dict(ks=127), INVALID),
    (dict(vs=1), INVALID), (dict(qs=255), INVALID), (dict(os=255), INVALID), (dict(flags=2), INVALID),
    (dict(dt=7), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(q=None), INVALID),
    (dict(q_out=None), INVALID), (dict(Hq=0), INVALID), (dict(f=None), INVALID), (dict(kp=None), INVALID),
    (dict(vp=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(pages=-1), INVALID),
    (dict(page=0), INVALID), (dict(width=-1), INVALID), (dict(ps=63), INVALID), (dict(ss=63), INVALID),
    (dict(hs=0), INVALID), (dict(hs=-64), INVALID), (dict(ps=1 << 62), INVALID), (dict(B=65536), UNSUPPORTED),
    (dict(T=1 << 30), UNSUPPORTED), (dict(d=1026, qs=8192, ks=8192, vs=8192, os=8192, ps=8192, ss=8192, hs=8192), UNSUPPORTED),
    (dict(k=A + 513), ALIGN), (dict(kp=A + 2 * GiB + 1), ALIGN), (dict(table=A + 4 * GiB + 2), ALIGN),
    (dict(lens=A + 5 * GiB + 1), ALIGN), (dict(cu=A + 8 * GiB + 2), ALIGN),
    (dict(vp=A + 2 * GiB), ALIAS), (dict(kp=A), ALIAS), (dict(vp=A + GiB), ALIAS), (dict(vp=A + 4 * GiB - 4096), ALIAS),
    (dict(q_out=A + 512, os=512), ALIAS), (dict(q_out=A, os=256), ALIAS), (dict(q_out=A + 6 * GiB), ALIAS),
    (dict(B=0), 0), (dict(T=0), 0)])
def test_append_rejects(L, kw, code):
    assert append(L, **kw) == code


def attention(L, **kw):
    a = dict(q=A, kp=A + 2 * GiB, vp=A + 3 * GiB, table=A + 4 * GiB, lens=A + 5 * GiB, cu=None, out=A + 6 * GiB,
             lse=A + 7 * GiB, B=2, T=5, Hq=4, Hk=2, d=64, qs=256, pages=8, page=16, width=4, ps=2048, ss=128, hs=64,
             scale=0.125, window=0, flags=0, dt=2, ws=A + 8 * GiB, wsb=GiB)
    a.update(kw)
    return L.gdn_paged_attention(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hk=0), INVALID), (dict(Hk=3), INVALID),
    (dict(d=0), INVALID), (dict(window=-1), INVALID), (dict(window=4, flags=1), INVALID), (dict(flags=2), INVALID),
    (dict(dt=5), INVALID), (dict(qs=255), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID),
    (dict(kp=None), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(page=0), INVALID),
    (dict(ss=32), INVALID), (dict(d=48, qs=512), UNSUPPORTED), (dict(d=256, qs=1024), UNSUPPORTED),
    (dict(B=65536), UNSUPPORTED), (dict(T=1 << 29), UNSUPPORTED), (dict(q=A + 1), ALIGN), (dict(out=A + 6 * GiB + 2), ALIGN),
    (dict(lse=A + 7 * GiB + 2), ALIGN), (dict(ws=A + 8 * GiB + 4), ALIGN), (dict(vp=A + 3 * GiB + 1), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(wsb=16), WORKSPACE), (dict(out=A), ALIAS), (dict(out=A + 2 * GiB), ALIAS),
    (dict(lse=A + 6 * GiB + 16), ALIAS), (dict(ws=A + 3 * GiB), ALIAS), (dict(B=0), 0), (dict(T=0), 0)])
def test_attention_rejects(L, kw, code):
    assert attention(L, **kw) == code


def test_workspace_size(L):
    size = L.gdn_paged_attention_workspace_size
    bad = (1 << 64) - 1
    for kw in ((-1, 1, 4, 2, 64, 2, 0), (1, 1, 4, 3, 64, 2, 0), (1, 1, 4, 2, 0, 2, 0), (1, 1, 4, 2, 64, 9, 0)):
        assert size(*kw) == bad
    assert 0 < size(1, 1, 4, 2, 64, 2, 0) < 1 << 32
    # only sizes that a call may have: as much for a short as for a long batch of the same kind
    assert size(1, 4096, 4, 2, 64, 2, 0) == size(16, 4096, 4, 2, 64, 2, 0)


def test_binding_checks_shapes_before_the_call():
    from gated_deltanet_recurrence_02_gb300 import gdn
    i32 = torch.int32
    x, f = torch.zeros(6, 4, 64), torch.zeros(32)
    pos = torch.zeros(6, dtype=i32)
    for kw in (dict(inv_freq=f.double()), dict(inv_freq=torch.zeros(33)), dict(positions=pos[:5]),
               dict(positions=pos.long()), dict(axes=pos), dict(out=x[:, :2]), dict(out=x.half()), dict()):
        a = {**dict(positions=pos, inv_freq=f), **kw}
        with pytest.raises(ValueError):
            gdn.gdn_rotary(x, a["positions"], a["inv_freq"], axes=a.get("axes"), out=a.get("out"))
    pages = torch.zeros(3, 16, 2, 64)
    table, lens = torch.zeros(2, 4, dtype=i32), torch.zeros(2, dtype=i32)
    k = torch.zeros(6, 2, 64)
    for kw in (dict(v=k[:5]), dict(v=k.half()), dict(kp=pages[:, :, :1]), dict(kp=pages.half(), vp=pages.half()),
               dict(vp=pages[:2]), dict(table=table[:1]), dict(lens=lens[:1]), dict(q=k[:5]), dict(q=k.half()),
               dict(q_out=k), dict(T=4), dict(cu_seqlens=lens), dict(vp=pages.transpose(0, 1).contiguous().transpose(0, 1)),
               dict()):
        a = {**dict(v=k, kp=pages, vp=pages, table=table, lens=lens), **kw}
        with pytest.raises(ValueError):
            gdn.gdn_paged_append(k, a["v"], a["kp"], a["vp"], a["table"], a["lens"], B=2, T=a.get("T"),
                                 cu_seqlens=a.get("cu_seqlens"), q=a.get("q"), q_out=a.get("q_out"))
    for kw in (dict(q=x[:, :, :32]), dict(q=x.half()), dict(out=x.half()), dict(lse=x[:, :, 0].half()), dict(T=4),
               dict(cu_seqlens=lens), dict(lens=lens[:1]), dict()):
        a = {**dict(q=x, lens=lens), **kw}
        with pytest.raises(ValueError):
            gdn.gdn_paged_attention(a["q"], pages, pages, table, a["lens"], B=2, T=a.get("T"),
                                    cu_seqlens=a.get("cu_seqlens"), out=a.get("out"), lse=a.get("lse"))
    for fn in (gdn.gdn_rotary, gdn.gdn_paged_append, gdn.gdn_paged_attention):
        assert "stream" in inspect.signature(fn).parameters
