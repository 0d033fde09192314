"""The fused norms against their formulas in 64 bits.

Tolerances: the result is rounded once (elementwise within half a unit in the
last place) and formed in fp32 before that; sums of up to 16384 squares, a
reciprocal root, an exponential and a divide leave it within 2^-19 of its
value.  So |error| <= (u + 2^-19) |value| with u = 2^-8 (bf16), 2^-11 (fp16;
below its normal range 2^-24 absolute), 0 (fp32); for x' = x + s g u the fp32
error is relative to the terms."""
import pytest
import torch

from gated_deltanet_recurrence_02_gb300 import gdn

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 0.0}
F = 2.0 ** -19


def near(got, want, terms=None):
    u = U[got.dtype]
    size = want.abs() if terms is None else terms
    tiny = 2.0 ** -24 if got.dtype == torch.float16 else 2.0 ** -126
    assert torch.isfinite(got).all()
    bad = (got.double() - want).abs() - (u * want.abs() + F * size + tiny)
    assert float(bad.max()) <= 0, float(bad.max())


def act(z, kind):
    s = torch.sigmoid(z)
    return {gdn.GDN_GATE_NONE: torch.ones_like(z), gdn.GDN_GATE_SILU: z * s, gdn.GDN_GATE_SIGMOID: s}[kind]


def rms(x, eps):
    return x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 5, 7), (7, 6, 80), (33, 4, 128), (2, 3, 129), (5, 1, 1000),
                                   (3, 2, 1024), (2, 1, 4099), (2, 1, 16384), (1, 1, 16383), (700, 32, 64)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("kind", [gdn.GDN_GATE_NONE, gdn.GDN_GATE_SILU, gdn.GDN_GATE_SIGMOID])
def test_gated(shape, dtype, kind):
    N, H, d = shape
    g = torch.Generator("cuda").manual_seed(d)
    x = torch.randn(N, H, d, device="cuda", generator=g).to(dtype)
    z = (3 * torch.randn(N, H, d, device="cuda", generator=g)).to(dtype) if kind else None
    wdt = torch.float32 if d % 2 else dtype
    w = torch.randn(d, device="cuda", generator=g).to(wdt)
    zd = act(z.double(), kind) if kind else 1.0
    y = gdn.gdn_gated_norm(x, z, w, eps=1e-5, gate=kind)
    near(y, rms(x.double(), 1e-5) * w.double() * zd)
    y = gdn.gdn_gated_norm(x, z, w, eps=1e-5, gate=kind | gdn.GDN_GATE_FIRST | gdn.GDN_NORM_UNIT_OFFSET)
    near(y, rms(x.double() * zd, 1e-5) * (1 + w.double()))
    y = gdn.gdn_gated_norm(x, z, None, eps=1e-5, gate=kind, out=x)  # in place, without weights
    assert y.data_ptr() == x.data_ptr()


@pytest.mark.parametrize("off,pad", [(0, 0), (8, 8), (3, 0), (1, 5)])
def test_gated_slices_of_wider_rows(off, pad):
    """x, z and out as slices of wider rows, on and off 16-byte boundaries."""
    N, H, d = 9, 3, 64
    wide = torch.randn(N, off + 2 * H * d + pad, device="cuda").bfloat16()
    x = wide[:, off:off + H * d].unflatten(1, (H, d))
    z = wide[:, off + H * d:off + 2 * H * d].unflatten(1, (H, d))
    buf = torch.full((N, H * d + 16), 7.0, device="cuda").bfloat16()
    w = torch.randn(d, device="cuda")
    gdn.gdn_gated_norm(x, z, w, out=buf[:, 8:8 + H * d].unflatten(1, (H, d)))
    zd = z.double()
    near(buf[:, 8:8 + H * d].unflatten(1, (H, d)), rms(x.double(), 1e-6) * w.double() * zd * torch.sigmoid(zd))
    assert (buf[:, :8] == 7).all() and (buf[:, 8 + H * d:] == 7).all()


def test_gated_zero_rows_extremes_and_none():
    x = torch.zeros(4, 1, 128, device="cuda")
    z = torch.full((4, 1, 128), 3.0, device="cuda")
    z[1], z[2] = -1e30, 1e4
    x[1:] = 2.0
    x[3, 0, 5] = float("nan")
    y = gdn.gdn_gated_norm(x, z, None, gate=gdn.GDN_GATE_SIGMOID)
    assert not y[:2].any()                      # a row of zeros, and a closed gate
    assert torch.allclose(y[2], torch.ones_like(y[2]))
    assert torch.isnan(y[3]).all() and torch.isfinite(y[:3]).all()
    assert gdn.gdn_gated_norm(x[:0], z[:0], None).shape == (0, 1, 128)


@pytest.mark.parametrize("dtype,res", [(torch.float32, torch.float32), (torch.float16, torch.float16),
                                       (torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16),
                                       (torch.float16, torch.float32)])
@pytest.mark.parametrize("N,D", [(1, 1), (3, 33), (5, 2047), (4, 2048), (130, 256), (2, 8192), (3, 16384), (2, 16383)])
@pytest.mark.parametrize("post,gate", [(True, True), (True, False), (False, True), (False, False)])
def test_residual(N, D, dtype, res, post, gate):
    g = torch.Generator("cuda").manual_seed(D)
    y, z = (torch.randn(N, D, device="cuda", generator=g).to(dtype) for _ in range(2))
    x = (2 * torch.randn(N, D, device="cuda", generator=g)).to(res)
    w1, w2 = (torch.randn(D, device="cuda", generator=g).to(dtype) for _ in range(2))
    a, h = gdn.gdn_residual_norm(y, x, post_weight=w1 if post else None, gate=z if gate else None,
                                 gate_act=gdn.GDN_GATE_SILU, res_scale=0.3, pre_weight=w2, eps=1e-5)
    u = rms(y.double(), 1e-5) * w1.double() if post else y.double()
    u = u * act(z.double(), gdn.GDN_GATE_SILU) if gate else u
    want = x.double() + 0.3 * u
    terms = x.double().abs() + 0.3 * u.abs()
    near(a, want, terms)
    near(h, rms(want, 1e-5) * w2.double(), rms(want, 1e-5).abs() * w2.double().abs() + terms / want.norm(dim=1, keepdim=True) * D ** 0.5 * w2.double().abs())
    # in place gives the same bits
    b, h2 = gdn.gdn_residual_norm(y, x, post_weight=w1 if post else None, gate=z if gate else None,
                                  gate_act=gdn.GDN_GATE_SILU, res_scale=0.3, pre_weight=w2, eps=1e-5, residual_out=x)
    assert b.data_ptr() == x.data_ptr() and torch.equal(a, b) and torch.equal(h, h2)


def test_residual_without_residual_offset_and_slices():
    wide = torch.randn(6, 700, device="cuda").bfloat16()
    y, z = wide[:, 5:261], wide[:, 300:556]
    w = torch.randn(256, device="cuda")
    a, h = gdn.gdn_residual_norm(y, None, post_weight=w, gate=z, unit_offset=True, pre_weight=w,
                                 residual_dtype=torch.float32)
    want = rms(y.double(), 1e-6) * (1 + w.double()) * torch.sigmoid(z.double())
    near(a, want)
    near(h, rms(want, 1e-6) * (1 + w.double()))
    assert gdn.gdn_residual_norm(y[:0], None)[1].shape == (0, 256)


def test_offsets_past_32_bits():
    """More than 2^31 elements in one call, the last rows checked."""
    N, H, d = 140000, 128, 128
    x = torch.empty(N, H, d, device="cuda", dtype=torch.bfloat16).fill_(2.0)
    x[-1] = torch.randn(H, d, device="cuda")
    y = gdn.gdn_gated_norm(x, x, None)
    xd = x[-1].double()
    near(y[-1], rms(xd, 1e-6) * xd * torch.sigmoid(xd))
    assert torch.allclose(y[:3].float(), torch.full((3, H, d), 1.7616, device="cuda"), atol=0.01)
    del y
    a, h = gdn.gdn_residual_norm(x.view(N, H * d), None)
    near(h[-1:], rms(x[-1].double().view(1, -1), 1e-6))
    assert torch.equal(a[-1], x[-1].view(-1))


def test_row_copies_that_run_out_are_reported():
    y = torch.randn(400, 4096, device="cuda").bfloat16()
    gdn.gdn_set_wait_limit_ns(1)
    try:
        gdn.gdn_residual_norm(y, y)
        with pytest.raises(gdn.GdnError) as e:
            gdn.gdn_device_errors()
        assert e.value.status == 6
    finally:
        gdn.gdn_set_wait_limit_ns(0)
    _, h = gdn.gdn_residual_norm(y, None)
    near(h, rms(y.double(), 1e-6))
    assert gdn.gdn_device_errors() == 0
