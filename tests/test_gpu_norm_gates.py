"""Gates at the ends of their range: sigmoid(+inf) = 1, sigmoid(-inf) = 0, silu(z) = z for
large z up to the type's largest value, and +inf for +inf.  Tolerances as in
test_gpu_norms."""
import pytest
import torch

from gated_deltanet_recurrence_02_gb300 import gdn
from test_gpu_norms import near, rms

pytestmark = pytest.mark.gpu

DTYPES = pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=["f32", "f16", "bf16"])


def gates(dtype, n):
    top = torch.finfo(dtype).max
    z = torch.linspace(-130, 130, n, device="cuda")
    z[1::5], z[2::5], z[3::7], z[4::11] = float("inf"), top, -float("inf"), -top
    z[6::13], z[8::13] = 0.75 * top, -0.75 * top
    return z.to(dtype)


@DTYPES
@pytest.mark.parametrize("d", [128, 129, 4096])
def test_sigmoid_ends(dtype, d):
    x = (1 + torch.rand(6, 2, d, device="cuda")).to(dtype)
    z = gates(dtype, 6 * 2 * d).view(6, 2, d)
    y = gdn.gdn_gated_norm(x, z, None, gate=gdn.GDN_GATE_SIGMOID)
    near(y, rms(x.double(), 1e-6) * torch.sigmoid(z.double()))
    y, x = y.view(12, d), x.view(12, d)
    a, h = gdn.gdn_residual_norm(x, None, gate=z.view(12, d), gate_act=gdn.GDN_GATE_SIGMOID)
    want = x.double() * torch.sigmoid(z.view(12, d).double())
    near(a, want)
    near(h, rms(want, 1e-6))


@DTYPES
@pytest.mark.parametrize("d", [128, 129])
def test_silu_of_large_gates(dtype, d):
    x = (1 + torch.rand(6, 2, d, device="cuda")).to(dtype)
    z = gates(dtype, 6 * 2 * d).view(6, 2, d)
    z[z.isinf()] = 1.0
    z *= 0.5  # (the norm of x is below 2)
    y = gdn.gdn_gated_norm(x, z, None, gate=gdn.GDN_GATE_SILU)
    zd = z.double()
    near(y, rms(x.double(), 1e-6) * zd * torch.sigmoid(zd))
    z[..., 5] = float("inf")
    y = gdn.gdn_gated_norm(x, z, None, gate=gdn.GDN_GATE_SILU)
    assert bool((y[..., 5] == float("inf")).all()) and bool(torch.isfinite(y[..., 6:]).all())
